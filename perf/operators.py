"""Cases that measure the packed attention (forward, single-token form and backward) and the norms around a block
(forward and backward), each in plain torch operations and through vision_sliding_window_b200.na2d.

Attention.  q, out [Tq][Hq][d]; k, v [Tk][Hk][d]; sequence s owns the rows cu_q[s] .. cu_q[s+1] of q and the keys from
cu_k[s] on, Lk of them (len_k[s] of the cu_k[s+1] - cu_k[s] slots of a cache).  Row i of a sequence stands at key
position p = i + Lk - Lq; it sees the keys [max(0, p - window + 1), p] when causal (window 0: from key 0), all Lk
otherwise.  out = softmax(scale q k^T) v, lse the logarithm of the softmax's sum; a row that sees no key gives zeros
and -inf.

Norms.  y = x + scale * gate . P(o), h = N(y) w + b, with N a LayerNorm or RMS norm over the last axis and P such a
norm with its own weight and bias, or the identity.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token for each of a few short conversations: nothing but latency.
        dict(name="decode_small", op="attend", lq="1 1 1 1", lk="37 400 129 255", cap=512, hq=8, hk=2, d=64,
             causal=True, window=0, dtype="bf16"),
        # One token for each of a batch of requests over long caches of unequal length.
        dict(name="decode_long", op="attend", lq="1 1 1 1 1 1 1 1 1 1 1 1 1 1 1 1",
             lk="16384 1 9001 12288 640 15999 7777 4096 11111 2049 16000 513 8192 14336 5000 10240",
             cap=16384, hq=32, hk=8, d=128, causal=True, window=0, dtype="bf16"),
        # Prompts of unequal length packed into one batch.
        dict(name="prompt_ragged", op="attend", lq="1 2500 17 640 1111 300 2047 129 900 64 255 1500",
             lk="1 2500 17 640 1111 300 2047 129 900 64 255 1500", cap=0, hq=16, hk=4, d=128, causal=True,
             window=0, dtype="bf16"),
        # Whole maps of unequal size packed together (7x7 to 56x56 and odd ones), every position seeing its whole map.
        dict(name="maps_packed", op="attend", lq="3136 784 196 49 1369 2209 400 3025",
             lk="3136 784 196 49 1369 2209 400 3025", cap=0, hq=8, hk=8, d=32, causal=False, window=0,
             dtype="f16"),
        # One long prompt of an odd length.
        dict(name="prompt_long", op="attend", lq="12001", lk="12001", cap=0, hq=16, hk=2, d=128, causal=True,
             window=0, dtype="bf16"),
        # Single precision with a sliding window.
        dict(name="window_f32", op="attend", lq="700 33 512 257", lk="700 33 512 257", cap=0, hq=8, hk=8, d=64,
             causal=True, window=200, dtype="f32"),
        # A training batch of packed documents.
        dict(name="train_ragged", op="attend_grad", lq="2000 511 1 1024 77 1300 640 1800",
             lk="2000 511 1 1024 77 1300 640 1800", cap=0, hq=16, hk=4, d=64, causal=True, window=0,
             dtype="bf16"),
        # A training step on one long document.
        dict(name="train_long", op="attend_grad", lq="6001", lk="6001", cap=0, hq=16, hk=4, d=128, causal=True,
             window=0, dtype="bf16"),
        # The norms around a block for the tokens of a small serving batch: latency.
        dict(name="norm_tokens", op="norm", rows=8, c=2048, gates=1, post=True, rms=True, bias=False, dtype="bf16"),
        # The same around the blocks of a long prompt: bandwidth.
        dict(name="norm_wide", op="norm", rows=16387, c=4096, gates=1, post=True, rms=True, bias=False, dtype="bf16"),
        # Gradients of the layer-scaled residual and LayerNorm of a batch of 32 56x56 maps, 64 channels.
        dict(name="norm_grad_map", op="norm_grad", rows=32 * 56 * 56, c=64, gates=1, post=False, rms=False, bias=True,
             dtype="f16"),
        # Gradients of both norms and of a gate for each of 8 packed documents of a training batch.
        dict(name="norm_grad_wide", op="norm_grad", rows=8 * 1021, c=4096, gates=8, post=True, rms=False, bias=True,
             dtype="bf16"),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("norm"):
        c = rng.choice([64, 96, 128, 200, 256, 333, 512, 768, 1000, 2048, 2500, 4096, _log_between(rng, 32, 4096)])
        rows = _log_between(rng, 1, min(110000, (16387 if op == "norm" else 8168) * 4096 // c))
        gates = rng.choice([0, 1, 1, rng.choice([2, 3, 5, 8, 32])])
        rows = max(1, rows // max(1, gates)) * max(1, gates)
        return dict(op=op, rows=rows, c=c, gates=gates, post=rng.random() < 0.5, rms=rng.random() < 0.5,
                    bias=rng.random() < 0.5, dtype=dtype)
    d = rng.choice([16, 32, 64, 64, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 7, 8])
    single = op == "attend" and rng.random() < 0.4
    longest = (8192 if single else 700 if dtype == "f32" else 2500)
    n = _log_between(rng, 1, 20)
    lk = [_log_between(rng, 1, longest) for _ in range(n)]
    while not single and n * hq * max(lk) ** 2 > 12 * 16 * 2500 ** 2:  # the most that a listed batch's plain form holds
        lk = [(x + 1) // 2 for x in lk]
    lq = [1] * n if single else list(lk)
    causal = rng.random() < 0.7
    cap = 0
    if single:
        cap = max(lk) + rng.randrange(64)
    elif op == "attend" and rng.random() < 0.3:  # prompts whose first part is in the cache already
        lq = [max(1, int(x * rng.uniform(0.1, 1.0))) for x in lk]
    window = _log_between(rng, 8, longest) if causal and rng.random() < 0.3 else 0
    return dict(op=op, lq=" ".join(map(str, lq)), lk=" ".join(map(str, lk)), cap=cap, hq=hq, hk=hk, d=d,
                causal=causal, window=window, dtype=dtype)


# --------------------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """The sequences' rows and keys, which a case lists in a text."""
    return [int(x) for x in case["lq"].split()], [int(x) for x in case["lk"].split()]


def _starts(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(t)

    s = dict(case=case)
    if case["op"].startswith("norm"):
        rows, c = case["rows"], case["c"]
        s["x"], s["o"] = normal(rows, c), normal(rows, c, std=0.7, mean=0.1)
        s["w"], s["pw"] = normal(c, std=0.1, mean=1.0), (normal(c, std=0.1, mean=1.0) if case["post"] else None)
        s["b"] = normal(c, std=0.1) if case["bias"] else None
        s["pb"] = normal(c, std=0.1) if case["bias"] and case["post"] else None
        s["gate"] = normal(case["gates"], c, std=0.1, mean=0.3) if case["gates"] else None
        if case["op"] == "norm_grad":  # x stands for the updated residual y, which the backward pass takes
            s["dy"], s["dh"] = normal(rows, c), normal(rows, c)
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    lq, lk = _lengths(case)
    slots = [case["cap"]] * len(lk) if case["cap"] else lk
    s["q"] = normal(sum(lq), hq, d)
    s["k"], s["v"] = normal(sum(slots), hk, d), normal(sum(slots), hk, d)
    s["cu_q"] = torch.tensor(_starts(lq), dtype=torch.int32, device="cuda")
    s["cu_k"] = torch.tensor(_starts(slots), dtype=torch.int32, device="cuda")
    s["len_k"] = torch.tensor(lk, dtype=torch.int32, device="cuda") if case["cap"] else None
    if case["op"] == "attend_grad":  # what the forward pass left behind, and the gradient that arrives
        s["out"], s["lse"] = _attend(s)
        s["dout"] = normal(sum(lq), hq, d)
    return s


# ----------------------------------------------------------------------------------------------------- plain forms
def _padded(s):
    """q [n, Hk, Lq*G, d], k and v [n, Hk, Lk, d] in 32 bits, padded to the longest sequence; the mask of what a row
    sees [n, 1, Lq*G, Lk]; which padded rows are real [n, Lq] and which padded keys [n, Lk]."""
    case = s["case"]
    lq, lk = _lengths(case)
    n, group, d = len(lq), case["hq"] // case["hk"], case["d"]
    dev = s["q"].device
    start_q, start_k = s["cu_q"].long(), s["cu_k"].long()
    length_q = start_q[1:] - start_q[:-1]
    length_k = s["len_k"].long() if s["len_k"] is not None else start_k[1:] - start_k[:-1]
    rows, keys = torch.arange(max(lq), device=dev), torch.arange(max(lk), device=dev)
    real_q, real_k = rows < length_q[:, None], keys < length_k[:, None]
    at_q = (start_q[:-1, None] + rows).clamp(max=s["q"].shape[0] - 1)
    at_k = (start_k[:-1, None] + keys).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][at_q].float().view(n, len(rows), case["hk"], group, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k, v = (s[x][at_k].float().permute(0, 2, 1, 3) for x in ("k", "v"))
    at = rows + (length_k - length_q)[:, None]  # a row's position among the keys
    sees = real_q[:, :, None] & real_k[:, None, :]
    if case["causal"]:
        sees &= keys <= at[:, :, None]
        if case["window"]:
            sees &= keys > at[:, :, None] - case["window"]
    return q, k, v, sees.repeat_interleave(group, 1)[:, None], real_q, real_k


def _weights(q, k, sees, scale):
    """The softmax's weights and the logarithm of its sum, 0 and -inf for rows that see nothing."""
    logits = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~sees, -math.inf)
    top = logits.amax(-1, keepdim=True)
    weights = logits.sub_(top.clamp(min=-3e38)).exp_()
    total = weights.sum(-1, keepdim=True)
    lse = total.log() + top.clamp(min=-3e38)
    return weights.div_(total.clamp(min=1e-37)), lse


def _unpadded(x, real, group):
    """[n, Hk, L*G, d] -> [T, Hk*G, d]: the real rows, sequence after sequence."""
    n, hk, rows, d = x.shape
    return x.view(n, hk, rows // group, group, d).permute(0, 2, 1, 3, 4).reshape(n, rows // group, hk * group, d)[real]


def _attend(s):
    case = s["case"]
    group = case["hq"] // case["hk"]
    q, k, v, sees, real_q, _ = _padded(s)
    weights, lse = _weights(q, k, sees, case["d"] ** -0.5)
    out = _unpadded(weights @ v, real_q, group).to(s["q"].dtype)
    return out, _unpadded(lse, real_q, group)[..., 0].t().contiguous()


def _attend_grad(s):
    case = s["case"]
    group, scale, t = case["hq"] // case["hk"], case["d"] ** -0.5, s["q"].dtype
    q, k, v, sees, real_q, real_k = _padded(s)
    dout = _padded(dict(s, q=s["dout"]))[0] * real_q.repeat_interleave(group, 1)[:, None, :, None]
    weights, _ = _weights(q, k, sees, scale)
    dv = weights.transpose(-1, -2) @ dout
    dweights = dout @ v.transpose(-1, -2)
    dlogits = (dweights - (weights * dweights).sum(-1, keepdim=True)) * weights * scale
    dq, dk = dlogits @ k, dlogits.transpose(-1, -2) @ q
    return _unpadded(dq, real_q, group).to(t), _unpadded(dk, real_k, 1).to(t), _unpadded(dv, real_k, 1).to(t)


EPS = 1e-5
SCALE = 0.5


def _normed(x, rms):
    """x normalised over its last axis, and the reciprocal deviation."""
    x = x if rms else x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r


def _float(x):
    return None if x is None else x.float()


def _affine(x, w, b):
    return x * w if b is None else x * w + b


def _per_row(gate, rows):
    return 1.0 if gate is None else gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _norm(s):
    case = s["case"]
    o = s["o"].float()
    if case["post"]:
        o = _affine(_normed(o, case["rms"])[0], _float(s["pw"]), _float(s["pb"]))
    y = s["x"].float() + SCALE * _per_row(s["gate"], case["rows"]) * o
    h = _affine(_normed(y, case["rms"])[0], _float(s["w"]), _float(s["b"]))
    return y.to(s["x"].dtype), h.to(s["x"].dtype)


def _norm_back(dn, n, r, rms):
    """The gradient of the norm's input from that of its output, n the output and r the reciprocal deviation."""
    dn = dn if rms else dn - dn.mean(-1, keepdim=True)
    return r * (dn - n * (dn * n).mean(-1, keepdim=True))


def _norm_grad(s):
    case, t = s["case"], s["x"].dtype
    dh, gate = s["dh"].float(), _per_row(s["gate"], case["rows"])
    n, r = _normed(s["x"].float(), case["rms"])
    dx = s["dy"].float() + _norm_back(dh * s["w"].float(), n, r, case["rms"])
    grads = dict(dx=dx.to(t), dw=(dh * n).sum(0), db=None if s["b"] is None else dh.sum(0))
    o = s["o"].float()
    if case["post"]:
        m, q = _normed(o, case["rms"])
        o = _affine(m, _float(s["pw"]), _float(s["pb"]))
    dp = SCALE * dx * gate
    if case["gates"]:
        grads["dgate"] = (SCALE * dx * o).view(case["gates"], -1, case["c"]).sum(1)
    if case["post"]:
        grads["dpw"], grads["dpb"] = (dp * m).sum(0), None if s["pb"] is None else dp.sum(0)
        dp = _norm_back(dp * s["pw"].float(), m, q, case["rms"])
    grads["do"] = dp.to(t)
    return {k: v for k, v in grads.items() if v is not None}


# -------------------------------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"attend": _attend, "attend_grad": _attend_grad, "norm": _norm, "norm_grad": _norm_grad}[case["op"]](state)


def _own(case, s):
    from vision_sliding_window_b200 import na2d

    if case["op"] == "attend":
        return na2d.packed_forward(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], len_k=s["len_k"],
                                   causal=case["causal"], window=case["window"])
    if case["op"] == "attend_grad":
        return na2d.packed_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu_q"], s["cu_k"],
                                    causal=case["causal"], window=case["window"])
    how = dict(o=s["o"], post=case["post"], post_w=s["pw"], post_b=s["pb"], gate=s["gate"], scale=SCALE, eps=EPS,
               rms=case["rms"])
    if case["op"] == "norm":
        return na2d.norm_forward(s["x"], s["w"], s["b"], **how)
    g = na2d.norm_backward(s["x"], s["dh"], s["dy"], s["w"], s["b"], **how)
    named = dict(dx=g.dx, dw=g.dw, db=g.db, dgate=g.dgate, dpw=g.dpost_w, dpb=g.dpost_b, do=g.do)
    return {k: v for k, v in named.items() if v is not None}


# ------------------------------------------------------------------------------------------------------------ work
def _pairs(case):
    """How many (row, key) pairs are seen, and how many keys are seen by a row at all."""
    pairs = keys = 0
    for lq, lk in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + lq * lk, keys + lk
            continue
        first = lk - lq
        window = case["window"] or lk
        for p in range(max(0, first), lk):
            pairs += min(p + 1, window)
        keys += lk - max(0, max(0, first) - window + 1)
    return pairs, keys


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n, c = case["rows"] * case["c"], case["c"]
        small = c * (1 + 2 * case["post"] + case["bias"] + case["gates"])
        if case["op"] == "norm":
            return {"bytes": e * (4 * n + small), "flops": 16 * n}
        return {"bytes": e * (6 * n + small) + 4 * small, "flops": 32 * n}
    pairs, keys = _pairs(case)
    rows = sum(_lengths(case)[0]) * case["hq"]
    q, kv = rows * case["d"], 2 * keys * case["hk"] * case["d"]
    if case["op"] == "attend":
        return {"bytes": e * (2 * q + kv) + 4 * rows, "flops": 4 * pairs * case["hq"] * case["d"]}
    return {"bytes": e * (4 * q + 2 * kv) + 4 * rows, "flops": 10 * pairs * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------------------------- the definition, 64 bits
def _visible(lq, lk, causal, window, dev):
    i = torch.arange(lk - lq, lk, device=dev)[:, None]
    j = torch.arange(lk, device=dev)[None, :]
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool, device=dev)
    return (j <= i) & (j > i - window) if window else j <= i


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    group = hq // hk
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    out, lse = torch.zeros_like(q), torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lengths = _lengths(case)
    slots = [case["cap"]] * len(lengths[1]) if case["cap"] else lengths[1]
    q0 = k0 = 0
    for lq, lk, slot in zip(*lengths, slots):
        hidden = ~_visible(lq, lk, case["causal"], case["window"], q.device)
        for h in range(hq):
            a, b, c = q[q0:q0 + lq, h], k[k0:k0 + lk, h // group], v[k0:k0 + lk, h // group]
            z = torch.einsum("id,jd->ij", a, b) / math.sqrt(d)
            z[hidden] = -math.inf
            l = torch.logsumexp(z, 1)
            z.sub_(l.nan_to_num(neginf=0.0)[:, None]).exp_()
            if case["op"] == "attend":
                lse[h, q0:q0 + lq] = l
                out[q0:q0 + lq, h] = torch.einsum("ij,jd->id", z, c)
                continue
            do = s["dout"][q0:q0 + lq, h].double()
            dv[k0:k0 + lk, h // group] += torch.einsum("ij,id->jd", z, do)
            dp = torch.einsum("id,jd->ij", do, c)
            dp.sub_(torch.einsum("ij,ij->i", dp, z)[:, None]).mul_(z).div_(math.sqrt(d))
            dq[q0:q0 + lq, h] = torch.einsum("ij,jd->id", dp, b)
            dk[k0:k0 + lk, h // group] += torch.einsum("ij,id->jd", dp, a)
        q0, k0 = q0 + lq, k0 + slot
    return (out, lse) if case["op"] == "attend" else (dq, dk, dv)


def _exact_norm(case, s):
    rows, c = case["rows"], case["c"]

    def norm(x):
        mean = 0.0 if case["rms"] else torch.sum(x, 1, keepdim=True) / c
        return (x - mean) / torch.sqrt(torch.sum((x - mean) ** 2, 1, keepdim=True) / c + EPS)

    names = ("o", "w", "b", "pw", "pb", "gate")
    leaf = {k: s[k].double().requires_grad_() for k in names if s[k] is not None}

    def branch():
        p = leaf["o"]
        if case["post"]:
            p = norm(p) * leaf["pw"] + leaf.get("pb", 0.0)
        if "gate" in leaf:
            p = (p.view(case["gates"], -1, c) * leaf["gate"][:, None]).reshape(rows, c)
        return SCALE * p

    if case["op"] == "norm":
        with torch.no_grad():
            y = s["x"].double() + branch()
            return y, norm(y) * leaf["w"] + leaf.get("b", 0.0)
    y = s["x"].double().requires_grad_()
    h = norm(y) * leaf["w"] + leaf.get("b", 0.0)
    dy = s["dy"].double()
    to = [y, leaf["w"]] + ([leaf["b"]] if "b" in leaf else [])
    first = torch.autograd.grad(h, to, s["dh"].double())
    dx = dy + first[0]
    got = dict(dx=dx, dw=first[1])
    if "b" in leaf:
        got["db"] = first[2]
    rest = [k for k in ("gate", "pw", "pb", "o") if k in leaf]
    got.update(("d" + k, v) for k, v in zip(rest, torch.autograd.grad(branch(), [leaf[k] for k in rest], dx)))
    return got
