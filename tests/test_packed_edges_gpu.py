"""The packed attention where it can go wrong: values that are not finite, rows
that see nothing, small float16 gradients, long sequences in the kernel for few
rows, and lengths that lie.  Bounds are derived as in plain64."""
import math

import pytest
import torch

from vision_sliding_window_b200 import build, na2d

from . import plain64
from .test_packed_gpu import TYPES, batch, check_forward, starts

pytestmark = pytest.mark.gpu

F = plain64.F


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    build.build()
    return na2d.load_library()


def synchronized():
    torch.cuda.synchronize()
    assert na2d.device_status() == na2d.NA_OK


# ------------------------------------------------- rows that see nothing, NaN
BLIND = [
    # lq, lk, hq, hk, d: causal, so that the first lq - lk rows see no key
    ([40, 200], [24, 100], 4, 2, 64),
    ([300], [200], 8, 1, 128),
    ([90, 5], [3, 1], 2, 2, 16),
    ([5], [2], 2, 2, 64),                                        # few rows
    ([9, 1, 1], [2, 300, 40], 4, 4, 32),
    ([5, 1], [2, 9000], 1, 1, 128),                              # few rows, keys cut into pieces
]


@pytest.mark.parametrize("lq,lk,hq,hk,d", BLIND)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_rows_without_keys_beside_values_that_are_not_finite(lq, lk, hq, hk, d, dtype, what):
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=d)
    v[0] = what
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True)
    synchronized()
    blind = lq[0] - lk[0]
    assert (out[:blind] == 0).all() and (lse[:, :blind] == -math.inf).all()
    assert not torch.isfinite(out[blind:lq[0]].float()).any()
    want, wlse, tol, ltol = plain64.forward(q, k, v, cu_q, cu_k, causal=True)
    plain64.check("out", out[lq[0]:], want[lq[0]:], tol[lq[0]:])
    plain64.check("lse", lse, wlse, ltol)


NOTHING = [
    # lq, lk, hq, hk, d, causal
    ([200, 30], [300, 150], 4, 2, 64, False),
    ([300], [300], 2, 2, 128, True),
    ([150], [2600], 2, 1, 32, False),          # keys cut into pieces
    ([1, 3], [300, 150], 4, 2, 64, False),     # few rows
    ([2], [9000], 2, 1, 128, False),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,causal", NOTHING)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", [1.0, math.inf])
def test_rows_whose_logits_are_all_minus_infinity(lq, lk, hq, hk, d, causal, dtype, value):
    """They have no weights, as if they saw no key."""
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=d)
    q[..., 0] = 1.0
    k[:lk[0], :, 0] = -math.inf
    v[:lk[0]] *= value
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=causal)
    synchronized()
    assert (out[:lq[0]] == 0).all() and (lse[:, :lq[0]] == -math.inf).all()
    want, wlse, tol, ltol = plain64.forward(q[lq[0]:], k[lk[0]:], v[lk[0]:], cu_q[1:] - lq[0], cu_k[1:] - lk[0],
                                            causal=causal)
    plain64.check("out", out[lq[0]:], want, tol)
    plain64.check("lse", lse[:, lq[0]:], wlse, ltol)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lq", [1, 150])
@pytest.mark.parametrize("lk,cut", [(600, 300), (9000, 4500)])
def test_logits_of_minus_infinity_before_others(dtype, lq, lk, cut):
    q, k, v, cu_q, cu_k, _ = batch([lq], [lk], 4, 2, 64, dtype, seed=7)
    q[..., 0] = 1.0
    k[:cut, :, 0] = -math.inf
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k)
    synchronized()
    want, wlse, tol, ltol = plain64.forward(q, k[cut:], v[cut:], cu_q, starts([lk - cut]))
    plain64.check("out", out, want, tol)
    plain64.check("lse", lse, wlse, ltol)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lq", [1, 150])
@pytest.mark.parametrize("lk", [600, 9000])
def test_a_value_that_is_seen_counts_however_small_its_weight(dtype, lq, lk):
    """0 * NaN: the first keys' weights vanish beside the later ones', wherever a
    tile, a warp's share or a piece ends."""
    q, k, v, cu_q, cu_k, _ = batch([lq], [lk], 2, 1, 64, dtype, seed=8)
    q[..., 0], k[..., 0] = 16.0, 0.0
    for cut in (1, 64, 200, 500):
        k[:cut, :, 0] = -300.0
        v[:cut] = 0.0
        v[0, :, 3] = math.nan
        out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k)
        synchronized()
        assert torch.isnan(out[..., 3]).all() and torch.isfinite(out[..., :3].float()).all()
        assert torch.isfinite(lse).all()


# ------------------------------------------------------------------ gradients
def bounds_of_gradients(q, k, v, out, lse, dout, cu_q, cu_k, causal, window, scale):
    """The gradients in 64 bits and their bounds, as plain64.backward, but with the
    sum over a row that a kernel takes: dout . out, of the out that was given, or,
    in the tensor-core kernel for a row tile whose keys lie in one tile, sum P dP.
    float16 weights' gradients are lifted so that dout's row (for dk the largest of
    the sequence and group) has a norm of 16 to 32: half a subnormal step of theirs
    is 2^-25 of a sixteenth of that norm at most; weights are lifted by 2^15."""
    d, hq, group = q.shape[2], q.shape[1], q.shape[1] // k.shape[1]
    half = q.dtype == torch.float16
    u = plain64.half_step(q.dtype)
    tensor_cores = q.dtype != torch.float32 and group <= 128
    zeros = [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v)]
    bound = [torch.zeros_like(t) for t in zeros]
    for q0, lq, k0, lk in plain64.spans(cu_q, cu_k, None):
        if lq == 0 or lk == 0:
            continue
        keep = plain64.visible(lq, lk, causal, window, q.device)
        per = 128 // max(group, 1) if tensor_cores else 1
        of_weights = torch.zeros(lq, 1, dtype=torch.bool, device=q.device)
        if tensor_cores:
            for a in range(0, lq, per):
                seen = keep[a:a + per].any(0).nonzero()
                if len(seen) and int(seen[-1]) - int(seen[0]) < 128:
                    of_weights[a:a + per] = True
        for h in range(hq):
            g = h // group
            a, go = q[q0:q0 + lq, h].double(), dout[q0:q0 + lq, h].double()
            b, c = k[k0:k0 + lk, g].double(), v[k0:k0 + lk, g].double()
            s, _, e = plain64._terms(a, b, keep, scale)
            l = lse[h, q0:q0 + lq].double()
            p = (s - l.nan_to_num(neginf=0.0)[:, None]).exp()
            e = e + 4 * F * l.nan_to_num(neginf=0.0).abs()[:, None]
            dp = go @ c.t()
            dp_err = (d + 4) * F * (go.abs() @ c.abs().t())
            o = out[q0:q0 + lq, h].double()
            delta = torch.where(of_weights, (p * dp).sum(1, keepdim=True), (go * o).sum(1, keepdim=True))
            delta_err = torch.where(of_weights, (p * (dp_err + (e + lk * F) * dp.abs())).sum(1, keepdim=True),
                                    (d + 4) * F * (go * o).abs().sum(1, keepdim=True))
            norm = dout[q0:q0 + lq, g * group:(g + 1) * group].double().norm(dim=-1).amax()
            sub = 2.0 ** -25 / 16 if half else 0.0
            ds = p * (dp - delta)
            ds_err = p * (dp_err + delta_err) + (e + u) * ds.abs()
            dq_err, dk_err = ds_err + sub * keep * go.norm(dim=1, keepdim=True), ds_err + sub * keep * norm
            p_err = p * (e + u) + (2.0 ** -40 * keep if half else 0.0)
            for n, at, value, error in (
                    (0, (slice(q0, q0 + lq), h), scale * (ds @ b), scale * (dq_err @ b.abs() + lk * F * (ds.abs() @ b.abs()))),
                    (1, (slice(k0, k0 + lk), g), scale * (ds.t() @ a),
                     scale * (dk_err.t() @ a.abs() + lq * group * F * (ds.abs().t() @ a.abs()))),
                    (2, (slice(k0, k0 + lk), g), p.t() @ go,
                     p_err.t() @ go.abs() + lq * group * F * (p.t() @ go.abs()))):
                zeros[n][at] += value
                bound[n][at] += error
    small = 1e-30 + (2.0 ** -25 if half else 0.0)  # the results' own subnormals
    bound = [t + u * z.abs() + small for t, z in zip(bound, zeros)]
    if half:  # what rounds to an infinity has to be one
        zeros = [torch.where(z.abs() >= 65520, z.sign() * math.inf, z) for z in zeros]
    return zeros, bound


def check_gradients(q, k, v, dout, cu_q, cu_k, causal=False, window=0, scale=None):
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=causal, window=window, scale=scale)
    got = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=causal, window=window, scale=scale)
    synchronized()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, tol = bounds_of_gradients(q, k, v, out, lse, dout, cu_q, cu_k, causal, window, scale)
    for name, *x in zip(("dq", "dk", "dv"), got, want, tol):
        plain64.check(name, *x)
    return got


GRADIENTS = [
    # lq, lk, hq, hk, d, dtype, causal, window
    ([5, 1, 130, 64], [5, 1, 130, 64], 4, 2, 64, "bf16", True, 0),
    ([257, 128, 3], [257, 128, 3], 8, 2, 128, "bf16", True, 0),
    ([300, 17, 511], [300, 17, 511], 6, 2, 64, "f16", False, 0),
    ([700, 90], [700, 90], 7, 1, 128, "bf16", True, 200),
    ([100, 33], [612, 333], 4, 4, 128, "f16", True, 0),
    ([40, 200], [24, 100], 4, 2, 64, "bf16", True, 0),
    ([129, 255], [129, 255], 3, 3, 16, "f16", True, 0),
    ([200, 65], [200, 65], 4, 2, 64, "f32", True, 0),
    ([31, 200], [31, 200], 130, 1, 16, "bf16", True, 0),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", GRADIENTS)
def test_gradients_with_the_sum_that_the_kernel_takes(lq, lk, hq, hk, d, dtype, causal, window):
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=d + hq)
    check_gradients(q, k, v, batch(lq, lk, hq, hk, d, dtype, seed=99)[0], cu_q, cu_k, causal, window)


@pytest.mark.parametrize("size", [1e-3, 1e-4, 2e-6, 3e3])
@pytest.mark.parametrize("qstd", [0.125, 8.0])
@pytest.mark.parametrize("causal", [False, True])
def test_small_and_large_float16_gradients(size, qstd, causal):
    """Weights of 1/2300 and gradients far below 1: their product is far below
    float16's normal numbers.  k's (q's) size brings dq (dk) back among them."""
    lens = [2300, 70]
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 2, 1, 64, "f16", seed=21)
    dout = batch(lens, lens, 2, 1, 64, "f32", seed=22)[0]
    if size < 1:
        dout[2300:] *= 1e-2  # a sequence of its own size
    dout[::3] *= 1e-3 if size > 1 else 1.0  # rows of theirs
    check_gradients((q * qstd), (k / qstd), v, (dout * size).half(), cu_q, cu_k, causal)


def test_float16_gradients_of_rows_of_zeros_and_of_all_sizes():
    lens = [300, 129]
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 4, 2, 64, "f16", seed=23)
    dout = batch(lens, lens, 4, 2, 64, "f32", seed=24)[0]
    dout *= (10.0 ** torch.linspace(-7, 1, len(q), device="cuda"))[:, None, None]
    dout[5::7] = 0.0
    check_gradients(q, k, v, dout.half(), cu_q, cu_k)
    grads = check_gradients(q, k, v, torch.zeros_like(q), cu_q, cu_k, causal=True)
    assert all((g == 0).all() for g in grads)


def test_float16_values_so_large_that_a_lifted_gradient_overflows():
    """Norms of 8000 along dout: |dS| reaches 2^17 before it is taken again in float32."""
    lens = [2, 3, 200]
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 2, 2, 64, "f16", seed=25)
    v = (v.float() * 1000).half()
    check_gradients(q, k, v, (v.float() * 1e-5).half(), cu_q, cu_k)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [40, 200])
def test_what_a_row_does_not_see_does_not_reach_its_gradients(dtype, bad):
    """A key, a value, a row and its gradient that are not finite, within the
    sequence; with a window of 16 they reach 16 rows and the keys of those."""
    lens, window = [300, 50], 16
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 4, 2, 64, dtype, seed=31)
    dout = torch.randn_like(q)
    kw = dict(causal=True, window=window)
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, **kw)
    want, tol = bounds_of_gradients(q, k, v, out, lse, dout, cu_q, cu_k, True, window, 0.125)
    k[bad], v[bad] = math.nan, math.inf
    q[bad + 60], dout[bad + 60] = math.nan, math.inf
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, **kw)
    got = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, **kw)
    synchronized()
    rows = torch.ones(len(q), dtype=torch.bool, device="cuda")
    rows[bad:bad + window] = False
    rows[bad + 60] = False
    keys = torch.ones(len(k), dtype=torch.bool, device="cuda")
    for r in (~rows).nonzero().flatten().tolist():
        keys[r - window + 1:r + 1] = False
    for name, g, w, t, clean in zip(("dq", "dk", "dv"), got, want, tol, (rows, keys, keys)):
        plain64.check(name, g[clean], w[clean], t[clean])
        assert not torch.isfinite(g[~clean].float()).all(-1).any() or name == "dv"
    again = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, **kw)
    for a, b, clean in zip(got, again, (rows, keys, keys)):
        assert torch.equal(a[clean], b[clean])


def test_many_float16_keys_of_small_weight():
    """139999 keys of weight e^-17.75 beside one of weight 1: together 0.3%, each
    below half of float16's smallest step."""
    n, d = 140000, 64
    for lq in (1, 40):
        q = torch.zeros(lq, 1, d, dtype=torch.float16, device="cuda")
        k, v = (torch.zeros(n, 1, d, dtype=torch.float16, device="cuda") for _ in range(2))
        q[..., 0] = 1.0
        k[1:, :, 0] = -17.75
        v[1:] = 1.0
        out, lse = na2d.packed_forward(q, k, v, starts([lq]), starts([n]), scale=1.0)
        synchronized()
        total = 1.0 + (n - 1) * math.exp(-17.75)
        want = (total - 1.0) / total
        # half a step of a weight lifted by 2^7, or of one beside a warp's own largest, is 2^-32; roundings of weights
        # and of out
        bound = n * 2.0 ** -32 + 2 * 2.0 ** -11 * want
        assert (out.double() - want).abs().max().item() <= bound
        assert (lse.double() - math.log(total)).abs().max().item() <= 1e-5


# ------------------------------------- long sequences in the kernel for few rows
LONG_AMONG_FEW = [
    # lq, lk, hq, hk, d, dtype, causal, window: 16 rows (of a group) a sequence on average
    ([17, 90, 400] + [1] * 60, [17, 1200, 400] + [33 * i + 1 for i in range(60)], 2, 2, 64, "bf16", True, 0),
    ([17, 90, 400] + [1] * 60, [300, 90, 700] + [33 * i + 1 for i in range(60)], 4, 4, 128, "f16", True, 100),
    ([1] * 40 + [37, 150], [65] * 40 + [2000, 150], 6, 3, 32, "bf16", False, 0),
    ([130, 0, 5] + [1] * 30, [64, 9, 0] + [700] * 30, 4, 2, 16, "f16", True, 0),       # rows without keys, no rows
    ([40, 1, 1, 1, 20], [9000, 5000, 6000, 12, 4097], 1, 1, 128, "bf16", True, 0),     # keys cut into pieces
    ([33, 1, 1], [9000, 5001, 40], 2, 2, 64, "f16", False, 0),
    ([40, 1, 1, 1, 20], [9000, 5000, 6000, 12, 4097], 1, 1, 128, "bf16", True, 4500),
    ([60] + [1] * 9, [2000] + [1500] * 9, 2, 1, 64, "f32", True, 0),                   # float32, in pieces
    ([50] + [1] * 9, [900] + [2500] * 9, 4, 2, 16, "f32", False, 0),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", LONG_AMONG_FEW)
@pytest.mark.parametrize("extra", [0, 3])
def test_long_sequences_among_single_tokens(lq, lk, hq, hk, d, dtype, causal, window, extra):
    assert (sum(lq) + extra) * (hq // hk) <= 16 * len(lq)
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=len(lq), extra=extra)
    out, lse = torch.full_like(q, 7.0), torch.full((hq, len(q)), 7.0, device="cuda")
    na2d.packed_forward(q, k, v, cu_q, cu_k, causal=causal, window=window, out=out, lse=lse)
    synchronized()
    want, wlse, tol, ltol = plain64.forward(q, k, v, cu_q, cu_k, causal=causal, window=window)
    plain64.check("out", out, want, tol)
    plain64.check("lse", lse, wlse, ltol)
    n = sum(lq)
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()


# --------------------------------------------------------------- lying lengths
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lq,lk", [([64, 100], [64, 100]), ([1, 1], [1, 1]), ([3, 1], [9000, 40]), ([70, 9], [2600, 30])])
def test_lengths_that_lie_write_nothing_outside(dtype, lq, lk):
    """Everything that a call writes lies between rows of a pattern that must stay."""
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, 4, 2, 64, dtype, seed=13)
    inside = []

    def guarded(shape, t):
        n = math.prod(shape)
        whole = torch.full((n + 2 * 4096,), 7.0, dtype=t, device="cuda")
        inside.append((whole, n))
        return whole[4096:4096 + n].view(shape)

    out, lse = guarded(q.shape, q.dtype), guarded((4, len(q)), torch.float32)
    grads = [guarded(t.shape, t.dtype) for t in (q, k, v)]
    sizes = (len(lq), len(q), len(k), 4, 2, 64, {"f32": 0, "f16": 1, "bf16": 2}[dtype])
    lib = na2d.load_library()
    ws = guarded((max(lib.na_packed_workspace_bytes(*sizes), 256) // 4,), torch.float32)
    back = guarded((max(lib.na_packed_backward_workspace_bytes(*sizes), 256) // 4,), torch.float32)
    far = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    for a, b in ((cu_q + 1000000, cu_k), (cu_q, cu_k + 1000000), (cu_q - 5000, cu_k - 5000), (cu_q, cu_k * 5),
                 (cu_q.flip(0).contiguous(), cu_k.flip(0).contiguous()), (cu_q * 7, cu_k * 5), (cu_q * 0, cu_k)):
        for causal in (False, True):
            na2d.packed_forward(q, k, v, a, b, far, causal=causal, out=out, lse=lse, workspace=ws)
            na2d.packed_backward(q, k, v, torch.zeros_like(q), torch.zeros_like(lse), q, a, b, causal=causal, grads=grads,
                                 workspace=back)
            synchronized()
            for whole, n in inside:
                assert (whole[:4096] == 7).all() and (whole[4096 + n:] == 7).all()


# ------------------------------------------------- numbers longer than 32 bits
def test_windows_of_more_than_32_bits():
    for dtype in ("bf16", "f32"):
        q, k, v, cu_q, cu_k, _ = batch([200, 9], [200, 9], 2, 2, 64, dtype, seed=41)
        want, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True)
        grads = na2d.packed_backward(q, k, v, want, lse, q, cu_q, cu_k, causal=True)
        for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 10 ** 30):
            assert torch.equal(na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True, window=window)[0], want)
            got = na2d.packed_backward(q, k, v, want, lse, q, cu_q, cu_k, causal=True, window=window)
            assert all(torch.equal(a, b) for a, b in zip(got, grads))
        for window in (-1, -2 ** 31 - 1, -2 ** 32):
            with pytest.raises(na2d.NA2DError):
                na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True, window=window)
    synchronized()


def test_sizes_of_more_than_32_bits_are_refused():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    q = torch.empty(1, 1, 2 ** 32 + 16, dtype=torch.bfloat16, device="cuda")
    cu = starts([1])
    for call in (lambda: na2d.packed_forward(q, q, q, cu, cu),
                 lambda: na2d.packed_backward(q, q, q, q, torch.zeros(1, 1, device="cuda"), q, cu, cu, grads=(q, q, q)),
                 lambda: na2d.norm_forward(q, h=q), lambda: na2d.norm_backward(q, q)):
        with pytest.raises(na2d.NA2DError) as e:
            call()
        assert e.value.status == na2d.NA_ERR_UNSUPPORTED
    synchronized()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_calls_without_rows_keys_or_sequences(dtype):
    for lq, lk, hq, hk in (([], [], 2, 1), ([0, 0], [5, 300], 4, 2), ([3, 70], [0, 0], 2, 2), ([0], [0], 1, 1)):
        q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, 64, dtype)
        out, lse = check_forward(q, k, v, cu_q, cu_k, causal=True)
        assert (out == 0).all() and (lse == -math.inf).all()
        grads = na2d.packed_backward(q, k, v, out, lse, q, cu_q, cu_k, causal=True)
        synchronized()
        assert all((g == 0).all() for g in grads)
