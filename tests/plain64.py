"""Packed attention and the norms around a block in 64 bits, from their
formulas, sequence by sequence, with the elementwise error that float32
arithmetic and roundings to the inputs' type allow.  Runs where its inputs lie.

Error model.  u is half a step of the type (2^-8, 2^-11, 2^-24), f = 2^-24.
A float32 dot product of length d is off by at most (d + 2) f sum |q||k|; that
times the scale, E, is the absolute error of a logit and so the relative one of
its weight, to which 2^-18 is added for exp, division and the running rescale.
Weights and their gradients are rounded to the type once (u), the result once
more (u); a sum of n terms in float32 adds n f of the terms' absolute sum.
float16 loses another half step of its subnormals, 2^-25, on each weight (whose
largest is at least 1 before division by the sum) and each gradient of one.
"""
import math

import torch

F = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def visible(lq, lk, causal, window, device="cpu"):
    i = torch.arange(lq, device=device)[:, None] + (lk - lq)
    j = torch.arange(lk, device=device)[None, :]
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool, device=device)
    m = j <= i
    return m & (j > i - window) if window else m


def spans(cu_q, cu_k, len_k):
    cu_q, cu_k = cu_q.tolist(), cu_k.tolist()
    for s in range(len(cu_q) - 1):
        lk = cu_k[s + 1] - cu_k[s]
        if len_k is not None:
            lk = min(lk, max(int(len_k[s]), 0))
        yield cu_q[s], cu_q[s + 1] - cu_q[s], cu_k[s], lk


def _terms(q, k, keep, scale):
    """Weights and lse of one head of one sequence, and the logits' error bound E."""
    s = (q @ k.t()) * scale
    err = ((q.abs() @ k.abs().t()) * scale).masked_fill(~keep, 0.0)
    e = (q.shape[1] + 8) * F * (err.amax(1, keepdim=True) if k.shape[0] else torch.zeros(len(q), 1, device=q.device))
    s = s.masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(s, 1) if k.shape[0] else torch.full((len(q),), -math.inf, dtype=q.dtype, device=q.device)
    return s, lse, 2 * e + 2.0 ** -18


def forward(q, k, v, cu_q, cu_k, len_k=None, causal=False, window=0, scale=None):
    """out, lse and the bounds on their errors; rows of no sequence are NaN with
    a bound of NaN."""
    d, hq, group = q.shape[2], q.shape[1], q.shape[1] // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    u, sub = half_step(q.dtype), (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((hq, q.shape[0]), math.nan, dtype=torch.float64, device=q.device)
    tol, ltol = out.clone(), lse.clone()
    for q0, lq, k0, lk in spans(cu_q, cu_k, len_k):
        keep = visible(lq, lk, causal, window, q.device)
        for h in range(hq):
            a = q[q0:q0 + lq, h].double()
            b, c = k[k0:k0 + lk, h // group].double(), v[k0:k0 + lk, h // group].double()
            c = c.masked_fill(~keep.any(0)[:, None], 0.0)
            s, l, e = _terms(a, b.masked_fill(~keep.any(0)[:, None], 0.0), keep, scale)
            p = (s - l.nan_to_num(neginf=0.0)[:, None]).exp()
            o, mag = p @ c, p @ c.abs()
            out[q0:q0 + lq, h], lse[h, q0:q0 + lq] = o, l
            tol[q0:q0 + lq, h] = (u + 2 * e + lk * F) * mag + u * o.abs() + sub * (keep.double() @ c.abs()) + 1e-30
            ltol[h, q0:q0 + lq] = e[:, 0] + lk * F + 4 * F * l.nan_to_num(neginf=0.0).abs() + 2.0 ** -20
    return out, lse, tol, ltol


def backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=False, window=0, scale=None):
    """(dq, dk, dv) from the lse given, and the bounds on their errors.

    dS = P (dP - sum P dP).  The sum equals dout . out, from which it may be taken:
    out is then off by what forward() bounds, so the sum by that times |dout|."""
    d, hq, group = q.shape[2], q.shape[1], q.shape[1] // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    u, sub = half_step(q.dtype), (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
    nan = dict(dtype=torch.float64, device=q.device)
    dq, tq = (torch.full(q.shape, math.nan, **nan) for _ in range(2))
    dk, dv, tk, tv = (torch.full(k.shape, math.nan, **nan) for _ in range(4))
    for q0, lq, k0, lk in spans(cu_q, cu_k, None):
        keep = visible(lq, lk, causal, window, q.device)
        for x in (dk, dv, tk, tv):
            x[k0:k0 + lk] = 0.0
        for h in range(hq):
            g = h // group
            a, go = q[q0:q0 + lq, h].double(), dout[q0:q0 + lq, h].double()
            b, c = k[k0:k0 + lk, g].double(), v[k0:k0 + lk, g].double()
            s, _, e = _terms(a, b, keep, scale)
            l = lse[h, q0:q0 + lq].double()
            p = (s - l.nan_to_num(neginf=0.0)[:, None]).exp()
            e = e + 4 * F * l.nan_to_num(neginf=0.0).abs()[:, None]
            dp = go @ c.t()
            delta = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - delta)
            mag = p @ c.abs()
            out_err = (u + 2 * e + lk * F) * mag + u * out[q0:q0 + lq, h].double().abs() + sub * (keep.double() @ c.abs())
            delta_err = (go.abs() * out_err).sum(1, keepdim=True)
            # errors of dp and delta (float32 sums) and of the weight
            ds_err = p * ((d + 4 + lk) * F * (go.abs() @ c.abs().t() + (go.abs() * mag).sum(1, keepdim=True)) + delta_err)
            ds_err = ds_err + ds.abs() * (e + u) + sub * keep
            p_err = p * (e + u) + sub * keep
            dq[q0:q0 + lq, h] = scale * (ds @ b)
            tq[q0:q0 + lq, h] = scale * (ds_err @ b.abs() + lk * F * (ds.abs() @ b.abs()))
            dk[k0:k0 + lk, g] += scale * (ds.t() @ a)
            tk[k0:k0 + lk, g] += scale * (ds_err.t() @ a.abs() + lq * group * F * (ds.abs().t() @ a.abs()))
            dv[k0:k0 + lk, g] += p.t() @ go
            tv[k0:k0 + lk, g] += p_err.t() @ go.abs() + lq * group * F * (p.t() @ go.abs())
    small = 1e-30 + sub  # a float16 result may be subnormal too
    return (dq, dk, dv), (tq + u * dq.abs() + small, tk + u * dk.abs() + small, tv + u * dv.abs() + small)


# ------------------------------------------------------------------------ norms
def _normed(x, rms, eps):
    """n, rstd and the bound on n's error in units of float32 steps."""
    mean = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    c = x - mean
    r = (c.square().mean(1, keepdim=True) + eps).rsqrt()
    # statistics: pairwise sums of up to 64 terms a lane, then log2 of the lanes
    n_err = 96 * F * ((x.abs() + mean.abs() + x.abs().mean(1, keepdim=True)) * r + (c * r).abs())
    return c * r, r, n_err


def _d(t):
    return None if t is None else t.double()


def _gate_rows(gate, rows):
    return 1.0 if gate is None else gate.double().view(-1, gate.shape[-1]).repeat_interleave(
        rows // (gate.numel() // gate.shape[-1]), 0)


def norm_forward(x, w=None, b=None, o=None, post=False, post_w=None, post_b=None, gate=None, scale=1.0, eps=1e-5,
                 rms=False):
    """(y, h) of [rows, C] tensors and the bounds on their errors."""
    u, rows = half_step(x.dtype), x.shape[0]
    y, yerr = x.double(), torch.zeros_like(x, dtype=torch.float64)
    sub = 2.0 ** -25 if x.dtype == torch.float16 else 1e-38
    if o is not None:
        t, terr = o.double(), yerr
        if post:
            n, _, nerr = _normed(t, rms, eps)
            pw = 1.0 if post_w is None else post_w.double()
            t, terr = n * pw, nerr * abs(pw)
            if post_b is not None:
                t = t + post_b.double()
            terr = terr + 4 * F * (t.abs() + (n * pw).abs())
        f = scale * _gate_rows(gate, rows)
        branch = f * t
        yerr = (terr * abs(f) if isinstance(f, float) else terr * f.abs()) + 4 * F * (branch.abs() + y.abs())
        y = y + branch
    n, r, nerr = _normed(y, rms, eps)
    nerr = nerr + 2 * r * (yerr + yerr.mean(1, keepdim=True)) + n.abs() * r * 2 * (n.abs() * yerr).mean(1, keepdim=True)
    h = n * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    herr = nerr * (1.0 if w is None else w.double().abs()) + 4 * F * (h.abs() + n.abs())
    return (y, h), (yerr + u * y.abs() + sub, herr + u * h.abs() + sub)


def norm_backward(y, dh, dy=None, w=None, b=None, o=None, post=False, post_w=None, post_b=None, gate=None, scale=1.0,
                  eps=1e-5, rms=False):
    """Gradients by name and the bounds on their errors."""
    u, (rows, C) = half_step(y.dtype), y.shape
    sub = 2.0 ** -25 if y.dtype == torch.float16 else 1e-38
    chain = (rows / 8 + 64) * F  # additions in a row's way to a sum over rows, at most
    g, t = {}, {}

    def back(dn, dn_err, n, r, nerr):
        m0 = 0.0 if rms else dn.mean(1, keepdim=True)
        m1 = (dn * n).mean(1, keepdim=True)
        out = r * (dn - m0 - n * m1)
        size = dn.abs() + (0.0 if rms else dn.abs().mean(1, keepdim=True)) + n.abs() * (dn * n).abs().mean(1, keepdim=True)
        err = r * (dn_err + dn_err.mean(1, keepdim=True) + n.abs() * (dn_err * n.abs()).mean(1, keepdim=True)
                   + nerr * m1.abs() + n.abs() * (dn.abs() * nerr).mean(1, keepdim=True)
                   + 96 * F * size)
        # a relative error of rstd
        return out, err + out.abs() * (2 * (n.abs() * nerr).mean(1, keepdim=True) + 8 * F)

    dx = torch.zeros(rows, C, dtype=torch.float64, device=y.device) if dy is None else dy.double()
    dxerr = torch.zeros_like(dx)
    if dh is not None:
        n, r, nerr = _normed(y.double(), rms, eps)
        dn = dh.double() * (1.0 if w is None else w.double())
        add, err = back(dn, 2 * F * dn.abs(), n, r, nerr)
        dx, dxerr = dx + add, err + 4 * F * (dx.abs() + add.abs())
        if w is not None:
            g["dw"] = (dh.double() * n).sum(0)
            t["dw"] = (dh.double().abs() * nerr).sum(0) + chain * (dh.double() * n).abs().sum(0) + 1e-30
        if b is not None:
            g["db"], t["db"] = dh.double().sum(0), chain * dh.double().abs().sum(0) + 1e-30
    g["dx"], t["dx"] = dx, dxerr + u * dx.abs() + sub
    if o is not None:
        f = _gate_rows(gate, rows)
        absf = abs(f) if isinstance(f, float) else f.abs()
        v, verr = o.double(), torch.zeros_like(dx)
        if post:
            m, q, merr = _normed(v, rms, eps)
            pw = torch.ones(C, dtype=torch.float64, device=y.device) if post_w is None else post_w.double()
            v = m * pw + (0.0 if post_b is None else post_b.double())
            verr = merr * pw.abs() + 4 * F * (v.abs() + (m * pw).abs())
        d = scale * dx
        derr = abs(scale) * dxerr + 4 * F * d.abs()
        if gate is not None:
            shape = (gate.numel() // C, -1, C)
            g["dgate"] = (d * v).view(shape).sum(1).view(gate.shape)
            t["dgate"] = ((derr * v.abs() + d.abs() * verr).view(shape).sum(1)
                          + chain * (d * v).abs().view(shape).sum(1)).view(gate.shape) + 1e-30
        dp, dperr = d * f, (derr + 4 * F * d.abs()) * absf
        if post:
            if post_w is not None:
                g["dpost_w"] = (dp * m).sum(0)
                t["dpost_w"] = (dperr * m.abs() + dp.abs() * merr).sum(0) + chain * (dp * m).abs().sum(0) + 1e-30
            if post_b is not None:
                g["dpost_b"], t["dpost_b"] = dp.sum(0), dperr.sum(0) + chain * dp.abs().sum(0) + 1e-30
            dp, dperr = back(dp * pw, dperr * pw.abs() + 4 * F * (dp * pw).abs(), m, q, merr)
        g["do"], t["do"] = dp, dperr + u * dp.abs() + sub
    return g, t


def check(name, got, want, bound):
    """got lies within bound of want, elementwise; where want is NaN nothing is said."""
    got, want, bound = (x.detach().double().cpu() for x in (got, want, bound))
    said = ~torch.isnan(want)
    same = got == want  # infinities
    ok = same | ((got - want).abs() <= bound)
    bad = said & ~ok
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        worst = ((got - want).abs() / bound)[bad].max().item()
        raise AssertionError(f"{name}: {int(bad.sum())} of {int(said.sum())} out of bounds, first at {at}: "
                             f"{got[at].item()} for {want[at].item()} +- {bound[at].item()} (worst {worst:.2f}x)")
