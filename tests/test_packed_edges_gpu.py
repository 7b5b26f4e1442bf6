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
