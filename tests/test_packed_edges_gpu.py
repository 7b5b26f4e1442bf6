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
