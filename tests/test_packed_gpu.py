"""Attention over packed sequences (na_packed_forward, na_packed_backward)
against the formulas in 64 bits, with bounds that plain64 derives."""
import math

import pytest
import torch

from vision_sliding_window_b200 import build, na2d

from . import plain64

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    build.build()
    return na2d.load_library()


def starts(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def batch(lq, lk, hq, hk, d, dtype, seed=0, cap=0, extra=0, std=1.0):
    """q, k, v, cu_q, cu_k, len_k; `extra` rows and slots behind the last sequence."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    slots = [cap] * len(lk) if cap else lk
    t = TYPES[dtype]

    def normal(n, h):
        return (torch.randn(n, h, d, generator=g, device="cuda") * std).to(t)

    q, k, v = normal(sum(lq) + extra, hq), normal(sum(slots) + extra, hk), normal(sum(slots) + extra, hk)
    len_k = torch.tensor(lk, dtype=torch.int32, device="cuda") if cap else None
    return q, k, v, starts(lq), starts(slots), len_k


def check_forward(q, k, v, cu_q, cu_k, len_k=None, **kw):
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, len_k, **kw)
    torch.cuda.synchronize()
    assert na2d.device_status() == na2d.NA_OK
    want, wlse, tol, ltol = plain64.forward(q, k, v, cu_q, cu_k, len_k, **kw)
    plain64.check("out", out, want, tol)
    plain64.check("lse", lse, wlse, ltol)
    return out, lse


FORWARD = [
    # lq, lk, hq, hk, d, dtype, causal, window
    ([1], [1], 1, 1, 64, "bf16", True, 0),
    ([5, 1, 130, 64], [5, 1, 130, 64], 4, 2, 64, "bf16", True, 0),
    ([257, 128, 3], [257, 128, 3], 8, 2, 128, "bf16", True, 0),
    ([300, 17, 511], [300, 17, 511], 6, 2, 64, "f16", False, 0),
    ([49, 196, 400], [49, 196, 400], 2, 2, 32, "f16", False, 0),
    ([129, 255], [129, 255], 3, 3, 16, "bf16", True, 0),
    ([700, 90], [700, 90], 7, 1, 128, "bf16", True, 200),       # a group that does not divide a tile
    ([333, 1025], [333, 1025], 8, 1, 64, "f16", True, 1),       # a window of one key: out = v
    ([100, 33], [612, 1033], 4, 4, 128, "bf16", True, 0),       # the first part is in the cache
    ([100, 33], [612, 1033], 4, 1, 64, "f16", True, 77),
    ([40, 200], [24, 100], 4, 2, 64, "bf16", True, 0),          # rows before the first key see nothing
    ([40, 200], [24, 100], 2, 2, 32, "f32", True, 0),
    ([3, 0, 70, 0], [3, 9, 0, 0], 2, 1, 64, "bf16", False, 0),  # lengths of zero
    ([3, 0, 70, 0], [3, 9, 0, 0], 2, 1, 64, "f32", True, 0),
    ([200, 65], [200, 65], 4, 2, 64, "f32", True, 0),
    ([77, 150], [77, 150], 3, 1, 128, "f32", False, 0),
    ([90, 300], [90, 300], 2, 2, 16, "f32", True, 50),
    ([2100], [2100], 2, 1, 128, "bf16", True, 0),
    ([1500, 600], [1500, 600], 4, 4, 128, "f16", False, 0),
    ([31, 900], [31, 900], 130, 1, 16, "bf16", True, 0),        # more heads in a group than a tile has rows
    ([100, 20], [3000, 40], 2, 1, 64, "f32", True, 0),          # keys cut into pieces
    ([70], [2500], 4, 2, 128, "f32", False, 0),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", FORWARD)
def test_forward(lq, lk, hq, hk, d, dtype, causal, window):
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=d + hq)
    check_forward(q, k, v, cu_q, cu_k, causal=causal, window=window)


SINGLE = [
    # lengths in the cache, capacity, hq, hk, d, dtype, window
    ([37, 400, 129, 255], 512, 8, 2, 64, "bf16", 0),
    ([1, 0, 64, 65, 1000], 1024, 8, 1, 128, "bf16", 0),
    ([4097, 3000, 17], 5000, 4, 4, 128, "f16", 0),
    ([4097, 3000, 17], 5000, 7, 1, 64, "bf16", 900),
    ([9000], 9001, 16, 2, 32, "f16", 0),
    ([2000, 5], 2048, 6, 3, 16, "bf16", 0),
    ([1500, 3], 1600, 8, 2, 64, "f32", 0),
    ([20000], 20011, 8, 1, 128, "bf16", 0),
    ([1300, 700], 1333, 20, 1, 64, "bf16", 0),   # more heads in a group than 16
]


@pytest.mark.parametrize("lk,cap,hq,hk,d,dtype,window", SINGLE)
def test_single_tokens_over_a_cache(lk, cap, hq, hk, d, dtype, window):
    q, k, v, cu_q, cu_k, len_k = batch([1] * len(lk), lk, hq, hk, d, dtype, seed=cap, cap=cap)
    for s, n in enumerate(lk):  # what a cache holds past its keys is anything
        k[s * cap + n:(s + 1) * cap] = math.nan
        v[s * cap + n:(s + 1) * cap] = math.inf
    check_forward(q, k, v, cu_q, cu_k, len_k, causal=True, window=window)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 32)])
def test_a_few_rows_over_a_cache(dtype, d):
    lk, cap = [700, 2049, 90, 5], 2100
    q, k, v, cu_q, cu_k, len_k = batch([4, 3, 90, 0], lk, 4, 2, d, dtype, seed=3, cap=cap)
    for s, n in enumerate(lk):
        k[s * cap + n:(s + 1) * cap] = math.inf
        v[s * cap + n:(s + 1) * cap] = math.nan
    check_forward(q, k, v, cu_q, cu_k, len_k, causal=True)
    check_forward(q, k, v, cu_q, cu_k, len_k, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_what_a_row_does_not_see_does_not_reach_it(dtype):
    """NaN and infinities in keys and values after a row, before its window, and
    in other sequences."""
    lens = [300, 200, 333]
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 4, 2, 64, dtype, seed=5)
    clean = check_forward(q, k, v, cu_q, cu_k, causal=True, window=64)[0]
    want, _, tol, _ = plain64.forward(q, k, v, cu_q, cu_k, causal=True, window=64)
    k[300:500], v[300:500] = math.nan, math.inf    # the middle sequence
    v[500 + 150], k[500 + 150] = math.inf, math.nan
    out, _ = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True, window=64)
    seen = torch.zeros(len(q), dtype=torch.bool, device="cuda")
    seen[300:500] = True
    seen[650:650 + 64] = True
    assert torch.equal(out[:300], clean[:300])
    plain64.check("out", out[~seen], want[~seen], tol[~seen])
    assert not torch.isfinite(out[650:650 + 64].float()).any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_large_and_rising_logits(dtype):
    """Maxima that move by more than any fixed margin from tile to tile, and logits
    far below zero."""
    q, k, v, cu_q, cu_k, _ = batch([400, 150], [400, 150], 2, 1, 64, dtype, seed=6)
    ramp = torch.linspace(0, 6, 550, device="cuda").to(k.dtype)[:, None, None]
    check_forward(q, k * ramp, v, cu_q, cu_k)
    check_forward(q, k * ramp.flip(0), v, cu_q, cu_k)
    up = torch.full_like(q, 4.0)
    check_forward(up, (k.abs() * ramp), v, cu_q, cu_k, causal=True)
    check_forward(up, -(k.abs() * ramp), v, cu_q, cu_k)


def test_rows_behind_the_last_sequence_stay():
    for dtype, lq in (("bf16", [70, 130]), ("f32", [20, 9]), ("bf16", [1, 1])):
        q, k, v, cu_q, cu_k, _ = batch(lq, lq, 4, 2, 64, dtype, extra=37)
        out, lse = torch.full_like(q, 7.0), torch.full((4, len(q)), 7.0, device="cuda")
        na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True, out=out, lse=lse)
        n = sum(lq)
        assert (out[n:] == 7).all() and (lse[:, n:] == 7).all() and (out[:n] != 7).any()
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        na2d.packed_backward(q, k, v, out, lse, torch.ones_like(q), cu_q, cu_k, causal=True, grads=grads)
        for g in grads:
            assert (g[n:] == 7).all() and torch.isfinite(g[:n].float()).all()


BACKWARD = [
    # lq, lk, hq, hk, d, dtype, causal, window
    ([1], [1], 1, 1, 64, "bf16", True, 0),
    ([5, 1, 130, 64], [5, 1, 130, 64], 4, 2, 64, "bf16", True, 0),
    ([257, 128, 3], [257, 128, 3], 8, 2, 128, "bf16", True, 0),
    ([300, 17, 511], [300, 17, 511], 6, 2, 64, "f16", False, 0),
    ([49, 196, 400], [49, 196, 400], 2, 2, 32, "f16", False, 0),
    ([129, 255], [129, 255], 3, 3, 16, "bf16", True, 0),
    ([700, 90], [700, 90], 7, 1, 128, "bf16", True, 200),
    ([333, 400], [333, 400], 8, 1, 64, "f16", True, 1),
    ([100, 33], [612, 333], 4, 4, 128, "bf16", True, 0),
    ([40, 200], [24, 100], 4, 2, 64, "bf16", True, 0),
    ([40, 200], [24, 100], 2, 2, 32, "f32", True, 0),
    ([3, 0, 70, 0], [3, 9, 0, 0], 2, 1, 64, "bf16", False, 0),
    ([3, 0, 70, 0], [3, 9, 0, 0], 2, 1, 64, "f32", True, 0),
    ([200, 65], [200, 65], 4, 2, 64, "f32", True, 0),
    ([77, 150], [77, 150], 3, 1, 128, "f32", False, 0),
    ([90, 300], [90, 300], 2, 2, 16, "f32", True, 50),
    ([1100], [1100], 2, 1, 128, "f16", True, 0),
    ([31, 200], [31, 200], 130, 1, 16, "bf16", True, 0),
    ([600, 40], [600, 40], 4, 1, 64, "f32", True, 0),           # walks over rows cut into pieces
    ([400, 33], [700, 50], 4, 2, 128, "f32", True, 100),
    ([300], [200], 8, 1, 32, "f32", False, 0),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype,causal,window", BACKWARD)
def test_backward(lq, lk, hq, hk, d, dtype, causal, window):
    q, k, v, cu_q, cu_k, _ = batch(lq, lk, hq, hk, d, dtype, seed=d + hq)
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=causal, window=window)
    dout = batch(lq, lk, hq, hk, d, dtype, seed=99)[0]
    got = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=causal, window=window)
    torch.cuda.synchronize()
    assert na2d.device_status() == na2d.NA_OK
    want, tol = plain64.backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=causal, window=window)
    for name, *x in zip(("dq", "dk", "dv"), got, want, tol):
        plain64.check(name, *x)
    again = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=causal, window=window)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_backward_of_non_finite_neighbours():
    """A sequence's gradients do not depend on what other sequences hold."""
    for dtype in ("bf16", "f16", "f32"):
        lens = [200, 100, 77]
        q, k, v, cu_q, cu_k, _ = batch(lens, lens, 4, 2, 64, dtype, seed=8)
        dout = torch.randn_like(q)

        def run():
            out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True)
            return na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=True)

        clean = run()
        for t in (q, k, v, dout):
            t[200:300] = math.nan
        for a, b in zip(run(), clean):
            assert torch.equal(a[:200], b[:200]) and torch.equal(a[300:], b[300:])


def test_gradients_against_differences():
    lens = [9, 20]
    q, k, v, cu_q, cu_k, _ = batch(lens, lens, 4, 2, 16, "f32", seed=11)
    dout = torch.randn_like(q)
    out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True, window=7)
    grads = na2d.packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal=True, window=7)
    inputs = [t.double() for t in (q, k, v)]

    def loss(args):
        return (plain64.forward(*args, cu_q, cu_k, causal=True, window=7)[0] * dout.double()).sum().item()

    g = torch.Generator().manual_seed(1)
    for n, grad in enumerate(grads):
        way = torch.randn(grad.shape, generator=g).double().cuda()
        h = 1e-5
        up, down = list(inputs), list(inputs)
        up[n], down[n] = inputs[n] + h * way, inputs[n] - h * way
        slope = (loss(up) - loss(down)) / (2 * h)
        dot = (grad.double() * way).sum().item()
        # float32 gradients: each entry off by some 1e-6 of its size, differences by h^2
        assert abs(slope - dot) <= 1e-5 * (grad.double() * way).abs().sum().item() + 1e-6


@pytest.mark.parametrize("lq,cap", [([300, 129], 0), ([1, 1], 3000)])
def test_captured_and_replayed_with_other_lengths(lq, cap):
    lk = [2500, 1999] if cap else lq
    q, k, v, cu_q, cu_k, len_k = batch(lq, lk, 8, 2, 64, "bf16", seed=12, cap=cap)
    args = (q, k, v, cu_q, cu_k, len_k)
    out, lse = na2d.packed_forward(*args, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        na2d.packed_forward(*args, causal=True, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        na2d.packed_forward(*args, causal=True, out=out, lse=lse)
    for change in range(2):
        q.normal_()
        if cap:
            len_k.copy_(torch.tensor([17 + change, 2999], dtype=torch.int32))
        else:
            cu_q.copy_(torch.tensor([0, 100 + change, 429], dtype=torch.int32))
            cu_k.copy_(cu_q)
        graph.replay()
        torch.cuda.synchronize()
        want, wlse, tol, ltol = plain64.forward(*args, causal=True)
        plain64.check("out", out, want, tol)
        plain64.check("lse", lse, wlse, ltol)
    assert na2d.device_status() == na2d.NA_OK


def test_lengths_that_leave_the_tensors_are_clamped():
    """Starts and lengths past the tensors, and falling ones, read and write inside them."""
    for dtype in ("bf16", "f32"):
        for lq in ([64, 100], [1, 1]):
            q, k, v, cu_q, cu_k, _ = batch(lq, lq, 4, 2, 64, dtype, seed=13)
            far = torch.tensor([2 ** 31 - 1, 2 ** 30], dtype=torch.int32, device="cuda")
            for a, b in ((cu_q + 1000000, cu_k), (cu_q, cu_k + 1000000), (cu_q - 5000, cu_k - 5000),
                         (cu_q.flip(0).contiguous(), cu_k.flip(0).contiguous()), (cu_q * 7, cu_k * 5)):
                out, lse = na2d.packed_forward(q, k, v, a, b, far, causal=True)
                na2d.packed_backward(q, k, v, torch.zeros_like(q), torch.zeros_like(lse), q, a, b, causal=True)
                torch.cuda.synchronize()
                assert na2d.device_status() == na2d.NA_OK


def test_two_streams_at_once():
    jobs = []
    for n, lq in enumerate(([900, 300], [1, 1, 1])):
        lk = lq if n == 0 else [2000, 40, 999]
        jobs.append(batch(lq, lk, 8, 2, 64, "bf16", seed=n, cap=0 if n == 0 else 2000))
    alone = [na2d.packed_forward(*j, causal=True)[0] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(3):
        for j, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(na2d.packed_forward(*j, causal=True)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, alone[i % 2])


def test_a_cache_whose_offsets_pass_32_bits():
    """Keys behind element 2^31 of the cache, whole sequences and single tokens."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of free device memory")
    d, hk, slots = 128, 8, (1 << 31) // (128 * 8) + 5000
    k, v = (torch.zeros(slots, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    tail = 3000
    k[-tail:] = torch.randn(tail, hk, d, generator=g, device="cuda").bfloat16()
    v[-tail:] = torch.randn(tail, hk, d, generator=g, device="cuda").bfloat16()
    for lq in (1, 300):
        q = torch.randn(lq, 16, d, generator=g, device="cuda").bfloat16()
        cu_q = torch.tensor([0, 0, lq], dtype=torch.int32, device="cuda")
        cu_k = torch.tensor([0, slots - tail, slots], dtype=torch.int32, device="cuda")
        out, lse = na2d.packed_forward(q, k, v, cu_q, cu_k, causal=True)
        near = starts([tail])
        want, wlse, tol, ltol = plain64.forward(q, k[-tail:], v[-tail:], starts([lq]), near, causal=True)
        plain64.check("out", out, want, tol)
        plain64.check("lse", lse, wlse, ltol)
    assert na2d.device_status() == na2d.NA_OK
