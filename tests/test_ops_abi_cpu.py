"""The packed attention, the norms and the layer without a GPU: arguments that
the library refuses, workspaces, empty calls, and the binding's own checks."""
import math

import pytest
import torch

from vision_sliding_window_b200 import build, na2d

from . import plain64

FAKE = 0x10000  # a 256-byte aligned address nothing ever dereferences: every call below fails first
BAD, OK, UNSUPPORTED = na2d.NA_ERR_INVALID_ARG, na2d.NA_OK, na2d.NA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return na2d.load_library()


def packed(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu_q=FAKE, cu_k=FAKE, len_k=None, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40,
             nseq=2, total_q=100, total_k=100, hq=4, hk=2, d=64, causal=1, window=0, scale=0.125, dt=na2d.NA_BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.na_packed_forward(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu_q=None), dict(cu_k=None), dict(q=FAKE + 8),
    dict(k=FAKE + 2), dict(v=FAKE + 4), dict(out=FAKE + 8), dict(cu_q=FAKE + 2), dict(len_k=FAKE + 1),
    dict(lse=FAKE + 2), dict(nseq=-1), dict(total_q=-1), dict(total_k=-5), dict(hq=0), dict(hk=0), dict(hq=3),
    dict(d=48), dict(d=0), dict(d=256), dict(causal=2), dict(window=-1), dict(causal=0, window=4), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(dt=3),
    dict(nseq=1, total_q=1, total_k=100000, ws=None), dict(nseq=1, total_q=1, total_k=100000, ws_bytes=255),
    dict(nseq=1, total_q=1, total_k=100000, ws=FAKE + 16),
])
def test_packed_forward_refuses(lib, kw):
    assert packed(lib, **kw) == BAD


def test_packed_forward_without_work(lib):
    none = dict(q=None, k=None, v=None, out=None, lse=None, cu_q=None, cu_k=None, ws=None, ws_bytes=0)
    assert packed(lib, nseq=0, **none) == OK
    assert packed(lib, total_q=0, **none) == OK
    assert packed(lib, total_q=2 ** 30, total_k=2 ** 30, hq=64, d=128) == UNSUPPORTED
    assert packed(lib, total_k=2 ** 30 + 1) == UNSUPPORTED
    assert packed(lib, hq=1 << 17, hk=1 << 17, d=16) == UNSUPPORTED


def test_packed_workspaces(lib):
    size = lib.na_packed_workspace_bytes
    assert size(2, 100, 100, 4, 3, 64, na2d.NA_BF16) == 0  # refused
    assert size(0, 0, 0, 4, 2, 64, na2d.NA_BF16) == 0
    assert size(1, 50000, 50000, 16, 4, 64, na2d.NA_BF16) == 0  # rows enough to fill the GPU
    for args in ((16, 16, 16 * 16384, 32, 8, 128), (1, 1, 1 << 20, 8, 1, 64), (4, 4, 4 * 512, 8, 2, 64)):
        need = size(*args, na2d.NA_BF16)
        assert need % 256 == 0 and need < 600 << 20, (args, need)
    back = lib.na_packed_backward_workspace_bytes(2, 100, 100, 4, 2, 64, na2d.NA_F16)
    assert back % 256 == 0 and back >= 100 * 4 * 8


def packed_back(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, dout=FAKE, cu_q=FAKE, cu_k=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             ws=FAKE, ws_bytes=1 << 40, nseq=2, total_q=100, total_k=100, hq=4, hk=2, d=64, causal=1, window=0,
             scale=0.125, dt=na2d.NA_BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.na_packed_backward(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(lse=None), dict(dout=None), dict(dq=None),
    dict(dk=None), dict(dv=None), dict(cu_q=None), dict(cu_k=None), dict(ws=None), dict(ws=FAKE + 16),
    dict(ws_bytes=3199), dict(dq=FAKE + 8), dict(dout=FAKE + 2), dict(lse=FAKE + 1), dict(hq=5), dict(d=8),
    dict(causal=0, window=1), dict(scale=math.nan), dict(dt=-1),
])
def test_packed_backward_refuses(lib, kw):
    assert packed_back(lib, **kw) == BAD


def test_packed_backward_without_work(lib):
    none = dict(q=None, k=None, v=None, out=None, lse=None, dout=None, dq=None, dk=None, dv=None, cu_q=None,
                cu_k=None, ws=None, ws_bytes=0)
    assert packed_back(lib, nseq=0, **none) == OK
    assert packed_back(lib, total_q=0, total_k=0, **none) == OK


def norm(lib, **kw):
    a = dict(x=FAKE, o=FAKE, post_w=None, post_b=None, gate=None, w=None, b=None, y=FAKE, h=FAKE, rows=10, C=64,
             gates=0, rms=0, post=0, eps=1e-5, scale=1.0, dt=na2d.NA_BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.na_norm_forward(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=FAKE + 8), dict(o=FAKE + 2), dict(y=None), dict(o=None), dict(o=None, y=None, h=None),
    dict(post_w=FAKE), dict(post_b=FAKE), dict(gate=FAKE), dict(gates=2), dict(gate=FAKE, gates=3),
    dict(gate=FAKE, gates=-1), dict(o=None, y=None, post=1), dict(o=None, y=None, gate=FAKE, gates=1),
    dict(h=None, w=FAKE), dict(h=None, b=FAKE), dict(w=FAKE + 4), dict(rows=-1), dict(C=0), dict(rms=2), dict(post=-1),
    dict(eps=-1.0), dict(eps=math.nan), dict(scale=math.inf), dict(dt=9),
])
def test_norm_forward_refuses(lib, kw):
    assert norm(lib, **kw) == BAD


def test_norm_without_work_and_too_large(lib):
    assert norm(lib, rows=0, x=None, o=None, y=None, h=None) == OK
    assert norm(lib, C=8193) == UNSUPPORTED
    assert norm(lib, rows=1 << 35, C=64) == UNSUPPORTED
    assert lib.na_norm_backward_workspace_bytes(0, 64, 0, na2d.NA_F32) == 0
    assert lib.na_norm_backward_workspace_bytes(10, 64, 3, na2d.NA_F32) == 0
    assert lib.na_norm_backward_workspace_bytes(10, 64, 2, na2d.NA_F32) >= 5 * 64 * 4


def norm_back(lib, **kw):
    a = dict(y=FAKE, o=FAKE, post_w=None, post_b=None, gate=None, w=None, dy=FAKE, dh=FAKE, dx=FAKE, d_o=FAKE, dw=None,
             db=None, dpost_w=None, dpost_b=None, dgate=None, ws=FAKE, ws_bytes=1 << 40, rows=10, C=64, gates=0, rms=0,
             post=0, eps=1e-5, scale=1.0, dt=na2d.NA_BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.na_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(dx=None), dict(d_o=None), dict(o=None), dict(dy=None, dh=None), dict(dh=None, w=FAKE),
    dict(dh=None, dw=FAKE), dict(dh=None, db=FAKE), dict(dgate=FAKE), dict(gate=FAKE), dict(dpost_w=FAKE),
    dict(dpost_b=FAKE), dict(post_w=FAKE), dict(ws=None), dict(ws_bytes=0), dict(ws=FAKE + 16), dict(dx=FAKE + 8),
    dict(dw=FAKE + 4), dict(C=-1), dict(eps=math.inf),
])
def test_norm_backward_refuses(lib, kw):
    assert norm_back(lib, **kw) == BAD


def test_norm_backward_of_no_rows(lib):
    assert norm_back(lib, rows=0) == UNSUPPORTED


def layer(lib, **kw):
    a = dict(x=FAKE, w=None, b=None, wqkv=FAKE, bqkv=None, wo=FAKE, bo=None, rpb=None, post_w=None, post_b=None,
             gate=None, y=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, H=8, W=8, heads=2, dh=32, ks=3, gates=0, rms=0, post=0,
             eps=1e-5, scale=1.0, dt=na2d.NA_BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.na2d_layer_forward(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(wqkv=None), dict(wo=None), dict(y=None), dict(ws=None), dict(ws_bytes=1000), dict(ws=FAKE + 16),
    dict(ks=4), dict(ks=9), dict(dh=24), dict(B=-1), dict(gate=FAKE), dict(gates=1), dict(gate=FAKE, gates=3),
    dict(post_w=FAKE), dict(w=FAKE + 2), dict(eps=-1.0), dict(rms=3), dict(dt=8),
])
def test_layer_refuses(lib, kw):
    assert layer(lib, **kw) == BAD


def test_layer_workspace_and_empty_batch(lib):
    need = lib.na2d_layer_workspace_bytes(2, 8, 8, 2, 32, 3, na2d.NA_BF16)
    block = lib.na2d_block_workspace_bytes(2, 8, 8, 2, 32, 3, na2d.NA_BF16)
    assert need == block + 2 * 2 * 8 * 8 * 64 * 2
    assert layer(lib, ws_bytes=need - 1) == BAD
    assert layer(lib, B=0, x=None, y=None, ws=None, ws_bytes=0) == OK


def test_the_binding_wants_cuda_tensors():
    q, cu = torch.zeros(4, 2, 16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        na2d.packed_forward(q, q, q, cu, cu)
    with pytest.raises(ValueError, match="CUDA"):
        na2d.packed_backward(q, q, q, q, torch.zeros(2, 4), q, cu, cu)
    x = torch.zeros(4, 8)
    for call in (lambda: na2d.norm_forward(x), lambda: na2d.norm_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---------------------------------------------- the 64-bit formulas themselves
def test_plain_gradients_are_those_of_autograd():
    torch.manual_seed(0)
    cu_q, cu_k = torch.tensor([0, 5, 12]), torch.tensor([0, 9, 16])
    q, k, v = (torch.randn(n, h, 16, dtype=torch.float64) for n, h in ((12, 4), (16, 2), (16, 2)))
    dout = torch.randn_like(q)
    for causal, window in ((False, 0), (True, 0), (True, 4)):
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        out, lse, _, _ = _differentiable(*leaves, cu_q, cu_k, causal, window)
        want = torch.autograd.grad(out, leaves, dout)
        o, l, _, _ = plain64.forward(q, k, v, cu_q, cu_k, causal=causal, window=window)
        assert torch.allclose(o, out.detach(), atol=1e-12)
        got, _ = plain64.backward(q, k, v, o, l, dout, cu_q, cu_k, causal=causal, window=window)
        for a, b in zip(got, want):
            assert torch.allclose(a, b, atol=1e-12)


def _differentiable(q, k, v, cu_q, cu_k, causal, window):
    outs = []
    for q0, lq, k0, lk in plain64.spans(cu_q, cu_k, None):
        heads = []
        for h in range(q.shape[1]):
            s = q[q0:q0 + lq, h] @ k[k0:k0 + lk, h // 2].t() * q.shape[2] ** -0.5
            s = s.masked_fill(~plain64.visible(lq, lk, causal, window), -math.inf)
            heads.append(torch.softmax(s, 1) @ v[k0:k0 + lk, h // 2])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs), None, None, None


def test_plain_norm_gradients_are_those_of_autograd():
    torch.manual_seed(0)
    x, o, dy, dh = (torch.randn(6, 10, dtype=torch.float64) for _ in range(4))
    kw = {n: torch.randn(10, dtype=torch.float64) for n in ("w", "b", "post_w", "post_b")}
    kw["gate"] = torch.randn(2, 10, dtype=torch.float64)
    for rms in (False, True):
        leaves = {"x": x, "o": o, **kw}
        leaves = {n: t.clone().requires_grad_() for n, t in leaves.items()}
        (y, h), _ = plain64.norm_forward(**leaves, post=True, scale=0.5, rms=rms)
        want = torch.autograd.grad([y, h], list(leaves.values()), [dy, dh])
        got, _ = plain64.norm_backward(y.detach(), dh, dy, o=o, **kw, post=True, scale=0.5, rms=rms)
        for n, t in zip(leaves, want):
            assert torch.allclose(got["d" + n], t, atol=1e-10), n
