"""The norms around a block (na_norm_forward, na_norm_backward) against their
formulas in 64 bits, and the layer made of them."""
import pytest
import torch

from vision_sliding_window_b200 import build, na2d
from vision_sliding_window_b200.inputs import make_block_inputs

from . import plain64

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    build.build()
    return na2d.load_library()


def make(rows, C, gates, post, bias, dtype, seed=0, mean=0.0, weights=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(TYPES[dtype])

    x = normal(rows, C, mean=mean)
    kw = dict(o=normal(rows, C, std=0.7, mean=mean), post=post)
    if weights:
        kw["w"] = normal(C, std=0.1, mean=1.0)
        kw["post_w"] = normal(C, std=0.1, mean=1.0) if post else None
    if bias:
        kw["b"] = normal(C, std=0.1)
        kw["post_b"] = normal(C, std=0.1) if post else None
    if gates:
        kw["gate"] = normal(gates, C, std=0.1, mean=0.3)
    return x, kw, normal(rows, C), normal(rows, C)


CASES = [
    # rows, C, gates, post, rms, bias, dtype
    (1, 64, 0, False, False, True, "bf16"),
    (7, 1, 1, True, True, False, "f32"),
    (33, 8, 3, True, False, True, "f16"),
    (100, 96, 1, False, False, True, "bf16"),
    (65, 200, 5, True, True, False, "f16"),
    (70, 333, 70, True, False, True, "bf16"),      # a gate row for each row
    (40, 256, 2, True, False, True, "f32"),
    (37, 512, 1, True, True, True, "bf16"),
    (300, 768, 3, True, False, True, "bf16"),
    (19, 1000, 0, True, False, False, "f32"),
    (24, 2048, 8, True, True, True, "bf16"),
    (9, 2500, 1, False, False, True, "f16"),
    (2600, 64, 2, False, False, True, "f16"),      # many rows a block
    (5000, 40, 1000, True, False, True, "bf16"),   # gate rows shorter than a block's share
    (700, 4096, 7, True, False, True, "bf16"),
    (6, 4096, 1, True, True, False, "f32"),
    (5, 8192, 1, True, False, True, "bf16"),
    (5, 8191, 5, True, True, True, "f16"),
    (3, 8192, 0, True, False, True, "f32"),
]


@pytest.mark.parametrize("rows,C,gates,post,rms,bias,dtype", CASES)
def test_norms_forward_and_backward(rows, C, gates, post, rms, bias, dtype):
    x, kw, dy, dh = make(rows, C, gates, post, bias, dtype, seed=rows + C)
    how = dict(kw, scale=0.5, eps=1e-5, rms=rms)
    y, h = na2d.norm_forward(x, **how)
    (wy, wh), (ty, th) = plain64.norm_forward(x, **how)
    plain64.check("y", y, wy, ty)
    plain64.check("h", h, wh, th)
    got = na2d.norm_backward(y, dh, dy, **how)
    want, tol = plain64.norm_backward(y, dh, dy, **how)
    for name in na2d.NormGrads._fields:
        assert (getattr(got, name) is not None) == (name in want), name
        if name in want:
            plain64.check(name, getattr(got, name), want[name], tol[name])
    again = na2d.norm_backward(y, dh, dy, **how)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("C", [64, 200, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_left_out(C, dtype):
    x, kw, dy, dh = make(21, C, 0, False, False, dtype, seed=C, weights=False)
    o = kw["o"]
    y, h = na2d.norm_forward(x)  # the norm alone
    assert y is x
    (_, wh), (_, th) = plain64.norm_forward(x)
    plain64.check("h", h, wh, th)
    y, none = na2d.norm_forward(x, o=o, norm=False, scale=-2.0)  # the residual alone
    assert none is None
    (wy, _), (ty, _) = plain64.norm_forward(x, o=o, scale=-2.0)
    plain64.check("y", y, wy, ty)
    for back in (dict(dh=dh), dict(dh=dh, dy=dy), dict(dh=None, dy=dy, o=o, scale=-2.0), dict(dh=dh, o=o)):
        got = na2d.norm_backward(x, **back)
        want, tol = plain64.norm_backward(x, **back)
        for name, t in want.items():
            plain64.check(name, getattr(got, name), t, tol[name])


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,mean", [("f32", 300.0), ("bf16", 30.0), ("f16", -100.0)])
def test_rows_far_from_zero_and_constant_rows(dtype, mean, rms):
    x, kw, dy, dh = make(40, 768, 2, True, True, dtype, seed=4, mean=mean)
    x[3] = mean
    kw["o"][5] = 0.0
    kw["o"][6] = mean
    how = dict(kw, scale=0.25, rms=rms)
    y, h = na2d.norm_forward(x, **how)
    (wy, wh), (ty, th) = plain64.norm_forward(x, **how)
    plain64.check("y", y, wy, ty)
    plain64.check("h", h, wh, th)
    got = na2d.norm_backward(y, dh, dy, **how)
    want, tol = plain64.norm_backward(y, dh, dy, **how)
    for name, t in want.items():
        plain64.check(name, getattr(got, name), t, tol[name])


@pytest.mark.parametrize("C", [64, 333, 768, 4096, 8188])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_begin_far_from_their_means(dtype, C):
    x, kw, dy, dh = make(40, C, 2, True, True, dtype, seed=C)
    x[::3, :8] += 1000.0
    kw["o"][1::3, :8] -= 500.0
    x[5, 0] = 3e4
    y, h = na2d.norm_forward(x, **kw)
    (wy, wh), (ty, th) = plain64.norm_forward(x, **kw)
    plain64.check("y", y, wy, ty)
    plain64.check("h", h, wh, th)
    got = na2d.norm_backward(x, dh, dy, **kw)
    want, tol = plain64.norm_backward(x, dh, dy, **kw)
    for name, t in want.items():
        plain64.check(name, getattr(got, name), t, tol[name])


def test_in_place():
    x, kw, dy, dh = make(33, 768, 1, True, True, "bf16", seed=9)
    y, h = na2d.norm_forward(x, **kw)
    x2, o2 = x.clone(), kw["o"].clone()
    na2d.norm_forward(x2, **dict(kw, o=o2), y=x2, h=o2)
    assert torch.equal(x2, y) and torch.equal(o2, h)


def test_a_row_of_nan_stays_in_its_row():
    x, kw, dy, dh = make(33, 96, 1, True, True, "bf16", seed=9)
    clean = na2d.norm_forward(x, **kw)
    x[7] = float("nan")
    kw["o"][8] = float("inf")
    got = na2d.norm_forward(x, **kw)
    keep = torch.ones(33, dtype=torch.bool)
    keep[7:9] = False
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(a[7:9].float()).any()


def test_gradients_against_differences():
    x, kw, dy, dh = make(12, 24, 3, True, True, "f32", seed=3)
    how = dict(scale=0.5, eps=1e-3, post=True)
    y, _ = na2d.norm_forward(x, **kw, scale=0.5, eps=1e-3)
    got = na2d.norm_backward(y, dh, dy, **kw, scale=0.5, eps=1e-3)
    base = dict(x=x, **{k: v for k, v in kw.items() if torch.is_tensor(v)})
    base = {k: v.double() for k, v in base.items()}
    named = dict(x=got.dx, o=got.do, w=got.dw, b=got.db, post_w=got.dpost_w, post_b=got.dpost_b, gate=got.dgate)

    def loss(t):
        (yy, hh), _ = plain64.norm_forward(**t, **how)
        return ((yy * dy.double()).sum() + (hh * dh.double()).sum()).item()

    for name, grad in named.items():
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        way = torch.randn(grad.shape, generator=g, device="cuda").double()
        step = 1e-5
        up, down = dict(base), dict(base)
        up[name], down[name] = base[name] + step * way, base[name] - step * way
        slope = (loss(up) - loss(down)) / (2 * step)
        # float32 gradients, and a y that was rounded to float32 before its norm was taken again
        assert abs(slope - (grad.double() * way).sum().item()) <= 2e-5 * (grad.double() * way).abs().sum().item() + 1e-6


def test_captured():
    x, kw, dy, dh = make(300, 768, 3, True, True, "bf16", seed=9)
    y, h = torch.empty_like(x), torch.empty_like(x)
    na2d.norm_forward(x, **kw, y=y, h=h)
    na2d.norm_backward(y, dh, dy, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        na2d.norm_forward(x, **kw, y=y, h=h)
        g = na2d.norm_backward(y, dh, dy, **kw)
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    ye, he = na2d.norm_forward(x, **kw)
    assert torch.equal(y, ye) and torch.equal(h, he)
    for a, b in zip(g, na2d.norm_backward(ye, dh, dy, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,post,rms,gates", [("f32", True, False, 1), ("bf16", True, True, 2), ("f16", False, False, 0)])
def test_layer_is_its_parts(dtype, post, rms, gates):
    B, H, W, heads, dh, ks = 2, 14, 12, 2, 32, 7
    x, wqkv, bqkv, wo, bo, rpb = (t.cuda() for t in make_block_inputs(B, H, W, heads, dh, ks, dtype, seed=1))
    C = heads * dh
    _, kw, _, _ = make(B * H * W, C, gates, post, True, dtype, seed=2)
    kw.pop("o")
    norms = {k: kw[k] for k in ("post", "post_w", "post_b", "gate") if kw.get(k) is not None}
    y = na2d.layer_forward(x, kw["w"], kw["b"], wqkv, bqkv, wo, bo, rpb, heads, ks, scale=0.5, rms=rms, **norms)
    _, h = na2d.norm_forward(x, kw["w"], kw["b"], rms=rms)
    o = na2d.block_forward(h, wqkv, bqkv, wo, bo, rpb, heads, ks)
    want, _ = na2d.norm_forward(x, o=o, norm=False, scale=0.5, rms=rms, **norms)
    assert torch.equal(y, want)
    assert na2d.device_status() == na2d.NA_OK
    # and the whole against 64 bits, from the block's own output
    x2 = x.view(-1, C)
    (wy, _), (ty, _) = plain64.norm_forward(x2, o=o.view(-1, C), scale=0.5, rms=rms, **norms)
    plain64.check("layer", y.view(-1, C), wy, ty)
