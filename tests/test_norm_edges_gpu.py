"""The norms around a block where they can go wrong."""
import pytest
import torch

from vision_sliding_window_b200 import build, na2d

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    build.build()
    return na2d.load_library()


@pytest.mark.parametrize("shape,gates", [((0, 64), 0), ((0, 5000), 1), ((2, 0, 96), 3)])
@pytest.mark.parametrize("post", [False, True])
def test_gradients_of_no_rows_are_zeros(shape, gates, post):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(shape[-1], dtype=x.dtype, device="cuda")
    kw = dict(w=w, b=w, o=x, post=post)
    if post:
        kw.update(post_w=w, post_b=w)
    if gates:
        kw["gate"] = w.repeat(gates, 1)
    y, h = na2d.norm_forward(x, **kw)
    assert y.shape == h.shape == x.shape
    assert na2d.norm_forward(x, o=x, norm=False)[0].shape == x.shape
    g = na2d.norm_backward(y, x, x, **kw)
    assert g.dx.shape == g.do.shape == x.shape
    for name in ("dw", "db", "dpost_w", "dpost_b", "dgate"):
        t, of = getattr(g, name), kw.get({"dw": "w", "db": "b", "dgate": "gate"}.get(name, name[1:]))
        assert (t is None) == (of is None), name
        if t is not None:
            assert t.dtype == torch.float32 and t.shape == of.shape and (t == 0).all(), name
