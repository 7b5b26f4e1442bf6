"""The norms of no rows, whose buffers have no addresses."""
import pytest

from vision_sliding_window_b200 import build, na2d

from .test_ops_abi_cpu import FAKE, norm


@pytest.fixture(scope="module")
def lib():
    build.build()
    return na2d.load_library()


@pytest.mark.parametrize("kw", [
    dict(w=FAKE, b=FAKE), dict(post=1, post_w=FAKE, post_b=FAKE), dict(gate=FAKE, gates=3), dict(h=None), dict(gates=2),
])
def test_norm_forward_of_no_rows_is_nothing(lib, kw):
    assert norm(lib, rows=0, **dict(dict(x=None, o=None, y=None, h=None), **kw)) == na2d.NA_OK


@pytest.mark.parametrize("kw", [dict(C=0), dict(eps=-1.0), dict(gates=-1), dict(dt=7), dict(post=2)])
def test_its_sizes_are_still_looked_at(lib, kw):
    assert norm(lib, rows=0, x=None, o=None, y=None, h=None, **kw) == na2d.NA_ERR_INVALID_ARG
