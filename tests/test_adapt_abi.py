"""The adapters' entry points on the host: arguments are checked before anything touches a GPU."""

import pytest
import torch

from spmm_row_sorted_gb300 import build as snack_build
from spmm_row_sorted_gb300 import snack

A = 1 << 20  # addresses that are never read: every call here is refused first
B = 1 << 24
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")


@pytest.fixture(scope="module")
def lib():
    snack_build.build()
    return snack.load()


def fwd(lib, x=A, x_ld=8, n=4, a=B, b=2 * B, k=2, rank=4, in_f=8, out_f=8, t=0, which=3 * B, which_t=1, scales=4 * B, base=5 * B,
        base_ld=8, y=6 * B, y_ld=8, h=7 * B, ws=8 * B, ws_bytes=1 << 20):
    return lib.snack_adapt_fwd(x, x_ld, n, a, b, k, rank, in_f, out_f, t, which, which_t, scales, base, base_ld, y, y_ld, h, ws, ws_bytes, None)


def bwd(lib, x=A, x_ld=8, n=4, a=B, b=2 * B, k=2, rank=4, in_f=8, out_f=8, t=0, which=3 * B, which_t=1, scales=4 * B, h=7 * B, dy=5 * B,
        dy_ld=8, dx=6 * B, dx_ld=8, da=9 * B, db=10 * B, ws=8 * B, ws_bytes=1 << 20):
    return lib.snack_adapt_bwd(x, x_ld, n, a, b, k, rank, in_f, out_f, t, which, which_t, scales, h, dy, dy_ld, 0, dx, dx_ld, da, db, ws,
                               ws_bytes, None)


BOTH = [
    (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(which=None), 1), (dict(ws=None), 1), (dict(ws=8 * B + 8), 1),
    (dict(n=-1), 1), (dict(k=0), 1), (dict(rank=0), 1), (dict(in_f=0), 1), (dict(out_f=0), 1), (dict(t=2), 1), (dict(which_t=2), 1),
    (dict(x_ld=7), 1), (dict(x=A + 2), 1), (dict(a=B + 2), 1), (dict(b=2 * B + 1), 1), (dict(which=3 * B + 4), 1), (dict(scales=4 * B + 2), 1),
    (dict(h=7 * B + 2), 1), (dict(n=1 << 24), 7), (dict(k=32769), 7), (dict(rank=257), 7), (dict(in_f=1 << 20, x_ld=1 << 20), 7),
    (dict(out_f=1 << 20), 7), (dict(ws_bytes=64), 4),
]


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(y=None), 1), (dict(y=6 * B + 2), 1), (dict(y_ld=7), 1), (dict(base_ld=7), 1), (dict(base=5 * B + 1), 1),
])
def test_adapt_fwd_refuses(lib, bad, status):
    assert fwd(lib, **bad) == status


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(dy=None), 1), (dict(dy=5 * B + 2), 1), (dict(dy_ld=7), 1), (dict(dx_ld=7), 1), (dict(dx=6 * B + 1), 1), (dict(da=9 * B + 2), 1),
    (dict(db=10 * B + 2), 1), (dict(h=None), 1),
])
def test_adapt_bwd_refuses(lib, bad, status):
    assert bwd(lib, **bad) == status


@NO_GPU
@pytest.mark.parametrize("bad", [
    dict(y=A), dict(y=B + 16), dict(y=2 * B), dict(y=3 * B), dict(y=4 * B), dict(y=5 * B + 32), dict(y=5 * B, y_ld=9), dict(y=7 * B), dict(y=8 * B),
    dict(h=A), dict(h=5 * B), dict(h=8 * B), dict(h=3 * B), dict(ws=A), dict(ws=B), dict(ws=3 * B), dict(ws=5 * B), dict(ws=4 * B),
])
def test_adapt_fwd_refuses_outputs_on_other_buffers(lib, bad):
    assert fwd(lib, **bad) == 1


@NO_GPU
@pytest.mark.parametrize("bad", [
    dict(dx=A), dict(dx=5 * B + 16), dict(dx=7 * B), dict(da=B), dict(db=2 * B), dict(da=6 * B), dict(db=9 * B + 64), dict(da=3 * B), dict(db=7 * B),
    dict(ws=A), dict(ws=5 * B), dict(ws=7 * B), dict(ws=9 * B), dict(da=4 * B), dict(db=8 * B + 64),
])
def test_adapt_bwd_refuses_outputs_on_other_buffers(lib, bad):
    assert bwd(lib, **bad) == 1


def test_adapt_without_rows_needs_nothing(lib):
    assert fwd(lib, n=0, x=None, a=None, b=None, which=None, base=None, y=None, h=None, ws=None, ws_bytes=0) == 0
    assert bwd(lib, n=0, x=None, a=None, b=None, which=None, dy=None, h=None, dx=None, da=None, db=None, ws=None, ws_bytes=0) == 0


def test_adapt_workspace_follows_the_shapes(lib):
    assert snack.snack_adapt_workspace_size(0, 4, 16) == 0
    prev = 0
    for n in (1, 63, 64, 65, 1000, 100000):
        size = snack.snack_adapt_workspace_size(n, 100, 16)
        assert size % 256 == 0 and size >= n * 17 * 4 and size > prev - 1
        prev = size
    for args, status in (((-1, 4, 16), 1), ((5, 0, 16), 1), ((5, 4, 0), 1), ((5, 4, 257), 7), ((5, 32769, 4), 7), ((1 << 24, 4, 4), 7)):
        with pytest.raises(snack.SnackError) as e:
            snack.snack_adapt_workspace_size(*args)
        assert e.value.status == status


def test_adapt_python_refusals():
    x, base = torch.zeros(4, 8), torch.zeros(4, 6)
    a, b, which = torch.zeros(2, 3, 8), torch.zeros(2, 6, 3), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        snack.adapt(x, base, a, b, which)
    with pytest.raises(ValueError, match="CUDA"):
        snack.adapt_grad(x, base, a, b, which, torch.zeros(4, 3))


def test_adapted_refuses_scales_that_want_a_gradient():
    """Before it looks at anything else, so that this runs without a GPU."""
    x, base = torch.zeros(4, 8), torch.zeros(4, 6)
    a, b, which = torch.zeros(2, 3, 8), torch.zeros(2, 6, 3), torch.zeros(4, dtype=torch.int64)
    scales = torch.ones(2, requires_grad=True)
    with pytest.raises(ValueError, match="scales"):
        snack.adapted(x, base, a, b, which, scales)
    for held in (scales.detach(), None):
        with pytest.raises(ValueError, match="CUDA"):
            snack.adapted(x, base, a, b, which, held)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        snack.adapted(x, base, a, b, which, scales)
