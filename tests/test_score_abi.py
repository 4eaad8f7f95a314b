"""The entry points of token log probabilities on the host: arguments are checked before anything touches a GPU."""

import ctypes

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


def fwd(lib, x=A, x_ld=8, n=4, w=B, w_ld=8, vocab=40, width=8, t=0, targets=2 * B, targets_t=1, logp=3 * B, entropy=4 * B, top=5,
        ids=5 * B, top_logp=6 * B, state=7 * B, ws=8 * B, ws_bytes=1 << 24):
    return lib.snack_score_fwd(x, x_ld, n, w, w_ld, vocab, width, t, targets, targets_t, logp, entropy, top, ids, top_logp, state, ws,
                               ws_bytes, None)


def bwd(lib, x=A, x_ld=8, n=4, w=B, w_ld=8, vocab=40, width=8, t=0, targets=2 * B, targets_t=1, state=7 * B, dlogp=3 * B, dentropy=4 * B,
        dx=5 * B, dx_ld=8, dw=6 * B, dw_ld=8, ws=8 * B, ws_bytes=1 << 24):
    return lib.snack_score_bwd(x, x_ld, n, w, w_ld, vocab, width, t, targets, targets_t, state, dlogp, dentropy, dx, dx_ld, dw, dw_ld, ws,
                               ws_bytes, None)


BOTH = [
    (dict(x=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(ws=8 * B + 8), 1), (dict(state=None), 1), (dict(state=7 * B + 2), 1),
    (dict(n=-1), 1), (dict(vocab=0), 1), (dict(width=0), 1), (dict(t=2), 1), (dict(targets_t=2), 1), (dict(x_ld=7), 1), (dict(w_ld=7), 1),
    (dict(x=A + 2), 1), (dict(w=B + 2), 1), (dict(targets=2 * B + 4), 1), (dict(n=1 << 24), 7), (dict(vocab=1 << 30), 7),
    (dict(width=1 << 20, x_ld=1 << 20, w_ld=1 << 20), 7), (dict(ws_bytes=64), 4),
]


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(top=-1), 1), (dict(top=41), 1), (dict(top=25), 7), (dict(ids=None), 1), (dict(top_logp=None), 1), (dict(targets=None), 1),
    (dict(logp=3 * B + 2), 1), (dict(entropy=4 * B + 1), 1), (dict(ids=5 * B + 4), 1), (dict(top_logp=6 * B + 2), 1),
])
def test_score_fwd_refuses(lib, bad, status):
    assert fwd(lib, **bad) == status


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(targets=None), 1), (dict(dlogp=3 * B + 2), 1), (dict(dentropy=4 * B + 2), 1), (dict(dx=5 * B + 2), 1), (dict(dw=6 * B + 1), 1),
    (dict(dx_ld=7), 1), (dict(dw_ld=7), 1),
])
def test_score_bwd_refuses(lib, bad, status):
    assert bwd(lib, **bad) == status


@NO_GPU
@pytest.mark.parametrize("bad", [
    dict(logp=A), dict(logp=4 * B), dict(entropy=B), dict(entropy=7 * B + 16), dict(ids=2 * B), dict(ids=6 * B), dict(top_logp=A), dict(state=B),
    dict(state=2 * B), dict(state=8 * B), dict(ws=A), dict(ws=B), dict(ws=2 * B), dict(ws=5 * B), dict(logp=8 * B + 64),
])
def test_score_fwd_refuses_outputs_on_other_buffers(lib, bad):
    assert fwd(lib, **bad) == 1


@NO_GPU
@pytest.mark.parametrize("bad", [
    dict(dx=A), dict(dx=7 * B), dict(dx=3 * B), dict(dw=B), dict(dw=2 * B), dict(dw=5 * B + 64), dict(dw=4 * B), dict(ws=A), dict(ws=7 * B),
    dict(ws=3 * B), dict(ws=6 * B), dict(dx=8 * B),
])
def test_score_bwd_refuses_outputs_on_other_buffers(lib, bad):
    assert bwd(lib, **bad) == 1


def test_score_without_rows_needs_nothing(lib):
    assert fwd(lib, n=0, x=None, w=None, targets=None, logp=None, entropy=None, ids=None, top_logp=None, state=None, ws=None, ws_bytes=0) == 0


def size(lib, n=100, vocab=1000, width=64, t=1, top=0, grad=0, x=A, x_ld=64, w=B, w_ld=64):
    b = ctypes.c_size_t(7)
    return lib.snack_score_workspace_size(x, x_ld, n, w, w_ld, vocab, width, t, top, grad, ctypes.byref(b)), b.value


def test_score_workspace_follows_the_shapes(lib):
    base = size(lib)[1]
    assert base % 256 == 0 and base > 0 and size(lib, n=0) == (0, 0)
    assert size(lib, top=1)[1] >= base + 100 * 1000 * 4      # the logits
    assert size(lib, top=24)[1] == size(lib, top=1)[1]
    assert size(lib, x_ld=65)[1] > base                      # rows off 16 bytes are laid out again
    assert size(lib, n=8192, vocab=1 << 17, top=8)[1] < (1500 << 20)  # a piece of the logits at a time
    assert size(lib, grad=1)[1] > size(lib, n=1, grad=1)[1]
    for bad, status in ((dict(top=-1), 1), (dict(top=1001), 1), (dict(top=25), 7), (dict(t=4), 1), (dict(n=-1), 1), (dict(vocab=1 << 30), 7)):
        assert size(lib, **bad)[0] == status


def test_score_python_refuses_cpu_tensors():
    x, w, t = torch.zeros(3, 8), torch.zeros(5, 8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: snack.score(x, w, t), lambda: snack.score_grad(x, w, t, torch.zeros(2, 3))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
