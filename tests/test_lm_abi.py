"""The language-model entry points on the host: arguments are checked before
anything touches a GPU, and workspace sizes follow the shapes."""

import ctypes

import pytest
import torch

from spmm_row_sorted_gb300 import build as snack_build
from spmm_row_sorted_gb300 import snack

A = 1 << 20  # an address that is never read: every call here is refused first
B = 1 << 24


@pytest.fixture(scope="module")
def lib():
    snack_build.build()
    return snack.load()


def embed_fwd(lib, ids=A, ids_t=1, n=4, table=B, ld=8, vocab=10, width=8, t=0, out=2 * B, out_ld=8):
    return lib.snack_embed_fwd(ids, ids_t, n, table, ld, vocab, width, t, 1.0, out, out_ld, None)


@pytest.mark.parametrize("bad", [
    dict(ids=None), dict(table=None), dict(out=None), dict(ids_t=2), dict(ids_t=-1), dict(t=3), dict(n=-1),
    dict(vocab=0), dict(vocab=2 ** 31), dict(width=0), dict(ld=7), dict(out_ld=7), dict(ids=A + 4), dict(table=B + 2),
    dict(out=2 * B + 1), dict(out=B + 32), dict(out=A),
])
def test_embed_fwd_refuses(lib, bad):
    assert embed_fwd(lib, **bad) == 1


def test_embed_fwd_without_tokens_needs_nothing(lib):
    assert embed_fwd(lib, n=0, ids=None, table=None, out=None) == 0


def embed_grad(lib, ids=A, ids_t=1, n=4, dout=B, ld=8, vocab=10, width=8, t=0, table=2 * B, table_ld=8, ws=3 * B, ws_bytes=1 << 20):
    return lib.snack_embed_grad(ids, ids_t, n, dout, ld, vocab, width, t, 1.0, 0, table, table_ld, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(ids=None), 1), (dict(dout=None), 1), (dict(table=None), 1), (dict(ws=None), 1), (dict(ws=3 * B + 8), 1),
    (dict(ids_t=5), 1), (dict(t=2), 1), (dict(n=-1), 1), (dict(vocab=-3), 1), (dict(width=-1), 1), (dict(ld=3), 1),
    (dict(table_ld=3), 1), (dict(table=B), 1), (dict(table=A), 1), (dict(ws_bytes=64), 4),
])
def test_embed_grad_refuses(lib, bad, status):
    assert embed_grad(lib, **bad) == status


def test_embed_grad_workspace(lib):
    prev = 0
    for n in (0, 1, 100, 4096, 4097, 65536, 65537, 1 << 20):
        size = snack.snack_embed_grad_workspace_size(n, 50000, 768)
        assert size % 256 == 0 and size >= 8 * n and size >= prev // 2
        prev = size
    for args in ((-1, 10, 8), (5, 0, 8), (5, 10, 0)):
        with pytest.raises(snack.SnackError) as e:
            snack.snack_embed_grad_workspace_size(*args)
        assert e.value.status == 1


def clip(lib, n=2, grads=(A, B), outs=(A, B), numel=(100, 50), types=(0, 1), max_norm=1.0, ws=3 * B, ws_bytes=1 << 24, norm=4 * B):
    arr = lambda c, v: None if v is None else (c * len(v))(*v)  # noqa: E731
    return lib.snack_clip_grad_norm(n, arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, numel),
                                    arr(ctypes.c_int, types), max_norm, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), 1), (dict(grads=None), 1), (dict(numel=None), 1), (dict(types=None), 1), (dict(numel=(100, -1)), 1),
    (dict(types=(0, 4)), 1), (dict(max_norm=-1.0), 1), (dict(max_norm=float("nan")), 1), (dict(grads=(A, None)), 1),
    (dict(outs=(A, None)), 1), (dict(outs=(A + 8, B)), 1), (dict(outs=(A + 2, B)), 1), (dict(grads=(A, B + 1)), 1),
    (dict(norm=4 * B + 2), 1), (dict(ws=None), 1), (dict(ws=3 * B + 16), 1), (dict(ws_bytes=64), 4),
])
def test_clip_refuses(lib, bad, status):
    assert clip(lib, **bad) == status


def xent_ws(lib, x=A, x_ld=64, n=100, w=B, w_ld=64, vocab=1000, width=64, t=1, grad=0):
    b = ctypes.c_size_t(7)
    return lib.snack_xent_workspace_size(x, x_ld, n, w, w_ld, vocab, width, t, grad, ctypes.byref(b)), b.value


@pytest.mark.parametrize("bad,status", [
    (dict(t=2), 1), (dict(n=-1), 1), (dict(vocab=0), 1), (dict(width=0), 1), (dict(x_ld=63), 1), (dict(w_ld=63), 1),
    (dict(x=A + 1), 1), (dict(w=B + 2, t=0), 1), (dict(vocab=1 << 30), 7), (dict(n=1 << 24), 7), (dict(width=1 << 20, x_ld=1 << 20, w_ld=1 << 20), 7),
])
def test_xent_workspace_refuses(lib, bad, status):
    assert xent_ws(lib, **bad)[0] == status


def test_xent_workspace_follows_the_shapes(lib):
    base = xent_ws(lib)[1]
    assert base % 256 == 0 and base > 0
    assert xent_ws(lib, n=0) == (0, 0)
    assert xent_ws(lib, x_ld=65)[1] > base        # rows off 16 bytes are laid out again
    assert xent_ws(lib, x=A + 2)[1] > base
    assert xent_ws(lib, w_ld=67)[1] >= base + 1000 * 64 * 2
    assert xent_ws(lib, t=0)[1] >= base + 3 * (1000 + 100) * 64 * 2  # three parts of both
    # the gradient keeps at most about 256 MB of dz
    assert xent_ws(lib, n=8192, vocab=1 << 17, grad=1)[1] < (600 << 20)


def xent(lib, fwd, x=A, n=4, w=B, targets=2 * B, targets_t=1, reduction=0, loss=3 * B, state=4 * B, dloss=5 * B, dx=6 * B, dw=7 * B,
         dx_ld=8, dw_ld=8, ws=8 * B, ws_bytes=1 << 26, t=0):
    if fwd:
        return lib.snack_xent_fwd(x, 8, n, w, 8, 10, 8, t, targets, targets_t, reduction, loss, state, ws, ws_bytes, None)
    return lib.snack_xent_bwd(x, 8, n, w, 8, 10, 8, t, targets, targets_t, reduction, state, dloss, dx, dx_ld, dw, dw_ld, ws,
                              ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(targets=None), 1), (dict(targets_t=9), 1), (dict(reduction=3), 1),
    (dict(reduction=-1), 1), (dict(loss=None), 1), (dict(state=None), 1), (dict(state=4 * B + 2), 1), (dict(ws=None), 1),
    (dict(ws=8 * B + 8), 1), (dict(t=7), 1), (dict(n=-2), 1), (dict(ws_bytes=128), 4),
])
def test_xent_fwd_refuses(lib, bad, status):
    assert xent(lib, True, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(targets=None), 1), (dict(state=None), 1), (dict(reduction=5), 1),
    (dict(dloss=None), 1), (dict(dloss=5 * B + 1), 1), (dict(dx=A), 1), (dict(dw=B), 1), (dict(dw=6 * B), 1), (dict(dx=6 * B + 2), 1),
    (dict(dx_ld=7), 1), (dict(dw_ld=7), 1), (dict(ws=None), 1), (dict(ws_bytes=128), 4),
])
def test_xent_bwd_refuses(lib, bad, status):
    assert xent(lib, False, **bad) == status


def test_python_functions_refuse_cpu_tensors():
    ids, table = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    for call in (lambda: snack.embed(ids, table), lambda: snack.embed_grad(ids, torch.zeros(3, 8), 4),
                 lambda: snack.xent(torch.zeros(3, 8), table, ids), lambda: snack.clip_grad_norm([table], 1.0)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("grads,outs", [
    ((A, A), (A, A)), ((A, A + 200), (A, A + 200)), ((A, B), (B, A)), ((A, B), (A + 4096, A + 4096)), ((A, B), (A + 4096, A)),
    ((B, A), (B, B + 396)),
])
def test_clip_refuses_outputs_on_other_tensors(lib, grads, outs):
    assert clip(lib, grads=grads, outs=outs) == 1
