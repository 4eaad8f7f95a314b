"""Outputs and workspaces of the language-model calls that lie on another buffer of the call are refused, before
anything is launched.  The addresses are made up, so this runs only where there is no GPU to launch on."""

import pytest
import torch

from spmm_row_sorted_gb300 import build as snack_build
from spmm_row_sorted_gb300 import snack

from test_lm_abi import A, B, clip, embed_grad, xent

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")


@pytest.fixture(scope="module")
def lib():
    snack_build.build()
    return snack.load()


@pytest.mark.parametrize("bad", [
    dict(dx=2 * B), dict(dw=4 * B + 16), dict(dx=5 * B), dict(dx=8 * B), dict(dw=8 * B + 64), dict(ws=A), dict(ws=2 * B),
    dict(ws=4 * B), dict(ws=5 * B), dict(ws=7 * B),
])
def test_xent_bwd_refuses_outputs_on_other_buffers(lib, bad):
    assert xent(lib, False, **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(loss=A), dict(loss=B + 64), dict(loss=2 * B), dict(loss=4 * B + 16), dict(loss=8 * B), dict(state=A), dict(state=2 * B + 16),
    dict(state=8 * B + 64), dict(ws=A), dict(ws=B), dict(ws=2 * B), dict(ws=3 * B), dict(ws=4 * B),
])
def test_xent_fwd_refuses_outputs_on_other_buffers(lib, bad):
    assert xent(lib, True, **bad) == 1


@pytest.mark.parametrize("bad", [dict(ws=A), dict(ws=B), dict(ws=2 * B)])
def test_embed_grad_refuses_a_workspace_on_other_buffers(lib, bad):
    assert embed_grad(lib, **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(ws=A), dict(ws=B), dict(norm=A + 4), dict(norm=B), dict(norm=3 * B + 512), dict(outs=None, ws=B), dict(outs=None, norm=A),
    dict(outs=(A, 6 * B), ws=6 * B), dict(outs=(A, 6 * B), norm=6 * B + 96),
])
def test_clip_refuses_its_norm_and_workspace_on_other_tensors(lib, bad):
    assert clip(lib, **bad) == 1
