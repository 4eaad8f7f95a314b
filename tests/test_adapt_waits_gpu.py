"""Adapters' products whose waits give up: the kernel returns, and its results are NaN where they are not right.

The library is built once more with few tries for k_adapt_up_tc's waits: none for the warp that fetches the matrix, which
gives up when it needs a stage for the second time, and 256 (a millisecond; a real wait is some microseconds) for the
warps that issue products and write results.  Every access stays where it is otherwise: the warp that fetches writes to no
stage that it has not waited for, nothing is issued without its operands, and every wait ends."""

import os
import subprocess
import sys

import pytest

from spmm_row_sorted_gb300 import build as snack_build

pytestmark = pytest.mark.gpu

CHILD = """
import sys
import torch
from spmm_row_sorted_gb300 import snack

g = torch.Generator(device="cuda").manual_seed(1)


def normal(*shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


# 11 tiles of 128 columns: five of them and more for a block, of which three have a stage without a wait
n, width, adapters, rank = 1300, 16384, 3, 16
x, wide = normal(n, 256), normal(n, width)
a, b = normal(adapters, rank, 256), normal(adapters, width, rank)
turned = b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous()
which = torch.randint(-1, adapters, (n,), device="cuda", generator=g)
h = torch.full((n, rank), 0.5, device="cuda")


def results():
    y = snack.adapt(x, wide, a, b, which)  # B's rows along the rank
    dx, da, db = snack.adapt_grad(wide, x, *turned, which, h)  # A's rows along the columns
    torch.cuda.synchronize()
    return y, dx, da, db


snack.load(sys.argv[1])
y, dx, da, db = results()
own = which >= 0
assert bool(torch.isnan(y[own]).any(1).all()) and bool(torch.isnan(dx[own]).any(1).all())
assert torch.equal(y[~own], wide[~own]) and bool((dx[~own] == 0).all())
assert bool(torch.isfinite(da).all()) and bool(torch.isfinite(db).all())
# what is no NaN is right
snack._lib = None
snack.load()
want = results()
assert bool((torch.isnan(y) | (y == want[0])).all()) and bool((torch.isnan(dx) | (dx == want[1])).all())
assert torch.equal(da, want[2]) and torch.equal(db, want[3]) and bool(torch.isfinite(want[0]).all())
print("returned")
"""


def test_rows_of_waits_that_gave_up_have_a_nan(tmp_path):
    lib = snack_build.build(extra_flags=["-DSNACK_UP_FETCH_WAITS=0", "-DSNACK_UP_WAITS=256"], out_dir=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", CHILD, lib], capture_output=True, text=True, timeout=300, cwd=snack_build.ROOT,
                       env=dict(os.environ, PYTHONPATH=snack_build.ROOT))
    assert r.returncode == 0 and "returned" in r.stdout, r.stdout + r.stderr
