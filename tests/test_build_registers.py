"""Registers of the cross entropy's product kernels, as the compiler reports them.

They move registers from one warpgroup to the other two by setmaxnreg, out of what the launch gave the block: with
fewer registers per thread than the split adds up to, a launch is refused at run time.  Here the compiler's own figures
say so when the library is built."""

import os
import re
import subprocess

import pytest

from spmm_row_sorted_gb300 import build as snack_build

SOURCE = os.path.join(snack_build.CSRC, "xent.cu")


def constant(text, name):
    return int(re.search(rf"\b{name} = (\d+)", text).group(1))


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("cubin") / "xent.cubin")
    r = subprocess.run([snack_build.nvcc(), *snack_build.NVCC_FLAGS, "-Xptxas", "-v", "-cubin", "-o", out, SOURCE],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = {}
    for part in r.stderr.split("Compiling entry function")[1:]:
        name = re.search(r"'(\w+)'", part).group(1)
        used, spilled = re.search(r"Used (\d+) registers", part), re.search(r"(\d+) bytes spill stores", part)
        kernels[name] = int(used.group(1)), int(spilled.group(1))
    return kernels


def test_product_kernels_launch_with_the_registers_they_split(report):
    with open(SOURCE) as f:
        text = f.read()
    epilogue, issue = constant(text, "kEpiRegs"), constant(text, "kIssueRegs")
    warps = constant(text, "kEpiWarps")
    products = {k: v for k, v in report.items() if re.search(r"6k_xentILi\d+EEEv", k)}
    assert len(products) == 4
    for name, (registers, spilled) in products.items():
        assert registers * (warps + 4) * 32 >= warps * 32 * epilogue + 128 * issue, name
        assert spilled == 0, name
