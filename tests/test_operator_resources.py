"""Register budget of the rotation, norm and feed-forward kernels, checked at
build time without a GPU: no instantiation may spill, and the feed-forward's
tiles must leave room for the wavefronts that their design counts on."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adaln_fwd_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def usage(tmp_path_factory):
    """{kernel: (spilled VGPRs, scratch bytes per lane, LDS bytes)}"""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    tmp = tmp_path_factory.mktemp("res")
    procs = {}
    for src in ("heads.hip", "glu.hip"):
        procs[src] = subprocess.Popen(
            [HIPCC, "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"),
             "-Rpass-analysis=kernel-resource-usage", "-c",
             os.path.join(CSRC, src), "-o", str(tmp / (src + ".o"))],
            stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    out = {}
    for src, p in procs.items():
        _, err = p.communicate(timeout=900)
        assert p.returncode == 0, err[-2000:]
        for block in err.split("remark: Function Name: ")[1:]:
            name = block.split("\n", 1)[0].split()[0]

            def read(what):
                return int(re.search(what + r": (\d+)", block).group(1))

            out[name] = (read("VGPRs Spill"),
                         read(r"ScratchSize \[bytes/lane\]"),
                         read(r"LDS Size \[bytes/block\]"))
    return out


def test_no_kernel_spills(usage):
    assert sum("heads_kernel" in n for n in usage) >= 100
    assert sum("product_kernel" in n for n in usage) >= 18
    assert sum("few_kernel" in n for n in usage) >= 12
    bad = {n: u for n, u in usage.items() if u[0] or u[1]}
    assert not bad, bad


def test_tiles_fit_the_lds(usage):
    for n, (_, _, lds) in usage.items():
        assert lds <= 160 * 1024, (n, lds)
