"""The wavefronts that the planners count on, checked at build time without a
GPU: the gated feed-forward's small and fine tiles run two workgroups to a CU
and its big ones two wavefronts to a SIMD, in registers and in LDS; the norm's
backward runs three workgroups of four wavefronts to a CU."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adaln_fwd_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
LDS = 160 * 1024  # of a CU

# tiling -> wavefronts of a workgroup, workgroups to a CU
TILINGS = {"small": (4, 2), "big": (8, 1), "deep": (4, 1), "fine": (2, 2)}
CODES = ["small", "big", "deep", "fine"]


def _usage(src, tmp):
    """{kernel: (wavefronts per SIMD by registers and LDS, LDS bytes)}"""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    err = subprocess.run(
        [HIPCC, "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"),
         "-Rpass-analysis=kernel-resource-usage", "-c",
         os.path.join(CSRC, src), "-o", str(tmp / "o.o")],
        stderr=subprocess.PIPE, text=True, check=True, timeout=900).stderr
    out = {}
    for block in err.split("remark: Function Name: ")[1:]:
        def read(what):
            return int(re.search(what + r": (\d+)", block).group(1))

        out[block.split()[0]] = (read(r"Occupancy \[waves/SIMD\]"),
                                 read(r"LDS Size \[bytes/block\]"))
    return out


def test_tiles_leave_room_for_the_workgroups_counted_on(tmp_path):
    usage = _usage("glu.hip", tmp_path)
    seen = dict.fromkeys(CODES, 0)
    for name, (waves, lds) in usage.items():
        # the tiling is the second number of a product, the first of both
        # gradients' kernel
        m = re.search(r"product_kernelI\w+?Li\d+ELi(\d)ELi\d+E", name) or \
            re.search(r"12grads_kernelI\w+?Li(\d)E", name)
        if not m:
            continue
        tiling = CODES[int(m.group(1))]
        seen[tiling] += 1
        of_group, groups = TILINGS[tiling]
        assert lds * groups <= LDS, (name, lds)
        assert 4 * waves >= of_group * groups, (name, waves)
    # two types: the forward and G, U again by two activations, dx, dW; and
    # the two in one launch
    assert seen["small"] >= 14 and seen["deep"] >= 14, seen
    assert seen["big"] >= 13 and seen["fine"] >= 8, seen


def test_backward_of_the_norm_leaves_room_for_three_workgroups(tmp_path):
    usage = _usage("heads.hip", tmp_path)
    seen = 0
    for name, (waves, lds) in usage.items():
        # (type, lanes per head, layout, pass: 2 is the norm's backward)
        if re.search(r"heads_kernelI\w+?Li\d+ELb[01]ELi2E", name):
            seen += 1
            # (its dynamic LDS, the sines, is at most 32 KiB)
            assert waves >= 3 and 3 * (lds + 32768) <= LDS, (name, waves, lds)
    assert seen >= 52
