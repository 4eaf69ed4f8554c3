"""The gated feed-forward's launch plans, on the host: that the sizes of the
GPU tests reach every combination of product, tiling, launch and kind of tile
that seeded random sizes reach, so that a change of the planner cannot leave a
kernel untested, and that each plan's tiles and slices cover the product.  CPU
only; needs hipcc."""

import math
import os
import random
import shutil
import subprocess

import pytest

from tests import glu_sizes
from tests.test_glu_gpu import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
TILINGS = ["small", "big", "deep", "fine"]
SIDE = {"small": 128, "big": 256, "deep": 128, "fine": 64}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """sizes -> their plans, as lists of whole numbers."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    tmp = tmp_path_factory.mktemp("plan")
    obj, exe = str(tmp / "plan.o"), str(tmp / "plan")
    subprocess.run([HIPCC, "-O1", "-std=c++17", "-fPIE", "--offload-host-only",
                    "-x", "hip", "-I", os.path.join(ROOT, "include"), "-c",
                    os.path.join(ROOT, "tests", "c", "glu_plan.hip"), "-o",
                    obj], check=True)
    # (the device code that the object refers to is nowhere)
    subprocess.run(["g++", obj, "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)

    def run(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        out = subprocess.run([exe], input=text, text=True, check=True,
                             stdout=subprocess.PIPE).stdout.splitlines()
        assert len(out) == len(sizes)
        return [[int(v) for v in line.split()] for line in out]

    return run


def _random_sizes(n):
    rng = random.Random(7)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    out = []
    while len(out) < n:
        s = (len(out) % 2, log(1, 40000), 8 * log(1, 800), 8 * log(1, 1728))
        if s[1] * s[2] * s[3] <= 1.2e12:
            out.append(s)
    return out


def _kind(full, rem):
    return "mixed" if full and rem else "sliced" if rem else "whole"


def _reached(size, plan):
    dtype, M, _, _ = size
    few, joint, ft, _, _, _, xt, xf, xr, _, wt, wf, wr, _ = plan
    fwd = f"few {16 if M <= 16 else 32 if M <= 32 else 64}" if few \
        else TILINGS[ft]
    launch = "one launch" if joint else "two"
    parts = "two parts" if dtype == glu_sizes.BF16 and M <= 64 else ""
    return {(dtype, "forward", fwd),
            (dtype, launch, "dx", parts, TILINGS[xt], _kind(xf, xr)),
            (dtype, launch, "dW", TILINGS[wt], _kind(wf, wr))}


def test_the_gpu_sizes_reach_every_kind_of_launch(plans):
    tested = [(dt, *s) for dt in (0, 1) for s in SIZES] + glu_sizes.SIZES
    covered = set()
    for s, p in zip(tested, plans(tested)):
        covered |= _reached(s, p)
    missing = {}
    sizes = _random_sizes(100000)
    for s, p in zip(sizes, plans(sizes)):
        for c in _reached(s, p) - covered:
            missing.setdefault(c, s)
    assert not missing, missing


def test_plans_cover_their_products(plans):
    sizes = _random_sizes(5000)
    for (dtype, M, D, F), p in zip(sizes, plans(sizes)):
        few, joint = p[:2]
        rows = 2 * M if dtype == glu_sizes.BF16 and M <= 64 else M
        for (t, full, rem, slices), (r, c, planes, steps) in zip(
                (p[2:6], p[6:10], p[10:14]),
                ((M, 2 * F, 1, D), (rows, D, 1, F), (F, D, 2, rows))):
            side = SIDE[TILINGS[t]]
            assert full + rem == -(-r // side) * -(-c // side) * planes
            assert slices >= 1 and (rem > 0 or slices == 1)
        if joint:
            assert p[6] == p[10]
