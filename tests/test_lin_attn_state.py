"""Which elements of a state the linear attention's lanes read, on the host:
none outside it, whatever the head's width, and each of its own once.  CPU only;
needs hipcc."""

import os
import shutil
import subprocess

import pytest

from adaln_fwd_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def test_no_lane_reads_outside_a_state(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    obj, exe = str(tmp_path / "state.o"), str(tmp_path / "state")
    subprocess.run([HIPCC, "-O1", "-std=c++17", "-fPIE", "--offload-host-only",
                    "-x", "hip", "-I", os.path.join(ROOT, "include"), "-c",
                    os.path.join(ROOT, "tests", "c", "lin_state.hip"), "-o",
                    obj], check=True)
    # (the device code that the object refers to is nowhere)
    subprocess.run(["g++", obj, "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)
    cases = [(dt, d, across) for dt, unit in ((_lib.F32, 4), (_lib.BF16, 8))
             for d in range(unit, 129, unit) for across in (0, 1)]
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    out = subprocess.run([exe], input=text, text=True, check=True,
                         stdout=subprocess.PIPE).stdout.splitlines()
    assert len(out) == len(cases)
    bad = {}
    for (dt, d, across), line in zip(cases, out):
        least, largest, loaded = map(int, line.split())
        if (least, largest, loaded) != (0, d * d - 1, d * d):
            bad[dt, d, across] = line
    assert not bad, bad
