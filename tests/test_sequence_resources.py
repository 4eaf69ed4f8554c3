"""What the linear attention, the gated join and the experts' kernels take of a
CU, and how the linear attention cuts its sequences, checked without a GPU: no
instantiation may spill, the workgroups that the planners count on fit, and the
stretches fill the GPU once or twice."""

import os
import random
import re
import shutil
import subprocess

import pytest
import torch

import adaln_fwd_amd as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adaln_fwd_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
LDS = 160 * 1024  # of a CU
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def usage(tmp_path_factory):
    """{kernel: (spilled VGPRs, scratch bytes, wavefronts per SIMD, LDS)}"""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    tmp = tmp_path_factory.mktemp("res")
    procs = [subprocess.Popen(
        [HIPCC, "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"),
         "-Rpass-analysis=kernel-resource-usage", "-c",
         os.path.join(CSRC, src), "-o", str(tmp / (src + ".o"))],
        stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        for src in ("lin_attn.hip", "residual.hip", "experts.hip")]
    out = {}
    for p in procs:
        _, err = p.communicate(timeout=900)
        assert p.returncode == 0, err[-2000:]
        for block in err.split("remark: Function Name: ")[1:]:
            def read(what):
                return int(re.search(what + r": (\d+)", block).group(1))

            out[block.split()[0]] = (
                read("VGPRs Spill"), read(r"ScratchSize \[bytes/lane\]"),
                read(r"Occupancy \[waves/SIMD\]"),
                read(r"LDS Size \[bytes/block\]"))
    return out


def test_no_kernel_spills(usage):
    for part, least in (("out_kernel", 32), ("state_kernel", 16),
                        ("step_kernel", 2), ("residual_kernel", 32),
                        ("move_kernel", 8), ("join_bwd_kernel", 4)):
        assert sum(part in n for n in usage) >= least, part
    bad = {n: u for n, u in usage.items() if u[0] or u[1]}
    assert not bad, bad


def test_workgroups_counted_on_fit_a_cu(usage):
    seen = 0
    for n, (_, _, waves, lds) in usage.items():
        assert lds <= LDS, (n, lds)
        m = re.search(r"out_kernelI(\w+?)Li(\d+)ELb[01]ELi([12])E", n)
        if not m:
            continue
        seen += 1
        # a workgroup has a wavefront for 32 features and each of its roles;
        # of bf16's forward two share a CU
        half, of_group = "bf16" in m[1], int(m[2]) // 32 * int(m[3])
        groups = 2 if half and m[3] == "1" else 1
        assert lds * groups <= LDS, (n, lds)
        assert 4 * waves >= of_group * groups, (n, waves)
    assert seen == 32
    for n, (_, _, waves, lds) in usage.items():
        if "residual_kernel" in n and lds:   # the backward
            assert 4 * waves * 64 >= 1280 and LDS // lds >= 5, (n, waves, lds)


def _stretches(B, N, H, d, dt, seg=None):
    return A.lin_attn_states_bytes(B, N, H, d, dt, seg) // (4 * H * d * d)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_stretches_fill_the_gpu_once_or_twice(dt):
    rnd = random.Random(5)
    most = 512 if dt == BF16 else 256
    for _ in range(400):
        B = rnd.choice([1, 1, 2, 5, 16, 300])
        N = rnd.choice([1, 31, 128, 129, 500, 1777, 8190, 75600])
        H = rnd.choice([1, 3, 12, 24, 40, 300])
        d = rnd.choice([8, 64, 72, 128])
        n = _stretches(B, N, H, d, dt)
        share = B * N * H // 256
        if N <= 128 or 3 * N <= 4 * share - 4:
            assert n == 0, (B, N, H)       # whole sequences
            continue
        if 3 * N <= 4 * share + 4:
            continue                       # (at the rule's edge)
        assert n % B == 0 and n >= B, (B, N, H, n)
        # each sequence's end is a stretch too (and the share is rounded down)
        assert n * H <= most * 33 / 32 + B * H, (B, N, H, n)
        # at least half of the CUs have work, if chunks of 32 suffice for it
        assert n * H >= min(128, B * H * ((N + 31) // 32) // 2), (B, N, H, n)


def test_equal_packed_sequences_are_cut_like_samples():
    for B, N, H, d, dt in ((4, 1560, 12, 128, BF16), (2, 1777, 10, 72, F32),
                           (16, 1560, 12, 128, BF16), (1, 32760, 24, 128, BF16)):
        seg = [i * N for i in range(B + 1)]
        assert (_stretches(1, B * N, H, d, dt, seg) ==
                _stretches(B, N, H, d, dt))


def test_one_long_sequence_among_short_ones_is_cut():
    seg = [0]
    for n in [40] * 50 + [20000] + [0] * 3:
        seg.append(seg[-1] + n)
    n = _stretches(1, seg[-1], 24, 64, BF16, seg)
    assert 53 + 8 <= n <= 53 + 100
