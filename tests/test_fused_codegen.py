"""Code-generation checks of the fused kernels (CPU only: hipcc cross-compiles
gfx950 assembly without a GPU)."""

from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_gemm_row_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["fused_nn.hip", "fused_nt.hip", "fused_tn.hip", "fused_tt.hip", "fused_pair.hip", "fused_rows.hip",
           "fused_parts.hip"]


@pytest.fixture(scope="module")
def build(tmp_path_factory):
    """(assembly, [(kernel, its arguments, bytes of scratch a lane, wavefronts a SIMD)])."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    filt = shutil.which("c++filt") or shutil.which("llvm-cxxfilt")
    assert filt, "c++filt not found"
    from concurrent.futures import ThreadPoolExecutor

    tmp = tmp_path_factory.mktemp("asm")

    def one(src):
        out = tmp / (src + ".s")
        cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Rpass-analysis=kernel-resource-usage", "--cuda-device-only", "-S",
               os.path.join(CSRC, src), "-o", str(out)]
        res = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
        assert res.returncode == 0, res.stderr[-2000:]
        return out.read_text(), res.stderr

    with ThreadPoolExecutor(max_workers=4) as ex:
        parts = list(ex.map(one, SOURCES))
    remarks = "\n".join(p[1] for p in parts)
    names = re.findall(r"Function Name: (\S+)", remarks)
    names = subprocess.run([filt], input="\n".join(names), capture_output=True, text=True).stdout.splitlines()
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", remarks)]
    waves = [int(x) for x in re.findall(r"Occupancy \[waves/SIMD\]: (\d+)", remarks)]
    assert len(names) == len(scratch) == len(waves) and len(names) > 60
    kernels = []
    for name, s, w in zip(names, scratch, waves):
        kind = re.search(r"(\w+_kernel)(?:<([^>]*)>)?", name)
        kernels.append((kind.group(1), tuple(a.strip() for a in (kind.group(2) or "").split(",")), s, w))
    return "\n".join(p[0] for p in parts), kernels


def test_no_packed_fp32_instructions(build):
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", build[0])


def test_spills_are_the_documented_ones(build):
    """The 256 x 256 tile holds 128 sums a lane and the next stages' values in 256
    registers; what it keeps in scratch is used outside its loops, but for two loads
    a stage."""
    for kind, args, scratch, _ in build[1]:
        large = kind == "tile_kernel" and args[2] == "4"
        assert scratch <= (288 if large else 0), f"{kind}<{', '.join(args)}>: {scratch} bytes a lane"


def test_workgroups_a_cu_that_the_choice_counts_on(build):
    """Wavefronts a SIMD for which the predicted times were measured: one
    workgroup of 8 of the largest tile, two and three of 4 of the others."""
    want = {"4": 2, "2": 2, "1": 3}
    tiles = [(args[2], waves) for kind, args, _, waves in build[1] if kind == "tile_kernel"]
    pairs = [(args[0], waves) for kind, args, _, waves in build[1] if kind == "tile_pair_kernel"]
    assert len(tiles) == 12 and len(pairs) == 4
    for fm, waves in tiles + pairs:
        assert waves == want[fm], (fm, waves)
