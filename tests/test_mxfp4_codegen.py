"""Code-generation checks of the MXFP4 tiles (CPU only: hipcc cross-compiles
gfx950 assembly without a GPU).

The product tile's barriers wait until all but the newest N vector-memory
instructions are done, and N counts on their order: the scale loads of a group
ahead of the first barrier of the loop, the code loads of two stages behind
each.  The compiler's scheduler may turn loads of one region around, and a scale load
ahead of a code load makes a wavefront read codes that have not landed.
"""

from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_gemm_row_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def build(tmp_path_factory):
    """(assembly, compiler remarks) of the MXFP4 sources."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
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

    with ThreadPoolExecutor(max_workers=3) as ex:
        parts = list(ex.map(one, ["mxfp4_product.hip", "mxfp4_weight.hip", "mxfp4_convert.hip"]))
    return "\n".join(p[0] for p in parts), "\n".join(p[1] for p in parts)


def demangled(names):
    filt = shutil.which("c++filt") or shutil.which("llvm-cxxfilt")
    assert filt, "c++filt not found"
    return subprocess.run([filt], input="\n".join(names), capture_output=True, text=True).stdout.splitlines()


def arguments(name):
    return [a.strip() for a in name[name.index("<") + 1:name.index(">")].split(",")]


def test_product_tile_waits_count_on_its_load_order(build):
    kernels = re.findall(r"^(_Z\S*product_tile_kernel\S*):[^\n]*\n(.*?)^\.Lfunc_end", build[0], re.S | re.M)
    assert len(kernels) == 4
    for name, body in zip(demangled([k[0] for k in kernels]), (k[1] for k in kernels)):
        # <FM, FN, WM, WN, workgroups a CU, WHOLE>
        fm, fn, wm, wn = (int(a) for a in arguments(name)[:4])
        rows, waves = 32 * (fm * wm + fn * wn), wm * wn
        code = rows // 8 // waves  # of two stages
        scale = -(-rows // 64 // waves) * (1 if arguments(name)[5] == "true" else 4)
        lines = [ln.strip() for ln in body.splitlines()]
        bars = [i for i, ln in enumerate(lines) if ln.startswith("s_barrier")]
        assert len(bars) == 3, f"{name}: {len(bars)} barriers"  # one ahead of the loop, two in it
        for k, want in ((1, scale), (2, 0)):
            before = [ln for ln in lines[bars[k - 1]:bars[k]] if ln.startswith("s_waitcnt") and "vmcnt" in ln]
            wait = int(re.search(r"vmcnt\((\d+)\)", before[-1]).group(1))
            assert wait == want, f"{name}: barrier {k} waits for {wait}"
        end = next(i for i in range(bars[2], len(lines)) if lines[i].startswith("buffer_store"))
        for k, first, last, want in ((0, bars[0], bars[1], "s" * scale), (1, bars[1], bars[2], "c" * code),
                                     (2, bars[2], end, "c" * code)):
            loads = "".join("c" if " lds" in ln else "s" for ln in lines[first:last] if ln.startswith("buffer_load"))
            assert loads == want, f"{name}: after barrier {k} loads {loads}"
        assert not any("vmcnt" in ln for ln in lines[bars[1]:bars[2] - 3] if ln.startswith("s_waitcnt")), name


def test_no_kernel_spills_registers(build):
    """A tile that spills runs at a fraction of its rate.  The one exception
    was measured: 24 registers of the 128 x 256 FP32 x MXFP4 tile (W
    transposed), for which a second workgroup fits on a CU."""
    names = re.findall(r"Function Name: (\S+)", build[1])
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", build[1])]
    assert len(names) == len(scratch) and len(names) > 20
    spilled = {n: s for n, s in zip(demangled(names), scratch) if s}
    allowed = [n for n in spilled if "weight_tile_kernel" in n and
               (arguments(n) == ["2", "4", "true", "true", "2"] or spilled[n] <= 16)]
    assert set(spilled) == set(allowed) and all(s <= 160 for s in spilled.values()), spilled


def test_no_packed_fp32_instructions(build):
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", build[0])


def test_spills_are_the_documented_ones(build):
    """24 registers (96 bytes a lane) of one tile, none of any other kernel's."""
    names = demangled(re.findall(r"Function Name: (\S+)", build[1]))
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", build[1])]
    for name, n in zip(names, scratch):
        documented = "weight_tile_kernel" in name and arguments(name) == ["2", "4", "true", "true", "2"]
        assert n <= (96 if documented else 0), f"{name}: {n} bytes a lane"


def test_workgroups_a_cu_that_the_choice_counts_on(build):
    """Wavefronts a SIMD for which the predicted times were measured."""
    names = demangled(re.findall(r"Function Name: (\S+)", build[1]))
    waves = [int(x) for x in re.findall(r"Occupancy \[waves/SIMD\]: (\d+)", build[1])]
    assert len(names) == len(waves)
    seen = {}
    for name, n in zip(names, waves):
        if "tile_kernel" in name:
            seen[(re.search(r"\w+_tile_kernel", name).group(0), *arguments(name))] = n
    # 8 wavefronts of 256 x 256 a CU, and two workgroups of 4 of 128 x 128
    for whole in ("true", "false"):
        assert seen["product_tile_kernel", "2", "4", "4", "2", "1", whole] == 2
        assert seen["product_tile_kernel", "2", "2", "2", "2", "2", whole] == 2
    # two of 128 x 256 (for which word loads of A leave one, W transposed),
    # two of 64 x 256, three of 64 x 128
    for bt in ("true", "false"):
        for quads in ("true", "false"):
            fits = "2" if bt == quads == "true" else "1"
            want = 1 if (bt, quads) == ("true", "false") else 2
            assert seen["weight_tile_kernel", "2", "4", bt, quads, fits] == want
            assert seen["weight_tile_kernel", "1", "4", bt, quads, "2"] == 2
            assert seen["weight_tile_kernel", "1", "2", bt, quads, "3"] == 3
