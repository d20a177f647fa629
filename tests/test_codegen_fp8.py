"""Code-generation guards of the 8-bit and root mean square norm kernels (CPU only: hipcc cross-compiles gfx950): no
scratch memory and no device function calls, no workgroup barrier reached with LDS reads outstanding, registers and LDS
that leave room for the workgroups a CU is meant to hold."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_codegen import CSRC, HIPCC, ROOT, _kernel_resources, barriers_with_pending_reads

SOURCES = ["fp8.hip", "fp8_gemm.hip", "fp8_gated.hip", "rms.hip"]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """{source: gfx950 assembly text}, the sources compiled in parallel."""
    if HIPCC is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm")

    def compile_one(src):
        dst = out / (src + ".s")
        cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S",
               "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               os.path.join(CSRC, src), "-o", str(dst)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return src, dst.read_text()

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        return dict(ex.map(compile_one, SOURCES))


@pytest.mark.parametrize("src", SOURCES)
def test_kernels_stay_in_registers(assembly, src):
    asm = assembly[src]
    assert "s_swappc_b64" not in asm, f"{src}: a kernel calls an outlined device function"
    sizes = [int(v) for v in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", asm)]
    assert sizes and max(sizes) == 0, f"{src}: private segment sizes {sizes}"
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", asm), f"{src}: packed float32 instructions"


@pytest.mark.parametrize("src", SOURCES)
def test_no_barrier_with_lds_reads_in_flight(assembly, src):
    assert not barriers_with_pending_reads(assembly[src])


@pytest.mark.parametrize("src,kernel,per_cu", [
    ("fp8_gemm.hip", "TileILi256ELi256", 1), ("fp8_gemm.hip", "TileILi128ELi128ELi2ELi2ELi2", 2),
    ("fp8_gemm.hip", "TileILi128ELi128ELi2ELi2ELi4", 1), ("fp8_gemm.hip", "TileILi64ELi128", 2),
    ("fp8_gemm.hip", "TileILi64ELi64", 2), ("fp8_gated.hip", "TileILi256ELi256", 1),
    ("fp8_gated.hip", "TileILi128ELi128ELi2ELi2ELi2", 2), ("fp8_gated.hip", "TileILi64ELi128", 2),
    ("fp8_gated.hip", "TileILi64ELi256", 1), ("fp8_gated.hip", "TileILi128ELi256", 1), ("fp8.hip", "fp8_rows_kernel", 2),
    ("fp8.hip", "fp8_quantize_t_kernel", 8),
])
def test_workgroups_fit_a_cu(assembly, src, kernel, per_cu):
    found = {k: v for k, v in _kernel_resources(assembly[src]).items() if kernel in k}
    assert found
    for name, f in found.items():
        waves = per_cu * f["max_flat_workgroup_size"] // 64
        assert -(-waves // 4) * (f["vgpr_count"] + f.get("agpr_count", 0)) <= 512, (name, f)
        assert per_cu * f["group_segment_fixed_size"] <= 160 * 1024, (name, f)
