"""Lanes of a wavefront that read what its other lanes wrote to LDS, without a workgroup barrier between: the gated kernels
tell the compiler so (CPU only; in what the compiler has before it optimizes)."""
import os
import re
import subprocess

import pytest

from fp8_dynamic_scaling_amd import build as hb


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    out = tmp_path_factory.mktemp("ir") / "gemm_gated.ll"
    cmd = [hb.HIPCC] + hb.COMMON + ["--cuda-device-only", "-S", "-emit-llvm", "-Xclang", "-disable-llvm-passes",
                                    os.path.join(hb.HERE, "csrc", "gemm_gated.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    parts = re.split(r"\n(?=define )", out.read_text())[1:]
    return {re.search(r"@(\w+)\(", p).group(1): p for p in parts}


def fences(text):
    return len(re.findall(r"call void @\w*wave_lds_fence", text))


def test_fence(functions):
    body = next(p for n, p in functions.items() if "wave_lds_fence" in n)
    assert 'fence syncscope("wavefront") acq_rel' in body and "llvm.amdgcn.wave.barrier" in body


def test_units_of_the_kernel_for_few_rows(functions):
    """Before the turned fragments are read, and before the next unit's codes take their place."""
    kernels = {m.group(1) for n in functions for m in [re.search(r"^_ZN\w*(k_gated_fewI\w+?EEE)v", n)] if m}
    assert kernels
    for k in kernels:
        assert [fences(p) for n, p in functions.items() if n.startswith("_ZZ") and k in n].count(2) == 1, k


def test_column_scales_of_the_epilogue(functions):
    epilogues = {n: p for n, p in functions.items() if re.match(r"_ZN6fp8dyn14gated_epilogueI", n)}
    assert epilogues
    for n, p in epilogues.items():  # activation, scales by rows or one, blocks
        assert fences(p) == (1 if re.search(r"gated_epilogueILb[01]ELb1E", n) else 0), n
