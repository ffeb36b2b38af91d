"""A call that finds its kernel not loaded, on the host: it fails, and the next one, when there is room, does not. The real
launchers run over a stand-in for the CUDA runtime (first_call.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_kernel_that_could_not_be_loaded_is_asked_for_again(tmp_path):
    from block_quantized_decode_nvfp4_gb300 import build
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    build.build(force=not os.path.exists(os.path.join(build.BUILD, "fp8_gemm.o")))
    objs = [os.path.join(build.BUILD, f"fp8_gemm{s}.o") for s in ("", "_tokens", "_pairs")]
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    exe = str(tmp_path / "first_call")
    subprocess.run(["g++", "-std=c++17", "-I", cuda, "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(HERE, "first_call.cpp"), *objs, "-o", exe, "-pthread"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(rows) == 10 and all(first != 0 and then == 0 for first, then in rows), out
