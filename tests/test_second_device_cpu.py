"""token_logprobs on several devices of one process, on the host: kernel attributes belong to a device, so each needs
its own. The real launcher runs over a stand-in for the CUDA runtime (two_devices.cpp)."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    from block_quantized_decode_nvfp4_gb300 import build
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    build.build()
    tmp = tmp_path_factory.mktemp("two_devices")
    obj = os.path.join(build.BUILD, "logprobs.o")
    if not os.path.exists(obj) or any(os.path.getmtime(p) > os.path.getmtime(obj) for p in build._deps()):
        obj = str(tmp / "logprobs.o")
        subprocess.run([build._nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", build.INCLUDE,
                                                       "-I", build.CSRC, "--expt-relaxed-constexpr", "-c",
                                                       os.path.join(build.CSRC, "logprobs.cu"), "-o", obj], check=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    exe = str(tmp / "two_devices")
    subprocess.run(["g++", "-std=c++17", "-I", cuda, "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(HERE, "two_devices.cpp"), obj, "-o", exe, "-pthread"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, re.findall(r"\d+", line))) for line in out.splitlines()]
    assert len(rows) == 12, out
    return rows


def test_every_device_may_launch_large_clusters(lines):
    for dev, kind, rows, status, cluster in lines[:9]:
        assert (status, cluster) == (0, 16 if rows == 1 else 9), (dev, kind, rows)


def test_many_rows_need_no_cluster(lines):
    assert lines[9][3:] == (0, 1)


def test_a_refusal_is_reported_and_not_kept(lines):
    assert lines[10][0] == lines[11][0] == 2
    assert lines[10][3] != 0 and lines[11][3:] == (0, 16)
