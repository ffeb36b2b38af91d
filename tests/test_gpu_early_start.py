"""Calls behind a kernel that lets its successor start at once and writes late (tests/early_writer.cu, a kernel of a
user's program): what it writes is read, however long it stays."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from tests.gpu_util import dev, need_gpu
from tests.test_gpu_nvfp4_gemm import _grouped_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert bqd.bqd_device_error() == 0  # no bounded wait ran out


@pytest.fixture(scope="module")
def write_late(tmp_path_factory):
    from block_quantized_decode_nvfp4_gb300 import build
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "early_writer.cu")
    lib = str(tmp_path_factory.mktemp("early") / "early_writer.so")
    subprocess.run([build._nvcc()] + build.ARCH + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", src, "-o", lib],
                   check=True)
    fn = C.CDLL(lib).early_writer
    fn.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_uint64, C.c_void_p]

    def write(pairs, us):
        """Copies `from` to `to` for pairs of tensors, after `us` microseconds, on the current stream."""
        n = len(pairs)
        for a, b in pairs:
            assert a.is_contiguous() and b.is_contiguous() and a.nbytes == b.nbytes
        to, frm = (C.c_void_p * n)(*[a.data_ptr() for a, _ in pairs]), (C.c_void_p * n)(*[b.data_ptr() for _, b in pairs])
        size = (C.c_int64 * n)(*[a.nbytes for a, _ in pairs])
        assert fn(to, frm, size, n, int(us * 1000), torch.cuda.current_stream().cuda_stream) == 0
    write([], 1)  # loaded
    torch.cuda.synchronize()
    return write


@pytest.fixture(params=[0, bqd.BQD_LAUNCH_PDL], ids=["plain", "dependent"])
def flags(request):
    old = bqd.set_launch_flags(request.param)
    yield request.param
    bqd.set_launch_flags(old)


@pytest.mark.parametrize("counts", [[0, 1, 15, 16, 17, 40, 3, 20], [0, 1, 63, 64, 65, 200, 3, 130]])
def test_offsets_of_a_grouped_product(counts, flags, write_late):
    E, M, K = 8, 384, 1024
    codes, scales, ts, offsets, x, P = _grouped_case(E, M, K, counts, seed=77)
    codes, scales, ts, x, offsets = dev(codes), dev(scales), dev(ts), dev(x), dev(offsets)
    want, got = torch.empty(P, M, device="cuda"), torch.full((P, M), 3.0, device="cuda")
    bqd.nvfp4_gemm_grouped(codes, scales, ts, x, offsets, want, E, M, K, P)
    late = torch.zeros_like(offsets)
    torch.cuda.synchronize()
    write_late([(late, offsets)], 200)
    bqd.nvfp4_gemm_grouped(codes, scales, ts, x, late, got, E, M, K, P)
    assert torch.equal(got, want)
    assert np.isfinite(want.cpu().numpy()).all()
