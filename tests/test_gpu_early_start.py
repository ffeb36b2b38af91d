"""Calls behind a kernel that lets its successor start at once and writes late (tests/early_writer.cu, a kernel of a
user's program): what it writes is read, however long it stays."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from block_quantized_decode_nvfp4_gb300 import synthetic as syn
from tests.gpu_util import dev, need_gpu
from tests.test_gpu_fp8_gemm import Data
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


class Product:
    """A product's inputs, and what it gives when they are there from the start."""

    def __init__(self, M, K, T, seed):
        self.M, self.K, self.T = M, K, T
        d = Data(M, K, T, n=2, seed=seed)
        self.inputs = {"x": d.x, "xs": d.dxs, "w": d.w[0], "ws": d.dws[0], "w2": d.w[1], "ws2": d.dws[1]}

    def run(self, gated, late=None):
        i = dict(self.inputs, **(late or {}))
        if gated:
            h = torch.zeros(self.T, self.M, dtype=torch.uint8, device="cuda")
            s = torch.zeros(-(-self.M // 128), self.T, device="cuda")
            bqd.fp8_b128_gemm_silu_mul(i["w"], i["ws"], i["w2"], i["ws2"], i["x"], i["xs"], h, bqd.BQD_E4M3, s, self.M, self.K,
                                       self.T)
            return h, s.view(torch.uint8)
        y = torch.zeros(self.T, self.M, device="cuda")
        bqd.fp8_b128_gemm(i["w"], i["ws"], i["x"], i["xs"], y, bqd.BQD_F32, self.M, self.K, self.T)
        return (y,)


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


# the kernels of up to 16, 32 and 64 tokens, of more and of many
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,T", [(640, 1), (640, 20), (640, 50), (640, 300), (5120, 1100)])
def test_products_read_what_is_written_late(M, T, gated, flags, write_late):
    p = Product(M, 1152, T, seed=51)
    want = p.run(gated)
    # tokens and scales always; weights' codes, where the flag lets them be read early, only without it
    for names in [("x",), ("xs",), ("ws",), ("x", "xs")] + ([] if flags else [("w",), ("w", "ws", "x", "xs")]):
        late = {n: torch.zeros_like(p.inputs[n]) for n in names}
        torch.cuda.synchronize()
        write_late([(late[n], p.inputs[n]) for n in names], 100)
        assert same(p.run(gated, late), want), names


@pytest.mark.parametrize("H", [272, 4096])
def test_rows_read_what_is_written_late(H, flags, write_late):
    T = 40
    g = torch.Generator(device="cuda").manual_seed(4)
    inputs = {n: torch.randn(s, generator=g, device="cuda") for n, s in
              (("x", (T, H)), ("gate", (T, H)), ("post", (H,)), ("pre", (H,)), ("res", (T, H)))}

    def norm(late):
        i = dict(inputs, **late)
        y, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(-(-H // 128), T, device="cuda")
        r = torch.zeros(T, H, device="cuda")
        bqd.residual_norm(i["x"], bqd.BQD_F32, H, i["post"], i["gate"], bqd.BQD_F32, H, 1.0, i["res"], r, bqd.BQD_F32, i["pre"],
                          1e-6, y, bqd.BQD_E4M3, s, H, T)
        return y, s, r

    def encode(late):
        y, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(-(-H // 128), T, device="cuda")
        bqd.fp8_x_encode(dict(inputs, **late)["x"], bqd.BQD_F32, H, y, s, H, T)
        return y, s
    for call, names in ((norm, ("x", "gate", "post", "pre", "res")), (encode, ("x",))):
        want = call({})
        for n in names:
            late = {n: torch.zeros_like(inputs[n])}
            torch.cuda.synchronize()
            write_late([(late[n], inputs[n])], 100)
            assert same(call(late), want), n


# longer than any bounded wait within a call may last (2^31 cycles, about a second)
LONG = 1_700_000


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,T", [(640, 1), (640, 20), (640, 50), (640, 300), (5120, 1100)])
def test_products_behind_a_long_kernel(M, T, gated, flags, write_late):
    p = Product(M, 1152, T, seed=52)
    want = p.run(gated)
    late = {"x": torch.zeros_like(p.inputs["x"])}
    torch.cuda.synchronize()
    write_late([(late["x"], p.inputs["x"])], LONG)
    assert same(p.run(gated, late), want)


@pytest.mark.parametrize("M,K,N,path", [(8000, 4096, 1, "STREAM"), (4000, 16384, 1, "STREAM"), (1024, 4096, 1, "DIRECT"),
                                        (1024, 4096, 8, "MMA"), (1024, 4096, 4, "TILES")])
def test_gemvs_behind_a_long_kernel(M, K, N, path, flags, write_late):
    w = syn.dense_nvfp4(M, K, N=N, seed=53)
    c, s, x = dev(w["codes"]), dev(w["scales"]), dev(w["x"])
    want, got, late = torch.zeros(N, M, device="cuda"), torch.zeros(N, M, device="cuda"), torch.zeros_like(x)
    path = getattr(bqd, "BQD_PATH_" + path)
    bqd.nvfp4_gemv_path(c, s, w["ts"], x, want, M, K, N, path)
    torch.cuda.synchronize()
    write_late([(late, x)], LONG)
    bqd.nvfp4_gemv_path(c, s, w["ts"], late, got, M, K, N, path)
    assert torch.equal(got, want)
