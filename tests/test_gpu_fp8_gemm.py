"""fp8_b128_gemm and fp8_b128_gemm_silu_mul against their fp64 definitions.

Bounds. Products of E4M3 values are exact. The tensor cores add a block's 128 of them in fp32 (or finer) in an order
and with a rounding of their own; nothing is assumed but that each of the 128 additions loses at most one unit of fp32
(2^-23) of the sum of magnitudes: 2^-16 of it. The blocks' sums, their scales and the output add KB + 4 half units.
So |y - exact| <= A (2^-16 + (KB + 4) 2^-24) + the output's rounding, A = sum |x w|. h carries both products' bounds
through SiLU(g) u (|SiLU'| < 1.1) and 2^-20 for the function itself."""
import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from oracle import fp8 as ref
from tests.fp8_util import HALF, TYPES, Out, check_codes, codes, scale_array
from tests.gpu_util import dev, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    yield
    assert bqd.bqd_device_error() == 0  # no bounded wait ran out


class Data:
    """Random activations and n weights of the same size, and their values."""

    def __init__(self, M, K, T, n=1, seed=0, lo=-12, hi=-2):
        self.M, self.K, self.T = M, K, T
        Mb, Kb = -(-M // 128), -(-K // 128)
        self.xc, self.xs = codes((T, K), seed), scale_array((Kb, T), seed + 1, lo, hi)
        self.wc = [codes((M, K), seed + 10 + i) for i in range(n)]
        self.ws = [scale_array((Mb, Kb), seed + 20 + i, lo, hi) for i in range(n)]
        self.upload()

    def upload(self):
        self.x, self.dxs = dev(self.xc), dev(self.xs)
        self.w, self.dws = [dev(c) for c in self.wc], [dev(s) for s in self.ws]

    def products(self, rows=None):
        """[(y, bound)] of each weight in fp64; rows: those of the tokens."""
        x = ref.scaled(self.xc, self.xs)
        x = x if rows is None else x[rows]
        out = []
        for c, s in zip(self.wc, self.ws):
            w = ref.weights(c, s)
            a = np.abs(x) @ np.abs(w).T
            out.append((x @ w.T, a * (2.0 ** -16 + (-(-self.K // 128) + 4) * 2.0 ** -24)))
        return out


def run_gemm(d, kind="f32", stream=None):
    y = Out((d.T, d.M), kind)
    bqd.fp8_b128_gemm(d.w[0], d.dws[0], d.x, d.dxs, y.ptr, TYPES[kind][1], d.M, d.K, d.T, stream)
    return y.get()


def check_gemm(d, kind="f32"):
    got = run_gemm(d, kind)
    (y, tol), = d.products()
    bad = ~(np.abs(got - y) <= tol + HALF[kind] * (np.abs(y) + tol))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}"


def check_ffn(d, kind):
    h, hs = Out((d.T, d.M), kind), Out((-(-d.M // 128), d.T), "f32")
    bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h.ptr, TYPES[kind][1],
                               hs.ptr if kind == "e4m3" else None, d.M, d.K, d.T)
    (g, tg), (u, tu) = d.products()
    with np.errstate(over="ignore"):
        want = ref.silu(g) * u
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(ref.silu(g)) * tu
    tol += 2.0 ** -20 * (np.abs(want) + tol)
    if kind == "e4m3":
        check_codes(h.get(), hs.get().astype(np.float32), want, tol, "h")
    else:
        bad = ~(np.abs(h.get() - want) <= tol + HALF[kind] * (np.abs(want) + tol))
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}"


SIZES = [(1, 16, 1), (128, 128, 1), (128, 128, 16), (130, 144, 3), (64, 4096, 1), (1000, 512, 8), (257, 1040, 17),
         (384, 2064, 32), (500, 384, 33), (129, 256, 64), (700, 640, 65), (256, 512, 128), (300, 1024, 129),
         (512, 128, 200), (1031, 272, 255), (256, 1536, 256), (2048, 144, 257), (384, 768, 513), (20000, 256, 5),
         (45000, 16, 2), (7, 16384, 2), (513, 384, 1030)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,T", SIZES)
def test_gemm_sizes(M, K, T, kind):
    check_gemm(Data(M, K, T, seed=M + K + T), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("I,K,T", SIZES[:-5] + [(20000, 128, 3), (513, 384, 1030)])
def test_ffn_sizes(I, K, T, kind):
    check_ffn(Data(I, K, T, n=2, seed=I + K + T, lo=-16, hi=-6), kind)


# more tiles than CTAs, so that each takes one after the other; a K of many blocks shared by eight CTAs
@pytest.mark.parametrize("M,K,T", [(40000, 272, 20), (40000, 144, 40), (30000, 272, 100), (20000, 144, 700), (130, 16384, 40),
                                   (130, 16384, 100), (130, 1152, 100)])
def test_gemm_many_tiles_and_long_k(M, K, T):
    check_gemm(Data(M, K, T, seed=21))
    if M < 30000:
        check_ffn(Data(M, K, T, n=2, seed=22, lo=-16, hi=-6), "e4m3")


# many tokens, tiles of 256 rows by 256 tokens: rows of y that start on 16 bytes and not, last tiles of a few rows or tokens
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,T", [(2600, 256, 2050), (2568, 128, 2049), (2692, 272, 2100), (2690, 128, 2304), (2816, 1040, 2303)])
def test_gemm_outputs_of_many_tokens(M, K, T, kind):
    check_gemm(Data(M, K, T, seed=23), kind)
    if M % 4 == 0 and K < 1000:
        check_ffn(Data(M // 2, K, T, n=2, seed=24, lo=-16, hi=-6), kind)


@pytest.mark.parametrize("M,K,T", [(12288, 4096, 1), (4096, 12288, 17), (4870, 4096, 333)])
def test_gemm_of_a_layer(M, K, T):
    check_gemm(Data(M, K, T, seed=7))


def test_gemm_of_a_prompt_sampled():
    d = Data(4096, 2048, 4100, seed=9)
    got = run_gemm(d, "bf16")
    rows = np.r_[0:5, 127:130, 255:258, 2047:2049, 4090:4100]
    (y, tol), = d.products(rows)
    assert (np.abs(got[rows] - y) <= tol + HALF["bf16"] * (np.abs(y) + tol)).all()
    assert np.isfinite(got).all() and np.array_equal(got, run_gemm(d, "bf16"))


@pytest.mark.parametrize("T", [1, 16, 40, 100, 300])
def test_one_hot_tokens_give_the_weights(T):
    # token t is 1.0 at k = 7 t + t / 3 with scale 2: y is exactly twice the weight's value
    M, K = 260, 1040
    d = Data(M, K, T, seed=4)
    at = (7 * np.arange(T) + np.arange(T) // 3) % K
    d.xc[:] = 0
    d.xc[np.arange(T), at] = 0x38
    d.xs[:] = 2.0
    d.ws[0][:] = np.exp2(np.round(np.log2(d.ws[0])))
    d.upload()
    want = 2 * ref.weights(d.wc[0], d.ws[0])[:, at].T
    assert np.array_equal(run_gemm(d), want)


@pytest.mark.parametrize("T", [2, 33, 200, 600])
def test_every_scale_meets_its_own_block(T):
    # all codes 1.0: y[t][m] = sum over blocks of 128 xs[kb][t] ws[m/128][kb], powers of two that tell the blocks apart
    M, K = 400, 640
    d = Data(M, K, T, seed=5)
    d.xc[:], d.wc[0][:] = 0x38, 0x38
    rng = np.random.default_rng(T)
    d.xs[:] = np.exp2(rng.integers(-3, 4, d.xs.shape))
    d.ws[0][:] = np.exp2(rng.integers(-3, 4, d.ws[0].shape))
    d.upload()
    want = 128.0 * (d.xs.T.astype(np.float64) @ d.ws[0].T.astype(np.float64))[:, np.arange(M) // 128]
    assert np.array_equal(run_gemm(d), want)


@pytest.mark.parametrize("T", [3, 70, 300])
def test_nan_spoils_its_row_and_column_alone(T):
    d = Data(300, 512, T, n=2, seed=6)
    clean = run_gemm(d)
    d.xc[1, 77] = 0x7F
    d.wc[0][200, 300] = 0xFF
    d.xs[2, 2] = np.nan
    d.upload()
    got = run_gemm(d)
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all() and np.isnan(got[:, 200]).all()
    keep = np.ones_like(got, bool)
    keep[1:3], keep[:, 200] = False, False
    assert np.array_equal(got[keep], clean[keep])
    h, hs = Out((T, 300), "e4m3"), Out((3, T), "f32")
    bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h.ptr, bqd.BQD_E4M3, hs.ptr, 300, 512, T)
    s = hs.get()
    assert np.isnan(s[:, 1:3]).all() and np.isnan(s[1]).all() and np.isfinite(s[0][[0] + list(range(3, T))]).all()
    assert (h.get()[0, 128:256] == 0x7F).all()


def test_zero_tokens_and_zero_weights():
    d = Data(256, 256, 40, n=2, seed=8)
    d.xc[3] = 0
    d.wc[1][:] = 0
    d.upload()
    assert (run_gemm(d)[3] == 0).all()
    h, hs = Out((40, 256), "e4m3"), Out((2, 40), "f32")
    bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h.ptr, bqd.BQD_E4M3, hs.ptr, 256, 256, 40)
    assert ((h.get() & 0x7F) == 0).all() and (hs.get() == 2.0 ** -126).all()


def test_large_gates():
    # g far below and above 0: SiLU goes to 0 and to g, nothing becomes NaN
    d = Data(128, 128, 20, n=2, seed=12, lo=-1, hi=1)
    h = Out((20, 128), "f32")
    bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h.ptr, bqd.BQD_F32, None, 128, 128, 20)
    got = h.get()
    (g, tg), (u, _) = d.products()
    assert np.isfinite(got).all() and (got[g < -200 - tg] == 0).all()
    far = g > 200 + tg
    assert far.any() and (np.abs(got[far] - (g * u)[far]) <= 1e-3 * np.abs(g * u)[far] + 1e-3 * np.abs(got).max()).all()


def test_halves_of_a_fused_weight():
    d = Data(512, 256, 19, seed=13)
    h = Out((19, 256), "f32")
    w, s = d.w[0], d.dws[0]
    bqd.fp8_b128_gemm_silu_mul(w, s, w[256:], s[2:], d.x, d.dxs, h.ptr, bqd.BQD_F32, None, 256, 256, 19)
    (y, tol), = d.products()
    g, u, tg, tu = y[:, :256], y[:, 256:], tol[:, :256], tol[:, 256:]
    with np.errstate(over="ignore"):
        want = ref.silu(g) * u
        bound = 1.1 * tg * (np.abs(u) + tu) + np.abs(ref.silu(g)) * tu
    assert (np.abs(h.get() - want) <= bound + 2.0 ** -19 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("M,K,T", [(1024, 2048, 4), (640, 512, 300), (4096, 4096, 1024)])
def test_same_bits_twice_on_any_stream_and_from_a_graph(M, K, T):
    d = Data(M, K, T, seed=14)
    y = [torch.zeros(T, M, device="cuda") for _ in range(3)]

    def call(out):
        bqd.fp8_b128_gemm(d.w[0], d.dws[0], d.x, d.dxs, out, bqd.BQD_F32, M, K, T)
    call(y[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(y[1])
        call(y[2])  # before the capture: nothing is set up within it
    torch.cuda.synchronize()
    y[2].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y[2])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_two_calls_at_once():
    a, b = Data(2048, 1024, 40, seed=15), Data(2048, 1024, 300, seed=16)
    alone = [run_gemm(a), run_gemm(b)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ya, yb = torch.empty(40, 2048, device="cuda"), torch.empty(300, 2048, device="cuda")
    for _ in range(20):
        bqd.fp8_b128_gemm(a.w[0], a.dws[0], a.x, a.dxs, ya, bqd.BQD_F32, 2048, 1024, 40, sa)
        bqd.fp8_b128_gemm(b.w[0], b.dws[0], b.x, b.dxs, yb, bqd.BQD_F32, 2048, 1024, 300, sb)
    torch.cuda.synchronize()
    assert np.array_equal(ya.cpu().double().numpy(), alone[0]) and np.array_equal(yb.cpu().double().numpy(), alone[1])


def test_beside_other_kernels_of_the_tensor_cores():
    # clusters here, clusters of the NVFP4 products there, on streams of their own: each ends, with its own answer
    M, K = 4096, 4096
    d = [Data(M, K, T, n=2, seed=30 + T) for T in (8, 40, 100)]
    codes_, scales = codes((M, K // 2), 40), np.full((M, K // 16), 0x38, np.uint8)
    nv, ns, x = dev(codes_), dev(scales), torch.randn(8, K, device="cuda").to(torch.bfloat16)
    y = [torch.empty(8, M, device="cuda")] + [torch.empty(e.T, M, device="cuda") for e in d]

    def calls(streams):
        bqd.nvfp4_gemv(nv, ns, 0.01, x, y[0], M, K, 8, streams[0])
        for e, o, s in zip(d, y[1:], streams[1:]):
            bqd.fp8_b128_gemm_silu_mul(e.w[0], e.dws[0], e.w[1], e.dws[1], e.x, e.dxs, o, bqd.BQD_F32, None, M, K, e.T, s)
    calls([None] * 4)
    torch.cuda.synchronize()
    want = [o.clone() for o in y]
    streams = [torch.cuda.Stream() for _ in y]
    for _ in range(30):
        calls(streams)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, y))


@pytest.mark.parametrize("norm", [False, True])
def test_dependent_launches(norm):
    # with programmatic dependent launch on: each call's activations come from the call before it. Without a norm
    # the values grow until they are NaN, so bits are compared
    T, K, I = 24, 1024, 512
    d = Data(I, K, T, n=2, seed=17)
    down = Data(K, I, T, seed=18)
    h, hs = torch.empty(T, I, dtype=torch.uint8, device="cuda"), torch.empty(I // 128, T, device="cuda")
    y, ones = torch.empty(T, K, device="cuda"), torch.ones(K, device="cuda")

    def step():
        bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h, bqd.BQD_E4M3, hs, I, K, T)
        bqd.fp8_b128_gemm(down.w[0], down.dws[0], h, hs, y, bqd.BQD_F32, K, I, T)
        if norm:
            bqd.residual_norm(y, bqd.BQD_F32, K, None, None, 0, 0, 1.0, None, None, bqd.BQD_F32, ones, 1e-6, d.x,
                              bqd.BQD_E4M3, d.dxs, K, T)
        else:
            bqd.fp8_x_encode(y, bqd.BQD_F32, K, d.x, d.dxs, K, T)
    got = []
    for flags in (0, bqd.BQD_LAUNCH_PDL):
        d.upload()
        old = bqd.set_launch_flags(flags)
        try:
            for _ in range(8):
                step()
            torch.cuda.synchronize()
        finally:
            bqd.set_launch_flags(old)
        got.append((y.clone(), d.x.clone(), d.dxs.clone()))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))
    assert not norm or bool(y.isfinite().all())


@pytest.mark.parametrize("T", [1, 40, 200, 1100])
def test_weights_written_by_the_call_before(T):
    # no early reads without the flag: each product's weights are written by the kernel before it, after a product has
    # let that kernel's neighbours start
    M, K, n = 1536, 1152, 6
    ds = [Data(M, K, T, seed=30 + i) for i in range(n)]
    want = []
    for d in ds:
        y = torch.empty(T, M, device="cuda")
        bqd.fp8_b128_gemm(d.w[0], d.dws[0], d.x, d.dxs, y, bqd.BQD_F32, M, K, T)
        torch.cuda.synchronize()
        want.append(y)
    w, s = torch.empty_like(ds[0].w[0]), torch.empty_like(ds[0].dws[0])
    rows = [d.w[0].float() for d in ds]  # (of code bytes: any kernel's output)
    for _ in range(20):
        got = [torch.empty(T, M, device="cuda") for _ in ds]
        for d, r, y in zip(ds, rows, got):
            s.copy_(d.dws[0])
            w.copy_(r)
            bqd.fp8_b128_gemm(w, s, d.x, d.dxs, y, bqd.BQD_F32, M, K, T)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [64, 300])
def test_weights_made_by_an_encoder_that_starts_early(T):
    # the same behind a call that lets the next one start: fp8_x_encode's codes are the product's weights
    M, K, n = 640, 1152, 5
    d = Data(M, K, T, seed=41)
    g = torch.Generator(device="cuda").manual_seed(2)
    src = [torch.randn(M, K, generator=g, device="cuda") for _ in range(n)]
    w, sc = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, M, device="cuda")

    def run(wait):
        out = []
        for _ in range(4):
            for x in src:
                y = torch.empty(T, M, device="cuda")
                bqd.fp8_x_encode(x, bqd.BQD_F32, K, w, sc, K, M)
                if wait:
                    torch.cuda.synchronize()
                bqd.fp8_b128_gemm(w, d.dws[0], d.x, d.dxs, y, bqd.BQD_F32, M, K, T)
                if wait:
                    torch.cuda.synchronize()
                out.append(y)
        return out
    assert all(torch.equal(a, b) for a, b in zip(run(True), run(False)))


@pytest.mark.parametrize("T", [300, 2500])
def test_dependent_launches_of_many_tokens(T):
    # outputs that leave after their kernel's last sums are complete for the next call: one call after the other,
    # against the same with a wait between
    K, I = 2048, 1024
    d = Data(I, K, T, n=2, seed=25)
    down = Data(K, I, T, seed=26)
    h, hs = torch.empty(T, I, dtype=torch.uint8, device="cuda"), torch.empty(I // 128, T, device="cuda")
    r, ones = torch.empty(T, K, dtype=torch.bfloat16, device="cuda"), torch.ones(K, device="cuda")
    got = []
    for wait in (True, False):
        for kind, code in ((torch.float32, bqd.BQD_F32), (torch.bfloat16, bqd.BQD_BF16)):
            d.upload()
            r.zero_()
            y = torch.empty(T, K, dtype=kind, device="cuda")
            calls = [
                lambda: bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h, bqd.BQD_E4M3, hs, I, K, T),
                lambda: bqd.fp8_b128_gemm(down.w[0], down.dws[0], h, hs, y, code, K, I, T),
                lambda: bqd.residual_norm(y, code, K, ones, None, 0, 0, 1.0, r, r, bqd.BQD_BF16, ones, 1e-6, d.x, bqd.BQD_E4M3,
                                          d.dxs, K, T)]
            for _ in range(6):
                for call in calls:
                    call()
                    if wait:
                        torch.cuda.synchronize()
            torch.cuda.synchronize()
            got.append((y.clone(), r.clone(), d.x.clone(), d.dxs.clone()))
    for a, b in zip(got[:2], got[2:]):
        assert all(torch.equal(v.view(torch.uint8), w.view(torch.uint8)) for v, w in zip(a, b))
        assert bool(b[0].isfinite().all()) and bool(b[1].isfinite().all())


@pytest.mark.parametrize("M,T", [(72000, 33000), (36000000, 64), (400000, 6000)])
def test_outputs_past_32_bits(M, T):
    # y holds more than 2^31 elements; sampled rows and columns against the definition
    K = 16
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 0x7E, (M, K), dtype=torch.uint8, generator=g, device="cuda")
    x = torch.randint(0, 0x7E, (T, K), dtype=torch.uint8, generator=g, device="cuda")
    ws, xs = torch.rand(-(-M // 128), 1, generator=g, device="cuda"), torch.rand(1, T, generator=g, device="cuda")
    y = torch.full((T, M), -1.0, dtype=torch.bfloat16, device="cuda")
    bqd.fp8_b128_gemm(w, ws, x, xs, y, bqd.BQD_BF16, M, K, T)
    ms = torch.tensor([0, 1, 127, M // 2, M // 2 + 1, M - 2, M - 1], device="cuda")
    ts = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    wv = w[ms].view(torch.float8_e4m3fn).double() * ws[ms // 128].double()
    xv = x[ts].view(torch.float8_e4m3fn).double() * xs[0, ts].double()[:, None]
    want, tol = xv @ wv.t(), (xv @ wv.t()) * (2.0 ** -8 + 2.0 ** -15)  # codes are not negative: the sum is its magnitude
    assert bool(((y[ts][:, ms].double() - want).abs() <= tol + 1e-30).all())
    assert bool((y >= 0).all())


# gated pairs of many tokens whose rows of h are whole 16 bytes and leave as boxes, several tiles for each pair of CTAs: a
# box of one tile may still be on its way when the next tile's is made, the sooner the fewer blocks of k there are
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("I,K,T", [(1288, 16, 8200), (2048, 128, 4100), (4096, 272, 4099), (4104, 16, 2050)])
def test_ffn_outputs_of_many_tiles(I, K, T, kind):
    d = Data(I, K, T, n=2, seed=27, lo=-16, hi=-6)
    check_ffn(d, kind)
    want = None
    for _ in range(10):
        h = torch.full((T, I), 7.0, dtype=TYPES[kind][0], device="cuda")
        bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h, TYPES[kind][1], None, I, K, T)
        assert want is None or torch.equal(h, want)
        want = h


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20, 50, 200, 2500])
def test_gates_far_below_zero_keep_their_bits(T, kind):
    # one k counts: g[i] = code value * (1 + i / 2^12 of a tile's scale), u = 2^70, so that h is a normal number from g = -120
    # on. The products are exact but for one rounding each of g's scale and sum: |dg| <= 2^-22 |g|, times |SiLU'| <= |g| e^g
    # for g < -2; e^-|g| and g e are off by a step of 2^-149 where they are subnormal, the rest by 2^-20
    I, K = 1100, 16
    d = Data(I, K, T, n=2, seed=28)
    d.xc[:], d.xc[:, 3] = 0, 0x38                       # 1.0
    d.xs[:] = 1.0
    d.wc[0][:], d.wc[1][:] = 0, 0
    gates = np.array([-2, -20, -40, -64, -72, -80, -88, -96, -104, 88, 0], np.float32)
    table = {float(v): c for c, v in enumerate(ref.VALUES) if v == v}
    d.wc[0][:, 3] = [table[float(g)] for g in np.resize(gates, I)]
    d.wc[1][:, 3] = 0x38
    d.ws[0][:, 0] = 1 + np.arange(len(d.ws[0])) * np.float32(2.0 ** -12)
    d.ws[1][:] = 2.0 ** 70
    d.upload()
    h = Out((T, I), kind)
    bqd.fp8_b128_gemm_silu_mul(d.w[0], d.dws[0], d.w[1], d.dws[1], d.x, d.dxs, h.ptr, TYPES[kind][1], None, I, K, T)
    g = np.resize(gates, I).astype(np.float64) * np.repeat(d.ws[0][:, 0].astype(np.float64), 128)[:I]
    want = ref.silu(g) * 2.0 ** 70
    tol = 2.0 ** -22 * np.maximum(np.abs(g), 1) * np.abs(want) + 2.0 ** -20 * np.abs(want) + (np.abs(g) + 1) * 2.0 ** (70 - 149)
    got = h.get()
    assert (np.abs(got - want) <= tol + HALF[kind] * (np.abs(want) + tol)).all()
    assert (got[:, (g < -60) & (g > -100)] < 0).all()


BETWEEN = {"direct": (1, "nvfp4", bqd.BQD_PATH_DIRECT), "stream": (1, "nvfp4", bqd.BQD_PATH_STREAM), "mma": (8, "nvfp4", bqd.BQD_PATH_MMA),
           "tiles": (4, "nvfp4", bqd.BQD_PATH_TILES), "gemm": (64, "gemm", None)}


@pytest.mark.parametrize("between", BETWEEN)
@pytest.mark.parametrize("T", [1, 50, 300])
def test_weights_written_two_calls_before_a_dependent_launch(T, between):
    # with the flag a product may read weights while the call before it runs; that call (a GEMV that writes something
    # else) lets it start only when the one before itself, the weights' encoder, is over
    M, K, n = 2048, 4096, 5
    N, form, path = BETWEEN[between]
    d = Data(128, K, T, seed=43)
    ws = torch.full((M // 128, K // 128), 0.01, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    src = [torch.randn(M, K, generator=g, device="cuda") for _ in range(n)]
    w, sc = torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, M, device="cuda")
    nv, ns = dev(codes((256, K // 2), 44)), dev(np.full((256, K // 16), 0x38, np.uint8))
    x, o = torch.randn(N, K, device="cuda").to(torch.bfloat16), torch.empty(N, 256, device="cuda")

    def run(wait):
        out = []
        for _ in range(6):
            for s in src:
                y = torch.empty(T, M, device="cuda")
                bqd.fp8_x_encode(s, bqd.BQD_F32, K, w, sc, K, M)
                if wait:
                    torch.cuda.synchronize()
                if form == "gemm":
                    bqd.nvfp4_gemm(nv, ns, 0.01, x, o, 256, K, N)
                else:
                    bqd.nvfp4_gemv_path(nv, ns, 0.01, x, o, 256, K, N, path)
                bqd.fp8_b128_gemm(w, ws, d.x, d.dxs, y, bqd.BQD_F32, M, K, T)
                if wait:
                    torch.cuda.synchronize()
                out.append(y)
        return out
    old = bqd.set_launch_flags(bqd.BQD_LAUNCH_PDL)
    try:
        got = run(False)
        torch.cuda.synchronize()
    finally:
        bqd.set_launch_flags(old)
    assert all(torch.equal(a, b) for a, b in zip(run(True), got))
