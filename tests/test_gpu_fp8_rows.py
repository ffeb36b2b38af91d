"""fp8_x_encode and residual_norm against their fp64 definitions."""
import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from oracle import fp8 as ref
from tests.fp8_util import HALF, TYPES, Out, check_codes, rows, to_type
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def run_encode(x, kind, T, K, pitch=None):
    c, s = Out((T, K), "e4m3"), Out((-(-K // 128), T), "f32")
    bqd.fp8_x_encode(x, TYPES[kind][1], pitch or K, c.ptr, s.ptr, K, T)
    return c.get(), s.get().astype(np.float32)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (1, 4096), (3, 144), (4, 256), (5, 1008), (17, 2064), (130, 512),
                                 (257, 112), (33, 12288)])
def test_encode_is_exact(kind, T, K):
    x, v = to_type(rows(T, K, T * 31 + K), kind)
    c, s = run_encode(x, kind, T, K)
    wc, wsc = ref.encode(v.astype(np.float32))
    assert np.array_equal(s, wsc) and np.array_equal(c, wc)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_encode_borders_between_codes(kind):
    # amax 7 * 2^j makes the scale a power of two, and the values lie on and beside the borders between codes
    grid = ref.VALUES[:0x7F]
    mids = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1e9))])
    n = -(-len(near) // 127)
    x = np.zeros((n, 128), np.float32)
    x[:, 0] = 448
    x[:, 1:] = np.resize(near, (n, 127)) * np.where(np.arange(127) % 2, 1, -1)
    x = np.concatenate([x * np.float32(2.0 ** e) for e in (-100, -62, -60, -30, 0, 5, 40, 100)])
    t, v = to_type(x, kind)
    c, s = run_encode(t, kind, *x.shape)
    wc, wsc = ref.encode(v.astype(np.float32))
    assert np.array_equal(s, wsc) and np.array_equal(c, wc)


def test_encode_small_large_and_bad_blocks():
    x = rows(9, 384, 3)
    x[0] = 0
    x[1] *= np.float32(2.0 ** -125)      # subnormal values: the scale stops at 2^-126
    x[2] = np.float32(2.0 ** -149)
    x[3] *= np.float32(2.0 ** 110)
    x[4, 7] = np.nan                     # spoils its block alone
    x[5, 200] = -np.inf
    x[6] = np.float32(3.4e38)
    x[7] *= np.float32(2.0 ** -70)       # scales below 2^-60
    t, v = to_type(x, "f32")
    c, s = run_encode(t, "f32", 9, 384)
    wc, wsc = ref.encode(v.astype(np.float32))
    assert np.array_equal(s, wsc, equal_nan=True) and np.array_equal(c, wc)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_encode_keeps_the_sign_of_zeros(kind):
    x = rows(6, 400, 11)
    x[:, 1::3] = -0.0
    x[:, 2::5] = 0.0
    x[1] *= np.float32(2.0 ** -80)       # by division
    x[2] = -0.0                          # nothing but zeros: the smallest scale
    x[3, :256] = 0.0
    x[4] *= np.float32(2.0 ** 100)
    t, v = to_type(x, kind)
    c, s = run_encode(t, kind, 6, 400)
    wc, wsc = ref.encode(v.astype(np.float32))
    assert (wc == 0x80).sum() > 400
    assert np.array_equal(s, wsc) and np.array_equal(c, wc)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_encode_of_a_slice_of_wider_rows(kind):
    x, v = to_type(rows(37, 1024, 5), kind)
    c, s = run_encode(x[:, 256:].data_ptr(), kind, 37, 272, pitch=1024)
    wc, wsc = ref.encode(v[:, 256:528].astype(np.float32))
    assert np.array_equal(s, wsc) and np.array_equal(c, wc)


def norm_case(T, H, x="f32", res="bf16", post=True, gate="full", gate_type="bf16", y="e4m3", scale=0.75, eps=1e-6, seed=0,
              pitch=None, in_place=False, y_out=True, r_out=True, pre=None):
    """One call, checked against the definition. Bounds: a row's sum of squares is added up in fp32 in chains of
    at most 8 pair sums a thread and a tree of 11, each rounding half a step, then a division, a sum, rsqrtf (2 units)
    and products: less than 2^-19 of the norm. z carries that and 4 roundings, r one more of itself, and y what r
    carries, r's own norm and 3 roundings."""
    rng = np.random.default_rng(seed)
    p = pitch or H
    xt = xv = gt = gv = None
    if x:
        xt, xv = to_type(rows(T, p, seed + 1), x)
        xv = xv[:, :H]
    if gate != "none":
        gt, gv = to_type(rng.random((T if gate == "full" else 1, p)).astype(np.float32), gate_type)
        gv = gv[:, :H]
    pw = to_type(1 + 0.2 * rng.standard_normal(H).astype(np.float32), "f32") if post else (None, None)
    w = to_type(1 + 0.2 * rng.standard_normal(H).astype(np.float32), "f32")
    rt = rv = None
    ro = Out((T, H), res)
    if res and in_place != "absent":
        rt, rv = to_type(4 * rows(T, H, seed + 2), res)
        if in_place:
            ro.buf[256:256 + ro.n] = rt.contiguous().view(torch.uint8).flatten()
            rt = ro.ptr
    yo, ys = Out((T, H), y), Out((-(-H // 128), T), "f32")
    bqd.residual_norm(xt, TYPES[x or "f32"][1], p, pw[0], gt, TYPES[gate_type][1], p if gate == "full" else 0, scale, rt,
                      ro.ptr if r_out else None, TYPES[res][1], w[0] if y_out else None, eps, yo.ptr if y_out else None,
                      TYPES[y][1], ys.ptr if y == "e4m3" and y_out else None, H, T)
    z, r, yv = ref.residual_norm(xv, rv, pw[1], gv, scale, w[1] if y_out else None, eps)
    dz = np.zeros_like(r) if z is None else np.abs(z) * (2.0 ** -19 + 4 * 2.0 ** -24)
    dr = dz + np.abs(r) * 2.0 ** -24
    got = ro.get()
    if r_out:
        assert (np.abs(got - r) <= dr + HALF[res] * (np.abs(r) + dr) + 1e-40).all(), "residual"
    else:
        assert np.array_equal(ro.buf.cpu().numpy(), np.full(ro.n + 512, 0x5A, np.uint8))
    if not y_out:
        return
    norm = np.sqrt((r * r).mean(1, keepdims=True) + eps)
    dy = np.abs(w[1]) / norm * dr + np.abs(yv) * (np.sqrt((dr * dr).mean(1, keepdims=True)) / norm + 2.0 ** -19 + 2.0 ** -22)
    if y == "e4m3":
        check_codes(yo.get(), ys.get().astype(np.float32), yv, dy, "y")
    else:
        assert (np.abs(yo.get() - yv) <= dy + HALF[y] * (np.abs(yv) + dy) + 1e-40).all(), "y"


@pytest.mark.parametrize("y", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,H", [(1, 16), (1, 128), (9, 240), (3, 256), (5, 272), (2, 512), (7, 1008), (4, 1024), (1, 2048),
                                 (130, 2064), (33, 4096), (2, 5120), (3, 8192), (2, 8208), (3, 16384)])
def test_norm_sizes(T, H, y):
    norm_case(T, H, y=y, seed=H + T)


@pytest.mark.parametrize("x,res,gate_type", [("f32", "f32", "f32"), ("bf16", "f32", "bf16"), ("f32", "bf16", "f32"),
                                             ("bf16", "bf16", "bf16")])
@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "row"), (False, "full"), (True, "none")])
@pytest.mark.parametrize("y", ["bf16", "e4m3"])
def test_norm_types_and_forms(x, res, gate_type, post, gate, y):
    norm_case(6, 528, x=x, res=res, gate_type=gate_type, post=post, gate=gate, y=y, seed=11)


@pytest.mark.parametrize("H", [144, 4096])
def test_norm_of_slices_and_in_place(H):
    norm_case(19, H, pitch=H + 64, in_place=True, seed=2)
    norm_case(19, H, x="bf16", res="f32", pitch=2 * H, in_place=True, y="bf16", seed=3)


def test_norm_without_parts():
    norm_case(5, 272, in_place="absent", seed=4)                        # no residual: the first block
    norm_case(5, 272, x=None, post=False, gate="none", seed=5)          # only the norm of the residual
    norm_case(5, 272, y_out=False, seed=6)                              # only the residual: the last block
    norm_case(5, 272, r_out=False, seed=7)
    norm_case(5, 272, scale=-1.5, seed=8)
    norm_case(5, 272, scale=0.0, seed=9)
    norm_case(5, 272, eps=0.1, seed=10)


def test_norm_of_zero_rows_and_bad_values():
    T, H = 4, 256
    x = torch.zeros(T, H, device="cuda")
    x[1, 130] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 1.0
    w = torch.ones(H, device="cuda")
    y, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(2, T, device="cuda")
    r = torch.empty(T, H, device="cuda")
    bqd.residual_norm(x, bqd.BQD_F32, H, None, None, 0, 0, 1.0, None, r, bqd.BQD_F32, w, 1e-6, y, bqd.BQD_E4M3, s, H, T)
    assert torch.equal(r.nan_to_num(5.0, 6.0), x.nan_to_num(5.0, 6.0))
    y, s = y.cpu(), s.cpu()
    assert (y[0] == 0).all() and (s[:, 0] == 2.0 ** -126).all()
    assert (y[1] == 0x7F).all() and s[:, 1].isnan().all()  # a NaN takes its row's norm with it
    assert (y[2, :128] == 0x7F).all() and s[0, 2].isnan()   # inf * 0; the others of its row are 0
    assert (y[3] == 0x7E).all()


def test_calls_are_the_same_twice_and_on_other_streams():
    x = torch.randn(300, 4096, device="cuda")
    out = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            c, s = torch.empty(300, 4096, dtype=torch.uint8, device="cuda"), torch.empty(32, 300, device="cuda")
            bqd.fp8_x_encode(x, bqd.BQD_F32, 4096, c, s, 4096, 300)
        stream.synchronize()
        out.append((c, s))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_rows_past_32_bits():
    # more than 2^31 elements in and out: the last rows are as alone
    T, H = 140000, 16384
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(3, H, device="cuda").to(torch.bfloat16)
    x[-3:] = last
    w = torch.ones(H, device="cuda")
    c, s = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(H // 128, T, device="cuda")
    bqd.fp8_x_encode(x, bqd.BQD_BF16, H, c, s, H, T)
    cl, sl = torch.empty(3, H, dtype=torch.uint8, device="cuda"), torch.empty(H // 128, 3, device="cuda")
    bqd.fp8_x_encode(last, bqd.BQD_BF16, H, cl, sl, H, 3)
    assert torch.equal(c[-3:], cl) and torch.equal(s[:, -3:], sl) and not bool(c[:-3].any())
    r = torch.empty_like(x)
    bqd.residual_norm(x, bqd.BQD_BF16, H, None, None, 0, 0, 1.0, None, r, bqd.BQD_BF16, w, 1e-6, c, bqd.BQD_E4M3, s, H, T)
    bqd.residual_norm(last, bqd.BQD_BF16, H, None, None, 0, 0, 1.0, None, None, bqd.BQD_BF16, w, 1e-6, cl, bqd.BQD_E4M3, sl,
                      H, 3)
    assert torch.equal(c[-3:], cl) and torch.equal(s[:, -3:], sl) and torch.equal(r[-3:], last) and not bool(c[:-3].any())


def test_a_tensor_of_the_host_is_refused():
    t = torch.zeros(16)
    d = torch.zeros(16, device="cuda")
    for x, c, y in ((t, d, d), (d, t, d), (d, d, t)):
        with pytest.raises(ValueError):
            bqd.fp8_x_encode(x, bqd.BQD_F32, 16, c, y, 16, 1)
    with pytest.raises(bqd.BqdError) as e:
        bqd.fp8_x_encode(d, bqd.BQD_F32, 16, d, d, 20, 1)
    assert e.value.status == 2


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [16, 144, 272, 4112, 8224])
def test_bad_weights_spoil_their_own_channels(H, bad):
    # weights of a few channels are no numbers: what they meet is none, the other blocks are as without them
    T, at = 9, [0, 5]
    x, _ = to_type(rows(T, H, H, spread=2), "f32")
    w = torch.ones(H, device="cuda")

    def run(post, pre):
        y, s = Out((T, H), "e4m3"), Out((-(-H // 128), T), "f32")
        r = Out((T, H), "f32")
        bqd.residual_norm(x, bqd.BQD_F32, H, post, None, 0, 0, 1.0, None, r.ptr, bqd.BQD_F32, pre, 1e-6, y.ptr, bqd.BQD_E4M3,
                          s.ptr, H, T)
        return y.get(), s.get(), r.get()
    v = w.clone()
    v[at] = bad
    y, s, r = run(None, w)
    by, bs, br = run(None, v)
    assert np.array_equal(br, r)
    assert (by[:, :128] == 0x7F).all() and np.isnan(bs[0]).all()
    assert np.array_equal(by[:, 128:], y[:, 128:]) and np.array_equal(bs[1:], s[1:])
    # the norm after the block: its bad channels enter the sum of squares; infinite ones leave zeros beside them
    y, s, r = run(w, w)
    by, bs, br = run(v, w)
    keep = np.ones(H, bool)
    keep[at] = False
    assert np.array_equal(br[:, keep], r[:, keep]) and not np.isfinite(br[:, ~keep]).any()
    assert (by[:, :128] == 0x7F).all() and np.isnan(bs[0]).all()
    if np.isnan(bad):
        assert (by == 0x7F).all() and np.isnan(bs).all()
    else:
        assert ((by[:, 128:] & 0x7F) == 0).all() and (bs[1:] == 2.0 ** -126).all()
