"""qk_norm_rope_cache on the GPU against the fp64 definition, and what it
leaves alone.

Tolerances: bf16 results round by at most 2^-8 |y|, E4M3 ones by 2^-4 |y| or
2^-10 (subnormal spacing 2^-9), saturating at 448; before that fp32: the mean
square (D terms), rsqrt, the weight and the rotation cost at most (D + 16)
2^-24 of the magnitudes that met, |a| + |b|."""
import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from oracle import attention as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def build(T, Hq, Hkv, D, rot, pairs=False, dtype="f32", cache="bf16", norm=True, page=16, layout="tokens", seed=0,
          gain=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    w = (Hq + 2 * Hkv) * D
    s = dict(T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, pairs=pairs, cache=cache, page=page, dtype=dtype)
    s["x"] = (gain * torch.randn(T, w + pad, generator=g)).to(dt).cuda()
    s["qw"] = (1 + 0.2 * torch.randn(D, generator=g)).cuda() if norm else None
    s["kw"] = (1 + 0.2 * torch.randn(D, generator=g)).cuda() if norm else None
    P = 501
    ang = torch.rand(P, max(rot // 2, 1), generator=g).double() * 40
    s["cs"] = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    s["pos"] = torch.randint(0, P, (T,), generator=g, dtype=torch.int32).cuda()
    pages = -(-T // page) + 3
    s["slots"] = torch.randperm(pages * page, generator=g)[:T].contiguous().cuda()
    ct = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    for n in "kv":
        c = torch.randn(pages, page, Hkv, D, generator=g).to(ct)
        c = c if cache == "bf16" else c.view(torch.uint8)
        s[n] = c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "heads" else c.cuda()
    s["ks"] = s["vs"] = None
    if cache == "e4m3":
        s["ks"] = (0.01 + 0.01 * torch.rand(Hkv, generator=g)).cuda()
        s["vs"] = (0.01 + 0.01 * torch.rand(Hkv, generator=g)).cuda()
    s["out"] = torch.full((T + 1, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    return s


def call(s, stream=None, **kw):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    item, base = s["x"].element_size(), s["x"].data_ptr()
    pitch = s["x"].shape[1]
    a = dict(q=base, k=base + Hq * D * item, v=base + (Hq + Hkv) * D * item,
             ty=bqd.BQD_F32 if s["dtype"] == "f32" else bqd.BQD_BF16, qp=pitch, kp=pitch, vp=pitch, qw=s["qw"],
             kw=s["kw"], eps=1e-5, cs=s["cs"], P=s["cs"].shape[0], rot=s["rot"],
             style=bqd.BQD_ROPE_PAIRS if s["pairs"] else bqd.BQD_ROPE_HALVES, pos=s["pos"], slots=s["slots"],
             out=s["out"], cache=bqd.kv_cache(s["k"], s["v"], s["ks"], s["vs"]), T=s["T"], Hq=Hq)
    a.update(kw)
    bqd.qk_norm_rope_cache(*a.values(), stream=stream)
    torch.cuda.synchronize()


def near(got, y, size, kind, D, what):
    err = (D + 16) * 2.0 ** -24 * size
    if kind == "bf16":
        tol = 2.0 ** -8 * np.abs(y) + 2 * err
    else:
        y = np.clip(y, -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + 2 * err
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (what, np.flatnonzero(bad)[:4], got[bad][:4], y[bad][:4])


def f64(t, kind):
    t = t.cpu().contiguous()
    return (t.double() if kind == "bf16" else t.view(torch.float8_e4m3fn).double()).numpy()


def check(s, rows=None):
    before = {n: s[n].clone() for n in "kv"}
    call(s)
    Hq, Hkv, D, rot = s["Hq"], s["Hkv"], s["D"], s["rot"]
    x = s["x"].double().cpu().numpy()
    cs = s["cs"].double().cpu().numpy()
    out = s["out"].double().cpu().numpy()
    flat = {n: f64(s[n], s["cache"]).reshape(-1, Hkv, D) for n in "kv"}
    w = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("qw", "kw")}
    for t in (range(s["T"]) if rows is None else rows):
        row, slot = cs[int(s["pos"][t])], int(s["slots"][t])
        heads = x[t, :(Hq + 2 * Hkv) * D].reshape(-1, D)
        for h in range(Hq):
            y, size = ref.norm_rope(heads[h], w["qw"], 1e-5, row, rot, s["pairs"])
            near(out[t, h], y, size, "bf16", D, ("q", t, h))
        for h in range(Hkv):
            y, size = ref.norm_rope(heads[Hq + h], w["kw"], 1e-5, row, rot, s["pairs"])
            f = 1.0 if s["ks"] is None else 1 / float(s["ks"][h])
            near(flat["k"][slot, h], y * f, size * f, s["cache"], D, ("k", t, h))
            y = heads[Hq + Hkv + h]
            f = 1.0 if s["vs"] is None else 1 / float(s["vs"][h])
            near(flat["v"][slot, h], y * f, np.abs(y * f), s["cache"], D, ("v", t, h))
    assert np.all(out[s["T"]:] == 5.0)
    used = np.zeros(flat["k"].shape[0], bool)
    used[s["slots"].cpu().numpy()] = True
    for n in "kv":  # other slots keep their bytes
        assert np.array_equal(flat[n][~used], f64(before[n], s["cache"]).reshape(-1, Hkv, D)[~used], equal_nan=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_dims_styles(D, dtype, cache, pairs):
    check(build(5, 6, 2, D, D, pairs, dtype, cache, seed=D))
    check(build(3, 3, 1, D, D // 4, pairs, dtype, cache, layout="heads", seed=D + 1))


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 80, 112, 128])
@pytest.mark.parametrize("pairs", [False, True])
def test_partial_rotation(rot, pairs):
    check(build(4, 2, 2, 128, rot, pairs, seed=rot))


@pytest.mark.parametrize("T", [1, 2, 3, 31, 33, 257])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (32, 8), (5, 5)])
def test_token_and_head_counts(T, Hq, Hkv):
    check(build(T, Hq, Hkv, 64, 64, seed=T), rows=sorted({0, T // 2, T - 1}))


def test_many_tokens():
    check(build(6000, 8, 2, 128, 64, dtype="bf16", seed=1), rows=[0, 1, 2999, 5998, 5999])


@pytest.mark.parametrize("page", [1, 2, 64, 1024])
def test_pages(page):
    check(build(9, 4, 2, 64, 64, page=page, seed=page))


def test_without_norm_and_padded_rows():
    check(build(4, 4, 2, 128, 128, norm=False, seed=2))
    check(build(4, 4, 2, 128, 128, pad=16, seed=3))


def test_e4m3_saturates():
    s = build(4, 2, 2, 64, 64, cache="e4m3", norm=False, gain=30.0, seed=4)
    check(s)
    assert (f64(s["v"], "e4m3") == 448).any()


def test_tiny_rows():
    s = build(3, 2, 1, 128, 128, seed=5)
    s["x"][1] = 0  # a zero head: 0 * rsqrt(eps) = 0
    s["x"][2] *= 1e-4
    check(s)


def test_padding_tokens_are_not_stored():
    s = build(6, 4, 2, 64, 64, seed=6)
    want = {n: s[n].clone() for n in "kv"}
    cap = s["k"].shape[0] * 16
    s["slots"][:] = torch.tensor([-1, cap, cap + 5, -7, 1 << 40, -(1 << 40)])
    call(s)
    assert all(torch.equal(s[n], want[n]) for n in "kv")
    assert (s["out"][:6].float().abs().sum((1, 2)) > 0).all()  # q does not need a slot
    s = build(3, 4, 2, 64, 64, seed=7)
    want = {n: s[n].clone() for n in "kv"}
    s["pos"][:] = torch.tensor([-1, 501, 2147483647], dtype=torch.int32)
    call(s)
    assert all(torch.equal(s[n], want[n]) for n in "kv") and torch.all(s["out"][:3] == 0)


def test_no_rotation_needs_no_positions():
    s = build(3, 4, 2, 64, 0, seed=8)
    call(s, pos=None, cs=None, P=0)
    a = s["out"].clone()
    call(s)
    assert torch.equal(a, s["out"])


def test_side_stream_and_same_bits():
    s = build(40, 8, 2, 128, 128, cache="e4m3", seed=9)
    call(s)
    a = [s[n].clone() for n in ("out", "k", "v")]
    call(s, stream=torch.cuda.Stream())
    assert all(torch.equal(x.view(torch.uint8), s[n].view(torch.uint8)) for x, n in zip(a, ("out", "k", "v")))


def test_slots_past_32_bits_of_elements():
    Hkv, D, page = 2, 128, 16
    pages = (1 << 31) // (page * Hkv * D) + 8
    s = build(4, 2, Hkv, D, D, seed=10)
    call(s)
    kv = [s["k"].view(-1, Hkv, D)[s["slots"]].clone(), s["v"].view(-1, Hkv, D)[s["slots"]].clone()]
    s["k"] = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    s["v"] = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    s["slots"] = pages * page - 1 - torch.arange(4, device="cuda") * 3
    call(s)
    for n, want in zip("kv", kv):
        assert torch.equal(s[n].view(-1, Hkv, D)[s["slots"]], want)


def test_refusals():
    s = build(2, 4, 2, 64, 64)
    call(s)
    x = s["x"].data_ptr()
    for status, kw in [(1, dict(q=None)), (1, dict(v=None)), (1, dict(slots=None)), (1, dict(out=None)),
                       (1, dict(pos=None)), (1, dict(cs=None)), (2, dict(ty=2)), (2, dict(ty=9)), (2, dict(qp=255)),
                       (2, dict(kp=126)), (2, dict(vp=130)), (2, dict(rot=8)), (2, dict(rot=80)), (2, dict(rot=-16)),
                       (2, dict(style=2)), (2, dict(T=-1)), (2, dict(Hq=0)), (2, dict(P=-1)), (3, dict(q=x + 4)),
                       (3, dict(out=s["out"].data_ptr() + 2)), (3, dict(cs=s["cs"].data_ptr() + 4))]:
        with pytest.raises(bqd.BqdError) as e:
            call(s, **kw)
        assert e.value.status == status, kw
    call(s, T=0)
    with pytest.raises(ValueError):
        bqd.kv_cache(s["k"], s["v"].transpose(1, 2))
    with pytest.raises(ValueError):
        bqd.kv_cache(s["k"].float(), s["v"].float())


@pytest.mark.parametrize("which", ["k", "v"])
def test_e4m3_stores_the_quotient_by_the_scale(which):
    # x = m * scale, exact in fp32, with m halfway between two neighbours: the quotient is m, and goes to the even one;
    # a product with the rounded reciprocal may land beside m
    mid = [(1 + (2 * i + 1) / 16) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1]
    mid += [2.0 ** -10, 3 * 2.0 ** -10]
    m = torch.tensor((mid + [-v for v in mid] + [0.0] * 256)[:256]).view(4, 64)
    scales = [n / 512 for n in (1, 3, 7, 13, 41, 47, 55, 61)]
    s = build(4, 1, 8, 64, 0, cache="e4m3", norm=False)
    s["ks"] = s["vs"] = torch.tensor(scales).cuda()
    x = m[:, None, :] * torch.tensor(scales)[None, :, None]
    assert torch.equal(x.double() / torch.tensor(scales).double()[None, :, None],
                       m.double()[:, None, :].expand(4, 8, 64))
    at = 64 * (1 if which == "k" else 9)
    s["x"][:, at:at + 512] = x.reshape(4, 512).cuda()
    call(s)
    got = f64(s[which], "e4m3").reshape(-1, 8, 64)[s["slots"].cpu().numpy()]
    want = m.to(torch.float8_e4m3fn).double().numpy()
    for h, scale in enumerate(scales):
        assert np.array_equal(got[:, h], want), (scale, np.argwhere(got[:, h] != want)[:4])


def test_e4m3_codes_are_those_of_fp32_quotients():
    scales = torch.tensor([0.0137, 1.7e-3, 1.0, 331.7, 1.3 * 2.0 ** -64, 1.1 * 2.0 ** 70, 1e-38, -0.021])
    T, g = 700, torch.Generator().manual_seed(11)
    s = build(T, 1, 8, 64, 0, cache="e4m3", norm=False)
    s["ks"] = s["vs"] = scales.cuda()
    m = torch.exp2(torch.rand(T, 8, 64, generator=g) * 22 - 12)
    m = m * torch.where(torch.rand(T, 8, 64, generator=g) < 0.5, 1, -1)
    x = m * scales[None, :, None]
    inf = float("inf")
    x[0, :, :8] = torch.tensor([inf, -inf, float("nan"), 3.4e38, -3.4e38, 0.0, -0.0, 1e-45])
    s["x"][:, 64 * 9:64 * 17] = x.reshape(T, 512).cuda()
    call(s)
    got = f64(s["v"], "e4m3").reshape(-1, 8, 64)[s["slots"].cpu().numpy()]
    want = (x / scales[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    for h in range(8):
        bad = ~((got[:, h] == want[:, h]) | (np.isnan(got[:, h]) & np.isnan(want[:, h])))
        assert not bad.any(), (float(scales[h]), x[:, h].numpy()[bad][:4], got[:, h][bad][:4], want[:, h][bad][:4])
