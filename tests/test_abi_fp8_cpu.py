"""Host-side argument checks of the calls on 8-bit activations (no GPU): the
documented status codes, before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def L():
    from block_quantized_decode_nvfp4_gb300 import build
    build.build()
    import block_quantized_decode_nvfp4_gb300 as bqd
    return bqd.lib()


A, U = 0x10000, 0x10008  # aligned to 16 bytes and to 8: never dereferenced (every call fails validation or has nothing to do)
F32, BF16, E4M3 = 0, 1, 2


def test_fp8_x_encode(L):
    def call(x=A, ty=BF16, pitch=256, c=A, s=A, K=256, T=3):
        return L.fp8_x_encode(x, ty, pitch, c, s, K, T, None)
    assert call(x=None) == 1 and call(c=None) == 1 and call(s=None) == 1
    assert call(ty=E4M3) == 2 and call(ty=-1) == 2 and call(pitch=248) == 2 and call(pitch=260) == 2
    assert call(pitch=1 << 31) == 2 and call(K=250) == 2 and call(K=-16) == 2 and call(T=-1) == 2
    assert call(K=(1 << 24) + 16, pitch=1 << 25) == 2 and call(T=(1 << 30) + 1) == 2
    assert call(K=1 << 24, pitch=1 << 24, T=1 << 20) == 2  # K T past 2^40
    assert call(x=U) == 3 and call(c=U) == 3 and call(s=U) == 3
    assert call(T=0, x=None) == 0 and call(K=0, c=None) == 0


def test_residual_norm(L):
    def call(x=A, xt=F32, xp=256, pw=A, g=A, gt=BF16, gp=256, sc=1.0, r=A, ro=A, rt=BF16, w=A, eps=1e-6, y=A, yt=BF16,
             ys=None, H=256, T=3):
        return L.residual_norm(x, xt, xp, pw, g, gt, gp, sc, r, ro, rt, w, eps, y, yt, ys, H, T, None)
    assert call(x=None, r=None, pw=None, g=None) == 1 and call(x=None) == 1 and call(x=None, g=None) == 1
    assert call(y=None, ro=None) == 1 and call(w=None) == 1 and call(yt=E4M3) == 1
    assert call(xt=E4M3) == 2 and call(gt=E4M3) == 2 and call(rt=E4M3) == 2 and call(yt=F32) == 2 and call(yt=3) == 2
    assert call(xp=240) == 2 and call(xp=258) == 2 and call(gp=128) == 2 and call(gp=260) == 2 and call(gp=-8) == 2
    assert call(xp=1 << 31) == 2 and call(gp=1 << 31) == 2 and call(H=250) == 2 and call(H=0) == 2
    assert call(H=16400, xp=16400, gp=0) == 2 and call(T=-1) == 2 and call(eps=-1.0) == 2 and call(eps=float("nan")) == 2
    for k in ("x", "pw", "g", "r", "ro", "w", "y"):
        assert call(**{k: U}) == 3, k
    assert call(yt=E4M3, ys=U) == 3
    assert call(T=0, x=None, r=None, pw=None, g=None) == 0


def test_fp8_b128_gemm(L):
    def call(c=A, s=A, x=A, xs=A, y=A, ty=F32, M=256, K=256, T=3):
        return L.fp8_b128_gemm(c, s, x, xs, y, ty, M, K, T, None)
    for k in ("c", "s", "x", "xs", "y"):
        assert call(**{k: None}) == 1 and call(**{k: U}) == 3, k
    assert call(ty=E4M3) == 2 and call(K=250) == 2 and call(K=0) == 2 and call(K=-16) == 2 and call(M=-1) == 2
    assert call(T=-1) == 2 and call(K=(1 << 24) + 16) == 2 and call(M=(1 << 30) + 1) == 2 and call(T=(1 << 30) + 1) == 2
    assert call(M=1 << 30, T=1 << 30) == 2
    assert call(M=0, c=None) == 0 and call(T=0, y=None) == 0


def test_fp8_b128_gemm_silu_mul(L):
    def call(gc=A, gs=A, uc=A, us=A, x=A, xs=A, h=A, ty=E4M3, hs=A, I=256, K=256, T=3):
        return L.fp8_b128_gemm_silu_mul(gc, gs, uc, us, x, xs, h, ty, hs, I, K, T, None)
    for k in ("gc", "uc", "x", "xs", "h", "hs"):
        assert call(**{k: None}) == 1 and call(**{k: U}) == 3, k
    for k in ("gs", "us"):  # halves of a fused weight's scales start at any fp32
        assert call(**{k: None}) == 1 and call(**{k: A + 2}) == 3, k
    assert call(ty=3) == 2 and call(K=250) == 2 and call(K=0) == 2 and call(I=-1) == 2 and call(T=-1) == 2
    assert call(I=0, gc=None) == 0 and call(T=0, h=None) == 0


def test_a_tensor_of_another_device_is_refused(L):
    import torch
    import block_quantized_decode_nvfp4_gb300 as bqd
    t = torch.zeros(16)
    if torch.cuda.is_available():
        with pytest.raises(ValueError):
            bqd.fp8_x_encode(t, F32, 16, t, t, 16, 1)
