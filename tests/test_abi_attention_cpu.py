"""Host-side argument checks of the calls around attention (no GPU): the
documented status codes, before any CUDA call."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from block_quantized_decode_nvfp4_gb300 import build
    build.build()
    import block_quantized_decode_nvfp4_gb300 as bqd
    return bqd.lib()


A, U = 0x10000, 0x10008  # aligned to 16 bytes and to 8: never dereferenced (every call fails validation or has nothing to do)


def cache(**kw):
    from block_quantized_decode_nvfp4_gb300 import KVCache
    f = dict(k=A, v=A, k_scale=None, v_scale=None, num_pages=8, page_stride=2048, token_stride=128, head_stride=64,
             page_size=16, heads=2, head_dim=64, type=1)
    f.update(kw)
    return C.byref(KVCache(*f.values()))


def test_paged_slots(L):
    def call(c=A, n=A, f=A, nf=4, t=A, R=2, W=3, page=16, d=None, o=A, s=A, p=A, cap=8, k=A):
        return L.paged_slots(c, n, f, nf, t, R, W, page, d, o, s, p, cap, k, None)
    assert call(c=None) == 1 and call(n=None) == 1 and call(f=None) == 1 and call(t=None) == 1
    assert call(o=None) == 1 and call(s=None) == 1 and call(p=None) == 1 and call(k=None) == 1
    assert call(R=-1) == 2 and call(R=1 << 24) == 2 and call(W=-1) == 2 and call(W=1 << 39) == 2
    assert call(page=0) == 2 and call(page=17) == 2 and call(page=8192) == 2
    assert call(nf=-1) == 2 and call(nf=1 << 31) == 2 and call(cap=-1) == 2 and call(cap=1 << 31) == 2
    assert call(s=A + 4) == 3 and call(c=A + 2) == 3


def test_qk_norm_rope_cache(L):
    def call(q=A, k=A, v=A, ty=0, qp=256, kp=128, vp=128, qw=A, kw=A, cs=A, P=64, rot=64, style=0, pos=A, sl=A, o=A,
             c=None, T=3, Hq=4):
        return L.qk_norm_rope_cache(q, k, v, ty, qp, kp, vp, qw, kw, 1e-6, cs, P, rot, style, pos, sl, o,
                                    c or cache(), T, Hq, None)
    assert call(q=None) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(sl=None) == 1 and call(o=None) == 1
    assert call(pos=None) == 1 and call(cs=None) == 1 and call(c=cache(k=None)) == 1
    assert call(ty=2) == 2 and call(qp=252) == 2 and call(kp=64) == 2 and call(vp=130) == 2 and call(ty=1, qp=260) == 2
    assert call(rot=80) == 2 and call(rot=24) == 2 and call(rot=-16) == 2 and call(style=2) == 2 and call(P=-1) == 2
    assert call(T=-1) == 2 and call(Hq=0) == 2
    for bad in (dict(head_dim=80), dict(page_size=24), dict(page_size=8192), dict(type=0), dict(type=3), dict(heads=0),
                dict(heads=1025), dict(num_pages=-1), dict(num_pages=1 << 40), dict(token_stride=-64),
                dict(token_stride=132), dict(type=2, head_stride=72), dict(page_stride=1 << 40)):
        assert call(c=cache(**bad)) == 2, bad
    assert call(q=U) == 3 and call(o=U) == 3 and call(c=cache(v=U)) == 3 and call(sl=A + 4) == 3 and call(cs=U) == 3
    assert call(T=0, q=None, o=None) == 0  # nothing to do


def test_tree_attention(L):
    size = L.tree_attention_workspace_bytes(2, 6, 4, 2, 64)
    assert size > 0

    def call(q=A, qp=256, c=None, t=A, W=4, ctx=A, off=A, mask=None, words=1, o=A, lse=None, ws=A, wsb=size, R=2, T=6,
             Hq=4):
        return L.tree_attention(q, qp, c or cache(), t, W, ctx, off, mask, words, 0.125, o, lse, ws, wsb, R, T, Hq, None)
    assert call(q=None) == 1 and call(t=None) == 1 and call(ctx=None) == 1 and call(off=None) == 1 and call(o=None) == 1
    assert call(qp=248) == 2 and call(qp=260) == 2 and call(Hq=3) == 2 and call(Hq=0) == 2 and call(T=-1) == 2
    assert call(R=-1) == 2 and call(W=-1) == 2 and call(mask=A, words=0) == 2 and call(T=1 << 30) == 2
    assert call(q=U) == 3 and call(o=U) == 3 and call(mask=A + 4) == 3 and call(off=A + 2) == 3
    assert call(ws=None) == 6 and call(ws=U) == 6 and call(wsb=size - 1) == 6
    assert call(T=0, q=None) == 0 and call(R=0) == 0
    assert L.tree_attention_workspace_bytes(1, 1, 130, 1, 64) == 0  # more than 64 query heads a kv head
    assert L.tree_attention_workspace_bytes(1, 1, 4, 2, 96) == 0


def test_token_logprobs(L):
    size = L.token_logprobs_workspace_bytes(3, 1000, 5)
    assert size > 0

    def call(x=A, ty=0, pitch=1000, tok=A, lp=A, ent=A, ids=A, top=A, k=5, ws=A, wsb=size, T=3, V=1000):
        return L.token_logprobs(x, ty, pitch, tok, lp, ent, ids, top, k, ws, wsb, T, V, None)
    assert call(x=None) == 1 and call(tok=None) == 1 and call(ids=None) == 1 and call(top=None) == 1
    assert call(ty=2) == 2 and call(pitch=999) == 2 and call(k=33) == 2 and call(k=-1) == 2 and call(T=-1) == 2
    assert call(V=0, k=0) == 2 and call(V=4) == 2 and call(V=1 << 31, pitch=1 << 31) == 2
    assert call(x=U) == 3 and call(lp=A + 2) == 3
    assert call(ws=None) == 6 and call(ws=U) == 6 and call(wsb=size - 1) == 6
    assert call(T=0) == 0
    assert L.token_logprobs_workspace_bytes(1, 4, 5) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (40, 8), (64, 1)])
def test_tree_attention_workspace_serves_smaller_calls(L, Hq, Hkv, D):
    # a program sizes it once, for its largest batch: a batch that shrinks to one wide draft needs no more
    sizes = [0, 1, 2, 3, 4, 7, 16, 17, 32, 33, 63, 64, 128, 129, 256, 1024, 8191]
    need = {(R, T): L.tree_attention_workspace_bytes(R, T, Hq, Hkv, D) for R in sizes[:-2] for T in sizes}
    assert all(n > 0 for n in need.values())
    for (R, T), n in need.items():
        for (r, t), m in need.items():
            assert m <= n or r > R or t > T, ((R, T, n), (r, t, m))
