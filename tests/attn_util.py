"""Shared builders of the tests around attention: a paged cache with its
tensors and fp64 values, requests of given lengths, and their checks."""
import numpy as np
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from oracle import attention as ref


class Cache:
    """Paged cache of given layout and type; `k64`, `v64` the stored values as fp64 [slots][heads][D]."""

    def __init__(self, pages, page, heads, D, kind="bf16", layout="tokens", seed=0, extra=0):
        rng = np.random.default_rng(seed)
        self.page, self.heads, self.D, self.kind, self.pages = page, heads, D, kind, pages
        shape = (pages, page, heads, D + extra)  # extra: elements between heads that belong to nobody

        def make():
            if kind == "bf16":
                t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)
            else:
                t = torch.from_numpy((40 * rng.standard_normal(shape)).astype(np.float32)).to(torch.float8_e4m3fn)
            raw = t if kind == "bf16" else t.view(torch.uint8)
            if layout == "heads":
                raw = raw.transpose(1, 2).contiguous().cuda().transpose(1, 2)
            else:
                raw = raw.cuda()
            return raw[..., :D]

        self.k, self.v = make(), make()
        self.ks = self.vs = None
        if kind == "e4m3":
            self.ks = torch.from_numpy(rng.uniform(0.01, 0.03, heads).astype(np.float32)).cuda()
            self.vs = torch.from_numpy(rng.uniform(0.01, 0.03, heads).astype(np.float32)).cuda()
        self.desc = bqd.kv_cache(self.k, self.v, self.ks, self.vs)

    def values(self, which):
        """The stored values, scaled, as fp64 [slots][heads][D]."""
        t = (self.k if which == "k" else self.v).cpu()
        t = t.double() if self.kind == "bf16" else t.contiguous().view(torch.float8_e4m3fn).double()
        t = t.reshape(-1, self.heads, self.D).numpy()
        if self.kind == "e4m3":
            t = t * (self.ks if which == "k" else self.vs).double().cpu().numpy()[:, None]
        return t


def table_for(lens, page, pages, seed=0, width=None):
    """Block table of requests of these total lengths over distinct, shuffled pages; -1 past their ends."""
    rng = np.random.default_rng(seed)
    ids = rng.permutation(pages)
    need = [-(-l // page) for l in lens]
    assert sum(need) <= pages
    width = max(need + [1]) if width is None else width
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for r, n in enumerate(need):
        table[r, :min(n, width)] = ids[at:at + min(n, width)]
        at += n
    return table


def run_attention(cache, q, table, ctx, off, mask, scale, T=None, stream=None, q_pitch=None, words=None, fill=7.0):
    T, Hq = (q.shape[0] if T is None else T), q.shape[1]
    R = len(ctx)
    out = torch.full((q.shape[0], Hq, cache.D), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], Hq), fill, dtype=torch.float32, device="cuda")
    wsb = bqd.tree_attention_workspace_bytes(R, T, Hq, cache.heads, cache.D)
    assert wsb > 0
    ws = torch.full((wsb,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing may be read unwritten
    dt = torch.from_numpy(np.ascontiguousarray(table)).cuda()
    dc = torch.tensor(list(ctx), dtype=torch.int32, device="cuda")
    do = torch.tensor(list(off), dtype=torch.int32, device="cuda")
    dm = None if mask is None else torch.from_numpy(np.ascontiguousarray(mask).view(np.int64)).cuda()
    bqd.tree_attention(q, q_pitch or Hq * cache.D, cache.desc, dt, table.shape[1], dc, do, dm,
                       words or (1 if mask is None else mask.shape[1]), scale, out, lse, ws, wsb, R, T, Hq, stream)
    torch.cuda.synchronize()
    return out, lse


def check_attention(cache, q, table, ctx, off, mask, scale, out, lse, rows=None, what=""):
    """Every (token, head) against the fp64 definition.

    |out - ref| <= 2^-8 |ref| (bf16 result) + sum p |v| (2^-8 (bf16 p) + 2 d + 2^-19 (exp2) + L 2^-23 (fp32 sums)),
    d = (D + 8) 2^-24 max sum |q k| scale: fp32 scores of exact products; |lse - ref| <= d + 2^-19 + L 2^-23 +
    2^-22 |lse|.
    """
    K, V = cache.values("k"), cache.values("v")
    qd = q.double().cpu().numpy()
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    G = q.shape[1] // cache.heads
    for r, c in enumerate(ctx):
        n = off[r + 1] - off[r]
        L = c + n
        l = np.arange(L)
        inside = l // cache.page < table.shape[1]
        pg = np.where(inside, table[r][np.minimum(l // cache.page, table.shape[1] - 1)], -1)
        good = (pg >= 0) & (pg < cache.pages)
        slot = np.where(good, pg * cache.page + l % cache.page, 0)
        for i in range(n):
            t = off[r] + i
            if rows is not None and t not in rows:
                continue
            seen = ref.seen_of(c, n, i, None if mask is None else mask[t].view(np.uint64)) & good
            for h in range(q.shape[1]):
                y, e, a, s = ref.attention(qd[t, h], K[slot, h // G], V[slot, h // G], seen, scale)
                d = (cache.D + 8) * 2.0 ** -24 * s
                tol = 2.0 ** -8 * np.abs(y) + a * (2.0 ** -8 + 2 * d + 2.0 ** -19 + L * 2.0 ** -23)
                bad = ~(np.abs(o[t, h] - y) <= tol)
                assert not bad.any(), (what, r, i, h, np.flatnonzero(bad)[:4], o[t, h][bad][:4], y[bad][:4], tol[bad][:4])
                if np.isneginf(e):
                    assert np.isneginf(z[t, h]), (what, r, i, h, z[t, h])
                else:
                    assert abs(z[t, h] - e) <= d + 2.0 ** -19 + L * 2.0 ** -23 + 2.0 ** -22 * abs(e), (what, r, i, h)


def random_tree_mask(news, seed=0, words=1):
    """Masks of random draft trees: each token sees itself and its ancestors."""
    rng = np.random.default_rng(seed)
    rows = []
    for n in news:
        m = []
        for j in range(n):
            p = int(rng.integers(max(-1, j - 6), j)) if j else -1
            m.append((m[p] if p >= 0 else 0) | (1 << j))
        for b in m:
            rows.append([(b >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)])
    return np.array(rows, np.uint64).reshape(-1, words)
