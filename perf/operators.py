"""The operators around attention in a decode or speculative-verify step, as cases to measure.

Four operators, in the order a step calls them:
 - slots: block table, cache slots and positions of a step's new tokens, from the requests' lengths;
 - qkrope: RMS norm of each query and key head, rotary positions, and the write of K and V into the paged cache;
 - attn: attention of drafted tokens (a chain or a tree) over the paged cache;
 - logprobs: log probability of given tokens, entropy and the top alternatives of each logits row.

Each has a plain form in elementary torch operations (32-bit arithmetic, rounded once), the framework's call (`own`),
and `exact`, the definition in 64 bits written apart from the plain form.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small batch: a launch's latency is all there is
        dict(name="slots_decode_8", op="slots", R=8, n=1, ctx=2000, page=16, tree=False),
        # a full server batch that appends ragged drafts and prompt chunks of up to 64 tokens
        dict(name="slots_chunks_1024", op="slots", R=1024, n=64, ctx=30000, page=16, tree=True),
        # one token of one request: fp32 rows as the GEMV leaves them, bf16 cache
        dict(name="qkrope_decode_1", op="qkrope", T=1, Hq=32, Hkv=8, D=128, rot=128, pairs=False, dtype="f32",
             cache="bf16", norm=True, page=16),
        # 16 requests verifying 8 drafted tokens each, 8-bit cache
        dict(name="qkrope_verify_128", op="qkrope", T=128, Hq=64, Hkv=8, D=128, rot=128, pairs=False, dtype="f32",
             cache="e4m3", norm=True, page=16),
        # a prompt of 8191 tokens, wide heads with a partial rotation
        dict(name="qkrope_prompt_8191", op="qkrope", T=8191, Hq=16, Hkv=2, D=256, rot=64, pairs=False, dtype="bf16",
             cache="bf16", norm=True, page=64),
        # single-token decode of one short conversation
        dict(name="attn_decode_1", op="attn", R=1, n=1, ctx=1023, Hq=32, Hkv=8, D=128, cache="bf16", page=16,
             tree=False),
        # 16 requests verifying 8 drafted tokens each
        dict(name="attn_verify_16x8", op="attn", R=16, n=8, ctx=8192, Hq=32, Hkv=8, D=128, cache="bf16", page=16,
             tree=True),
        # single-token decode of a batch over an 8-bit cache
        dict(name="attn_decode_64_e4m3", op="attn", R=64, n=1, ctx=8192, Hq=64, Hkv=8, D=128, cache="e4m3", page=64,
             tree=False),
        # four long contexts, each with a draft tree of 64 tokens: 512 query rows share a kv head
        dict(name="attn_tree_64_long", op="attn", R=4, n=64, ctx=32768, Hq=64, Hkv=8, D=128, cache="bf16", page=64,
             tree=True),
        # the answer of one decode step over the LM head's 151936 logits
        dict(name="logprobs_decode_1", op="logprobs", T=1, V=151936, k=20, dtype="f32"),
        # 16 requests x 8 drafted tokens
        dict(name="logprobs_verify_128", op="logprobs", T=128, V=151936, k=8, dtype="f32"),
        # scoring a long prompt, bf16 logits
        dict(name="logprobs_prompt_2047", op="logprobs", T=2047, V=151936, k=5, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["slots", "qkrope", "attn", "attn", "logprobs"])
    if op == "slots":
        return dict(op=op, R=_log_int(rng, 1, 1024), n=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 30000),
                    page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.5)
    if op == "qkrope":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
        most = 8191 * (16 + 2 * 2) * 256 // ((Hq + 2 * Hkv) * D)  # no more rows than the largest listed case
        return dict(op=op, T=_log_int(rng, 1, max(1, min(16384, most // 2))), Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2, D // 4]), pairs=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]),
                    cache=rng.choice(["bf16", "e4m3"]), norm=rng.random() < 0.8, page=rng.choice([16, 64]))
    if op == "attn":
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8])
        R = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, 64)
        most = 4 * 64 * 32768 * 64 * 128 // (R * n * Hq * D)   # no more products than the largest listed case,
        most = min(most, 64 * 8192 * 8 * 128 // (R * Hkv * D))  # no more cache than the batched ones
        return dict(op=op, R=R, n=n, ctx=_log_int(rng, 1, max(1, min(32768, most))), Hq=Hq, Hkv=Hkv, D=D,
                    cache=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.5)
    V = _log_int(rng, 1000, 262144)
    return dict(op=op, T=_log_int(rng, 1, min(2047, max(1, 2047 * 151936 // (2 * V)))), V=V, k=rng.randint(0, 32),
                dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------- lengths and trees (host)
def _lens(case):
    """Context and new-token counts of each request: ragged, the same for every seed."""
    r = random.Random(case["R"] * 1000003 + case["ctx"] * 101 + case["n"])
    ctx = [case["ctx"]] + [r.randint(case["ctx"] // 2, case["ctx"]) for _ in range(case["R"] - 1)]
    new = [case["n"]] + [r.randint((case["n"] + 1) // 2, case["n"]) for _ in range(case["R"] - 1)]
    return ctx, new


def _trees(new, seed):
    """A random draft tree per request: depth of each token and the bits of the tokens it sees (itself, its ancestors)."""
    r = random.Random(seed)
    depth, mask = [], []
    for n in new:
        d, m = [], []
        for j in range(n):
            p = r.randint(max(-1, j - 8), j - 1)
            d.append(0 if p < 0 else d[p] + 1)
            m.append((0 if p < 0 else m[p]) | (1 << j))
        depth += d
        mask += [b - (1 << 64) if b >= 1 << 63 else b for b in m]
    return depth, mask


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=dtype)

    if op == "slots":
        ctx, new = _lens(case)
        p = case["page"]
        have = [-(-c // p) for c in ctx]
        need = [-(-(c + n) // p) - h for c, n, h in zip(ctx, new, have)]
        width = max(h + n for h, n in zip(have, need)) + 3
        ids = torch.randperm(sum(have) + sum(need) + 8, generator=g, device=DEV).to(torch.int32)
        hv = torch.tensor(have, device=DEV)
        cols = torch.arange(width, device=DEV)[None]
        first = (torch.cumsum(hv, 0) - hv)[:, None]
        table = torch.where(cols < hv[:, None], ids[(first + cols).clamp(max=ids.numel() - 1)], -1).to(torch.int32)
        T = sum(new)
        s.update(ctx=_i32(ctx), new=_i32(new), free=ids[sum(have):].contiguous(), table=table.contiguous(), T=T,
                 cap=T + 5, depths=None)
        if case["tree"]:
            s["depths"] = _i32(_trees(new, seed)[0] + [0] * 5)
    elif op == "qkrope":
        T, Hq, Hkv, D, p = case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["qkv"] = randn(T, (Hq + 2 * Hkv) * D).to(dt)  # one row per token as a fused projection leaves it
        s["qw"] = 1 + 0.1 * randn(D) if case["norm"] else None
        s["kw"] = 1 + 0.1 * randn(D) if case["norm"] else None
        P = max(4096, T)
        rot = case["rot"]
        f = torch.pow(torch.tensor(1e6, dtype=torch.float64, device=DEV),
                      -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        a = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * f[None]
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        s["pos"] = torch.randint(0, P, (T,), generator=g, device=DEV, dtype=torch.int32)
        pages = -(-T // p) + 4
        s["slots"] = torch.randperm(pages * p, generator=g, device=DEV)[:T].contiguous()
        ct = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
        s["k"] = randn(pages, p, Hkv, D).to(ct)
        s["v"] = randn(pages, p, Hkv, D).to(ct)
        s["ks"] = s["vs"] = None
        if case["cache"] == "e4m3":
            s["ks"] = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
            s["vs"] = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
    elif op == "attn":
        ctx, new = _lens(case)
        p, Hq, Hkv, D = case["page"], case["Hq"], case["Hkv"], case["D"]
        npg = [-(-(c + n) // p) for c, n in zip(ctx, new)]
        width = max(npg) + 1
        pages = sum(npg) + 2
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        nv = torch.tensor(npg, device=DEV)
        cols = torch.arange(width, device=DEV)[None]
        first = (torch.cumsum(nv, 0) - nv)[:, None]
        s["table"] = torch.where(cols < nv[:, None], ids[(first + cols).clamp(max=pages - 1)], -1).to(torch.int32)
        T = sum(new)
        s["T"] = T
        s["ctx"] = _i32(ctx)
        s["off"] = _i32([0] + list(np.cumsum(new)))
        s["q"] = (2 * randn(T, Hq, D)).to(torch.bfloat16)  # scores of a few units, as after a norm with weights
        s["ks"] = s["vs"] = None
        if case["cache"] == "bf16":
            s["k"] = randn(pages, p, Hkv, D, dtype=torch.bfloat16)
            s["v"] = randn(pages, p, Hkv, D, dtype=torch.bfloat16)
        else:
            s["k"] = (randn(pages, p, Hkv, D, dtype=torch.bfloat16) * 64).to(torch.float8_e4m3fn)
            s["v"] = (randn(pages, p, Hkv, D, dtype=torch.bfloat16) * 64).to(torch.float8_e4m3fn)
            s["ks"] = (1 + 0.2 * torch.rand(Hkv, generator=g, device=DEV)) / 64
            s["vs"] = (1 + 0.2 * torch.rand(Hkv, generator=g, device=DEV)) / 64
        s["scale"] = 1.0 / math.sqrt(D)
        s["mask"] = None
        if case["tree"]:
            s["mask"] = torch.tensor(_trees(new, seed)[1], dtype=torch.int64, device=DEV)[:, None].contiguous()
    else:
        T, V = case["T"], case["V"]
        x = randn(T, V) * 2.5
        s["x"] = x if case["dtype"] == "f32" else x.to(torch.bfloat16)
        s["tok"] = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what a program keeps from step to step: output buffers, workspaces, the cache's descriptor
        import block_quantized_decode_nvfp4_gb300 as bqd
        s["bqd"] = bqd
        op = case["op"]
        if op == "slots":
            s["off"] = torch.empty(case["R"] + 1, dtype=torch.int32, device=DEV)
            s["slots"] = torch.empty(s["cap"], dtype=torch.int64, device=DEV)
            s["pos"] = torch.empty(s["cap"], dtype=torch.int32, device=DEV)
            s["counts"] = torch.empty(4, dtype=torch.int32, device=DEV)
        elif op == "qkrope":
            s["cache"] = bqd.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
            s["q_out"] = torch.empty(case["T"], case["Hq"], case["D"], dtype=torch.bfloat16, device=DEV)
        elif op == "attn":
            s["cache"] = bqd.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
            s["out"] = torch.empty(s["T"], case["Hq"], case["D"], dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(s["T"], case["Hq"], dtype=torch.float32, device=DEV)
            s["wsb"] = bqd.tree_attention_workspace_bytes(case["R"], s["T"], case["Hq"], case["Hkv"], case["D"])
            s["ws"] = torch.empty(max(16, s["wsb"]), dtype=torch.uint8, device=DEV)
        else:
            T, k = case["T"], case["k"]
            s["lp"] = torch.empty(T, dtype=torch.float32, device=DEV)
            s["ent"] = torch.empty(T, dtype=torch.float32, device=DEV)
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["tlp"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
            s["wsb"] = bqd.token_logprobs_workspace_bytes(T, case["V"], k)
            s["ws"] = torch.empty(max(16, s["wsb"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _RUN[s["case"]["op"], bool(own)](s)


def _slots_own(s):
    c = s["case"]
    s["bqd"].paged_slots(s["ctx"], s["new"], s["free"], s["free"].numel(), s["table"], c["R"], s["table"].shape[1],
                         c["page"], s["depths"], s["off"], s["slots"], s["pos"], s["cap"], s["counts"])
    return {"table": s["table"], "off": s["off"], "slots": s["slots"], "pos": s["pos"], "counts": s["counts"]}


def _slots_plain(s):
    p, cap = s["case"]["page"], s["cap"]
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    have = (ctx + p - 1) // p
    need = (ctx + new + p - 1) // p - have
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(table.shape[1], device=DEV)[None]
    take = (cols >= have[:, None]) & (cols < (have + need)[:, None])
    at = (first[:, None] + cols - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(take, s["free"][at], table)
    ends = torch.cumsum(new, 0)
    off = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(cap, device=DEV)
    r = torch.searchsorted(ends, t, right=True).clamp(max=ctx.numel() - 1)
    j = t - off[r]
    live = t < ends[-1]
    lin = torch.where(live, ctx[r] + j, 0)
    slots = torch.where(live, table[r, lin // p].long() * p + lin % p, -1)
    step = j if s["depths"] is None else s["depths"].long()
    pos = torch.where(live, ctx[r] + step, -1).to(torch.int32)
    zero = torch.zeros_like(ends[-1])
    counts = torch.stack([ends[-1], need.sum(), zero, zero]).to(torch.int32)
    return {"table": table, "off": off.to(torch.int32), "slots": slots, "pos": pos, "counts": counts}


def _qkrope_own(s):
    c, b = s["case"], s["bqd"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    qkv = s["qkv"]
    base, item, pitch = qkv.data_ptr(), qkv.element_size(), (Hq + 2 * Hkv) * D
    b.qk_norm_rope_cache(base, base + Hq * D * item, base + (Hq + Hkv) * D * item,
                         b.BQD_F32 if c["dtype"] == "f32" else b.BQD_BF16, pitch, pitch, pitch, s["qw"], s["kw"], 1e-6,
                         s["cos_sin"], s["cos_sin"].shape[0], c["rot"],
                         b.BQD_ROPE_PAIRS if c["pairs"] else b.BQD_ROPE_HALVES, s["pos"], s["slots"], s["q_out"],
                         s["cache"], c["T"], Hq)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _norm_rope(x, w, cos, sin, rot, pairs):
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    y, rest = x[..., :rot], x[..., rot:]
    if pairs:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _store(cache, slots, x, scale):
    flat = cache.view(-1, *cache.shape[2:])
    if scale is None:
        flat[slots] = x.to(torch.bfloat16)
    else:
        x = (x / scale[None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        flat.view(torch.uint8)[slots] = x.view(torch.uint8)


def _qkrope_plain(s):
    c = s["case"]
    T, Hq, Hkv, D, rot = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"][s["pos"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _norm_rope(x[:, :Hq], s["qw"], cos, sin, rot, c["pairs"])
    k = _norm_rope(x[:, Hq:Hq + Hkv], s["kw"], cos, sin, rot, c["pairs"])
    _store(s["k"], s["slots"], k, s["ks"])
    _store(s["v"], s["slots"], x[:, Hq + Hkv:], s["vs"])
    return {"q": q.to(torch.bfloat16), "k": s["k"], "v": s["v"]}


def _attn_own(s):
    c, t = s["case"], s["table"]
    s["bqd"].tree_attention(s["q"], c["Hq"] * c["D"], s["cache"], t, t.shape[1], s["ctx"], s["off"], s["mask"], 1,
                            s["scale"], s["out"], s["lse"], s["ws"], s["wsb"], c["R"], s["T"], c["Hq"])
    return {"out": s["out"], "lse": s["lse"]}


def _gather(cache, table, width, scale):
    x = cache.view(torch.uint8)[table] if cache.dtype == torch.float8_e4m3fn else cache[table]
    x = x.view(cache.dtype).flatten(1, 2)[:, :width].float()
    return x if scale is None else x * scale[:, None]


def _attn_plain(s):
    c = s["case"]
    R, n, Hq, Hkv, D, T = c["R"], c["n"], c["Hq"], c["Hkv"], c["D"], s["T"]
    off, ctx = s["off"].long(), s["ctx"].long()
    new = off[1:] - off[:-1]
    L = min(c["ctx"] + n, s["table"].shape[1] * c["page"])  # the longest request's tokens
    table = s["table"].long().clamp(min=0)
    k = _gather(s["k"], table, L, s["ks"])
    v = _gather(s["v"], table, L, s["vs"])
    j = torch.arange(n, device=DEV)
    at = (off[:-1, None] + j).clamp(max=T - 1)  # token of (request, draft)
    q = s["q"].float()[at].view(R, n, Hkv, Hq // Hkv, D)
    l = torch.arange(L, device=DEV)
    d = l[None, None] - ctx[:, None, None]  # draft index of a cache position
    if s["mask"] is None:
        seen = d <= j[None, :, None]
    else:
        seen = ((s["mask"][at].expand(R, n, 1) >> d.clamp(0, 63)) & 1).bool() | (d < 0)
    seen = seen & (d < new[:, None, None])
    v = v * (l[None] < (ctx + new)[:, None])[..., None, None]
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * (Hq // Hkv), D), k.permute(0, 2, 3, 1))
    x = x.view(R, Hkv, n, Hq // Hkv, L) * s["scale"]
    x = x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m0).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hkv, n * (Hq // Hkv), L), v.permute(0, 2, 1, 3)).view(R, Hkv, n, Hq // Hkv, D)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, D)
    lse = (m0 + torch.log(z)).squeeze(-1).permute(0, 2, 1, 3).reshape(R, n, Hq)
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[r]
    return {"out": o[r, i].to(torch.bfloat16), "lse": lse[r, i].contiguous()}


def _logprobs_own(s):
    c, b = s["case"], s["bqd"]
    b.token_logprobs(s["x"], b.BQD_F32 if c["dtype"] == "f32" else b.BQD_BF16, c["V"], s["tok"], s["lp"], s["ent"],
                     s["ids"], s["tlp"], c["k"], s["ws"], s["wsb"], c["T"], c["V"])
    return {"lp": s["lp"], "entropy": s["ent"], "ids": s["ids"], "top": s["tlp"]}


def _logprobs_plain(s):
    V, k = s["case"]["V"], s["case"]["k"]
    x = s["x"].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    lp = x.gather(1, s["tok"].long()[:, None]) - lse
    ent = torch.log(z) - (e * torch.where(e > 0, x - m, 0.0)).sum(-1, keepdim=True) / z
    # equal values go to the lowest index: order by (value, -index) in one integer
    bits = (x + 0.0).view(torch.int32)
    key = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = (key.long() << 32) | (V - 1 - torch.arange(V, device=DEV))
    ids = V - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
    return {"lp": lp[:, 0], "entropy": ent[:, 0], "ids": ids.to(torch.int32), "top": x.gather(1, ids) - lse}


_RUN = {("slots", True): _slots_own, ("slots", False): _slots_plain,
        ("qkrope", True): _qkrope_own, ("qkrope", False): _qkrope_plain,
        ("attn", True): _attn_own, ("attn", False): _attn_plain,
        ("logprobs", True): _logprobs_own, ("logprobs", False): _logprobs_plain}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "slots":
        ctx, new = _lens(case)
        p, R, T = case["page"], case["R"], sum(new)
        taken = sum(-(-(c + n) // p) - -(-c // p) for c, n in zip(ctx, new))
        # lengths and the free pages read, the new table entries, offsets, slots and positions written; a request's
        # partly filled page and the depths read
        return {"bytes": R * 8 + taken * 8 + (R + 1) * 4 + (T + 5) * 12 + R * 4 + (T * 4 if case["tree"] else 0) + 16,
                "flops": 0}
    if op == "qkrope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        e, ce = (4 if case["dtype"] == "f32" else 2), (2 if case["cache"] == "bf16" else 1)
        b = T * (Hq + 2 * Hkv) * D * e + T * Hq * D * 2 + T * 2 * Hkv * D * ce + T * 12 + T * case["rot"] * 4
        return {"bytes": b, "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    if op == "attn":
        ctx, new = _lens(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        e = 2 if case["cache"] == "bf16" else 1
        T = sum(new)
        kv = sum(c + n for c, n in zip(ctx, new))
        b = kv * Hkv * D * 2 * e + T * Hq * (4 * D + 4) + sum(-(-(c + n) // case["page"]) for c, n in zip(ctx, new)) * 4
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        return {"bytes": b, "flops": 4 * D * Hq * pairs}
    T, V, k = case["T"], case["V"], case["k"]
    return {"bytes": T * (V * (4 if case["dtype"] == "f32" else 2) + 12 + 8 * k), "flops": 6 * T * V}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return {"slots": _slots_exact, "qkrope": _qkrope_exact, "attn": _attn_exact, "logprobs": _logprobs_exact}[
        case["op"]](s)


def _slots_exact(s):
    p = s["case"]["page"]
    ctx, new, free = s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
    table = s["table"].cpu().numpy().copy()
    depths = None if s["depths"] is None else s["depths"].tolist()
    off, slots, pos, used = [0], [], [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(-(-c // p), -(-(c + n) // p)):
            table[r, b] = free[used]
            used += 1
        for j in range(n):
            slots.append(int(table[r, (c + j) // p]) * p + (c + j) % p)
            pos.append(c + (j if depths is None else depths[off[-1] + j]))
        off.append(off[-1] + n)
    pad = s["cap"] - off[-1]
    return {"table": table, "off": np.array(off, np.int32), "slots": np.array(slots + [-1] * pad, np.int64),
            "pos": np.array(pos + [-1] * pad, np.int32), "counts": np.array([off[-1], used, 0, 0], np.int32)}


def _qkrope_exact(s):
    c = s["case"]
    T, Hq, Hkv, D, rot = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    out = x[:, :Hq + Hkv].clone()
    for lo, hi, w in ((0, Hq, s["qw"]), (Hq, Hq + Hkv, s["kw"])):
        if w is not None:
            y = out[:, lo:hi]
            out[:, lo:hi] = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
    cs = s["cos_sin"].double()[s["pos"].long()]
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]  # a rotation is a product of complex numbers
    i = torch.arange(rot // 2, device=DEV)
    re, im = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + rot // 2)
    z = torch.complex(out[..., re], out[..., im]) * turn
    out[..., re], out[..., im] = z.real, z.imag
    done = {"q": out[:, :Hq]}
    for name, y, scale in (("k", out[:, Hq:], s["ks"]), ("v", x[:, Hq + Hkv:], s["vs"])):
        full = s[name].double()
        full.view(-1, Hkv, D)[s["slots"]] = y if scale is None else y / scale.double()[:, None]
        done[name] = full
    return done


def _attn_exact(s):
    c = s["case"]
    Hq, Hkv, D, p = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    ctx, off = s["ctx"].tolist(), s["off"].tolist()
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    for r, cl in enumerate(ctx):
        a, b = off[r], off[r + 1]
        L = cl + b - a
        l = torch.arange(L, device=DEV)
        at = s["table"][r].long()[l // p] * p + l % p
        hide = torch.zeros(b - a, L, dtype=torch.bool, device=DEV)
        for j in range(b - a):
            if s["mask"] is None:
                hide[:j, cl + j] = True
            else:
                hide[:, cl + j] = ((s["mask"][a:b, 0] >> j) & 1) == 0
        for h in range(Hkv):
            K = s["k"].flatten(0, 1)[:, h].view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16)[at]
            V = s["v"].flatten(0, 1)[:, h].view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16)[at]
            K, V = K.view(s["k"].dtype).double(), V.view(s["v"].dtype).double()
            if s["ks"] is not None:
                K, V = K * s["ks"][h].double(), V * s["vs"][h].double()
            for e in range(h * G, h * G + G):
                x = (s["q"][a:b, e].double() @ K.T) * s["scale"]
                x[hide] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[a:b, e] = z
                out[a:b, e] = torch.exp(x - z[:, None]) @ V
    return {"out": out, "lse": lse}


def _logprobs_exact(s):
    k = s["case"]["k"]
    got = {"lp": [], "entropy": [], "ids": [], "top": []}
    for a in range(0, s["case"]["T"], 128):
        x = s["x"][a:a + 128]
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        lp = torch.log_softmax(x.double(), 1)
        got["lp"].append(lp[torch.arange(lp.shape[0], device=DEV), s["tok"][a:a + 128].long()])
        got["entropy"].append(-(lp.exp() * lp).sum(1))
        got["ids"].append(order.to(torch.int32))
        got["top"].append(lp.gather(1, order))
    return {name: torch.cat(v) for name, v in got.items()}
