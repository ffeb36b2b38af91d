"""One speculative-verify step of a small random transformer block, as a program would run it.

The library's calls in the order of a step: the new tokens' places in the paged cache from the requests' lengths
(paged_slots), the query/key/value projection with NVFP4 weights (nvfp4_gemm), norm, rotary positions and the cache
write (qk_norm_rope_cache), attention over cache and drafts (tree_attention), the output projection and the vocabulary
head (nvfp4_gemm), and the drafted tokens' log probabilities (token_logprobs). PyTorch holds the memory and makes the
random weights.

    python examples/verify_step.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_decode_nvfp4_gb300 as bqd  # noqa: E402


class Linear:
    """NVFP4 weights [M][K] of a random matrix; __call__: bf16 [T][K] -> fp32 [T][M]."""

    def __init__(self, M, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = (torch.randn(M, K, generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
        self.M, self.K, self.ts = M, K, float(w.float().abs().max()) / (448.0 * 6.0)
        self.codes = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(M, K // 16, dtype=torch.uint8, device="cuda")
        bqd.nvfp4_encode(w, self.ts, self.codes, self.scales, M, K)

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.M, device="cuda")
        bqd.nvfp4_gemm(self.codes, self.scales, self.ts, x, y, self.M, self.K, x.shape[0])
        return y


class Model:
    """Embedding, one attention block and a vocabulary head, with a paged cache for `pages` pages of 16 tokens."""

    def __init__(self, hidden=512, Hq=8, Hkv=2, D=64, vocab=4096, pages=256, cache="bf16", seed=0):
        self.Hq, self.Hkv, self.D, self.vocab, self.page = Hq, Hkv, D, vocab, 16
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.qkv = Linear((Hq + 2 * Hkv) * D, hidden, seed + 1)
        self.out = Linear(hidden, Hq * D, seed + 2)
        self.head = Linear(vocab, hidden, seed + 3)
        self.q_weight, self.k_weight = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        angle = torch.arange(4096, device="cuda")[:, None] / 1e4 ** (torch.arange(0, D, 2, device="cuda")[None] / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
        self.k = torch.zeros(pages, self.page, Hkv, D, dtype=dtype, device="cuda")
        self.v = torch.zeros(pages, self.page, Hkv, D, dtype=dtype, device="cuda")
        scales = [None, None] if cache == "bf16" else [torch.full((Hkv,), s, device="cuda") for s in (0.02, 0.02)]
        self.cache = bqd.kv_cache(self.k, self.v, *scales)

    def step(self, tokens, places, table, context, mask):
        """Logits [T][vocab] of a step's tokens; their keys and values go into the cache at places["slots"]."""
        T, R, Hq, Hkv, D = tokens.numel(), context.numel(), self.Hq, self.Hkv, self.D
        x = self.embedding[tokens]
        qkv = self.qkv(x)
        pitch, row = qkv.shape[1], qkv.data_ptr()
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        bqd.qk_norm_rope_cache(row, row + 4 * Hq * D, row + 4 * (Hq + Hkv) * D, bqd.BQD_F32, pitch, pitch, pitch,
                               self.q_weight, self.k_weight, 1e-6, self.cos_sin, self.cos_sin.shape[0], D,
                               bqd.BQD_ROPE_HALVES, places["positions"], places["slots"], q, self.cache, T, Hq)
        o = torch.empty_like(q)
        size = bqd.tree_attention_workspace_bytes(R, T, Hq, Hkv, D)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        bqd.tree_attention(q, Hq * D, self.cache, table, table.shape[1], context, places["offsets"], mask, 1,
                           D ** -0.5, o, None, work, size, R, T, Hq)
        h = (x.float() + self.out(o.view(T, Hq * D))).to(torch.bfloat16)
        return self.head(h)


def place(context, new, free, table, page, depths=None):
    """paged_slots with its outputs: offsets, slots and positions of the step's tokens, the pages taken."""
    R, T = context.numel(), int(new.sum())
    i32 = dict(dtype=torch.int32, device="cuda")
    out = {"offsets": torch.empty(R + 1, **i32), "positions": torch.empty(T, **i32), "counts": torch.empty(4, **i32),
           "slots": torch.empty(T, dtype=torch.int64, device="cuda")}
    bqd.paged_slots(context, new, free, free.numel(), table, R, table.shape[1], page, depths, out["offsets"],
                    out["slots"], out["positions"], T, out["counts"])
    return out


def score(logits, tokens, topk=4):
    """Log probability of `tokens` under the rows of `logits`, entropy, and the topk alternatives."""
    T, V = logits.shape
    lp, entropy = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ids = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    alternatives = torch.empty(T, topk, device="cuda")
    size = bqd.token_logprobs_workspace_bytes(T, V, topk)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    bqd.token_logprobs(logits, bqd.BQD_F32, V, tokens, lp, entropy, ids, alternatives, topk, work, size, T, V)
    return lp, entropy, ids, alternatives


def main():
    model = Model()
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(256, device="cuda").to(torch.int32)
    table = torch.full((2, 16), -1, **i32)
    context = torch.zeros(2, **i32)
    # two prompts, as chains
    new = torch.tensor([37, 20], **i32)
    places = place(context, new, free, table, model.page)
    model.step(torch.randint(0, model.vocab, (57,), device="cuda"), places, table, context, None)
    free, context = free[int(places["counts"][1]):], context + new
    # a drafted tree for each: 0 -> 1 -> 2 and 0 -> 3 -> 4 (token 0 is the one already accepted)
    tree = torch.tensor([0b00001, 0b00011, 0b00111, 0b01001, 0b11001], device="cuda").repeat(2)[:, None].contiguous()
    depths = torch.tensor([0, 1, 2, 1, 2] * 2, **i32)
    new = torch.tensor([5, 5], **i32)
    places = place(context, new, free, table, model.page, depths)
    drafted = torch.randint(0, model.vocab, (10,), device="cuda")
    logits = model.step(drafted, places, table, context, tree)
    # draft j is scored by the logits of its parent
    parent = torch.tensor([0, 1, 0, 3, 5, 6, 5, 8], device="cuda")
    child = torch.tensor([1, 2, 3, 4, 6, 7, 8, 9], device="cuda")
    lp, entropy, ids, _ = score(logits[parent].contiguous(), drafted[child].to(torch.int32))
    for p, c, l, e, i in zip(parent.tolist(), child.tolist(), lp.tolist(), entropy.tolist(), ids.tolist()):
        print(f"token {c} after {p}: log probability {l:.3f}, entropy {e:.3f}, best {i}")


if __name__ == "__main__":
    main()
