"""tree_attention on the GPU against the fp64 definition: head layouts, head
dimensions, cache types and layouts, lengths from none to long, chains, trees
and empty rows, what is hidden, and the calls' surroundings."""
import numpy as np
import pytest
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from tests.attn_util import Cache, check_attention, random_tree_mask, run_attention, table_for
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def queries(T, Hq, D, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (gain * torch.randn(T, Hq, D, generator=g)).to(torch.bfloat16).cuda()


def case(ctx, new, Hq=8, Hkv=2, D=128, kind="bf16", page=16, layout="tokens", tree=False, seed=0, words=1, gain=1.0,
         rows=None, extra=0):
    lens = [c + n for c, n in zip(ctx, new)]
    pages = sum(-(-l // page) for l in lens) + 3
    cache = Cache(pages, page, Hkv, D, kind, layout, seed, extra)
    table = table_for(lens, page, pages, seed)
    off = [0] + list(np.cumsum(new))
    q = queries(off[-1], Hq, D, seed + 1, gain)
    mask = random_tree_mask(new, seed, words) if tree else None
    scale = D ** -0.5
    out, lse = run_attention(cache, q, table, ctx, off, mask, scale)
    check_attention(cache, q, table, ctx, off, mask, scale, out, lse, rows, f"{ctx} {new} {Hq}/{Hkv} {D} {kind} {page}")
    return cache, q, table, off, mask, scale, out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (7, 1), (16, 1)])
def test_heads_types_dims(D, kind, Hq, Hkv):
    case([37, 130], [1, 3], Hq, Hkv, D, kind, seed=D + Hq)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 511, 1023, 2049])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_single_token_lengths(ctx, kind):
    case([ctx], [1], 8, 2, 128, kind, seed=ctx)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 48, 63, 64])
@pytest.mark.parametrize("tree", [False, True])
def test_draft_widths(n, tree):
    case([50], [n], 8, 2, 64, seed=n, tree=tree)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [8, 20, 64])
def test_wide_trees(D, kind, n):
    # up to 512 query rows share a kv head, in tiles with a ragged end
    case([300, 5], [n, n // 2 + 1], 8, 1, D, kind, seed=n + D, tree=True)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 32, 64, 256, 1024])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("n", [2, 24])
def test_pages_and_layouts(page, layout, n):
    case([200, 33, 0], [n, 1, n], 8, 2, 128, "bf16", page, layout, seed=page, tree=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_padded_strides(kind):
    case([70, 9], [3, 30], 8, 2, 64, kind, 16, seed=5, extra=16)


@pytest.mark.parametrize("group", [3, 5, 6, 12, 64])
def test_odd_groups(group):
    case([90, 200], [3, 11], group, 1, 64, seed=group, tree=True)


def test_long_context_few_rows():
    case([20000, 17, 9001], [1, 1, 2], 4, 1, 128, seed=3)


def test_long_context_many_rows():
    case([9000, 100], [64, 40], 8, 1, 128, seed=4, tree=True, rows={0, 17, 63, 64, 103})


def test_many_ragged_requests():
    rng = np.random.default_rng(6)
    ctx, new = rng.integers(0, 90, 150).tolist(), rng.integers(0, 4, 150).tolist()
    case(ctx, new, 4, 2, 64, seed=6)


def test_requests_without_new_tokens():
    case([40, 20, 60, 10], [0, 2, 0, 0], 4, 2, 64, seed=7)


def test_large_scores():
    # scores of hundreds: the running maximum carries the sums
    case([500, 100], [2, 20], 8, 2, 128, seed=8, gain=40.0)


def test_more_than_64_drafts():
    case([30], [100], 4, 1, 64, seed=9, tree=True, words=2)
    case([30], [100], 4, 1, 64, seed=9, tree=True, words=1)  # drafts past the words are hidden
    case([30, 2], [200, 130], 4, 1, 64, seed=9)              # a chain needs no words


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 5, 40])
@pytest.mark.parametrize("ctx", [0, 21])
def test_rows_that_see_nothing(kind, n, ctx):
    cache, q, table, off, mask, scale, _, _ = case([ctx], [n], 8, 2, 128, kind, seed=n, tree=True)
    mask = mask.copy()
    mask[n // 2] = 0
    mask[0] = 0
    out, lse = run_attention(cache, q, table, [ctx], off, mask, scale)
    check_attention(cache, q, table, [ctx], off, mask, scale, out, lse, what="empty rows")
    if ctx == 0:
        assert torch.all(out[0] == 0) and torch.all(lse[0] == -float("inf"))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 9, 40])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_hidden_places_have_no_influence(kind, n, bad):
    if kind == "e4m3" and bad == "inf":
        pytest.skip("E4M3 has no infinities")
    D, ctx = 128, 53
    cache, q, table, off, mask, scale, out, lse = case([ctx], [n], 8, 2, D, kind, seed=n, tree=True)
    poison = (float("nan") if bad == "nan" else float("inf")) if kind == "bf16" else 0x7F
    # everything outside the request's tokens, and draft 1 for those that do not see it
    slots = [int(table[0, l // 16]) * 16 + l % 16 for l in range(ctx + n)]
    rest = [s for s in range(cache.pages * 16) if s not in set(slots)]
    for t in (cache.k, cache.v):
        for s in rest + [slots[ctx + 1]]:
            t[s // 16, s % 16] = poison
    out2, lse2 = run_attention(cache, q, table, [ctx], off, mask, scale)
    sees = np.array([(int(m[0]) >> 1) & 1 for m in mask], bool)
    assert sees[1] and not sees.all()
    hid = torch.from_numpy(~sees).cuda()
    assert torch.isfinite(out2[hid].float()).all()
    check_attention(cache, q, table, [ctx], off, mask, scale, out2, lse2, rows=set(np.flatnonzero(~sees).tolist()))
    assert not torch.isfinite(out2[~hid].float()).any(), "a token that sees it shows it"


@pytest.mark.parametrize("n", [2, 30])
def test_infinite_value_that_is_seen(n):
    cache, q, table, off, mask, scale, _, _ = case([40], [n], 8, 2, 64, seed=2)
    s = int(table[0, 40 // 16]) * 16 + 40 % 16  # the first draft, seen by all
    cache.v[s // 16, s % 16, :, 5] = float("inf")
    cache.v[s // 16, s % 16, :, 6] = -float("inf")
    out, _ = run_attention(cache, q, table, [40], off, None, scale)
    assert torch.all(out[..., 5] == float("inf")) and torch.all(out[..., 6] == -float("inf"))
    assert torch.isfinite(out[..., 7:].float()).all()


def test_bad_pages_and_short_tables_are_not_seen():
    cache, q, table, off, mask, scale, _, _ = case([100, 80], [2, 18], 8, 2, 64, seed=11)
    t2 = table.copy()
    t2[0, 1], t2[1, 3] = -5, cache.pages + 7
    out, lse = run_attention(cache, q, t2, [100, 80], off, None, scale)
    check_attention(cache, q, t2, [100, 80], off, None, scale, out, lse, what="bad pages")
    t3 = np.ascontiguousarray(table[:, :4])
    out, lse = run_attention(cache, q, t3, [100, 80], off, None, scale)
    check_attention(cache, q, t3, [100, 80], off, None, scale, out, lse, what="short table")


def test_tokens_of_no_request_are_not_written():
    cache, q, table, off, mask, scale, out, lse = case([30, 40], [2, 3], 8, 2, 64, seed=12)
    qq = torch.cat([q, q, q])
    o2, l2 = run_attention(cache, qq, table, [30, 40], off, None, scale)
    check_attention(cache, qq, table, [30, 40], off, None, scale, o2, l2, what="padded")
    assert torch.all(o2[5:] == 7.0) and torch.all(l2[5:] == 7.0)
    # offsets past T are clamped to it
    o3, l3 = run_attention(cache, q, table, [30, 40], [0, 2, 9], None, scale)
    assert torch.isfinite(o3.float()).all()


def test_row_pitch_and_no_lse():
    cache, q, table, off, mask, scale, out, lse = case([30], [3], 8, 2, 64, seed=13)
    wide = torch.zeros(3, 8 * 64 + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = q.view(3, 512)
    o2 = torch.empty_like(out)
    wsb = bqd.tree_attention_workspace_bytes(1, 3, 8, 2, 64)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bqd.tree_attention(wide, 536, cache.desc, torch.from_numpy(table).cuda(), table.shape[1], dev([30]), dev(off), None,
                       1, scale, o2, None, ws, wsb, 1, 3, 8)
    assert torch.equal(o2, out)


@pytest.mark.parametrize("n", [1, 6, 40])
def test_same_bits_every_time_and_on_a_side_stream(n):
    cache, q, table, off, mask, scale, out, lse = case([700, 31, 300], [n, 1, n], 8, 2, 128, seed=14, tree=True)
    for stream in (None, torch.cuda.Stream()):
        o2, l2 = run_attention(cache, q, table, [700, 31, 300], off, mask, scale, stream=stream)
        assert torch.equal(o2.view(torch.int16), out.view(torch.int16)) and torch.equal(l2, lse)


def test_graph_replay_with_other_lengths():
    # lengths are read on the device: one captured launch serves a growing context
    cache, q, table, off, mask, scale, _, _ = case([150, 90], [2, 2], 8, 2, 128, seed=15)
    dt, do = torch.from_numpy(table).cuda(), torch.tensor(off, dtype=torch.int32, device="cuda")
    dc = torch.tensor([150, 90], dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(4, 8, device="cuda")
    wsb = bqd.tree_attention_workspace_bytes(2, 4, 8, 2, 128)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    go = lambda: bqd.tree_attention(q, 1024, cache.desc, dt, table.shape[1], dc, do, None, 1, scale, out, lse, ws, wsb,  # noqa: E731
                                    2, 4, 8)
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for ctx in ([150, 90], [3, 0], [77, 88]):
        dc.copy_(torch.tensor(ctx, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_attention(cache, q, table, ctx, off, None, scale, out, lse, what=f"replay {ctx}")


def test_offsets_past_32_bits():
    # 2^31 elements and more in each of K and V: the pages used lie at the far end
    page, Hkv, D = 16, 2, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    k = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    small = Cache(40, page, Hkv, D, seed=16)
    k[-40:] = small.k
    v[-40:] = small.v
    desc = bqd.kv_cache(k, v)
    lens, off = [70, 200], [0, 2, 20]
    table = table_for([72, 218], page, 40, 16)
    q = queries(20, 8, D, 17)
    out, lse = run_attention(small, q, table, lens, off, None, D ** -0.5)
    far = np.where(table >= 0, table + pages - 40, -1).astype(np.int32)
    small.desc = desc
    out2, lse2 = run_attention(small, q, far, lens, off, None, D ** -0.5)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_refusals():
    cache = Cache(4, 16, 2, 64)
    q = queries(2, 4, 64)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ctx, off = i32([[0, 1]]), i32([5]), i32([0, 2])
    out = torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    wsb = bqd.tree_attention_workspace_bytes(1, 2, 4, 2, 64)
    ws = torch.empty(wsb + 16, dtype=torch.uint8, device="cuda")

    def call(**kw):
        a = dict(q=q, q_pitch=256, cache=cache.desc, table=table, width=2, ctx=ctx, off=off, mask=None, words=1,
                 scale=0.125, out=out, lse=None, ws=ws, wsb=wsb, R=1, T=2, Hq=4)
        a.update(kw)
        bqd.tree_attention(*a.values())

    call()
    for status, kw in [(1, dict(q=None)), (1, dict(out=None)), (1, dict(ctx=None)), (1, dict(table=None)),
                       (2, dict(q_pitch=248)), (2, dict(q_pitch=260)), (2, dict(Hq=3)), (2, dict(Hq=0)),
                       (2, dict(T=-1)), (2, dict(R=-1)), (2, dict(mask=ctx, words=0)), (2, dict(width=-1)),
                       (3, dict(q=q.data_ptr() + 2)), (3, dict(out=out.data_ptr() + 8)),
                       (6, dict(ws=None)), (6, dict(wsb=wsb - 1)), (6, dict(ws=ws.data_ptr() + 4))]:
        with pytest.raises(bqd.BqdError) as e:
            call(**kw)
        assert e.value.status == status, kw
    for field, value in [("head_dim", 96), ("page_size", 12), ("page_size", 0), ("type", 0), ("heads", 0),
                         ("token_stride", 65), ("num_pages", -1)]:
        c = Cache(4, 16, 2, 64)
        setattr(c.desc, field, value)
        with pytest.raises(bqd.BqdError) as e:
            call(cache=c.desc)
        assert e.value.status == 2, field
    call(T=0)
    call(R=0)
    assert bqd.tree_attention_workspace_bytes(1, 1, 3, 2, 64) == 0


@pytest.mark.parametrize("ctx", [0, 1, 37, 64, 91, 127, 300])
@pytest.mark.parametrize("D,page", [(64, 8), (128, 16), (128, 64)])
def test_masks_of_several_words(ctx, D, page):
    """Random bits over more drafts than a block of tokens holds, the first of them anywhere in a block."""
    n, words = 210, 4
    rng = np.random.default_rng(ctx + D + page)
    pages = -(-(ctx + n) // page) + 3
    cache = Cache(pages, page, 1, D, "bf16", "tokens", ctx, 0)
    table = table_for([ctx + n], page, pages, ctx)
    q = queries(n, 2, D, ctx)
    mask = rng.integers(0, 2 ** 64, (n, words), dtype=np.uint64, endpoint=False)
    mask[5] = 0
    rows = {0, 5, 31, 63, 64, 100, 128, 160, 191, 209}
    out, lse = run_attention(cache, q, table, [ctx], [0, n], mask, D ** -0.5)
    check_attention(cache, q, table, [ctx], [0, n], mask, D ** -0.5, out, lse, rows, f"{ctx} {D} {page}")


@pytest.mark.parametrize("gain", [1e4, 1e7, 1e9, 3e10, 1e20])
@pytest.mark.parametrize("kind,D,n", [("bf16", 64, 2), ("bf16", 128, 10), ("bf16", 128, 40), ("bf16", 256, 10),
                                      ("e4m3", 128, 2), ("e4m3", 128, 40)])
def test_scores_of_any_size(kind, D, n, gain):
    # scores far apart: each token's largest takes all, whatever the scores' size (two keys are equal)
    ctx, Hq, Hkv, page = [300], 8, 2, 16
    cache = Cache(40, page, Hkv, D, kind, seed=3)
    table = table_for([ctx[0] + n], page, 40, 3)
    q = queries(n, Hq, D, 4, gain)
    pg, at = int(table[0, 0]), 0
    cache.k[int(table[0, 0]), 1] = cache.k[pg, at]
    out, lse = run_attention(cache, q, table, ctx, [0, n], None, D ** -0.5)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    K, V = cache.values("k"), cache.values("v")
    slot = table[0][np.arange(ctx[0] + n) // page] * page + np.arange(ctx[0] + n) % page
    o = out.double().cpu().numpy()
    for t in range(n):
        for h in range(Hq):
            k, v = K[slot[:ctx[0] + t + 1], h // (Hq // Hkv)], V[slot[:ctx[0] + t + 1], h // (Hq // Hkv)]
            s = (k @ q[t, h].double().cpu().numpy()) * D ** -0.5
            order = np.argsort(-s, kind="stable")
            best, second = s[order[0]], s[order[2 if order[0] == 0 else 1]]
            size = float((np.abs(k) @ np.abs(q[t, h].double().cpu().numpy())).max()) * D ** -0.5
            err = 2 * (D + 8) * 2.0 ** -24 * size
            if best - second <= 40 + err:
                continue  # another token may be as large once rounded
            y = (v[0] + v[1]) / 2 if order[0] in (0, 1) else v[order[0]]
            assert np.all(np.abs(o[t, h] - y) <= 2.0 ** -7 * np.abs(y) + 2.0 ** -7 * 2.0 ** -8), (t, h)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
def test_sums_of_one_seen_token(kind, n):
    # lse is the one score itself: what p is shifted or scaled by leaves no trace, whatever the score's size
    for seed, gain in enumerate([0.01, 0.1, 1.0, 3.0, 10.0, 100.0]):
        case([1], [n], 64, 1, 64, kind, tree=False, seed=seed, gain=gain, rows={0, n - 1})
        cache, q, table, off, _, scale, _, _ = case([1], [n], 64, 1, 64, kind, seed=seed + 50, gain=gain, rows={0})
        mask = np.zeros((n, 1), np.uint64)
        out, lse = run_attention(cache, q, table, [1], off, mask, scale)
        check_attention(cache, q, table, [1], off, mask, scale, out, lse, None, f"{gain}")
