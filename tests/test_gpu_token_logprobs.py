"""token_logprobs on the GPU against the fp64 definition.

Tolerances: a sum of V positive terms along chains of at most 1024 additions
costs 1024 2^-24 = 2^-14 of itself, exp 2^-21 of each term, the subtraction
2^-23 of the values: |lse| is good to 2^-13 + 2^-22 max |x|; the entropy's
second sum has terms of one sign, so 2^-13 (1 + entropy) more. Indices are
exact."""
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


def run(x, tok, k, stream=None, V=None, base=None, pitch=None):
    T = x.shape[0]
    V = x.shape[1] if V is None else V
    o = [torch.full((T + 1,), 5.0, device="cuda"), torch.full((T + 1,), 5.0, device="cuda"),
         torch.full((T + 1, max(k, 1)), 5, dtype=torch.int32, device="cuda"),
         torch.full((T + 1, max(k, 1)), 5.0, device="cuda")]
    wsb = bqd.token_logprobs_workspace_bytes(T, V, k)
    ws = torch.full((wsb,), 0xFF, dtype=torch.uint8, device="cuda")
    bqd.token_logprobs(x if base is None else base, bqd.BQD_F32 if x.dtype == torch.float32 else bqd.BQD_BF16,
                       pitch or x.stride(0) or V, tok, o[0], o[1], o[2], o[3], k, ws, wsb, T, V, stream)
    torch.cuda.synchronize()
    assert torch.all(o[0][T:] == 5) and torch.all(o[1][T:] == 5)
    if k:
        assert torch.all(o[2].view(-1)[T * k:] == 5) and torch.all(o[3].view(-1)[T * k:] == 5)
    return (o[0][:T].cpu().numpy(), o[1][:T].cpu().numpy(), o[2].view(-1)[:T * k].view(T, k).cpu().numpy(),
            o[3].view(-1)[:T * k].view(T, k).cpu().numpy())


def same(a, b, tol):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    fin = np.isfinite(b)
    assert np.array_equal(a[~fin], b[~fin], equal_nan=True), (a, b)
    assert np.all(np.abs(a[fin] - b[fin]) <= tol), (a, b, tol)


def check(x, tok, k, rows=None, **kw):
    lp, ent, ids, top = run(x, torch.tensor(tok, dtype=torch.int32, device="cuda"), k, **kw)
    xs = x.float().cpu().numpy()
    for t in (range(x.shape[0]) if rows is None else rows):
        e = ref.logprobs(xs[t], tok[t], k)
        fin = xs[t][np.isfinite(xs[t])]
        tol = 2.0 ** -13 + 2.0 ** -22 * (np.abs(fin).max() if fin.size else 0)
        assert ids[t].tolist() == list(e[2]), (t, ids[t], e[2])
        same(lp[t:t + 1], [e[0]], tol)
        same(top[t], e[3], tol)
        same(ent[t:t + 1], [e[1]], tol + 2.0 ** -13 * (1 + abs(e[1]) if np.isfinite(e[1]) else 1))
    return lp, ent, ids, top


def logits(T, V, dtype="f32", seed=0, gain=3.0):
    x = gain * torch.randn(T, V, generator=torch.Generator().manual_seed(seed))
    return (x if dtype == "f32" else x.to(torch.bfloat16)).cuda()


@pytest.mark.parametrize("V", [1, 2, 3, 7, 31, 32, 33, 127, 1000, 1024, 4095, 4097, 32000, 50257])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_vocabulary_sizes(V, dtype):
    T = 3  # odd V: rows start at every alignment
    check(logits(T, V, dtype, V), [0, V - 1, V // 2], min(V, 20))


@pytest.mark.parametrize("T", [1, 2, 5, 16, 40, 153, 700])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_counts(T, dtype):
    check(logits(T, 9973, dtype, T), [(7 * t) % 9973 for t in range(T)], 5, rows=sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("V", [151936, 262143])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 9, 200])
def test_large_vocabularies(V, dtype, T):
    check(logits(T, V, dtype, 1), [V - 1] * T, 20, rows=[0, T - 1])


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("T", [1, 300])
def test_topk(k, T):
    check(logits(T, 20011, "f32", k), [5] * T, k, rows=[0, T - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5000, 151936])
def test_ties_go_to_the_lowest_index(dtype, V):
    x = torch.randint(-3, 4, (4, V), generator=torch.Generator().manual_seed(2)).float()
    x[0] = 0.0
    x[0, 1::2] = -0.0  # equal to +0
    x[1] = 2.5
    check((x if dtype == "f32" else x.to(torch.bfloat16)).cuda(), [0, 1, 2, 3], 32)


@pytest.mark.parametrize("order", ["ascending", "descending"])
@pytest.mark.parametrize("T", [1, 200])
def test_sorted_rows(order, T):
    # ascending: every logit is a new maximum and a new candidate
    x = torch.linspace(-20, 20, 100003).repeat(T, 1)
    check((x if order == "ascending" else x.flip(1)).contiguous().cuda(), [17] * T, 32, rows=[0, T - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    x = logits(8, 40007, dtype, 3)
    inf = float("inf")
    x[0] = -inf                       # nothing left
    x[1] = -inf
    x[1, 39999] = 2.0                 # one left
    x[2, 100:] = -inf
    x[3, :-3] = -inf                  # fewer than topk left
    x[4] = torch.finfo(x.dtype).min   # the lowest value, as masks use it: a uniform row
    x[5, ::2] = torch.finfo(x.dtype).min
    x[6] = -inf
    x[6, 5] = torch.finfo(x.dtype).min
    check(x, [3, 39999, 50, 2, 1, 1, 5, 0], 8)


@pytest.mark.parametrize("T", [1, 160])
def test_nan_and_inf(T):
    x = logits(max(T, 4), 30011, "f32", 4)
    x[0, 20000] = float("nan")
    x[1 % T, 7] = float("inf")
    x[2 % T, [3, 9, 30000]] = float("nan")
    check(x[:T].contiguous(), [1] * T, 20, rows=[0, T - 1, 1 % T, 2 % T])
    y = torch.full((1, 50), float("nan"), device="cuda")
    check(y, [0], 7)


def test_extreme_ranges():
    x = logits(4, 20000, "f32", 5)
    x[0] *= 1e4     # one token holds everything
    x[1] += 1e5
    x[2] *= 1e-6    # uniform: entropy log V
    x[3, 77] = 3e38
    check(x, [1, 2, 3, 77], 10)


def test_tokens_outside_the_vocabulary():
    lp, *_ = check(logits(4, 1000, "f32", 6), [-1, 1000, 2147483647, -2147483648], 2)
    assert np.all(lp == -np.inf)


@pytest.mark.parametrize("off", [0, 1, 3, 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_pitch(off, dtype):
    big = logits(5, 9000 + off, dtype, 7)
    check(big[:, :8990], [1, 2, 3, 4, 5], 6)


def test_optional_outputs():
    x = logits(3, 5000, "f32", 8)
    wsb = bqd.token_logprobs_workspace_bytes(3, 5000, 0)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda")
    ent = torch.empty(3, device="cuda")
    bqd.token_logprobs(x, bqd.BQD_F32, 5000, None, None, ent, None, None, 0, ws, wsb, 3, 5000)
    same(ent.cpu().numpy(), [ref.logprobs(r, 0, 0)[1] for r in x.cpu().numpy()], 2.0 ** -9)
    bqd.token_logprobs(x, bqd.BQD_F32, 5000, None, None, None, None, None, 0, ws, wsb, 3, 5000)
    torch.cuda.synchronize()


def test_same_bits_every_time_and_on_a_side_stream():
    for T, V in ((1, 151936), (16, 50257), (300, 32000)):
        x, tok = logits(T, V, "f32", T), torch.zeros(T, dtype=torch.int32, device="cuda")
        a, b = run(x, tok, 20), run(x, tok, 20, stream=torch.cuda.Stream())
        assert all(np.array_equal(u, v) for u, v in zip(a, b))


def test_graph_replay():
    x, tok = logits(2, 151936, "f32", 9), torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    o = [torch.empty(2, device="cuda"), torch.empty(2, device="cuda"),
         torch.empty(2, 4, dtype=torch.int32, device="cuda"), torch.empty(2, 4, device="cuda")]
    wsb = bqd.token_logprobs_workspace_bytes(2, 151936, 4)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    go = lambda: bqd.token_logprobs(x, bqd.BQD_F32, 151936, tok, *o, 4, ws, wsb, 2, 151936)  # noqa: E731
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for seed in (10, 11, 12):
        x.copy_(logits(2, 151936, "f32", seed))
        g.replay()
        torch.cuda.synchronize()
        assert o[2].cpu().numpy().tolist() == [ref.logprobs(r, 0, 4)[2] for r in x.cpu().numpy()]


def test_rows_past_32_bits():
    T, V = 3, 1000
    pitch = (1 << 31) - 8
    x = torch.empty(2 * pitch + V, device="cuda")
    rows = logits(T, V, "f32", 13)
    for t in range(T):
        x[t * pitch:t * pitch + V] = rows[t]
    tok = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    a, b = run(rows, tok, 9), run(rows, tok, 9, base=x, pitch=pitch)
    assert all(np.array_equal(u, v) for u, v in zip(a, b))


def test_refusals():
    x, tok = logits(2, 100), torch.zeros(4, dtype=torch.int32, device="cuda")
    f, i = torch.empty(64, device="cuda"), torch.empty(64, dtype=torch.int32, device="cuda")
    wsb = bqd.token_logprobs_workspace_bytes(2, 100, 4)
    ws = torch.empty(wsb + 16, dtype=torch.uint8, device="cuda")

    def call(**kw):
        a = dict(x=x, ty=0, pitch=100, tok=tok, lp=f, ent=f, ids=i, top=f, k=4, ws=ws, wsb=wsb, T=2, V=100)
        a.update(kw)
        bqd.token_logprobs(*a.values())

    call()
    for status, kw in [(1, dict(x=None)), (1, dict(tok=None)), (1, dict(ids=None)), (1, dict(top=None)),
                       (2, dict(ty=2)), (2, dict(pitch=99)), (2, dict(k=33)), (2, dict(k=-1)), (2, dict(V=0, k=0)),
                       (2, dict(V=3, k=4)), (2, dict(T=-1)), (3, dict(x=x.data_ptr() + 4)),
                       (3, dict(ent=f.data_ptr() + 2)), (6, dict(ws=None)), (6, dict(wsb=wsb - 1))]:
        with pytest.raises(bqd.BqdError) as e:
            call(**kw)
        assert e.value.status == status, kw
    call(T=0)
    assert bqd.token_logprobs_workspace_bytes(1, 10, 11) == 0


def tie_with_the_end(V, T, dtype, k, low=0.0):
    """Constant rows but for k - 1 larger logits at the row's start and two equal ones: the row's last, and one of the
    second thousand 16-byte windows, which the same warp meets later and which has the lower index."""
    n = 4 if dtype == "f32" else 8
    x = torch.full((T, V), low)
    x[:, :k - 1] = 6.0
    x[:, 1025 * n] = 5.0
    x[:, V - 1] = 5.0
    return (x if dtype == "f32" else x.to(torch.bfloat16)).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [32769, 50257, 151937, 151939])
@pytest.mark.parametrize("k", [2, 20, 32])
@pytest.mark.parametrize("T", [1, 200])
def test_ties_with_the_end_of_the_row(dtype, V, k, T):
    # odd V: rows begin and end at every alignment
    check(tie_with_the_end(V, T, dtype, k), [V - 1] * T, k, rows=sorted({0, min(1, T - 1), min(6, T - 1), T - 1}))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 13, 21, 16385, 32769, 50257])
@pytest.mark.parametrize("T", [1, 4])
def test_coarse_rows_of_any_end(dtype, V, T):
    x = torch.randint(-3, 4, (T, V), generator=torch.Generator().manual_seed(V)).float()
    x[:, -3:] = 3.0  # the end ties with the largest
    for k in (1, min(5, V), min(32, V)):
        check((x if dtype == "f32" else x.to(torch.bfloat16)).cuda(), [V - 1] * T, k)


def check_masked(x, tok, k):
    """Rows of a few distinct values whose gaps are 0 or more than 1000: the entropy is that of the largest's copies,
    good to 2^-12 (1 + entropy) and 2^-13 of the shift that the maximum's product with log2(e) leaves, at most 64."""
    rows = [0, 1, 2, 3, 4, x.shape[0] - 1]
    _, ent, _, _ = check(x, tok, k, rows=rows)
    for t in rows:
        row = x[t].double().cpu().numpy()
        H = np.log((row == row.max()).sum())
        shift = min(64.0, np.abs(row.max()) * 2.0 ** -23)
        assert abs(ent[t] - H) <= 2.0 ** -12 * (1 + H) + 2.0 ** -13 * shift, (t, ent[t], H)


@pytest.mark.parametrize("low", [-1e5, -1e9, -3e9, -1e10, -1e20, -1e30, -9e37, -1.1e38])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 200])
def test_rows_masked_by_a_large_value(low, dtype, T):
    # what a mask other than -inf or the type's lowest value leaves: all of a row hidden, one logit, a few, a half
    V = 40007
    x = torch.full((T, V), low)
    x[1, 39999] = 2.0
    x[2, 100:104] = 1.0
    x[3, V // 2:] = 0.5
    x[4, :] = -low
    x = (x if dtype == "f32" else x.to(torch.bfloat16)).cuda()
    tok = [3, 39999, 102, V - 1, 7] + [0] * (T - 5)
    check_masked(x, tok, 8)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tokens_outside_the_vocabulary_of_a_row_without_an_answer(bad):
    x = logits(3, 1000, "f32", 14)
    x[:, 500] = bad
    lp, *_ = check(x, [-1, 1000, 7], 3)
    assert np.isneginf(lp[:2]).all() and np.isnan(lp[2])
