"""paged_slots on the GPU against the definition: integers, equal throughout."""
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


def dev(a, dt=torch.int32):
    return torch.tensor(np.asarray(a).tolist(), dtype=dt, device="cuda")


def run(ctx, new, free, table, page, cap, depths=None, stream=None):
    R, W = np.asarray(table).shape
    t = dev(table).reshape(R, W)
    off = torch.full((R + 1 + 8,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((cap + 8,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((cap + 8,), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    bqd.paged_slots(dev(ctx), dev(new), dev(free), len(free), t, R, W, page, None if depths is None else dev(depths),
                    off, slots, pos, cap, counts, stream)
    torch.cuda.synchronize()
    for x, n in ((off, R + 1), (slots, cap), (pos, cap)):
        assert torch.all(x[n:] == 77), "written past the end"
    return dict(table=t.cpu().numpy(), offsets=off[:R + 1].cpu().numpy(), slots=slots[:cap].cpu().numpy(),
                positions=pos[:cap].cpu().numpy(), counts=counts.cpu().numpy())


def check(ctx, new, page, free_extra=3, width_extra=2, cap_extra=4, tree=False, seed=0, short=0):
    rng = np.random.default_rng(seed)
    c, n = np.maximum(ctx, 0), np.maximum(new, 0)
    have, want = -(-c // page), -(-(c + n) // page)
    W = max(0, int(want.max(initial=0)) + width_extra)
    ids = rng.permutation(int(have.sum() + (want - have).sum()) + free_extra + 5)
    table, at = np.full((len(c), W), -1, np.int32), 0
    for r in range(len(c)):
        m = min(int(have[r]), W)
        table[r, :m] = ids[at:at + m]
        at += m
    free = ids[at:][:max(0, int((want - have).sum()) + free_extra - short)]
    cap = max(0, int(n.sum()) + cap_extra)
    depths = rng.integers(0, 50, cap) if tree else None
    got = run(ctx, new, free, table, page, cap, depths)
    want_ = ref.slots(ctx, new, free, table, page, cap, depths)
    for k in want_:
        assert np.array_equal(got[k], want_[k]), (k, got[k], want_[k])
    return got


@pytest.mark.parametrize("R", [1, 2, 7, 31, 32, 33, 255, 256, 257, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("page", [1, 16, 256])
def test_request_counts(R, page):
    rng = np.random.default_rng(R)
    check(rng.integers(0, 300, R), rng.integers(0, 9, R), page, seed=R, tree=R % 2 == 0)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 64, 1000, 70000])
def test_token_counts(n):
    check(np.array([33, 0, 16]), np.array([n, 1, n]), 16, seed=n)


def test_nothing_new_and_negative_lengths():
    check(np.array([5, 0, 40]), np.array([0, 0, 0]), 16)
    check(np.array([-3, 7, 40]), np.array([2, -9, 1]), 16)


@pytest.mark.parametrize("short", [1, 2, 5, 100])
def test_too_few_free_pages(short):
    got = check(np.array([5, 31, 0, 64]), np.array([30, 2, 60, 17]), 16, free_extra=0, short=short)
    assert got["counts"][2] == min(short, 9)


@pytest.mark.parametrize("less", [1, 3])
def test_table_too_narrow(less):
    got = check(np.array([5, 31, 0, 64]), np.array([30, 2, 90, 17]), 16, width_extra=-less)
    assert got["counts"][3] & bqd.BQD_SLOTS_TABLE_FULL


@pytest.mark.parametrize("cap_extra", [-1, -7, -29, -1000])
def test_more_tokens_than_room(cap_extra):
    got = check(np.array([5, 31]), np.array([20, 9]), 16, cap_extra=cap_extra, tree=True)
    assert got["counts"][3] == bqd.BQD_SLOTS_TOKENS_CUT


def test_no_requests():
    got = run([], [], [1, 2], np.zeros((0, 4), np.int32), 16, 3)
    assert got["offsets"].tolist() == [0] and got["slots"].tolist() == [-1] * 3
    assert got["counts"].tolist() == [0, 0, 0, 0]


def test_large_values():
    # page ids and contexts near 2^31: slots past 32 bits, sums that stop at 2^31 - 1
    got = run([100, 3], [5, 1], [2147483000, 2147483600], np.array([[2147483647, -1], [7, -1]], np.int32), 64, 8)
    want = ref.slots([100, 3], [5, 1], [2147483000, 2147483600], [[2147483647, -1], [7, -1]], 64, 8)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    got = run([2147483647, 0], [2147483647, 2147483647], [], np.zeros((2, 1), np.int32), 1024, 2)
    assert got["offsets"].tolist() == [0, 2147483647, 2147483647] and got["counts"][0] == 2147483647
    assert got["counts"][3] == 3


def test_graph_replay_on_a_side_stream():
    ctx, new, free = dev([3, 20]), dev([2, 1]), dev([9, 8, 7])
    table, off = dev([[1, -1, -1], [2, 3, -1]]), torch.zeros(3, dtype=torch.int32, device="cuda")
    slots, pos = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    counts = torch.zeros(4, dtype=torch.int32, device="cuda")
    go = lambda: bqd.paged_slots(ctx, new, free, 3, table, 2, 3, 16, None, off, slots, pos, 8, counts)  # noqa: E731
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for n in ([2, 1], [5, 3], [0, 8]):
        new.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = ref.slots([3, 20], n, [9, 8, 7], table.cpu().numpy(), 16, 8)
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(off.cpu().numpy(), want["offsets"])


def test_refusals():
    a = torch.zeros(64, dtype=torch.int64, device="cuda")

    def call(**kw):
        v = dict(c=a, n=a, f=a, nf=1, t=a, R=2, W=2, page=16, d=None, off=a, s=a, p=a, cap=4, counts=a)
        v.update(kw)
        bqd.paged_slots(*v.values())

    call()
    for status, kw in [(1, dict(c=None)), (1, dict(n=None)), (1, dict(f=None)), (1, dict(t=None)), (1, dict(off=None)),
                       (1, dict(s=None)), (1, dict(p=None)), (1, dict(counts=None)), (2, dict(R=-1)), (2, dict(W=-1)),
                       (2, dict(page=0)), (2, dict(page=24)), (2, dict(page=8192)), (2, dict(cap=-1)), (2, dict(nf=-1)),
                       (2, dict(R=1 << 24)), (2, dict(W=1 << 40)), (3, dict(s=a.data_ptr() + 4)), (3, dict(f=a.data_ptr() + 2))]:
        with pytest.raises(bqd.BqdError) as e:
            call(**kw)
        assert e.value.status == status, kw
