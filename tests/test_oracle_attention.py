"""Pins of the fp64 definitions around attention: hand-worked examples and
invariants (CPU)."""
import numpy as np
import pytest
import torch

from oracle import attention as ref


def test_slots_worked_example():
    # page size 4. Request 0: 5 cached (2 pages), 4 new -> positions 5..8, one more page.
    # Request 1: nothing cached, 1 new -> one page. Request 2: 8 cached (2 full pages), none new.
    table = [[7, 3, -1], [-1, -1, -1], [5, 6, -1]]
    got = ref.slots([5, 0, 8], [4, 1, 0], [9, 2, 4], table, 4, 7)
    assert got["table"].tolist() == [[7, 3, 9], [2, -1, -1], [5, 6, -1]]
    assert got["offsets"].tolist() == [0, 4, 5, 5]
    assert got["slots"].tolist() == [13, 14, 15, 36, 8, -1, -1]
    assert got["positions"].tolist() == [5, 6, 7, 8, 0, -1, -1]
    assert got["counts"].tolist() == [5, 2, 0, 0]


def test_slots_short_of_pages_and_columns():
    got = ref.slots([0, 0], [5, 5], [8], [[-1, -1], [-1, -1]], 2, 8)
    assert got["table"].tolist() == [[8, -1], [-1, -1]]
    assert got["slots"].tolist() == [16, 17, -1, -1, -1, -1, -1, -1]
    assert got["counts"].tolist() == [10, 1, 3, 3]


def test_e4m3_table_matches_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_table(), t, equal_nan=True)


def test_bf16_rounding_matches_torch():
    x = np.random.default_rng(0).standard_normal(4096).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(ref.f32_to_bf16(x), want)


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_rotation(pairs):
    rng = np.random.default_rng(1)
    x, ang = rng.standard_normal(64), rng.uniform(0, 6, 16)
    cs = np.concatenate([np.cos(ang), np.sin(ang)])
    y, _ = ref.norm_rope(x, None, 0.0, cs, 32, pairs)
    back, _ = ref.norm_rope(y, None, 0.0, np.concatenate([np.cos(ang), -np.sin(ang)]), 32, pairs)
    assert np.allclose(back, x, atol=1e-12) and np.array_equal(y[32:], x[32:])
    # a quarter turn sends (a, b) to (-b, a)
    q, _ = ref.norm_rope([1.0, 2.0, 3.0, 4.0], None, 0.0, [0.0, 0.0, 1.0, 1.0], 4, pairs)
    assert q.tolist() == ([-2.0, 1.0, -4.0, 3.0] if pairs else [-3.0, -4.0, 1.0, 2.0])


def test_norm_makes_unit_mean_square():
    x = np.random.default_rng(2).standard_normal(128) * 7
    y, _ = ref.norm_rope(x, np.full(128, 2.0), 0.0, [], 0, False)
    assert abs(np.mean(y * y) - 4.0) < 1e-12


def test_attention_worked_example():
    # scores log 1, log 3 over values 0 and 4: out = 3, lse = log 4
    k = np.array([[0.0], [np.log(3.0)], [50.0]])
    v = np.array([[0.0], [4.0], [np.nan]])
    out, lse, _, _ = ref.attention(np.array([1.0]), k, v, np.array([True, True, False]), 1.0)
    assert abs(out[0] - 3.0) < 1e-12 and abs(lse - np.log(4.0)) < 1e-12
    out, lse, _, _ = ref.attention(np.array([1.0]), k, v, np.zeros(3, bool), 1.0)
    assert out[0] == 0.0 and lse == -np.inf


def test_seen():
    assert ref.seen_of(2, 3, 1).tolist() == [True, True, True, True, False]
    assert ref.seen_of(1, 3, 0, [0b101]).tolist() == [True, True, False, True]
    assert ref.seen_of(0, 65, 0, [1 << 63])[63:].tolist() == [True, False]


def test_logprobs_worked_example():
    x = np.log(np.array([1, 2, 1, 4], np.float64)).astype(np.float32)
    lp, ent, ids, top = ref.logprobs(x, 1, 4)
    assert abs(lp - np.log(0.25)) < 1e-6 and ids == [3, 1, 0, 2]
    assert abs(ent - 1.75 * np.log(2)) < 1e-6 and abs(top[0] - np.log(0.5)) < 1e-6
    assert ref.logprobs(np.full(3, -np.inf), 0, 2)[:3] == (-np.inf, 0.0, [0, 1])
    assert ref.logprobs(np.array([1.0, np.nan, np.inf, -np.inf]), 0, 4)[2] == [2, 0, 3, 1]
    assert ref.logprobs(x, 9, 0)[0] == -np.inf


def test_logprobs_of_a_token_outside_the_vocabulary():
    for x in ([0.0, 1.0], [0.0, np.nan], [0.0, np.inf], [-np.inf, -np.inf]):
        assert ref.logprobs(x, 2, 0)[0] == ref.logprobs(x, -1, 0)[0] == -np.inf
