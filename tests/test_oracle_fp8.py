"""Pins of the fp64 definitions of the calls on 8-bit activations."""
import numpy as np
import torch

from oracle import fp8 as ref


def test_e4m3_codes_are_torchs_rounding():
    grid = ref.VALUES[:0x7F]
    mids = (grid[1:] + grid[:-1]) / 2
    near = np.concatenate([grid, mids, np.nextafter(mids.astype(np.float32), np.float32(0)).astype(np.float64),
                           np.nextafter(mids.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    x = np.concatenate([near, -near]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_codes(x), want)
    assert ref.e4m3_codes(np.array([1e30, -1e30, np.nan]))[:2].tolist() == [0x7E, 0xFE]
    assert ref.e4m3_codes(np.array([np.nan])) == 0x7F


def test_encode_by_hand():
    # amax 448: scale 1, codes of the values themselves; a block of its own after 128 channels
    x = np.zeros((1, 144), np.float32)
    x[0, :4] = [448, 1, -0.5, 2.0 ** -10]  # 2^-10 is half the smallest code: to even, 0
    x[0, 128] = -7
    codes, scales = ref.encode(x)
    assert codes[0, :4].tolist() == [0x7E, 0x38, 0xB0, 0x00] and codes[0, 128] == 0xFE
    assert scales.shape == (2, 1) and scales[0, 0] == 1 and scales[1, 0] == np.float32(7) / np.float32(448)
    codes, scales = ref.encode(np.zeros((2, 16), np.float32))
    assert not codes.any() and (scales == ref.TINY).all()
    for bad in (np.nan, np.inf, -np.inf):
        codes, scales = ref.encode(np.full((1, 16), bad, np.float32))
        assert (codes == 0x7F).all() and np.isnan(scales).all()


def test_a_code_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((5, 400)) * np.exp2(rng.integers(-30, 30, (5, 1)))).astype(np.float32)
    codes, scales = ref.encode(x)
    v = ref.scaled(codes, scales)
    s = np.repeat(scales.T.astype(np.float64), 128, 1)[:, :400]
    assert (np.abs(v - x) <= np.abs(x) * (2.0 ** -4 + 2.0 ** -20) + s * 2.0 ** -10).all()


def test_weights_and_silu():
    codes = np.full((130, 144), 0x38, np.uint8)  # 1.0
    w = ref.weights(codes, [[2, 3], [5, 7]])
    assert w[0, 0] == 2 and w[127, 128] == 3 and w[128, 127] == 5 and w[129, 143] == 7
    assert ref.silu(0.0) == 0 and abs(ref.silu(1.0) - 0.7310585786300049) < 1e-15


def test_residual_norm():
    rng = np.random.default_rng(1)
    x, res, w = rng.standard_normal((3, 32)), rng.standard_normal((3, 32)), rng.standard_normal(32)
    z, r, y = ref.residual_norm(x, res, np.ones(32), None, 0.5, w, 0.0)
    assert np.allclose((2 * z) ** 2 @ np.ones(32), 32) and np.array_equal(r, res + z)
    assert np.allclose(((y / w) ** 2).mean(1), 1)
    assert np.allclose(ref.residual_norm(4 * x, None, None, None, 1.0, w, 0.0)[2],
                       ref.residual_norm(x, None, None, None, 1.0, w, 0.0)[2])  # a norm knows no size
    assert np.array_equal(ref.residual_norm(None, res, None, None, 9.0, None, 0.0)[1], res)
