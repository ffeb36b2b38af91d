"""Shared pieces of the tests of the calls on 8-bit activations: outputs with guard rows, random codes, and the
bounds of codes."""
import numpy as np
import torch

import block_quantized_decode_nvfp4_gb300 as bqd
from oracle import fp8 as ref

TYPES = {"f32": (torch.float32, bqd.BQD_F32), "bf16": (torch.bfloat16, bqd.BQD_BF16), "e4m3": (torch.uint8, bqd.BQD_E4M3)}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # a rounding is off by at most this much of the value
GUARD = 256


class Out:
    """A device output of a shape between two guard bands that nothing may touch."""

    def __init__(self, shape, kind, fill=0x5A):
        self.shape, self.dt = shape, TYPES[kind][0]
        self.n = int(np.prod(shape)) * torch.empty(0, dtype=self.dt).element_size()
        self.buf = torch.full((self.n + 2 * GUARD,), fill, dtype=torch.uint8, device="cuda")
        self.fill = fill

    @property
    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def get(self):
        raw = self.buf.cpu()
        assert (raw[:GUARD] == self.fill).all() and (raw[GUARD + self.n:] == self.fill).all(), "written past the output"
        t = raw[GUARD:GUARD + self.n].clone().view(self.dt).view(self.shape)
        return t.numpy() if self.dt == torch.uint8 else t.double().numpy()


def rows(T, K, seed, spread=6):
    """fp32 rows of different size, a few channels far larger than the rest."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-spread, spread + 1, (T, 1)))
    return (x * (1 + 30 * (rng.random(K) < 0.02))).astype(np.float32)


def to_type(x, kind):
    """Device tensor of a type, and its values."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[kind][0])
    return t.cuda(), t.double().numpy()


def codes(shape, seed):
    """E4M3 codes of all kinds but NaN."""
    c = np.random.default_rng(seed).integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 0x7F) == 0x7F, c & 0x81, c).astype(np.uint8)


def scale_array(shape, seed, lo=-12, hi=-2):
    return np.exp2(np.random.default_rng(seed).uniform(lo, hi, shape)).astype(np.float32)


def check_codes(got, got_s, want, slack, what=""):
    """Codes and scales of values known to within `slack` (an array as `want`): the scale is that of some value
    within the slack, and a code's value is within half a step of one: 2^-4 of the value, or 2^-10 of the scale
    among the subnormal codes."""
    m, d = ref.block_max(want), ref.block_max(slack)
    lo, hi = np.maximum((m - d) / 448, ref.TINY), np.maximum((m + d) / 448, ref.TINY)
    s = got_s.astype(np.float64).T
    assert (s >= lo * (1 - 2.0 ** -23)).all() and (s <= hi * (1 + 2.0 ** -23)).all(), what + ": scales"
    full = np.repeat(s, 128, 1)[:, :want.shape[1]]
    err = np.abs(ref.scaled(got, got_s) - want)
    # the largest value may have been rounded above 448 s by the scale's own rounding and saturated: 2^-23 of it
    tol = slack + 2.0 ** -4 * (np.abs(want) + slack) + full * 2.0 ** -10 + np.abs(want) * 2.0 ** -22
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} codes outside, first {np.argwhere(bad)[0]}, err {err[bad][0]} tol {tol[bad][0]}"
