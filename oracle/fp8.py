"""fp64 definitions of the calls on 8-bit activations (fp8_x_encode,
residual_norm, fp8_b128_gemm, fp8_b128_gemm_silu_mul): numpy, straight from
the formulas in include/bqd.h."""
import numpy as np

from oracle.attention import e4m3_table

TINY = np.float32(2.0 ** -126)
VALUES = e4m3_table()


def e4m3_codes(x):
    """Codes of fp32 values rounded to E4M3, to nearest even, saturated at 448; NaN is 0x7F. By the grid: every
    value between two neighbours of the table goes to the nearer, halfway to the even code."""
    x = np.asarray(x, np.float64)
    grid = VALUES[:0x7F]  # 0 .. 448, ascending
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    left, right = a - grid[lo], grid[hi] - a
    code = np.where(left < right, lo, np.where(right < left, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def block_max(x):
    """Largest magnitude of each block of 128 columns: [T][ceil(K/128)]; NaN or infinity if the block has one."""
    T, K = x.shape
    return np.stack([np.abs(x[:, j:j + 128]).max(1) for j in range(0, K, 128)], 1)


def encode(x):
    """Codes [T][K] and scales [ceil(K/128)][T] of fp32 rows: the scale and the quotients are fp32 operations."""
    x = np.asarray(x, np.float32)
    m = block_max(x)
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum(m / np.float32(448), TINY)
        s = np.where(np.isfinite(m), s, np.float32(np.nan)).astype(np.float32)
        q = x / np.repeat(s, 128, 1)[:, :x.shape[1]]
    return e4m3_codes(q), np.ascontiguousarray(s.T)


def scaled(codes, scales):
    """The values of 8-bit activations: codes [T][K], scales [ceil(K/128)][T]."""
    return VALUES[codes] * np.repeat(np.asarray(scales, np.float64).T, 128, 1)[:, :codes.shape[1]]


def weights(codes, scales):
    """The values of FP8 block-128 weights: codes [M][K], scales [ceil(M/128)][ceil(K/128)]."""
    M, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), 128, 0)[:M], 128, 1)[:, :K]
    return VALUES[codes] * s


def silu(g):
    return g / (1 + np.exp(-g))


def residual_norm(x, residual, post_weight, gate, scale, pre_weight, eps):
    """z scaled and gated, r and y as fp64 [T][H]; None stands for what a call leaves out."""
    z = None
    if x is not None:
        z = np.asarray(x, np.float64)
        if post_weight is not None:
            z = z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * np.asarray(post_weight, np.float64)
        if gate is not None:
            z = z * np.asarray(gate, np.float64)
        z = scale * z
    r = 0.0 if residual is None else np.asarray(residual, np.float64)
    r = r if z is None else r + z
    y = None
    if pre_weight is not None:
        y = r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * np.asarray(pre_weight, np.float64)
    return z, r, y
