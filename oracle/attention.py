"""fp64 definitions of the operators around attention (paged_slots,
qk_norm_rope_cache, tree_attention, token_logprobs): plain numpy loops over
requests, tokens and heads, straight from the formulas in include/bqd.h."""
import numpy as np

NEG = -np.inf


# ---------------------------------------------------------------- number formats
def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16(x):
    """Round fp32 to bf16 bit patterns, to nearest even (finite inputs)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def e4m3_table():
    """The 256 values of E4M3 (OCP FP8 v1.0, no infinities, NaN at S.1111.111)."""
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if (e == 15 and m == 7) else (-v if s else v)
    return t


# ---------------------------------------------------------------- paged_slots
def slots(context, fresh, free, table, page, capacity, depths=None):
    table = np.array(table, np.int32).copy()
    R, width = table.shape
    off, slot, pos, used, flags = [0], [], [], 0, 0
    for r in range(R):
        c, n = max(0, int(context[r])), max(0, int(fresh[r]))
        have, want = -(-c // page), -(-(c + n) // page)
        if n and want > width:
            flags |= 1
        for b in range(have, min(want, width)):
            table[r, b] = free[used] if used < len(free) else -1
            used += 1
        for j in range(n):
            b = (c + j) // page
            s = -1
            if b < width and table[r, b] >= 0:
                s = int(table[r, b]) * page + (c + j) % page
            t = off[-1] + j
            slot.append(s)
            pos.append(c + (int(depths[t]) if depths is not None and t < capacity else j))
        off.append(off[-1] + n)
    total = off[-1]
    if total > capacity:
        flags |= 2
    pad = max(0, capacity - total)
    return dict(table=table, offsets=np.array(off, np.int32),
                slots=np.array(slot[:capacity] + [-1] * pad, np.int64),
                positions=np.array(pos[:capacity] + [-1] * pad, np.int32),
                counts=np.array([total, min(used, len(free)), max(0, used - len(free)), flags], np.int32))


# ---------------------------------------------------------------- norm and rotation
def norm_rope(x, weight, eps, cos_sin_row, rot, pairs):
    """One head x [D] -> (y [D], size [D]): size bounds the magnitudes that met in each y."""
    y = np.array(x, np.float64)
    D = y.size
    if weight is not None:
        y = y / np.sqrt(np.sum(y * y) / D + eps) * np.asarray(weight, np.float64)
    out, size = y.copy(), np.abs(y)
    h = rot // 2
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + h)
        c, s = float(cos_sin_row[i]), float(cos_sin_row[h + i])
        out[a] = y[a] * c - y[b] * s
        out[b] = y[b] * c + y[a] * s
        size[a] = size[b] = abs(y[a]) + abs(y[b])
    return out, size


# ---------------------------------------------------------------- attention
def attention(q, k, v, seen, scale):
    """One (token, head): q [D], k, v [L][D], seen [L] bool -> out [D], lse, sum p |v| [D], max sum |q k|."""
    k, v = k[seen], v[seen]
    D = q.size
    if k.shape[0] == 0:
        return np.zeros(D), NEG, np.zeros(D), 0.0
    s = scale * (k @ q)
    m = s.max()
    e = np.exp(s - m)
    z = e.sum()
    p = e / z
    return p @ v, m + np.log(z), p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(scale))


def seen_of(ctx, n, i, mask_words=None):
    """Which of ctx + n logical positions draft i sees."""
    seen = np.zeros(ctx + n, bool)
    seen[:ctx] = True
    for j in range(n):
        if mask_words is None:
            seen[ctx + j] = j <= i
        elif j // 64 < len(mask_words):
            seen[ctx + j] = (int(mask_words[j // 64]) >> (j % 64)) & 1
    return seen


# ---------------------------------------------------------------- log probabilities
def logprobs(x, token, topk):
    """One row (fp32 values): logprob, entropy, top ids, their log probabilities."""
    x = np.asarray(x, np.float32)
    d = x.astype(np.float64)
    key = np.where(np.isnan(x), NEG, d)
    order = sorted(range(x.size), key=lambda i: (bool(np.isnan(x[i])), -key[i], i))[:topk]
    if np.isnan(d).any() or np.isposinf(d).any():
        nan = float("nan")
        return nan if 0 <= token < x.size else NEG, nan, order, np.full(topk, nan)
    m = d.max()
    if m == NEG:
        return NEG, 0.0, order, np.full(topk, NEG)
    e = np.exp(d - m)
    z = e.sum()
    lse = m + np.log(z)
    p = e[e > 0] / z
    lp = d[token] - lse if 0 <= token < x.size else NEG
    return lp, float(-(p * np.log(p)).sum()), order, d[order] - lse
