"""Plain 64-bit reference of the 4-bit paged cache: the row format, the sparse attention over held
rows, and the page calls as sequential bookkeeping.  numpy only; shares nothing with the library."""
from __future__ import annotations

import numpy as np

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite non-negative e4m3 values by code: subnormals m / 8 * 2^-6, then (1 + m / 8) * 2^(e - 7)
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def page_bytes(rows: int, D: int) -> int:
    return rows * (D // 2 + D // GROUP + 4)


def _nearest(v, levels):
    """Code of the level nearest to v >= 0; a tie goes to the even code; beyond the last, the last."""
    lo = np.clip(np.searchsorted(levels, v, side="right") - 1, 0, len(levels) - 1)
    hi = np.minimum(lo + 1, len(levels) - 1)
    below, above = v - levels[lo], levels[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where((hi > lo) & up, hi, lo)


def encode(x):
    """codes uint8 [N, D / 2], scale codes uint8 [N, D / 16], row scales float32 [N] of rows x (float64 [N, D])."""
    N, D = x.shape
    codes = np.zeros((N, D // 2), np.uint8)
    s8 = np.zeros((N, D // GROUP), np.uint8)
    r = np.zeros(N)
    for i in range(N):
        e = -100
        while np.abs(x[i]).max() > 6.0 * 448.0 * 2.0 ** e:
            e += 1
        r[i] = 2.0 ** e
        g = (x[i] / r[i]).reshape(-1, GROUP)
        s8[i] = _nearest(np.abs(g).max(1) / 6.0, E4M3)
        s = E4M3[s8[i]][:, None]
        c = _nearest(np.abs(g) / np.where(s > 0, s, 1.0), E2M1) * (s > 0)
        c = (c + 8 * np.signbit(x[i].reshape(-1, GROUP))).reshape(-1).astype(np.uint8)
        codes[i] = c[0::2] | (c[1::2] << 4)
    return codes, s8, r.astype(np.float32)


def decode(codes, s8, r):
    """float64 values [..., D] of held rows."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = E4M3[np.minimum(s8 & 0x7F, 126)]
    return v * np.repeat(s, GROUP, -1) * np.asarray(r, np.float64)[..., None]


def put_row(cache, page, at, rows, D, codes, s8, r):
    """One held row into a pool's bytes (uint8 [P, page bytes])."""
    a, b = rows * D // 2, rows * (D // 2 + D // GROUP)
    cache[page, at * D // 2:(at + 1) * D // 2] = codes
    cache[page, a + at * D // GROUP:a + (at + 1) * D // GROUP] = s8
    cache[page, b + 4 * at:b + 4 * at + 4] = np.frombuffer(np.float32(r).tobytes(), np.uint8)


def get_row(cache, page, at, rows, D):
    a, b = rows * D // 2, rows * (D // 2 + D // GROUP)
    return (cache[page, at * D // 2:(at + 1) * D // 2], cache[page, a + at * D // GROUP:a + (at + 1) * D // GROUP],
            np.frombuffer(cache[page, b + 4 * at:b + 4 * at + 4].tobytes(), np.float32)[0])


def place(table, P, rows, seq, pos):
    """(page, row in it) of row pos of sequence seq, or None."""
    R, M = table.shape
    if not (0 <= seq < R and 0 <= pos < M * rows):
        return None
    page = int(table[seq, pos // rows])
    return (page, pos % rows) if 0 <= page < P else None


def attend(q, kv, sink, scale):
    """One token: q [H, D], kv [n, D] (its listed rows), float64.  Returns out [H, D], lse [H], p [H, n], x [H, n]."""
    H, D = q.shape
    x = scale * (q @ kv.T)
    s = np.full((H, 1), -np.inf) if sink is None else np.asarray(sink, np.float64)[:, None]
    m = np.maximum(x.max(1, initial=-np.inf, keepdims=True), s)
    m = np.where(np.isinf(m), 0.0, m)
    w = np.exp(x - m)
    z = w.sum(1, keepdims=True) + np.exp(s - m)
    p = w / np.where(z > 0, z, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(z))[:, 0]
    return p @ kv, lse, p, x


def attend_tolerance(q, kv, r, p, x, out, lse, scale):
    """Bounds of |out - exact| [H, D] and |lse - exact| [H] for the kernel's arithmetic (u = 2^-24):
      * the output's rounding to bf16: 2^-8 |o|;
      * the weight of row j comes out within a factor e^(+-E_j): its score is a D-term fp32 sum of exact
        products, off by at most 4 D u scale sum |q||kv_j| (each addition rounded or cut, 2 u); its exponent, of
        magnitude X_j = |x_j| log2 e + |log2 r_j|, carries a few fp32 roundings (8 u X_j), the hardware exponential
        2^-22, the row scale's logarithm 2^-22, their sum over n rows 2 n u.  With p_j the exact share, the output
        moves by sum_j dp_j (|kv_j| + |o|), dp_j = p_j (e^(2 E_j) - 1) and at most 1, and lse by
        ln sum_j p_j e^(2 E_j);
      * weights rounded to fp16: half a step, 2^-11 of each, and below 2^-14 of the unit 2^-25 of it.  The unit is
        at most the largest r e^x, so relative to the denominator at most U = max r p, and it multiplies |kv| / r.
    """
    u = 2.0 ** -24
    D, n = q.shape[1], kv.shape[0]
    flat = 8 * u * np.abs(np.where(np.isinf(lse), 0, lse)) + 2.0 ** -21
    if n == 0:
        return np.zeros_like(out) + 1e-30, flat
    X = np.abs(x) * 1.4427 + np.abs(np.log2(r))[None, :]
    E = 4 * D * u * scale * (np.abs(q) @ np.abs(kv).T) + 8 * u * X + 2.0 ** -20 + 2 * n * u
    logp = x - lse[:, None]
    dp = np.exp(np.minimum(logp + 2 * E, 0.0)) - np.exp(np.minimum(logp, 0.0))
    U = (p * r[None, :]).max(1, keepdims=True)
    tol = (2.0 ** -8 * np.abs(out) + dp @ np.abs(kv) + dp.sum(1, keepdims=True) * np.abs(out)
           + 2.0 ** -11 * (p @ np.abs(kv)) + n * 2.0 ** -25 * U * (np.abs(kv) / r[:, None]).max(0)[None, :])
    top = (logp + 2 * E).max(1, keepdims=True)
    grow = top[:, 0] + np.log(np.exp(logp + 2 * E - top).sum(1) + np.exp(np.log1p(-np.minimum(p.sum(1), 1 - 1e-16)) - top[:, 0]))
    return tol * 1.01 + 1e-30, np.maximum(grow, 0) + flat


# ------------------------------------------------------------------------------------- page calls


def counts(table, P):
    t = table[(table >= 0) & (table < P)]
    return np.bincount(t.reshape(-1), minlength=P).astype(np.int32)


def fork(table, parent, ref):
    """(table, ref) after dsa_fork_pages, one row at a time."""
    R, M = table.shape
    out, ref = np.full_like(table, -1), ref.copy()
    P = len(ref)
    for r in range(R):
        if 0 <= parent[r] < R:
            out[r] = table[parent[r]]
        for a, b in zip(table[r], out[r]):
            if 0 <= b < P:
                ref[b] += 1
            if 0 <= a < P:
                ref[a] -= 1
    return out, ref


def reserve(table, ref, begin, end, rows):
    """(table, ref, src, dst, lacking) after dsa_reserve_pages, one page at a time."""
    R, M = table.shape
    P = len(ref)
    free = [p for p in range(P) if ref[p] <= 0]
    needs = []
    for r in range(R):
        b, e = max(0, int(begin[r])), min(int(end[r]), M * rows)
        if b < e:
            for j in range(b // rows, (e - 1) // rows + 1):
                p = int(table[r, j])
                if not 0 <= p < P or ref[p] > 1:
                    needs.append((r, j, p if 0 <= p < P else -1, b, e))
    src, dst = np.full(2 * R, -1, np.int32), np.full(2 * R, -1, np.int32)
    if len(needs) > len(free):
        return table.copy(), ref.copy(), src, dst, len(needs) - len(free)
    table, new = table.copy(), ref.copy()
    for (r, j, old, b, e), page in zip(needs, free):
        table[r, j] = page
        new[page] = 1
        if old >= 0:
            new[old] -= 1
            if b > j * rows or e < (j + 1) * rows:  # some of its rows are not about to be written
                i = 2 * r + (0 if j == b // rows else 1)
                src[i], dst[i] = old, page
    return table, new, src, dst, 0


def compact(table, ref):
    """(table, ref, src, dst, n_live) after dsa_compact_pages."""
    P = len(ref)
    used = [p for p in range(P) if ref[p] > 0]
    L = len(used)
    to = {p: p for p in used if p < L}
    moves = [p for p in used if p >= L]
    gaps = [p for p in range(L) if ref[p] <= 0]
    src, dst = np.full(P // 2, -1, np.int32), np.full(P // 2, -1, np.int32)
    for k, (a, b) in enumerate(zip(moves, gaps)):
        to[a] = b
        src[k], dst[k] = a, b
    new = np.zeros_like(ref)
    for p in used:
        new[to[p]] = ref[p]
    t = np.array([to.get(int(p), -1) for p in table.reshape(-1)], np.int32).reshape(table.shape)
    return t, new, src, dst, L
