"""Plain references, in 64 bits, of the bf16 paged cache's calls and of the drafts' check, and makers of pools and tables."""
from __future__ import annotations

import math

import numpy as np
import torch


def pool(lens, rows, D, rng, M=None, spare=2, fill=float("nan"), device="cuda"):
    """A pool of pages (bf16 [P, rows, D], `fill` where nobody wrote), the table of sequences of these lengths, their rows in
    float64 and the generator's rows written in place."""
    need = [-(-int(n) // rows) for n in lens]
    M = M if M is not None else max(need + [1])
    P = sum(need) + spare
    ids = rng.permutation(P)
    table = np.full((len(lens), M), -1, np.int32)
    pages = torch.full((P, rows, D), fill, dtype=torch.bfloat16)
    kv, at = [], 0
    for r, n in enumerate(lens):
        table[r, :need[r]] = ids[at:at + need[r]]
        x = torch.from_numpy(rng.standard_normal((int(n), D)) * 2.0 ** rng.integers(-2, 3, (int(n), 1))).to(torch.bfloat16)
        for i in range(need[r]):
            part = x[i * rows:(i + 1) * rows]
            pages[ids[at + i], :len(part)] = part
        kv.append(x.double())
        at += need[r]
    return pages.to(device), torch.from_numpy(table).to(device), kv


def attn(q, kv, seq, pos, window, first, sink, scale, skip=None):
    """out, lse and A = sum of weight * |kv| (all float64) of q [T, H, D] over the sequences' rows kv[r]; rows in `skip` (pairs
    sequence, row) are not there."""
    T, H, D = q.shape
    out, size = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    q = q.double().cpu()
    err = torch.zeros(T, H, dtype=torch.float64)  # sum |q| |k| of the largest score
    for t in range(T):
        r, p = int(seq[t]), int(pos[t])
        j = torch.zeros(0, dtype=torch.long)
        if 0 <= r < len(kv) and p >= 0:
            j = torch.arange(min(p + 1, len(kv[r])))
            if window:
                j = j[(j > p - window) | (j < first)]
            if skip:
                j = j[torch.tensor([(r, int(i)) not in skip for i in j], dtype=torch.bool)]
        x = scale * (q[t] @ kv[r][j].T) if len(j) else torch.zeros(H, 0, dtype=torch.float64)
        z = x if sink is None else torch.cat([x, sink.double().cpu()[:, None]], 1)
        if z.shape[1] == 0:
            continue
        lse[t] = torch.logsumexp(z, 1)
        w = torch.exp(x - lse[t][:, None])
        if len(j):
            out[t], size[t] = w @ kv[r][j], w @ kv[r][j].abs()
            err[t] = (abs(scale) * (q[t].abs() @ kv[r][j].abs().T)).amax(1)
    return out, lse, size, err


def check_attn(got, lse, ref, D, worst=None):
    """Bounds.  A score is a sum of D products of bf16 values (exact in fp32) in fp32, in any order, and may lose half a step, 2^-24 of
    what was summed, or a whole one where it is cut off, with each: E = D 2^-23 sum |q k| scale at most; the scaling to
    log2 units, the bound's subtraction (exponents up to 2^7 with steps of 2^-17) and the exponential add 2^-16.  Both the weights and
    their sum have that error: 2 (E + 2^-16); a weight is rounded to bf16: 2^-8; the weighted sum of n terms in fp32 adds
    n 2^-23 at most, 2^-8 of it for n up to 2^15.  The output is rounded to bf16: 2^-8 of it."""
    o, l, size, err = ref
    e = D * 2.0 ** -23 * err + 2.0 ** -16
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2 * e)[..., None] * size + 1e-30
    d = (got.double().cpu() - o).abs()
    assert not torch.isnan(d).any()
    assert (d <= tol).all(), f"out: worst {float((d / tol).max()):.3g} of the bound"
    if lse is not None:
        a, b = lse.double().cpu(), l
        assert torch.equal(a == -math.inf, b == -math.inf)
        some = b > -math.inf
        d = (a - b).abs()[some]
        assert (d <= (e + 2.0 ** -20 * (1 + b.abs()))[some]).all()


def maps(held, added, T):
    seq, pos, ks, ke = (np.full(T, v, np.int64) for v in (-1, -1, 0, 0))
    t = base = 0
    for r, (h, a) in enumerate(zip(held, added)):
        h, a = max(0, int(h)), max(0, int(a))
        n = max(0, min(a, T - t))
        seq[t:t + n], pos[t:t + n], ks[t:t + n] = r, h + np.arange(n), base
        ke[t:t + n] = base + h + np.arange(n) + 1
        t += a
        base += h + a
    top = 2 ** 31 - 1
    return [np.minimum(x, top) for x in (seq, pos, ks, ke)]


def slots(table, P, rows, seq, start, idx):
    R, M = table.shape
    out = np.full(idx.shape, -1, np.int64)
    for t in range(idx.shape[0]):
        for k in range(idx.shape[1]):
            v, s = int(idx[t, k]), int(seq[t])
            j = v - (int(start[t]) if start is not None else 0)
            if v >= 0 and j >= 0 and 0 <= s < R and j // rows < M and 0 <= table[s, j // rows] < P:
                out[t, k] = int(table[s, j // rows]) * rows + j % rows
    return out


UNIT = 2 ** 55


def units(p):
    """fp32 probabilities in whole multiples of 2^-55, the nearest ones, as Python ints."""
    p = np.asarray(p, np.float32)
    p = np.where(p > 0, np.minimum(p, np.float32(1)), np.float32(0)).astype(np.float64)  # (no number: 0)
    return [int(v) for v in np.rint(p * UNIT)]  # (the product is exact: 24 bits times a power of two; ties to even)


def verify(target, draft, tokens, count, u):
    """Accepted and following token, in whole numbers and fractions of them."""
    from fractions import Fraction

    R, G = tokens.shape
    V = target.shape[2]
    accepted, token = [], []
    for r in range(R):
        n = min(int(count[r]), G)
        if n < 0:
            accepted.append(0), token.append(-1)
            continue
        a = 0
        while a < n:
            d = int(tokens[r, a])
            if not 0 <= d < V or not float(u[r, a]) * float(draft[r, a, d]) < float(target[r, a, d]):
                break
            a += 1
        p = units(target[r, a])
        w = p
        if a < n:
            w = [max(0, x - y) for x, y in zip(p, units(draft[r, a]))]
            w = w if any(w) else p
        s, x = 0, min(max(Fraction(float(u[r, G])), Fraction(0)), 1 - Fraction(1, 2 ** 64)) * sum(w)
        at = -1
        for v, y in enumerate(w):
            s += y
            if s > x:
                at = v
                break
        accepted.append(a), token.append(at)
    return np.array(accepted), np.array(token)
