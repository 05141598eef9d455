"""The 4-bit paged cache on the GPU: rows in and back, and the sparse attention over them, against the
64-bit reference (tests/kv4_ref.py).  Held rows are compared byte for byte; the attention within
kv4_ref.attend_tolerance, which derives its bounds from the kernel's arithmetic."""
import numpy as np
import pytest

import kv4_ref as K4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_indexer_e4m3_gb300 as m
    from sparse_attention_indexer_e4m3_gb300 import build

    build.build()
    m.load()
    return m


def dev(a, t=None):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a if t is None else np.asarray(a, t))).cuda()


def bf16(a):
    """(the bf16 tensor nearest to a, its values in 64 bits)"""
    import torch

    t = torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def rows_of(rng, n, D, spread=6):
    x = rng.standard_normal((n, D)) * 2.0 ** rng.integers(-spread, spread + 1, (n, 1))
    x[:, ::7] *= rng.choice([1.0, 30.0], (n, 1))
    x[rng.random(x.shape) < 0.05] = 0.0
    return x


def make_pool(rng, R, M, D, B, rows, spare=3, fill=0xFF):
    """A pool with a shuffled table [R, M] whose every page is mapped and bytes `fill` (NaN scales)."""
    P = R * M + spare
    table = rng.permutation(P)[:R * M].reshape(R, M).astype(np.int32)
    return table, np.full((P, K4.page_bytes(B, D)), fill, np.uint8)


# ------------------------------------------------------------------------------------ the codec


@pytest.mark.parametrize("D,B,N", [(64, 16, 1), (64, 256, 333), (128, 32, 77), (256, 64, 130), (512, 64, 61), (512, 128, 259)])
def test_codec_bytes_and_values(dsa, D, B, N):
    rng = np.random.default_rng(D + B + N)
    R, M = 3, max(2, -(-N // B))
    table, cache = make_pool(rng, R, M, D, B, N)
    table[1, 0] = -1  # no page
    table[2, M - 1] = len(cache) + 4  # no page either
    where = rng.permutation(R * M * B)[:N]
    seq, pos = where // (M * B), where % (M * B)
    if N > 8:
        seq[3], seq[4], pos[5], pos[6] = -1, R, -1, M * B
    x = rows_of(rng, N, D)
    if N > 20:
        x[7] = 0.0
        x[8] = -0.0
        x[9] = rng.standard_normal(D) * 2.0 ** -126   # below what the least row scale resolves: all codes 0
        x[10] = 2.0 ** 120 * rng.standard_normal(D)
        x[11] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], D)  # borders between codes
        x[12] = np.repeat(2.0 ** -np.arange(D // 16), 16) * rng.choice([-6.0, 6.0, 1.0], D)  # scales down to nothing
        x[13] = 1.0
    t, x = bf16(x)
    ct = dev(cache)
    want = cache.copy()
    codes, s8, r = K4.encode(x)
    held = K4.decode(codes, s8, r)
    for i in range(N):
        at = K4.place(table, len(cache), B, int(seq[i]), int(pos[i]))
        if at is None:
            held[i] = 0.0
        else:
            K4.put_row(want, *at, B, D, codes[i], s8[i], r[i])
    assert dsa.quantize_kv4(t, ct, dev(table), dev(seq, np.int32), dev(pos, np.int32)) is ct
    assert np.array_equal(ct.cpu().numpy(), want)  # every other byte stays
    back = dsa.dequantize_kv4(ct, dev(table), dev(seq, np.int32), dev(pos, np.int32), D)
    assert np.array_equal(back.double().cpu().numpy(), held)


def test_codec_every_exponent_and_mantissa(dsa):
    """Every bf16 magnitude as a row's largest value, with a fixed set of fractions of it beside it."""
    import torch

    D, B = 64, 256
    bits = np.arange(1, 0x7F80, dtype=np.uint16)
    top = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    rng = np.random.default_rng(5)
    frac = np.concatenate([[1.0, -1.0, 0.5, 1 / 24, 1 / 6, 5 / 12, 7 / 24, 0.0], rng.uniform(-1, 1, D - 8)])
    t, x = bf16(top[:, None] * frac[None, :])
    N = len(top)
    M = -(-N // B)
    table = np.arange(M, dtype=np.int32)[None, :]
    ct = torch.zeros(M, K4.page_bytes(B, D), dtype=torch.uint8, device="cuda")
    pos, seq = np.arange(N), np.zeros(N)
    dsa.quantize_kv4(t, ct, dev(table), dev(seq, np.int32), dev(pos, np.int32))
    got = dsa.dequantize_kv4(ct, dev(table), dev(seq, np.int32), dev(pos, np.int32), D).double().cpu().numpy()
    held = K4.decode(*K4.encode(x))
    # a scale rounded up can take values next to the largest bf16 past it: the nearest bf16 is infinity there
    held = np.where(np.abs(held) >= 511 * 2.0 ** 119, np.copysign(np.inf, held), held)
    assert np.isinf(held[-20:]).any() and np.isfinite(held[:-256]).all()
    assert np.array_equal(got, held)


def test_codec_row_scales_of_others(dsa):
    """Rows whose scale is no power of two (another writer's): r s c rounded to bf16 (half a step, 2^-8)."""
    rng = np.random.default_rng(1)
    D, B, N = 128, 16, 16
    cache = rng.integers(0, 256, (1, K4.page_bytes(B, D)), dtype=np.uint8)
    cache[0, B * D // 2:] &= 0x77  # scale codes without sign, none NaN
    r = rng.uniform(0.01, 3.0, N).astype(np.float32)
    held = np.zeros((N, D))
    for i in range(N):
        c, s, _ = K4.get_row(cache, 0, i, B, D)
        K4.put_row(cache, 0, i, B, D, c, s, r[i])
        held[i] = K4.decode(c, s, r[i])
    table = np.zeros((1, 1), np.int32)
    got = dsa.dequantize_kv4(dev(cache), dev(table), dev(np.zeros(N), np.int32), dev(np.arange(N), np.int32), D)
    # fp32 product (2^-24), then bf16 (2^-8)
    assert np.all(np.abs(got.double().cpu().numpy() - held) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(held))


# ------------------------------------------------------------------------------------ the attention


class Case:
    """A pool with R sequences of `length` written rows each, T tokens and their lists."""

    def __init__(self, seed, T, H, D, K, B, R=2, length=300, sink=False, q_scale=1.0, spread=3, start=True, one_each=False):
        rng = self.rng = np.random.default_rng(seed)
        self.D, self.B, self.T, self.H, self.K, self.R = D, B, T, H, K, R
        M = -(-length // B) + 1
        self.table, self.cache = make_pool(rng, R, M, D, B, length)
        self.table[:, M - 1] = [-1, 10 ** 9][:1] * R  # the last page of every sequence is not mapped
        self.kv = np.zeros((R, M * B, D))
        self.r = np.zeros((R, M * B))
        for s in range(R):
            _, x = bf16(rows_of(rng, length, D, spread))
            codes, s8, r = K4.encode(x)
            self.kv[s, :length] = K4.decode(codes, s8, r)
            self.r[s, :length] = r
            for i in range(length):
                K4.put_row(self.cache, *K4.place(self.table, len(self.cache), B, s, i), B, D, codes[i], s8[i], r[i])
        self.length = length
        self.seq = rng.integers(0, R, T)
        self.start = rng.integers(0, 1000, T) if start else np.zeros(T, np.int64)
        self.idx = rng.integers(0, length, (T, K)) + self.start[:, None]
        self.q_t, self.q = bf16(rng.standard_normal((T, H, D)) * q_scale)
        self.sink = rng.standard_normal(H).astype(np.float32) * 2 if sink else None
        self.scale = 0.6 / (np.sqrt(D) * q_scale)
        self.use_start = start

    def listed(self, t):
        """kv rows and row scales that token t attends to."""
        kv, r = [], []
        for v in self.idx[t]:
            p = int(v) - int(self.start[t])
            if v >= 0 and K4.place(self.table, len(self.cache), self.B, int(self.seq[t]), p) is not None:
                kv.append(self.kv[self.seq[t], p])
                r.append(self.r[self.seq[t], p])
        return np.array(kv).reshape(-1, self.D), np.array(r)

    def run(self, dsa, **kw):
        import torch

        lse = torch.full((self.T, self.H), 77.0, device="cuda")
        out = dsa.sparse_attn_kv4(self.q_t, dev(self.cache), dev(self.table), dev(self.seq, np.int32),
                                  dev(self.idx, np.int32), start=dev(self.start, np.int32) if self.use_start else None,
                                  attn_sink=None if self.sink is None else dev(self.sink), scale=self.scale, lse=lse, **kw)
        assert dsa.get_device_error() == 0
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, out, lse, rows=None):
        for t in range(self.T) if rows is None else rows:
            kv, r = self.listed(t)
            o, l, p, x = K4.attend(self.q[t], kv, self.sink, self.scale)
            to, tl = K4.attend_tolerance(self.q[t], kv, r, p, x, o, l, self.scale)
            bad = np.argwhere(~(np.abs(out[t] - o) <= to))
            assert len(bad) == 0, (t, len(bad), bad[0], out[t][tuple(bad[0])], o[tuple(bad[0])], to[tuple(bad[0])])
            same = (lse[t] == l) | (np.abs(lse[t] - l) <= tl)
            assert np.all(same), (t, lse[t][~same], l[~same])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("H,K,B,sink", [(1, 1, 16, False), (20, 77, 32, True), (64, 129, 64, False), (65, 128, 256, True)])
def test_attention_shapes(dsa, D, H, K, B, sink):
    c = Case(D + H + K, 5, H, D, K, B, sink=sink, length=200)
    c.check(*c.run(dsa))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_attention_shared_lists(dsa, D):
    """One token and three: a cluster of CTAs shares each list (8, 4 and 2 shares)."""
    for T, H, K in ((1, 64, 2048), (3, 130, 700), (30, 64, 400)):
        c = Case(D + T, T, H, D, K, 64, sink=T == 3, length=500)
        c.check(*c.run(dsa))


@pytest.mark.parametrize("D", [128, 512])
@pytest.mark.parametrize("K", [300, 385, 600, 900, 1100, 1500, 1900, 5000])
def test_attention_share_counts(dsa, D, K):
    """Lists of 3 to 40 blocks for one token: 3, 4, 5, 8, 9, 12, 15 and 14 shares of one to three blocks (as far as the device
    has such clusters), ragged lists whose last shares hold nothing, an empty one."""
    c = Case(D + K, 4, 20, D, K, 64, length=500, sink=True)
    for t in range(c.T):
        c.idx[t, [K, K // 2, 130, 0][t]:] = -1
    c.check(*c.run(dsa))


def test_attention_workspace(dsa):
    import torch

    c = Case(21, 2, 64, 512, 700, 64, length=500)
    need = dsa.sparse_attn_kv4_workspace_size(c.T, c.H, c.D, c.K)
    assert need > 0 and dsa.sparse_attn_kv4_workspace_size(4096, 64, 512, 2048) == 0
    want = c.run(dsa)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.run(dsa, workspace=ws)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    for bad in (ws[:need - 16], ws[8:]):
        with pytest.raises(dsa.DsaError) as e:
            c.run(dsa, workspace=bad)
        assert e.value.status == 3


@pytest.mark.parametrize("D,H,T", [(64, 64, 400), (128, 20, 400), (256, 130, 170), (512, 64, 330)])
def test_attention_many_tokens(dsa, D, H, T):
    """More units than SMs, ragged lists with holes, entries out of range, rows without a key at the first and last
    token and between, repeated entries, unmapped pages, pages and sequences that do not exist."""
    c = Case(D + H, T, H, D, 300, 32, R=3, sink=True, length=280)
    rng = c.rng
    c.idx[rng.random(c.idx.shape) < 0.15] = -1
    for t in range(T):
        c.idx[t, 300 - (t * 7) % 301:] = -1
    c.idx[0] = c.idx[T // 2] = c.idx[T - 1] = -1
    c.idx[3, :5] = c.idx[3, 5]
    c.idx[4, ::3] = c.start[4] + 290        # the unmapped page (rows 288 to 319)
    c.idx[5, ::2] = c.start[5] + 10 ** 6    # behind the table's row
    c.idx[6, ::2] = np.maximum(c.start[6] - 3, 0)  # before the sequence
    c.idx[7] = 2 ** 31 - 1
    c.seq[8], c.seq[9] = -1, 3
    c.table[1, 2] = len(c.cache)
    c.table[2, 0] = -(2 ** 31)
    out, lse = c.run(dsa)
    c.check(out, lse, rows=list(range(12)) + list(range(12, T, 9)) + [T // 2, T - 1])
    for t in (0, 7, 8, 9, T // 2, T - 1):
        assert np.all(out[t] == 0.0) and np.allclose(lse[t], c.sink, rtol=2.0 ** -22)


@pytest.mark.parametrize("D,H", [(64, 16), (128, 64), (256, 65), (512, 64)])
def test_attention_mostly_empty_lists(dsa, D, H):
    """Long runs of tokens without entries between tokens with one to three blocks."""
    c = Case(31 + D, 1300, H, D, 300, 32, R=3, length=200, sink=True)
    rng = c.rng
    keep = rng.random(c.T) < 0.3
    keep[400:800] = False
    keep[1299] = True
    c.idx[~keep] = -1
    for t in np.flatnonzero(keep):
        c.idx[t, rng.integers(1, 301):] = -1
    out, lse = c.run(dsa)
    assert np.all(out[~keep] == 0.0) and np.allclose(lse[~keep], c.sink, rtol=2.0 ** -22)
    c.check(out, lse, rows=np.flatnonzero(keep)[::17])


def test_attention_very_long_list(dsa):
    """70,000 entries over 500 rows: every row counts about 140 times."""
    c = Case(41, 2, 5, 128, 70000, 64, length=500)
    c.idx[1, 65000:] = -1
    c.check(*c.run(dsa))


def test_attention_no_keys_at_all(dsa):
    c = Case(1, 3, 5, 128, 4, 16)
    c.idx[:] = -1
    out, lse = c.run(dsa)
    assert np.all(out == 0) and np.all(lse == -np.inf)
    c.idx = c.idx[:, :0]
    out, lse = c.run(dsa)
    assert np.all(out == 0) and np.all(lse == -np.inf)
    c.sink = np.array([0.0, 3.0, -200.0, 300.0, -np.inf], np.float32)
    out, lse = c.run(dsa)
    assert np.all(out == 0) and np.allclose(lse, c.sink, rtol=2.0 ** -22)
    import torch

    c.T, c.q_t, c.idx, c.seq, c.start = 0, c.q_t[:0], c.idx[:0], c.seq[:0], c.start[:0]
    assert c.run(dsa)[0].shape == (0, 5, 128)
    e = torch.empty(0, K4.page_bytes(16, 128), dtype=torch.uint8, device="cuda")
    q, _ = bf16(np.ones((2, 5, 128)))
    out = dsa.sparse_attn_kv4(q, e, dev(np.zeros((0, 4), np.int32)), dev(np.zeros(2, np.int32)), dev(np.ones((2, 9), np.int32)))
    assert torch.all(out == 0)  # an empty pool and an empty table


@pytest.mark.parametrize("q_scale", [2.0 ** -70, 1e-3, 300.0, 2.0 ** 90])
@pytest.mark.parametrize("T", [2, 160])
def test_attention_q_range(dsa, q_scale, T):
    c = Case(3, T, 9, 128, 200, 32, q_scale=q_scale, sink=True)
    c.check(*c.run(dsa), rows=range(0, T, 13))


@pytest.mark.parametrize("T", [2, 160])
def test_attention_row_scales(dsa, T):
    """Rows of very different size in one list, rows of zeros (their score is 0: they count in the denominator), and
    a row much larger than the rest that its score all but excludes."""
    c = Case(4, T, 33, 256, 300, 32, spread=0, sink=False)
    rng = c.rng
    for s in range(c.R):
        x = rows_of(rng, c.length, c.D, 0)
        x[::3] *= 2.0 ** -40
        x[1::6] = 0.0
        x[5] *= 2.0 ** 20
        _, x = bf16(x)
        codes, s8, r = K4.encode(x)
        c.kv[s, :c.length], c.r[s, :c.length] = K4.decode(codes, s8, r), r
        for i in range(c.length):
            K4.put_row(c.cache, *K4.place(c.table, len(c.cache), c.B, s, i), c.B, c.D, codes[i], s8[i], r[i])
    c.idx[:, :] = rng.integers(0, c.length, c.idx.shape) + c.start[:, None]
    c.idx[(c.idx - c.start[:, None]) == 5] = -1
    c.idx[0, 7] = c.start[0] + 5
    c.idx[1] = (rng.integers(0, c.length // 6, c.K) * 6 + 1) + c.start[1]  # only rows of zeros
    out, lse = c.run(dsa)
    assert np.all(out[1] == 0.0) and np.allclose(lse[1], np.log(c.K), rtol=1e-6)
    c.check(out, lse, rows=[0] + list(range(2, T, 11)))


@pytest.mark.parametrize("T,K", [(1, 900), (170, 400)])
def test_attention_growing_scores(dsa, T, K):
    """Scores that rise along the list, so that the running bound moves and earlier blocks are rescaled; and a
    wide range of scores, where single keys take all the weight."""
    c = Case(6, T, 64, 128, K, 64, length=900, spread=1, start=False)
    c.scale *= 8.0
    order = np.argsort(np.einsum("d,srd->sr", c.q[0, 0], c.kv[:, :900]), axis=1)
    for t in range(T):
        c.idx[t] = order[c.seq[t]][np.linspace(0, 899, K).astype(int)]
    c.check(*c.run(dsa), rows=range(0, T, 13))


def test_attention_sinks(dsa):
    c = Case(7, 4, 6, 128, 150, 32)
    c.sink = np.array([0.0, 60.0, -60.0, 150.0, -np.inf, 5.0], np.float32)
    c.check(*c.run(dsa))


def test_attention_full_width(dsa):
    """The serving shape: 64 heads of 512, lists of 2048 over 5000 rows."""
    for T, H in ((2, 128), (160, 64)):
        c = Case(8, T, H, 512, 2048, 64, length=5000 if T == 2 else 2500, R=1)
        c.check(*c.run(dsa), rows=range(0, T, 40))


def test_attention_same_bits_every_time(dsa):
    for T in (2, 170):
        c = Case(9, T, 64, 512, 500, 64)
        a, b = c.run(dsa), c.run(dsa)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_codec_and_attention_behind_4_gib(dsa):
    """Pages whose bytes lie more than 2^32 into the pool."""
    import torch

    D, B, T, H, K = 512, 64, 3, 16, 100
    P = (9 << 29) // K4.page_bytes(B, D)
    cache = torch.zeros(P, K4.page_bytes(B, D), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    table = np.array([[P - 1, 0, P - 2, P // 2]], np.int32)
    t, x = bf16(rows_of(rng, 4 * B, D, 2))
    seq, pos = dev(np.zeros(4 * B), np.int32), dev(np.arange(4 * B), np.int32)
    dsa.quantize_kv4(t, cache, dev(table), seq, pos)
    codes, s8, r = K4.encode(x)
    kv = K4.decode(codes, s8, r)
    assert np.array_equal(dsa.dequantize_kv4(cache, dev(table), seq, pos, D).double().cpu().numpy(), kv)
    q_t, q = bf16(rng.standard_normal((T, H, D)))
    idx = rng.integers(0, 4 * B, (T, K))
    out = dsa.sparse_attn_kv4(q_t, cache, dev(table), dev(np.zeros(T), np.int32), dev(idx, np.int32))
    assert dsa.get_device_error() == 0
    sc = 1 / np.sqrt(D)
    for i in range(T):
        o, l, p, xx = K4.attend(q[i], kv[idx[i]], None, sc)
        to, _ = K4.attend_tolerance(q[i], kv[idx[i]], r[idx[i]].astype(np.float64), p, xx, o, l, sc)
        assert np.all(np.abs(out[i].double().cpu().numpy() - o) <= to)


def test_attention_on_streams_and_in_a_graph(dsa):
    """Two calls at once on two streams, and a captured call replayed on changed inputs."""
    import torch

    a, b = Case(11, 3, 64, 512, 600, 64, length=400), Case(12, 200, 20, 128, 200, 32)
    want = [c.run(dsa) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    args = []
    for c in (a, b):
        args.append((c.q_t, dev(c.cache), dev(c.table), dev(c.seq, np.int32), dev(c.idx, np.int32), dev(c.start, np.int32)))
    torch.cuda.synchronize()
    for _ in range(3):
        outs = [dsa.sparse_attn_kv4(*x[:5], start=x[5], scale=c.scale, stream=s) for x, c, s in zip(args, (a, b), streams)]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(o.double().cpu().numpy(), w[0])
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(a.q_t)
    with torch.cuda.graph(g):
        dsa.sparse_attn_kv4(*args[0][:5], start=args[0][5], scale=a.scale, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0][0])
    a.idx = (a.idx - a.start[:, None] + 17) % 400 + a.start[:, None]
    args[0][4].copy_(dev(a.idx, np.int32))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), a.run(dsa)[0])
    assert dsa.get_device_error() == 0
