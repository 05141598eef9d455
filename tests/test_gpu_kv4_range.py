"""The 4-bit cache's attention at the ends of its range: rows of any size beside one another, scores of any size,
q of any size head by head.  The bounds are those of kv4_ref.attend_tolerance."""
import numpy as np
import pytest

import kv4_ref as K4
from test_gpu_kv4 import Case, bf16, dsa, rows_of  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def hold(c, s, x):
    """Sequence s of case c holds the rows x from its first row on."""
    _, x = bf16(x)
    codes, s8, r = K4.encode(x)
    c.kv[s, :len(x)], c.r[s, :len(x)] = K4.decode(codes, s8, r), r
    for i in range(len(x)):
        K4.put_row(c.cache, *K4.place(c.table, len(c.cache), c.B, s, i), c.B, c.D, codes[i], s8[i], r[i])


# ------------------------------------------------------------------------------------ row scales


@pytest.mark.parametrize("order", ["mixed", "large first", "large last", "one large"])
@pytest.mark.parametrize("q", ["ordinary", "zeros"])
@pytest.mark.parametrize("big", [40, 80, 124])
@pytest.mark.parametrize("T,K", [(2, 900), (1, 300), (160, 300)])
def test_attention_small_rows_beside_large_ones(dsa, T, K, big, q, order):  # noqa: F811
    """Rows of zeros and of size 2^-60 beside rows of size 2^big, with scores of order 1 (or all 0): each counts in the
    denominator by its score alone, however far apart the row scales are (up to 2^-100 and 2^115)."""
    c = Case(big + T, T, 20, 128, K, 32, spread=0, sink=T == 1)
    rng, n = c.rng, c.length
    for s in range(c.R):
        x = rng.standard_normal((n, c.D))
        x[:100] *= 2.0 ** big
        x[100:200] = 0.0
        x[200:] *= 2.0 ** -60
        hold(c, s, x)
    large, small = lambda k: rng.integers(0, 100, k), lambda k: rng.integers(100, n, k)  # noqa: E731
    for t in range(T):
        part = {"mixed": rng.integers(0, n, K), "large first": np.concatenate([large(K // 2), small(K - K // 2)]),
                "large last": np.concatenate([small(K - K // 2), large(K // 2)]),
                "one large": np.concatenate([large(1), small(K - 1)])}[order]
        c.idx[t] = part + c.start[t]
    if q == "zeros":
        c.q_t.zero_()
        c.q[:] = 0.0
    else:
        c.scale *= 2.0 ** -big
    c.check(*c.run(dsa), rows=range(0, T, 13))


@pytest.mark.parametrize("D", [64, 256, 512])
def test_attention_zero_rows_behind_an_orthogonal_large_one(dsa, D):  # noqa: F811
    """A large row that q does not see, and K - 1 rows of zeros: every one of the K rows has the weight 1 / K."""
    c = Case(D, 170, 9, D, 2048, 64, spread=0, R=1, start=False)
    x = np.zeros((c.length, D))
    x[0, :16] = 2.0 ** 60
    hold(c, 0, x)
    c.q_t[:, :, :16] = 0.0
    c.q[:, :, :16] = 0.0
    c.idx[:] = np.concatenate([[0], c.rng.integers(1, c.length, c.K - 1)])
    c.idx[1] = c.rng.permutation(c.idx[1])
    c.idx[2] = c.idx[2][::-1]
    out, lse = c.run(dsa)
    # the bound m and log2 of the sum in its units, each at most 60, with a few fp32 roundings each: 4 2^-24 60
    assert np.allclose(lse, np.log(c.K), rtol=0, atol=2.0 ** -16)
    assert np.all(np.abs(out[:, :, 0] - c.kv[0, 0, 0] / c.K) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -19) * c.kv[0, 0, 0] / c.K)
    assert np.all(out[:, :, 16:] == 0.0)


def test_attention_sequence_of_growing_rows(dsa):  # noqa: F811
    """Row sizes that rise from 2^-80 to 2^120 along the list, so that every block raises the bounds by a great deal; one
    CTA for a list, and a list shared by several."""
    for T, K in ((3, 1200), (170, 700)):
        c = Case(T, T, 33, 256, K, 64, spread=0, length=400, start=False, sink=True)
        for s in range(c.R):
            hold(c, s, c.rng.standard_normal((c.length, c.D)) * 2.0 ** np.linspace(-80, 120, c.length)[:, None])
        c.idx[:] = np.sort(c.rng.integers(0, c.length, c.idx.shape), axis=1)
        c.scale *= 2.0 ** -119
        c.check(*c.run(dsa), rows=range(0, T, 23))


# ------------------------------------------------------------------------------------ scores


@pytest.mark.parametrize("T,K", [(2, 1), (2, 900), (170, 1)])
def test_attention_very_negative_scores(dsa, T, K):  # noqa: F811
    """A key whose score is -1e33 or so (q 2^60, kv -2^55, scale 0.05) is a key: alone in its list it has all the weight."""
    c = Case(T + K, T, 10, 128, K, 32, start=False)
    for s in range(c.R):
        hold(c, s, -np.abs(c.rng.standard_normal((c.length, c.D))) * 2.0 ** 55)
    c.q_t, c.q = bf16(np.abs(c.q) * 2.0 ** 60)
    c.idx[:, 1:] = -1
    if K > 1:
        c.idx[1] = np.roll(c.idx[1], K - 1)  # the only entry is the last
    out, lse = c.run(dsa)
    assert np.all(lse < -1e31)
    c.check(out, lse, rows=range(0, T, 13))


# ------------------------------------------------------------------------------------ q
#
# A head's q enters as fp16 times a power of two: each value is off by at most 2^-23 of the head's largest.  Beside
# attend_tolerance's 4 D 2^-24 of sum |q| |kv| that is little where the head's values are of one size (the largest of D normal
# values is below 6 times their mean), and where they are not, the tests below hold values that are exact all the same
# (8 significant bits, 2^19 below a largest value of 2^-4 or more).


@pytest.mark.parametrize("D,H,T", [(64, 7, 2), (128, 64, 3), (256, 20, 160), (512, 70, 2), (512, 64, 160)])
@pytest.mark.parametrize("low", [-20, -40, -100])
def test_attention_heads_of_different_size(dsa, D, H, T, low):  # noqa: F811
    """Heads whose q is 2^low of the others', with a scale at which their scores count: a head is as exact as alone."""
    c = Case(D + H + T, T, H, D, 200, 32, sink=True, spread=0)
    size = np.where(np.arange(H) % 3 == 1, 2.0 ** low, 1.0)
    c.q_t, c.q = bf16(c.q * size[None, :, None])
    c.scale *= 2.0 ** -low
    for t in range(0, T, 13):  # (the other heads' scores are beyond what fp32 tells apart, those of the small ones are not)
        out, lse = c.run(dsa) if t == 0 else (out, lse)
        kv, r = c.listed(t)
        small = np.flatnonzero(size < 1.0)
        q, sink = c.q[t][small], c.sink[small]
        o, l, p, x = K4.attend(q, kv, sink, c.scale)
        to, tl = K4.attend_tolerance(q, kv, r, p, x, o, l, c.scale)
        assert np.all(np.abs(out[t][small] - o) <= to) and np.all(np.abs(lse[t][small] - l) <= tl)
    assert np.all(np.isfinite(out))


@pytest.mark.parametrize("base", [0, -20, 30])
@pytest.mark.parametrize("T", [2, 160])
def test_attention_heads_about_the_widest_common_factor(dsa, T, base):  # noqa: F811
    """Heads 2^9 and 2^10, 2^14 to 2^16 and 2^19 below the largest: where one factor serves all of them and where not."""
    for spread in (0, 9, 10, 14, 15, 16, 19):
        c = Case(T + spread, T, 66, 128, 150, 32, sink=True, spread=0)
        size = 2.0 ** (base - spread * (np.arange(66) % 2))
        c.q_t, c.q = bf16(c.q * size[None, :, None])
        for part in (0, 1):
            c.scale = 0.6 / np.sqrt(c.D) * 2.0 ** (spread * part - base)
            out, lse = c.run(dsa)
            for t in range(0, T, 31):
                kv, r = c.listed(t)
                q, sink = c.q[t][part::2], c.sink[part::2]
                o, l, p, x = K4.attend(q, kv, sink, c.scale)
                to, tl = K4.attend_tolerance(q, kv, r, p, x, o, l, c.scale)
                assert np.all(np.abs(out[t][part::2] - o) <= to) and np.all(np.abs(lse[t][part::2] - l) <= tl), (spread, part)


@pytest.mark.parametrize("top", [0.0625, 1.0, 2.0, 200.0, 40000.0])
@pytest.mark.parametrize("T", [2, 160])
def test_attention_small_values_beside_a_large_one(dsa, T, top):  # noqa: F811
    """One value of each head's q far above the others, where the rows are zero: the others alone make the scores, and
    their lowest bits count."""
    c = Case(T, T, 12, 128, 200, 32, sink=True, spread=0)
    for s in range(c.R):
        x = c.rng.standard_normal((c.length, c.D))
        x[:, :16] = 0.0
        hold(c, s, x)
    tiny = top * 2.0 ** -19 * (1.0 + c.rng.integers(0, 128, c.q.shape) / 128.0) * c.rng.choice([-1.0, 1.0], c.q.shape)
    tiny[:, :, :16] = 0.0
    tiny[:, :, 3] = top
    c.q_t, c.q = bf16(tiny)
    c.scale = 2.0 / (np.sqrt(c.D) * top * 2.0 ** -19)
    c.check(*c.run(dsa), rows=range(0, T, 13))


def test_attention_heads_of_extreme_size(dsa):  # noqa: F811
    """Heads of zeros, of the least and of the largest bf16 values in one token."""
    for T in (2, 160):
        c = Case(T, T, 9, 64, 100, 16, sink=True, spread=0)
        size = 2.0 ** np.array([0, -133, -126, -30, 30, 100, 126, 0, 0], np.float64)
        q = np.clip(c.q, -2.0, 2.0) * 0.9 * size[None, :, None]
        q[:, 7] = 0.0
        c.q_t, c.q = bf16(q)
        for e, heads in ((0, [0, 7, 8, 3]), (100, [1, 2]), (-30, [4]), (-100, [5]), (-120, [6])):
            c.scale = 0.3 * 2.0 ** e
            out, lse = c.run(dsa)
            for t in range(0, T, 13):
                kv, r = c.listed(t)
                q, sink = c.q[t][heads], c.sink[heads]
                o, l, p, x = K4.attend(q, kv, sink, c.scale)
                to, tl = K4.attend_tolerance(q, kv, r, p, x, o, l, c.scale)
                assert np.all(np.abs(out[t][heads] - o) <= to) and np.all(np.abs(lse[t][heads] - l) <= tl), (T, e)


# ------------------------------------------------------------------------------------ list lengths


@pytest.mark.parametrize("at", [0, 2 ** 25 + 7])
def test_attention_longest_list(dsa, at):  # noqa: F811
    """2^26 entries, of which one names a row."""
    import torch

    c = Case(5, 1, 3, 64, 1, 16, start=False, R=1)
    want = c.run(dsa)
    long = torch.full((1, 2 ** 26), -1, dtype=torch.int32, device="cuda")
    long[0, at] = int(c.idx[0, 0])
    table, cache = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.cache).cuda()
    seq, lse = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 3, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    out = dsa.sparse_attn_kv4(c.q_t, cache, table, seq, long, scale=c.scale, lse=lse)
    b.record()
    assert dsa.get_device_error() == 0
    print(f"{a.elapsed_time(b):.1f} ms")
    assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.allclose(lse.double().cpu().numpy(), want[1], rtol=2.0 ** -20)


# ------------------------------------------------------------------------------------ workspaces


def test_attention_workspace_alignment_and_size(dsa):  # noqa: F811
    """Of the right size but 8 bytes off, 16 bytes short, and 16 bytes into a larger buffer."""
    import torch

    c = Case(21, 2, 64, 512, 700, 64, length=500)
    need = dsa.sparse_attn_kv4_workspace_size(c.T, c.H, c.D, c.K)
    big = torch.full((need + 32,), 0xFF, dtype=torch.uint8, device="cuda")
    assert need > 0 and big.data_ptr() % 16 == 0
    for bad in (big[8:8 + need], big[4:], big[:need - 16], big[:need - 1]):
        with pytest.raises(dsa.DsaError) as e:
            c.run(dsa, workspace=bad)
        assert e.value.status == 3
    want, got = c.run(dsa), c.run(dsa, workspace=big[16:16 + need])
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert bool((big[:16] == 0xFF).all()) and bool((big[16 + need:] == 0xFF).all())


@pytest.mark.parametrize("size", ["small", "mixed"])
@pytest.mark.parametrize("T,K", [(2, 900), (160, 300)])
def test_attention_own_factors_beside_rows_far_apart(dsa, T, K, size):  # noqa: F811
    """Heads that need powers of two of their own, over lists of rows whose scales lie far apart."""
    c = Case(T + K, T, 20, 128, K, 32, spread=0, sink=True)
    for s in range(c.R):
        x = c.rng.standard_normal((c.length, c.D))
        x[:100] *= 2.0 ** 50
        x[100:200] = 0.0
        hold(c, s, x)
    head = 2.0 ** -30 * np.ones(20) if size == "small" else np.where(np.arange(20) % 2, 2.0 ** -25, 1.0)
    c.q_t, c.q = bf16(c.q * head[None, :, None])
    c.scale *= 2.0 ** -50 / head.min()
    heads = np.flatnonzero(head == head.min())
    out, lse = c.run(dsa)
    for t in range(0, T, 13):
        kv, r = c.listed(t)
        q, sink = c.q[t][heads], c.sink[heads]
        o, l, p, x = K4.attend(q, kv, sink, c.scale)
        to, tl = K4.attend_tolerance(q, kv, r, p, x, o, l, c.scale)
        assert np.all(np.abs(out[t][heads] - o) <= to) and np.all(np.abs(lse[t][heads] - l) <= tl)
