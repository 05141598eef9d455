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
