"""More of what the bf16 paged cache's and the drafts' calls refuse, and of what their documents say, without a GPU."""
import pytest

from test_paged_host import INVALID, UNSUPPORTED, a, lib  # noqa: F401  (fixtures)


@pytest.fixture
def at(a):  # noqa: F811
    return [a + (i << 20) for i in range(16)]  # (addresses apart; none is read)


def test_stored_pages_over_what_is_read(lib, at):  # noqa: F811
    """Pages of 2 x 64 rows of 128 values: 32 KB."""

    def f(kv=at[0], seq=at[1], pos=at[2], pages=at[3], table=at[4], lacking=at[5]):
        return lib.dsa_store_kv(kv, 128, seq, pos, 4, 128, pages, 2, 64, table, 1, 2, lacking, None)

    for k in ("kv", "seq", "pos", "table", "lacking"):
        assert f(**{k: at[3] + 32752}) == INVALID and f(**{k: at[3]}) == INVALID, k
    assert f(seq=at[3] - 12) == f(table=at[3] - 4) == INVALID


def test_attention_over_what_is_read(lib, at):  # noqa: F811
    """Outputs of 2 x 4 x 128 values (2 KB), logs of 32 bytes."""

    def f(q=at[0], pages=at[1], table=at[2], seq=at[3], pos=at[4], sink=at[5], out=at[6], lse=at[7]):
        return lib.dsa_paged_attn(q, pages, 2, 64, table, 1, 2, seq, pos, sink, 2, 4, 128, 0, 0, 1.0, out, lse, None, 0, None)

    for k in ("pages", "table", "seq", "pos", "sink"):
        assert f(**{k: at[6] + 2032}) == f(**{k: at[7] + 16}) == INVALID, k
    assert f(lse=at[6] + 2044) == f(lse=at[6] - 28) == f(lse=at[0]) == f(lse=at[0] + 2044) == f(out=at[0] + 16) == INVALID


def test_drafts_over_the_probabilities(lib, at):  # noqa: F811
    """Two rows of 4 x 5 probabilities of the target (160 bytes), 3 x 5 of the draft (120)."""

    def f(target=at[0], draft=at[1], accepted=at[5], token=at[6], R=2, G=3, V=5):
        return lib.dsa_verify_drafts(target, draft, at[2], at[3], at[4], R, G, V, accepted, token, None)

    for k in ("accepted", "token"):
        assert f(**{k: at[0] + 156}) == f(**{k: at[0] - 4}) == f(**{k: at[1] + 116}) == f(**{k: at[1]}) == INVALID, k
    assert f(R=2 ** 27, G=2 ** 20, V=2 ** 30) == f(R=2 ** 10, G=2 ** 20 - 1, V=2 ** 30) == UNSUPPORTED


def test_strides_past_what_memory_holds(lib, at):  # noqa: F811
    """A last row whose place no 64-bit count of bytes reaches: refused before it is formed."""
    f = lambda stride, N=4: lib.dsa_store_kv(at[0], stride, at[1], at[2], N, 128, at[3], 2, 64, at[4], 1, 2, None, None)  # noqa: E731
    assert f(2 ** 60) == f(2 ** 62) == f(2 ** 63 - 8) == f(2 ** 61 // 3 // 8 * 8 + 8, N=3) == f(2 ** 31, N=2 ** 31 - 1) == INVALID
