"""More of what the bf16 paged cache's and the drafts' calls refuse, and of what their documents say, without a GPU."""
import os
import re
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import paged_ref as PR
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


def test_documented_step():
    """The README's step over a bf16 cache, its calls replaced by the references: places without a sequence stay as they are, more
    drafts than there is room for count as that many, and a step whose pool fell short leaves the lengths."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    start = text.index("A step over a bf16 cache")
    code = "\n".join(re.findall(r"^    (.*)$", text[start:text.index("## ", start)], re.M))
    assert "dsa.step_maps(held, added, T)" in code and "dsa.verify_drafts(" in code
    R, G, V, T = 5, 3, 7, 24
    rng = np.random.default_rng(0)
    t = lambda x: torch.from_numpy(np.asarray(x, np.int32))  # noqa: E731
    held = t([4, 0, 100, 7, 33])
    for step, (count, short) in enumerate((([2, -1, 3, 0, -5], 0), ([-1, 9, 0, 1, 2], 0), ([1, 1, 1, 1, 1], 4), ([0, 3, -1, -1, 3], 0))):
        before, seen = held.clone(), {}
        target, draft = rng.random((R, G + 1, V)).astype(np.float32), rng.random((R, G, V)).astype(np.float32)
        tokens, u = rng.integers(0, V, (R, G)), rng.random((R, G + 1)).astype(np.float32)

        def reserve_pages(table, ref, begin, end, rows):
            seen.update(begin=begin.clone(), end=end.clone())
            return None, None, t([short])

        def step_maps(h, a, n):
            assert h.dtype == a.dtype == torch.int32
            seen.update(maps=[t(x) for x in PR.maps(h.tolist(), a.tolist(), n)])
            return seen["maps"]

        def verify_drafts(p, q, d, n, x):
            seen.update(checked=PR.verify(p, q, d, n.numpy(), x))
            return [t(x) for x in seen["checked"]]

        calls = SimpleNamespace(reserve_pages=reserve_pages, step_maps=step_maps, verify_drafts=verify_drafts,
                                **{k: lambda *a, **k: None for k in ("copy_pages", "store_kv", "paged_attn", "index_topk", "page_slots",
                                                                     "sparse_attn")})
        pages = torch.zeros(2, 64, 1)
        names = dict(torch=torch, dsa=calls, G=G, T=T, held=held, count=t(count), pages=pages, target=target, draft=draft, tokens=tokens, u=u,
                     **{k: None for k in ("table", "ref", "kv", "q", "q_e4m3", "w", "k_e4m3", "k_scale")})
        exec(code, names)
        live = np.array(count) >= 0
        rows = np.where(live, np.minimum(count, G) + 1, 0)
        assert seen["begin"].tolist() == before.tolist() and (seen["end"] - seen["begin"]).tolist() == rows.tolist()
        seq, pos, ks, _ = (x.numpy() for x in seen["maps"])
        assert (seq >= 0).sum() == rows.sum() and np.array_equal(np.bincount(seq[seq >= 0], minlength=R), rows)
        grown = np.where(live & (short == 0), seen["checked"][0] + 1, 0)
        assert (held - before).tolist() == grown.tolist() and names["held"] is held, step
