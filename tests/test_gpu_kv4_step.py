"""A decoding step over the 4-bit cache on the device: reserve, copy, write, attend, with and without enough pages."""
import numpy as np
import pytest

import kv4_ref as K4
from test_gpu_kv4 import bf16, dev, dsa, rows_of  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu

R, M, B, D = 4, 3, 16, 64


def state(rng, P):
    """Sequences 0 and 1 share their pages, 2 and 3 hold one each; P pages in all."""
    table = np.full((R, M), -1, np.int32)
    table[0, :2] = table[1, :2] = [0, 1]
    table[2, 0], table[3, 0] = 2, 3
    return table, K4.counts(table, P), rng.integers(0, 128, (P, K4.page_bytes(B, D)), dtype=np.uint8)


def step(m, a, P):
    """One new row for every sequence, in the documented order."""
    src, dst, lacking = m.reserve_pages(a["table"], a["ref"], a["begin"], a["end"], B)
    m.copy_pages(a["cache"], src, dst)
    m.quantize_kv4(a["kv"], a["cache"], a["table"], a["seq"], a["pos"], lacking=lacking)
    return lacking


def expected(table, ref, cache, begin, x):
    t, r, src, dst, lack = K4.reserve(table, ref, begin, begin + 1, B)
    want = cache.copy()
    if lack == 0:
        for s, d in zip(src, dst):
            if s >= 0:
                want[d] = cache[s]
        codes, s8, sc = K4.encode(x)
        for i in range(R):
            K4.put_row(want, *K4.place(t, len(cache), B, i, int(begin[i])), B, D, codes[i], s8[i], sc[i])
    return t, r, want, lack


def arguments(rng, P, begin):
    import torch

    table, ref, cache = state(rng, P)
    kv, x = bf16(rows_of(rng, R, D))
    a = dict(table=dev(table), ref=dev(ref), cache=dev(cache), begin=dev(begin, np.int32), end=dev(begin + 1, np.int32), kv=kv,
             seq=dev(np.arange(R), np.int32), pos=dev(begin, np.int32))
    torch.cuda.synchronize()
    return a, expected(table, ref, cache, begin, x)


def same(a, want):
    for got, w in zip((a["table"], a["ref"], a["cache"]), want):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("P,lack", [(5, 2), (6, 1), (7, 0), (40, 0)])
def test_step_writes_nothing_where_the_pool_falls_short(dsa, P, lack):  # noqa: F811
    """Rows 20 of sequences 0 and 1 lie in a page that both hold, row 16 of 2 in a new one: three pages, or nothing at all."""
    a, want = arguments(np.random.default_rng(P), P, np.array([20, 20, 16, 5]))
    lacking = step(dsa, a, P)
    assert lacking.item() == lack == want[3]
    same(a, want)
    # without a look at `lacking` the two branches' rows would have met in the page they share
    assert lack == 0 or int(a["ref"][1]) == 2


def test_captured_step_with_and_without_enough_pages(dsa):  # noqa: F811
    import torch

    P = 7
    begin = np.array([20, 20, 16, 5])
    a, want = arguments(np.random.default_rng(1), P, begin)
    first = {k: v.clone() for k, v in a.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lacking = step(dsa, a, P)
    for short in (False, True, False):
        for k, v in first.items():
            a[k].copy_(v)
        if short:
            a["ref"][6] = 1  # a page less
        g.replay()
        torch.cuda.synchronize()
        assert lacking.item() == int(short)
        if short:
            for k in ("table", "cache"):
                assert torch.equal(a[k], first[k])
        else:
            same(a, want)


def test_lacking_guards_every_row_size_and_count(dsa):  # noqa: F811
    import torch

    rng = np.random.default_rng(2)
    for Dx in (64, 128, 256, 512):
        for N in (1, 37, 4000):
            pages = -(-N // 64)
            table = dev(rng.permutation(pages)[None, :], np.int32)
            kv, x = bf16(rows_of(rng, N, Dx))
            seq, pos = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")
            caches = [torch.full((pages, K4.page_bytes(64, Dx)), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
            flags = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (3, -(2 ** 31), 0)]
            for c, f in zip(caches, flags):
                assert dsa.quantize_kv4(kv, c, table, seq, pos, lacking=f) is c
            assert bool((caches[0] == 7).all()) and bool((caches[1] == 7).all())
            plain = torch.full_like(caches[2], 7)
            dsa.quantize_kv4(kv, plain, table, seq, pos)
            assert torch.equal(caches[2], plain)
