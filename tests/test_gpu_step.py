"""The paged bf16 cache's small calls and the drafts' check against plain references; all results are whole numbers or copies."""
import numpy as np
import pytest
import torch

import paged_ref as PR
import sparse_attention_indexer_e4m3_gb300 as dsa

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("R,T,most", [(0, 5, 1), (1, 1, 1), (3, 7, 4), (61, 64, 1), (61, 40, 1), (1000, 2500, 5), (1025, 1024, 2), (2500, 9000, 7), (5, 5000, 2000), (4, 0, 3)])
def test_step_maps(R, T, most):
    rng = np.random.default_rng(R + T)
    held, added = rng.integers(-2, 5000, R), rng.integers(-1, most + 1, R)
    got = dsa.step_maps(i32(held), i32(added), T)
    for g, w in zip(got, PR.maps(held, added, T)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w)


def test_step_maps_sums_past_an_int():
    top = 2 ** 31 - 1
    held, added = np.array([top, top, 5, top - 2]), np.array([2, 0, 3, top])
    for g, w in zip(dsa.step_maps(i32(held), i32(added), 9), PR.maps(held, added, 9)):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("T,K,rows", [(1, 1, 16), (5, 7, 32), (9, 64, 64), (3, 4, 256), (200, 2048, 64)])
@pytest.mark.parametrize("start", [False, True])
def test_page_slots(T, K, rows, start):
    rng = np.random.default_rng(T + K)
    R, M, P = 4, 9, 20
    table = rng.integers(-2, P + 2, (R, M))
    seq = rng.integers(-1, R + 1, T)
    st = rng.integers(-5, 100, T) if start else None
    idx = rng.integers(-3, M * rows + 20, (T, K))
    pages = torch.empty(P, rows, 3, device="cuda")
    some = min(T, 9)
    want = PR.slots(table, P, rows, seq[:some], st[:some] if start else None, idx[:some])
    x = i32(idx)
    got = dsa.page_slots(pages, i32(table), i32(seq), x, start=i32(st) if start else None)
    assert np.array_equal(got[:some].cpu().numpy(), want)
    dsa.page_slots(pages, i32(table), i32(seq), x, start=i32(st) if start else None, out=x)  # in place
    assert torch.equal(x, got)
    one = dsa.page_slots(pages, i32(table), i32(seq), i32(idx[:, 0]), start=i32(st) if start else None)
    assert torch.equal(one, got[:, 0].contiguous())


@pytest.mark.parametrize("D,rows", [(64, 16), (128, 64), (256, 256), (512, 32)])
def test_store_kv(D, rows):
    rng = np.random.default_rng(D)
    R, M, P, N = 3, 6, 14, 77
    table = np.full((R, M), -1)
    table[:, :4] = rng.permutation(12).reshape(R, 4)
    table[0, 0], table[1, 1] = P, -5
    at = rng.permutation(R * M * rows)[:N]
    seq, pos = at // (M * rows), at % (M * rows)
    seq[:4], pos[:4] = [-1, R, 0, 1], [3, 3, -1, M * rows]
    wide = torch.randn(N, D + 24, device="cuda").to(torch.bfloat16)
    before = torch.randn(P, rows, D, device="cuda").to(torch.bfloat16)
    slot = PR.slots(table, P, rows, seq, None, pos[:, None])[:, 0]
    slot[2:4] = -1
    for kv in (wide[:, 8:8 + D], wide[:, :D].contiguous()):
        want = before.clone().view(-1, D)
        want[torch.from_numpy(slot[slot >= 0]).cuda()] = kv[torch.from_numpy(np.flatnonzero(slot >= 0)).cuda()]
        pages = before.clone()
        dsa.store_kv(kv, pages, i32(table), i32(seq), i32(pos), lacking=i32([3]))
        assert torch.equal(pages, before)
        assert dsa.store_kv(kv, pages, i32(table), i32(seq), i32(pos), lacking=i32([0])) is pages
        assert torch.equal(pages.view(-1, D), want)
        pages = before.clone()
        dsa.store_kv(kv, pages, i32(table), i32(seq), i32(pos))
        assert torch.equal(pages.view(-1, D), want)


def probs(shape, rng, peak):
    x = rng.standard_normal(shape) * peak
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("R,G,V", [(1, 1, 1), (1, 0, 5), (3, 2, 33), (40, 4, 127), (5, 35, 128), (7, 3, 4097), (2, 5, 50257), (700, 2, 130), (1, 3, 300001)])
@pytest.mark.parametrize("peak", [0.5, 4.0])
def test_verify(R, G, V, peak):
    rng = np.random.default_rng(R + G + V)
    target = probs((R, G + 1, V), rng, peak)
    draft = probs((R, G, V), rng, peak)
    near = rng.random((R, G)) < 0.6
    draft[near] = target[:, :G][near]  # the same: accepted whatever the number
    tokens = rng.integers(0, V, (R, G))
    if G > 1 and R > 2:
        tokens[0, 0], tokens[1, 1] = -1, V  # (no such token)
    count = rng.integers(-1, G + 2, R)
    u = rng.random((R, G + 1)).astype(np.float32)
    u[0, G] = 0.0
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    a, k = dsa.verify_drafts(t(target), t(draft), i32(tokens), i32(count), t(u))
    wa, wk = PR.verify(target, draft, tokens, count, u)
    assert np.array_equal(a.cpu().numpy(), wa) and np.array_equal(k.cpu().numpy(), wk)


def test_verify_borders():
    """Sums that the drawn number meets exactly, values that are no probabilities, rows where nothing is left."""
    V = 1024
    flat = np.full((1, 1, V), 1 / V, np.float32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    none = np.zeros((1, 0, V), np.float32)
    run = lambda tg, dr, tok, n, u: [int(x) for x in dsa.verify_drafts(t(tg), t(dr), i32(tok).reshape(1, -1), i32([n]), t(u))]  # noqa: E731
    for v in (0, 1, 127, 128, 511, 1023):
        assert run(flat, none, [], 0, np.array([[v / V]], np.float32)) == [0, v]
        assert run(flat, none, [], 0, np.array([[np.nextafter(np.float32((v + 1) / V), np.float32(0))]])) == [0, v]
    odd = np.zeros((1, 1, V), np.float32)
    odd[0, 0, [3, 5, 9, 700]] = [np.nan, -1.0, 0.25, 0.75]
    assert run(odd, none, [], 0, np.array([[0.24]], np.float32)) == [0, 9]
    assert run(odd, none, [], 0, np.array([[0.25]], np.float32)) == [0, 700]
    for u in (1.0, 2.0, np.inf):
        assert run(odd, none, [], 0, np.array([[u]], np.float32)) == [0, 700]
    for u in (-1.0, np.nan):
        assert run(odd, none, [], 0, np.array([[u]], np.float32)) == [0, 9]
    assert run(0 * flat, none, [], 0, np.array([[0.5]], np.float32)) == [0, -1]
    # refused with nothing left over the draft: from the target
    two = np.concatenate([flat, odd], 1)
    assert run(two, flat, [4], 1, np.array([[1.0, 0.5]], np.float32)) == [0, 512]
    assert run(two, flat, [4], 1, np.array([[0.999, 0.5]], np.float32)) == [1, 700]
