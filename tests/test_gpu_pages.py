"""The page calls on the GPU against sequential bookkeeping (tests/kv4_ref.py), equal in every entry; and a
serving run in which indexer, cache, attention and page calls work together."""
import numpy as np
import pytest

import kv4_ref as K4
from test_gpu_kv4 import bf16, dev, dsa, rows_of  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu


def host(*ts):
    return [t.cpu().numpy() for t in ts]


def random_state(rng, R, M, P, fill=0.6, share=0.4, junk=True):
    """A table whose rows hold some pages, part of them shared, and its counts."""
    table = np.full((R, M), -1, np.int32)
    ids = list(rng.permutation(P)[:int(P * fill)])
    for r in range(R):
        n = int(rng.integers(0, M + 1))
        for j in range(n):
            if r > 0 and rng.random() < share and table[r - 1, j] >= 0:
                table[r, j] = table[r - 1, j]
            elif ids:
                table[r, j] = ids.pop()
    ref = K4.counts(table, P)
    if junk and R * M > 4:  # entries that name no page
        k = rng.integers(0, R * M, 3)
        for i, v in zip(k, (P, -7, 2 ** 31 - 1)):
            old = table.reshape(-1)[i]
            if 0 <= old < P:
                ref[old] -= 1
            table.reshape(-1)[i] = v
    return table, ref.astype(np.int32)


SIZES = [(1, 1, 1), (1, 5, 3), (7, 9, 40), (33, 65, 900), (300, 31, 9000), (5, 700, 3000), (600, 3, 65537), (700, 190, 20000)]


@pytest.mark.parametrize("R,M,P", SIZES)
def test_fork(dsa, R, M, P):  # noqa: F811
    rng = np.random.default_rng(R + M + P)
    for trial in range(3):
        table, ref = random_state(rng, R, M, P)
        parent = rng.integers(-1, R, R)
        if trial == 1:
            parent = np.arange(R)
        if trial == 2:
            parent[rng.random(R) < 0.3] = R + 5
            parent[0] = -(2 ** 31)
        t, r = dev(table), dev(ref)
        out = dsa.fork_pages(t, dev(parent, np.int32), r)
        want, want_ref = K4.fork(table, parent, ref)
        assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(r.cpu().numpy(), want_ref)
        assert np.array_equal(t.cpu().numpy(), table)


@pytest.mark.parametrize("B", [16, 64])
@pytest.mark.parametrize("R,M,P", SIZES)
def test_reserve(dsa, R, M, P, B):  # noqa: F811
    rng = np.random.default_rng(R * M + P + B)
    short = 0
    for trial in range(4):
        table, ref = random_state(rng, R, M, P, fill=(0.3, 0.6, 0.97, 0.5)[trial])
        begin = rng.integers(-5, M * B + 5, R)
        end = begin + rng.integers(-2, (2, 3 * B, M * B, 2 * B)[trial], R)
        if trial == 3:  # whole pages
            begin, end = begin // B * B, end // B * B
            end[0] = 2 ** 31 - 1
            begin[0] = 0
        t, r = dev(table), dev(ref)
        src, dst, lack = dsa.reserve_pages(t, r, dev(begin, np.int32), dev(end, np.int32), B)
        want = K4.reserve(table, ref, begin, end, B)
        assert lack.item() == want[4]
        for got, w in zip(host(t, r, src, dst), want[:4]):
            assert np.array_equal(got, w)
        short += want[4] > 0
    assert short < 4


def test_reserve_exact_fit_and_shortage(dsa):  # noqa: F811
    """As many needs as free pages succeeds; one more changes nothing and says by how many pages."""
    table = np.full((3, 4), -1, np.int32)
    table[0, 0] = 5
    for P, lack in ((9, 0), (8, 1), (6, 3)):
        ref = K4.counts(table, P)
        t, r = dev(table), dev(ref)
        src, dst, n = dsa.reserve_pages(t, r, dev([16, 0, 0], np.int32), dev([64, 48, 32], np.int32), 16)
        want = K4.reserve(table, ref, [16, 0, 0], [64, 48, 32], 16)
        assert n.item() == lack == want[4]
        assert all(np.array_equal(a, b) for a, b in zip(host(t, r, src, dst), want[:4]))


@pytest.mark.parametrize("R,M,P", SIZES)
def test_compact(dsa, R, M, P):  # noqa: F811
    rng = np.random.default_rng(R + M * P)
    for trial in range(3):
        table, ref = random_state(rng, R, M, P, fill=(0.2, 0.9, 1.0)[trial])
        if trial == 1:
            ref[rng.random(P) < 0.05] = -3  # counts below zero are free; entries naming them end as -1
        t, r = dev(table), dev(ref)
        src, dst, n = dsa.compact_pages(t, r)
        want = K4.compact(table, ref)
        assert n.item() == want[4]
        for got, w in zip(host(t, r, src, dst), want[:4]):
            assert np.array_equal(got, w)


@pytest.mark.parametrize("shape,t", [((5, 16), "uint8"), ((40, 33, 8), "float32"), ((300, 18688), "uint8"), ((9, 40, 512), "int64"),
                                     ((3, 16400), "uint8")])
def test_copy(dsa, shape, t):  # noqa: F811
    import torch

    rng = np.random.default_rng(shape[0])
    P = shape[0]
    pages = dev(rng.integers(0, 100, shape)).to(getattr(torch, t))
    perm = rng.permutation(P)
    n = P // 2
    src, dst = perm[:n].copy(), perm[n:2 * n].copy()
    src, dst = np.concatenate([src, [-1, 0, P, 2, -9]]), np.concatenate([dst, [0, -1, 1, P + 3, -9]])
    want = pages.cpu().numpy().copy()
    for a, b in zip(src, dst):
        if 0 <= a < P and 0 <= b < P:
            want[b] = want[a]
    assert dsa.copy_pages(pages, dev(src, np.int32), dev(dst, np.int32)) is pages
    assert np.array_equal(pages.cpu().numpy(), want)


def test_page_calls_in_a_graph_and_on_a_stream(dsa):  # noqa: F811
    import torch

    rng = np.random.default_rng(8)
    R, M, P, B = 9, 20, 400, 16
    table, ref = random_state(rng, R, M, P, junk=False)
    parent = rng.integers(-1, R, R)
    begin = rng.integers(0, M * B - 8, R)
    t, r, par, b, e = dev(table), dev(ref), dev(parent, np.int32), dev(begin, np.int32), dev(begin + 5, np.int32)
    cache = dev(rng.integers(0, 256, (P, 640), dtype=np.uint8))

    def step(stream=None):
        out = dsa.fork_pages(t, par, r, stream=stream)
        src, dst, lack = dsa.reserve_pages(out, r, b, e, B, stream=stream)
        dsa.copy_pages(cache, src, dst, stream=stream)
        s2, d2, n = dsa.compact_pages(out, r, stream=stream)
        dsa.copy_pages(cache, s2, d2, stream=stream)
        return out, src, dst, lack, s2, d2, n

    def want(c):
        w_t, w_r = K4.fork(table, parent, ref)
        w_t, w_r, a, d, lack = K4.reserve(w_t, w_r, begin, begin + 5, B)
        for i, j in zip(a, d):
            if i >= 0:
                c[j] = c[i]
        w_t, w_r, a2, d2, n = K4.compact(w_t, w_r)
        for i, j in zip(a2, d2):
            if i >= 0:
                c[j] = c[i]
        return [w_t, a, d, np.array([lack]), a2, d2, np.array([n])], w_r, c

    def same(got, c0):
        w, w_r, c = want(c0)
        assert all(np.array_equal(x, y) for x, y in zip(host(*got), w))
        assert np.array_equal(r.cpu().numpy(), w_r) and np.array_equal(cache.cpu().numpy(), c)

    c0 = cache.cpu().numpy().copy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.synchronize()
    same(got, c0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        r.copy_(dev(ref))
        c0 = cache.cpu().numpy().copy()
        g.replay()
        torch.cuda.synchronize()
        same(got, c0)


def test_serving_run(dsa):  # noqa: F811
    """Prompts into the cache, selection by the indexer, attention; a sequence branches, the branches write
    their own next rows, one is freed, the pool is compacted: after each step the attention over the cache
    equals the 64-bit attention over rows kept beside it, and compaction changes no bit."""
    import torch

    import workloads as W

    rng = np.random.default_rng(3)
    R, M, B, D, P, H, topk = 4, 6, 32, 128, 20, 12, 48
    HI, DI = 4, 64  # the indexer's heads
    cache = torch.full((P, K4.page_bytes(B, D)), 0xFF, dtype=torch.uint8, device="cuda")
    table, ref = torch.full((R, M), -1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    kv = [np.zeros((0, D)) for _ in range(R)]  # the rows that each sequence holds, and their scales
    scales = [np.zeros(0) for _ in range(R)]
    keys = [np.zeros((0, DI)) for _ in range(R)]

    def write(grow):
        begin = np.array([len(k) for k in kv])
        end = begin + grow
        src, dst, lack = dsa.reserve_pages(table, ref, dev(begin, np.int32), dev(end, np.int32), B)
        assert lack.item() == 0
        dsa.copy_pages(cache, src, dst)
        seq = np.repeat(np.arange(R), grow)
        pos = np.concatenate([np.arange(b, e) for b, e in zip(begin, end)])
        t, x = bf16(rows_of(rng, len(seq), D, 2))
        dsa.quantize_kv4(t, cache, table, dev(seq, np.int32), dev(pos, np.int32))
        codes, s8, r = K4.encode(x)
        held = K4.decode(codes, s8, r)
        for s in range(R):
            kv[s] = np.concatenate([kv[s], held[seq == s]])
            scales[s] = np.concatenate([scales[s], r[seq == s]])
            keys[s] = np.concatenate([keys[s], rng.standard_normal((grow[s], DI))])
        assert np.array_equal(ref.cpu().numpy(), K4.counts(table.cpu().numpy(), P))

    def attend():
        live = [s for s in range(R) if len(kv[s])]
        lens = np.array([len(kv[s]) for s in live])
        off = np.concatenate([[0], np.cumsum(lens)])[:-1]
        kt, _ = bf16(np.concatenate([keys[s] for s in live]))
        codes, ksc = dsa.quantize_k(kt)
        qi = torch.from_numpy(W.normal(5, 1, len(live) * HI * DI).reshape(len(live), HI, DI)).cuda().to(torch.float8_e4m3fn)
        w = torch.ones(len(live), HI, device="cuda")
        start = dev(off, np.int32)
        idx = dsa.index_topk(qi, w, codes, ksc, start, dev(off + lens, np.int32), topk)
        qt, q = bf16(np.random.default_rng(9).standard_normal((len(live), H, D)))
        out = dsa.sparse_attn_kv4(qt, cache, table, dev(live, np.int32), idx, start=start)
        assert dsa.get_device_error() == 0
        got, sel = out.double().cpu().numpy(), idx.cpu().numpy()
        for i, s in enumerate(live):
            at = sel[i][sel[i] >= 0] - off[i]
            assert len(at) == min(topk, lens[i]) and at.min() >= 0 and at.max() < lens[i]
            o, l, p, x = K4.attend(q[i], kv[s][at], None, 1 / np.sqrt(D))
            to, _ = K4.attend_tolerance(q[i], kv[s][at], scales[s][at], p, x, o, l, 1 / np.sqrt(D))
            assert np.all(np.abs(got[i] - o) <= to)
        return got

    write(np.array([70, 33, 0, 0]))
    attend()
    parent = np.array([0, 1, 0, 0])
    table = dsa.fork_pages(table, dev(parent, np.int32), ref)  # sequences 2 and 3 branch off sequence 0
    kv, scales, keys = ([x[p].copy() for p in parent] for x in (kv, scales, keys))
    attend()
    for _ in range(3):
        write(np.array([1, 2, 1, 5]))
        attend()
    parent = np.array([0, -1, 2, 2])
    table = dsa.fork_pages(table, dev(parent, np.int32), ref)  # sequence 1 is freed, 3 restarts from 2
    kv, scales, keys = ([x[p].copy() if p >= 0 else x[0][:0] for p in parent] for x in (kv, scales, keys))
    write(np.array([4, 0, 1, 20]))
    before = attend()
    src, dst, n = dsa.compact_pages(table, ref)
    dsa.copy_pages(cache, src, dst)
    assert n.item() == int((ref > 0).sum()) and bool((ref[n.item():] == 0).all()) and int(table.max()) < n.item()
    cache[n.item():] = 0xFF  # nothing above the live pages is read
    assert np.array_equal(attend(), before)
    write(np.array([1, 40, 1, 1]))
    attend()
