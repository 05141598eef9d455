"""The 4-bit cache's calls next to other work of their streams.  They are launched before the stream's earlier work
has ended and wait for it themselves: here each follows at once on what writes its inputs (a long kernel whose last
elements they are, a copy, a fill), eagerly, across streams and in captured graphs, and the result has to be, bit
for bit, that of the same calls with a synchronisation before each."""
import numpy as np
import pytest

import kv4_ref as K4
from test_gpu_kv4 import dev, dsa  # noqa: F401

pytestmark = pytest.mark.gpu

R, M, B, D, H, K, T = 5, 6, 64, 128, 24, 300, 5
P = R * M * 2 + 3


def inputs(seed):
    """One step's inputs, as a list of tensors on the GPU in the order of `step`."""
    import torch

    rng = np.random.default_rng(seed)
    n = R * 250
    x = torch.from_numpy(rng.standard_normal((n, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    seq, pos = np.repeat(np.arange(R), 250), np.tile(np.arange(250), R)
    table = np.full((R, M), -1, np.int32)
    table[:, :4] = rng.permutation(P)[:R * 4].reshape(R, 4)
    ref = np.zeros(P, np.int32)
    ref[table[:, :4].ravel()] = 1
    idx = rng.integers(-1, 250, (T, K))
    i32 = [dev(a, np.int32) for a in (seq, pos, table, ref, idx, rng.permutation(R), rng.integers(0, R, R),
                                      np.full(R, 250), np.full(R, 300))]
    return [x, q] + i32


def step(dsa, a, cache, between=lambda: None, stream=None):  # noqa: F811
    """Write rows, attend, read back, branch, grow, copy and compact; `between` runs ahead of each call."""
    import torch

    x, q, seq, pos, table, ref, idx, tok, parent, begin, end = a
    between()
    dsa.quantize_kv4(x, cache, table, seq, pos, stream=stream)
    between()
    lse = torch.empty((T, H), device="cuda")
    out = dsa.sparse_attn_kv4(q, cache, table, tok, idx, lse=lse, stream=stream)
    between()
    back = dsa.dequantize_kv4(cache, table, seq, pos, D, stream=stream)
    between()
    forked = dsa.fork_pages(table, parent, ref, stream=stream)
    between()
    src, dst, lack = dsa.reserve_pages(forked, ref, begin, end, B, stream=stream)
    between()
    dsa.copy_pages(cache, src, dst, stream=stream)
    between()
    s2, d2, live = dsa.compact_pages(forked, ref, stream=stream)
    between()
    dsa.copy_pages(cache, s2, d2, stream=stream)
    between()
    back2 = dsa.dequantize_kv4(cache, forked, seq, pos, D, stream=stream)
    return out, lse, back, forked, src, dst, lack, s2, d2, live, back2, cache, ref


def empty_cache():
    import torch

    return torch.zeros((P, K4.page_bytes(B, D)), dtype=torch.uint8, device="cuda")


def synced(dsa, seed):  # noqa: F811
    import torch

    a = inputs(seed)
    torch.cuda.synchronize()
    return [t.clone() for t in step(dsa, a, empty_cache(), torch.cuda.synchronize)]


def same(got, want):
    import torch

    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8)), i


@pytest.mark.parametrize("how", ["kernel", "copy"])
def test_calls_follow_at_once(dsa, how):  # noqa: F811
    """Each call right behind the kernel or the copy that brings all its inputs."""
    import torch

    want = [synced(dsa, s) for s in (1, 2)]
    sets = [inputs(s) for s in (1, 2)]
    sizes = [(t.numel() * t.element_size() + 255) // 256 * 256 for t in sets[0]]
    total, pad = sum(sizes), 256 << 20

    def packed(ts):
        big = torch.zeros(pad + total, dtype=torch.uint8, device="cuda")
        at = pad
        for t, n in zip(ts, sizes):
            big[at:at + t.numel() * t.element_size()] = t.contiguous().view(torch.uint8).view(-1)
            at += n
        return big

    big = [packed(ts) for ts in sets]
    live = torch.zeros_like(big[0])
    views, at = [], pad
    for t, n in zip(sets[0], sizes):
        views.append(live[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape))
        at += n
    torch.cuda.synchronize()
    for r in range(6):
        cache = empty_cache()
        if how == "kernel":
            torch.bitwise_or(big[r & 1], 0, out=live)
        else:
            live.copy_(big[r & 1])
        same(step(dsa, views, cache), want[r & 1])
    assert dsa.get_device_error() == 0


def test_calls_follow_on_another_stream(dsa):  # noqa: F811
    """Inputs made on one stream, the calls on another that waits for an event, and back."""
    import torch

    want = [synced(dsa, s) for s in (3, 4)]
    sets = [inputs(s) for s in (3, 4)]
    live = [torch.zeros_like(t) for t in sets[0]]
    busy = torch.zeros(64 << 20, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(6):
        cache = empty_cache()
        for _ in range(4):
            busy.add_(1.0)
        for t, s in zip(live, sets[r & 1]):
            t.copy_(s)
        side.wait_stream(torch.cuda.current_stream())
        got = step(dsa, live, cache, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        same([t.clone() for t in got], want[r & 1])
    assert dsa.get_device_error() == 0


def test_calls_in_a_graph_behind_copies_fills_and_joins(dsa):  # noqa: F811
    """Captured: each call behind a fill, a copy, a kernel, and behind a side stream that wrote another cache; two
    graphs of the same calls replayed in turn on changed inputs."""
    import torch

    want = [synced(dsa, s) for s in (5, 6)]
    sets = [inputs(s) for s in (5, 6)]
    graphs = []
    for _ in range(2):
        live, cache, other = [t.clone() for t in sets[0]], empty_cache(), empty_cache()
        staged = [t.clone() for t in sets[0]]
        scratch, copied = torch.zeros(4096, device="cuda"), torch.zeros(4096, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.zero_()
            for t, s in zip(live, staged):
                t.copy_(s)
            turn = [0]

            def between():
                turn[0] += 1
                if turn[0] % 4 == 0:
                    scratch.zero_()
                elif turn[0] % 4 == 1:
                    copied.copy_(scratch)
                elif turn[0] % 4 == 2:
                    scratch.add_(1.0)
                else:
                    here = torch.cuda.current_stream()
                    side.wait_stream(here)
                    with torch.cuda.stream(side):
                        dsa.quantize_kv4(live[0], other, live[4], live[2], live[3])
                    here.wait_stream(side)

            got = step(dsa, live, cache, between)
        graphs.append((g, staged, got))
    for r in range(4):
        for k, (g, staged, got) in enumerate(graphs):
            for t, s in zip(staged, sets[(r + k) & 1]):
                t.copy_(s)
            g.replay()
        for k, (_, _, got) in enumerate(graphs):
            same(got, want[(r + k) & 1])
    assert dsa.get_device_error() == 0
