"""Calls with stream=: what they allocate belongs to that stream, so that work still running on the current one, on memory that
was freed there, and the call do not meet in one buffer."""
import numpy as np
import pytest

import kv4_ref as K4
from test_gpu_kv4 import dev, dsa, rows_of, bf16  # noqa: F401  (dsa: the fixture)

pytestmark = pytest.mark.gpu

T, H, D, K, N, B, R = 2, 64, 512, 700, 640, 64, 1


@pytest.fixture(scope="module")
def world():
    import torch

    rng = np.random.default_rng(1)
    P = N // B + 2
    kv, _ = bf16(rows_of(rng, N, D, 2))
    q, _ = bf16(rng.standard_normal((T, H, D)))
    return dict(kv=kv, q=q, cache=torch.zeros(P, K4.page_bytes(B, D), dtype=torch.uint8, device="cuda"),
                table=dev(np.arange(N // B)[None, :], np.int32), seq=dev(np.zeros(N), np.int32), pos=dev(np.arange(N), np.int32),
                tok=dev(np.zeros(T), np.int32), idx=dev(rng.integers(0, N, (T, K)), np.int32),
                ref=dev(K4.counts(np.arange(N // B, dtype=np.int32)[None, :], P)), parent=dev([0], np.int32),
                begin=dev([5], np.int32), end=dev([70], np.int32))


def calls(m, w):
    """(call, shapes and type of what it allocates to return) of every call of the 4-bit cache that allocates."""
    i32, P = "int32", w["ref"].numel()
    return {
        "dequantize_kv4": (lambda s: m.dequantize_kv4(w["cache"], w["table"], w["seq"], w["pos"], D, stream=s), (N, D), "bfloat16"),
        "sparse_attn_kv4": (lambda s: m.sparse_attn_kv4(w["q"], w["cache"], w["table"], w["tok"], w["idx"], stream=s), (T, H, D), "bfloat16"),
        "fork_pages": (lambda s: m.fork_pages(w["table"], w["parent"], w["ref"], stream=s), (R, N // B), i32),
        "reserve_pages": (lambda s: m.reserve_pages(w["table"], w["ref"], w["begin"], w["end"], B, stream=s)[0], (4 * R + 1 + 2 * P,), i32),
        "compact_pages": (lambda s: m.compact_pages(w["table"], w["ref"], stream=s)[0], (2 * (P // 2) + 1 + P,), i32),
    }


NAMES = ["dequantize_kv4", "sparse_attn_kv4", "fork_pages", "reserve_pages", "compact_pages"]


def check(f, shape, t):
    """What the current stream freed is not what the call on another stream is given; and the other way round."""
    import torch

    side = torch.cuda.Stream()
    want = f(None).clone()
    f(side)
    torch.cuda.synchronize()
    freed = torch.empty(shape, dtype=getattr(torch, t), device="cuda")
    here = freed.untyped_storage().data_ptr()
    del freed
    got = f(side)
    torch.cuda.synchronize()
    assert got.untyped_storage().data_ptr() != here
    assert torch.equal(got, want)
    there = got.untyped_storage().data_ptr()
    del got
    again = torch.empty(shape, dtype=getattr(torch, t), device="cuda")
    assert again.untyped_storage().data_ptr() != there


@pytest.mark.parametrize("name", NAMES)
def test_allocations_of_the_4_bit_cache_s_calls(dsa, world, name):  # noqa: F811
    dsa.quantize_kv4(world["kv"], world["cache"], world["table"], world["seq"], world["pos"])
    check(*calls(dsa, world)[name])


def test_captured_call_on_a_side_stream(dsa, world):  # noqa: F811
    """stream= naming a stream that takes part in a capture: the allocation is the graph's."""
    import torch

    dsa.quantize_kv4(world["kv"], world["cache"], world["table"], world["seq"], world["pos"])
    want = dsa.sparse_attn_kv4(world["q"], world["cache"], world["table"], world["tok"], world["idx"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = dsa.sparse_attn_kv4(world["q"], world["cache"], world["table"], world["tok"], world["idx"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
    out.zero_()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert dsa.get_device_error() == 0


# ------------------------------------------------------------------------------------ the other calls


def small(m):
    """Calls of the indexer and the bf16 attention that allocate, as in `calls`; the outputs are compared where the call
    writes all of them."""
    import torch

    rng = np.random.default_rng(2)
    t, h, d, n, k = 40, 8, 64, 512, 32
    q = torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)).cuda().to(torch.float8_e4m3fn)
    key = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda().to(torch.bfloat16)
    codes, scale = m.quantize_k(key)
    w = torch.ones(t, h, device="cuda")
    ks, ke = dev(np.zeros(t), np.int32), dev(np.full(t, n), np.int32)
    logits = m.index_score(q, w, codes, scale, ks, ke)
    idx = m.index_topk(q, w, codes, scale, ks, ke, k)
    qb, _ = bf16(rng.standard_normal((t, h, 128)))
    kb, _ = bf16(rng.standard_normal((n, 128)))
    lse = torch.empty(t, h, device="cuda")
    out = m.sparse_attn(qb, kb, idx, lse=lse)

    def run(s):
        plan = m.index_topk_plan(ks, ke, n, h, d, k, stream=s)
        return m.index_topk_run(q, w, codes, scale, ks, ke, k, plan, stream=s)

    return {
        "index_score": (lambda s: m.index_score(q, w, codes, scale, ks, ke, stream=s), (t, n), "float32"),
        "index_score_kres": (lambda s: m.index_score_kres(q, w, codes, scale, ks, ke, stream=s), (t, n), "float32"),
        "topk": (lambda s: m.topk(logits, ks, ke, k, stream=s), (t, k), "int32"),
        "index_topk": (lambda s: m.index_topk(q, w, codes, scale, ks, ke, k, stream=s), (t, k), "int32"),
        "index_topk_plan, _run": (run, (t, k), "int32"),
        "quantize_k": (lambda s: m.quantize_k(key, stream=s)[0], (n, d), "uint8"),
        "sparse_attn": (lambda s: m.sparse_attn(qb, kb, idx, stream=s), (t, h, 128), "bfloat16"),
        "sparse_attn_bwd": (lambda s: m.sparse_attn_bwd(qb, kb, idx, out, lse, out, stream=s)[0], (t, h, 128), "float32"),
    }


@pytest.mark.parametrize("name", ["index_score", "index_score_kres", "topk", "index_topk", "index_topk_plan, _run", "quantize_k",
                                  "sparse_attn", "sparse_attn_bwd"])
def test_allocations_of_the_other_calls(dsa, name):  # noqa: F811
    check(*small(dsa)[name])
    assert dsa.get_device_error() == 0


def test_nothing_is_allocated_when_the_caller_brings_everything(dsa, world):  # noqa: F811
    import torch

    w, P = world, world["ref"].numel()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    src, dst, one, ws = i32(2 * R), i32(2 * R), i32(1), u8(dsa.reserve_pages_workspace_size(P))
    s2, d2, n2, ws2 = i32(P // 2), i32(P // 2), i32(1), u8(dsa.compact_pages_workspace_size(P))
    none = i32(0)
    empty, e_begin = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32(0)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = count()
    got = dsa.reserve_pages(w["table"], w["ref"], w["begin"], w["end"], B, src=src, dst=dst, lacking=one, workspace=ws)
    assert got[0] is src and got[1] is dst and got[2] is one
    got = dsa.compact_pages(w["table"], w["ref"], src=s2, dst=d2, n_live=n2, workspace=ws2)
    assert got[0] is s2 and got[1] is d2 and got[2] is n2
    assert count() == before
    # some of them, and lists of no entries
    for kw in ({}, dict(src=src), dict(dst=dst, workspace=ws), dict(lacking=one, workspace=ws), dict(src=src, dst=dst, workspace=ws),
               dict(src=src, dst=dst, lacking=one)):
        got = dsa.reserve_pages(w["table"], w["ref"], w["begin"], w["end"], B, **kw)
        assert [t.numel() for t in got] == [2 * R, 2 * R, 1] and got[2].item() == 0 and bool((got[0] == -1).all())
    for kw in (dict(lacking=one, workspace=ws), dict(src=none, lacking=one, workspace=ws), {}):
        got = dsa.reserve_pages(empty, w["ref"], e_begin, e_begin, B, **kw)
        assert [t.numel() for t in got] == [0, 0, 1] and got[2].item() == 0


def pool_of(t):
    """The stream whose pool the tensor's memory belongs to."""
    import torch

    p = t.untyped_storage().data_ptr()
    found = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"]]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("name", NAMES + ["index_score", "topk", "quantize_k", "sparse_attn", "sparse_attn_bwd"])
def test_allocations_from_the_right_pool(dsa, world, name):  # noqa: F811
    """For another stream, for the default stream (whose handle is 0) beside another current one, and without stream=."""
    import torch

    f = (calls(dsa, world) if name in NAMES else small(dsa))[name][0]
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert pool_of(f(side)) == side.cuda_stream
    assert pool_of(f(torch.cuda.ExternalStream(side.cuda_stream))) == side.cuda_stream
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert pool_of(f(torch.cuda.default_stream())) == 0
        assert pool_of(f(third)) == third.cuda_stream
        assert pool_of(f(None)) == side.cuda_stream
        assert pool_of(f(side)) == side.cuda_stream
    torch.cuda.synchronize()
    assert pool_of(f(torch.cuda.current_stream())) == 0 and pool_of(f(None)) == 0
    torch.cuda.synchronize()
