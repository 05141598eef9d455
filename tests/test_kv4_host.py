"""The 4-bit paged cache without a GPU: the reference of its tests against hand-made values and torch's
e4m3, the C ABI's synchronous refusals, and the binding's checks of arguments on CPU tensors, which get as far as the
device check."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as K4
import sparse_attention_indexer_e4m3_gb300 as dsa


# ------------------------------------------------------------------------------------ the reference


def test_reference_levels():
    assert np.array_equal(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), K4.E4M3)
    v = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 3.5, 5.0, 5.01, 9.0])
    assert list(K4._nearest(v, K4.E2M1)) == [0, 0, 1, 2, 2, 3, 4, 4, 6, 6, 7, 7]


def test_reference_worked_row():
    """One group 0, -6, 3, 2.5, .25, ... whose largest value is 6 * 1: r is the least power of two with
    6 <= 2688 r, 2^-8 (2688 / 256 = 10.5); s = 6 / 6 / r = 256; codes of x / 256 / 2^-8 = x."""
    x = np.zeros((1, 16))
    x[0, :6] = [0.0, -6.0, 3.0, 2.5, 0.25, -0.25]
    c, s8, r = K4.encode(x)
    assert r[0] == 2.0 ** -8 and K4.E4M3[s8[0, 0]] == 256.0
    assert list(c[0, :3]) == [0 | 15 << 4, 5 | 4 << 4, 0 | 8 << 4]
    assert np.array_equal(K4.decode(c, s8, r)[0, :6], [0, -6, 3, 2, 0, 0])
    z = K4.encode(np.zeros((1, 16)))
    assert z[2][0] == 2.0 ** -100 and not z[0].any() and not z[1].any()


def test_reference_pages():
    t = np.array([[4, 1, -1], [4, 5, -1], [-1, -1, -1]], np.int32)
    ref = K4.counts(t, 7)
    assert list(ref) == [0, 1, 0, 0, 2, 1, 0]
    t2, r2 = K4.fork(t, [0, 0, 1], ref)
    assert t2.tolist() == [[4, 1, -1], [4, 1, -1], [4, 5, -1]] and np.array_equal(r2, K4.counts(t2, 7))
    # rows [6, 9) of 4-row pages: page 1 (shared) keeps rows 4, 5; page 2 is missing
    t3, r3, src, dst, lack = K4.reserve(t2, r2, [6, 0, 8], [9, 0, 8], 4)
    assert lack == 0 and t3.tolist() == [[4, 0, 2], [4, 1, -1], [4, 5, -1]] and np.array_equal(r3, K4.counts(t3, 7))
    assert src.tolist() == [1, -1, -1, -1, -1, -1] and dst.tolist() == [0, -1, -1, -1, -1, -1]
    t4, r4, src, dst, n = K4.compact(t3, r3)
    assert n == 5 and t4.tolist() == [[4, 0, 2], [4, 1, -1], [4, 3, -1]] and np.array_equal(r4, K4.counts(t4, 7))
    assert src.tolist() == [5, -1, -1] and dst.tolist() == [3, -1, -1]


# ------------------------------------------------------------------------------------ C ABI refusals


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_e4m3_gb300 import build

    build.build()
    lib = ctypes.CDLL(dsa.library_path())
    p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.dsa_quantize_kv4.argtypes = [p, p, p, i, i, p, i, i, p, i, i, p]
    lib.dsa_dequantize_kv4.argtypes = [p, i, i, p, i, i, p, p, i, i, p, p]
    lib.dsa_sparse_attn_kv4.argtypes = [p, p, i, i, p, i, i, p, p, p, p, i, i, i, i, ctypes.c_float, p, p, p, sz, p]
    lib.dsa_sparse_attn_kv4_workspace_size.argtypes, lib.dsa_sparse_attn_kv4_workspace_size.restype = [i] * 4, sz
    lib.dsa_fork_pages.argtypes = [p, p, i, i, i, p, p, p]
    lib.dsa_reserve_pages.argtypes = [p, p, p, p, i, i, i, i, p, p, p, p, sz, p]
    lib.dsa_reserve_pages_workspace_size.restype = lib.dsa_compact_pages_workspace_size.restype = sz
    lib.dsa_compact_pages.argtypes = [p, p, i, i, i, p, p, p, p, sz, p]
    lib.dsa_copy_pages.argtypes = [p, sz, i, p, p, i, p]
    return lib


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(256)
    at = (ctypes.addressof(buf) + 63) // 64 * 64
    return buf, at


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def test_page_bytes(lib):
    for rows in (16, 32, 64, 128, 256):
        for D in (64, 128, 256, 512):
            assert dsa.kv4_page_bytes(rows, D) == K4.page_bytes(rows, D) and K4.page_bytes(rows, D) % 16 == 0
    assert dsa.kv4_page_bytes(8, 128) == dsa.kv4_page_bytes(48, 128) == dsa.kv4_page_bytes(512, 128) == 0
    assert dsa.kv4_page_bytes(64, 96) == 0


def test_codec_refusals(lib, mem):
    _, a = mem
    w = lambda kv=a, seq=a, pos=a, N=4, D=128, cache=a, P=2, rows=64, table=a, R=1, M=2: lib.dsa_quantize_kv4(  # noqa: E731
        kv, seq, pos, N, D, cache, P, rows, table, R, M, None)
    r = lambda kv=a, seq=a, pos=a, N=4, D=128, cache=a, P=2, rows=64, table=a, R=1, M=2: lib.dsa_dequantize_kv4(  # noqa: E731
        cache, P, rows, table, R, M, seq, pos, N, D, kv, None)
    for f in (w, r):
        assert f(D=96) == f(rows=48) == f(rows=8) == f(rows=512) == f(M=1 << 25) == UNSUPPORTED
        assert f(N=-1) == f(P=-1) == f(R=-1) == f(M=-1) == INVALID
        assert f(kv=None) == f(seq=None) == f(pos=None) == f(cache=None) == f(table=None) == INVALID
        assert f(kv=a + 8) == f(cache=a + 8) == f(table=a + 2) == f(seq=a + 1) == f(pos=a + 2) == INVALID
        assert f(N=0, kv=None, seq=None, pos=None) == OK


def test_attention_refusals(lib, mem):
    _, a = mem

    def f(q=a, cache=a, P=2, rows=64, table=a, R=1, M=2, seq=a, start=None, sink=None, idx=a, T=2, H=4, D=128, K=3, out=a,
          lse=None):
        return lib.dsa_sparse_attn_kv4(q, cache, P, rows, table, R, M, seq, start, sink, idx, T, H, D, K, 1.0, out, lse, None, 0, None)

    assert f(D=96) == f(rows=24) == f(M=1 << 26) == f(T=1 << 30, H=256) == UNSUPPORTED
    assert f(T=-1) == f(H=0) == f(K=-1) == f(P=-1) == f(R=-3) == INVALID
    assert f(q=None) == f(out=None) == f(seq=None) == f(idx=None) == f(cache=None) == f(table=None) == INVALID
    assert f(q=a + 8) == f(cache=a + 4) == f(out=a + 1) == f(start=a + 1) == f(sink=a + 2) == f(lse=a + 1) == f(idx=a + 2) == INVALID
    assert f(T=0, q=None, out=None, seq=None, idx=None) == OK


def test_attention_workspace_of_extreme_counts(lib):
    """Head and block counts near the largest int neither wrap nor ask for memory: so many units share no list."""
    top = 2 ** 31 - 1
    for T, H, K in [(1, top, 2048), (1, top - 63, top), (top, top, top), (3, top - 1, 1)]:
        for D in (64, 128, 256, 512):
            assert lib.dsa_sparse_attn_kv4_workspace_size(T, H, D, K) == 0
    assert lib.dsa_sparse_attn_kv4_workspace_size(0, 64, 128, 64) == lib.dsa_sparse_attn_kv4_workspace_size(1, 64, 96, 64) == 0


def test_page_call_refusals(lib, mem):
    _, a = mem
    fork = lambda table=a, parent=a, R=2, M=2, P=3, ref=a, out=a + 64: lib.dsa_fork_pages(table, parent, R, M, P, ref, out, None)  # noqa: E731
    assert fork(R=-1) == fork(M=-1) == fork(P=-1) == INVALID
    assert fork(table=None) == fork(parent=None) == fork(ref=None) == fork(out=None) == fork(out=a + 66) == INVALID
    assert fork(out=a) == fork(out=a + 8) == fork(table=a + 68) == INVALID  # the tables overlap
    assert fork(R=0) == fork(M=0) == OK
    assert lib.dsa_reserve_pages_workspace_size(10) >= 80 and lib.dsa_reserve_pages_workspace_size(0) == 0

    def res(table=a, ref=a, begin=a, end=a, R=2, M=2, P=3, rows=64, src=a, dst=a, lack=a, ws=a, nb=1 << 10):
        return lib.dsa_reserve_pages(table, ref, begin, end, R, M, P, rows, src, dst, lack, ws, nb, None)

    assert res(R=-1) == res(M=-1) == res(P=-1) == INVALID
    assert res(rows=63) == res(M=1 << 28) == UNSUPPORTED
    for k in ("table", "ref", "begin", "end", "src", "dst", "lack"):
        assert res(**{k: None}) == INVALID and res(**{k: a + 2}) == INVALID, k
    assert res(ws=None) == res(nb=8) == res(ws=a + 2) == WORKSPACE

    def com(table=a, ref=a, R=2, M=2, P=3, src=a, dst=a, n=a, ws=a, nb=1 << 10):
        return lib.dsa_compact_pages(table, ref, R, M, P, src, dst, n, ws, nb, None)

    assert com(R=-1) == com(M=-1) == com(P=-1) == INVALID
    for k in ("table", "ref", "src", "dst", "n"):
        assert com(**{k: None}) == INVALID and com(**{k: a + 2}) == INVALID, k
    assert com(ws=None) == com(nb=8) == com(ws=a + 2) == WORKSPACE
    copy = lambda pages=a, nb=32, P=2, src=a, dst=a, n=1: lib.dsa_copy_pages(pages, nb, P, src, dst, n, None)  # noqa: E731
    assert copy(nb=0) == copy(nb=24) == copy(nb=1 << 41) == UNSUPPORTED
    assert copy(P=-1) == copy(n=-1) == copy(pages=None) == copy(pages=a + 8) == copy(src=None) == copy(dst=a + 1) == INVALID
    assert copy(n=0, src=None, dst=None) == copy(P=0, pages=None) == OK


# ------------------------------------------------------------------------------------ the binding

T, H, D, K, P, B, R, M = 6, 5, 128, 7, 9, 32, 3, 4
i32, bf16 = torch.int32, torch.bfloat16


def z(*shape, t=i32):
    return torch.zeros(shape, dtype=t)


CACHE = lambda: z(P, K4.page_bytes(B, D), t=torch.uint8)  # noqa: E731


@pytest.mark.parametrize("call", [
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M), z(T), z(T)),
    lambda: dsa.dequantize_kv4(CACHE(), z(R, M), z(T), z(T), D, out=z(T, D, t=bf16)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), start=z(T), attn_sink=torch.zeros(H),
                                lse=torch.zeros(T, H), out=z(T, H, D, t=bf16)),
    lambda: dsa.fork_pages(z(R, M), z(R), z(P), table_out=z(R, M)),
    lambda: dsa.reserve_pages(z(R, M), z(P), z(R), z(R), B, src=z(2 * R), dst=z(2 * R), lacking=z(1), workspace=z(99, t=torch.uint8)),
    lambda: dsa.compact_pages(z(R, M), z(P), src=z(P // 2), dst=z(P // 2), n_live=z(1), workspace=z(99, t=torch.uint8)),
    lambda: dsa.copy_pages(torch.zeros(P, 4, 4), z(3), z(3)),
])
def test_binding_accepts_shapes_and_wants_cuda(lib, call):
    """Arguments that are right in every other respect get as far as the device check."""
    with pytest.raises(ValueError, match="CUDA"):
        call()


@pytest.mark.parametrize("call", [
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M), z(T - 1), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M), z(T), z(T, 1)),
    lambda: dsa.quantize_kv4(z(T, 96, t=bf16), CACHE(), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), z(P, K4.page_bytes(B, D) + 16, t=torch.uint8), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), z(P, 24 * (D // 2 + D // 16 + 4), t=torch.uint8), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R * M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, 2 * D, t=bf16)[:, ::2], CACHE(), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(D, t=bf16), CACHE(), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=torch.float16), CACHE(), z(R, M), z(T), z(T)),
    lambda: dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M, t=torch.int64), z(T), z(T)),
    lambda: dsa.dequantize_kv4(CACHE(), z(R, M), z(T), z(T), D, out=z(T, D + 1, t=bf16)),
    lambda: dsa.dequantize_kv4(CACHE(), z(R, M), z(T, 1), z(T, 1), D),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T - 1, K)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T + 1), z(T, K)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), start=z(T - 1)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), attn_sink=torch.zeros(H + 1)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), out=z(T, H, D - 1, t=bf16)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), lse=torch.zeros(H, T)),
    lambda: dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K, t=torch.int64)),
    lambda: dsa.sparse_attn_kv4(z(T, H, 2 * D, t=bf16), CACHE(), z(R, M), z(T), z(T, K)),
    lambda: dsa.fork_pages(z(R, M), z(R + 1), z(P)),
    lambda: dsa.fork_pages(z(R, M), z(R), z(P, 1)),
    lambda: dsa.fork_pages(z(R, M), z(R), z(P), table_out=z(R, M + 1)),
    lambda: dsa.reserve_pages(z(R, M), z(P), z(R - 1), z(R), B),
    lambda: dsa.reserve_pages(z(R, M), z(P), z(R), z(R), B, src=z(R)),
    lambda: dsa.reserve_pages(z(R, M), z(P), z(R), z(R), B, lacking=z(2)),
    lambda: dsa.reserve_pages(z(R, M), z(P), z(R), z(R), B, workspace=z(99)),
    lambda: dsa.compact_pages(z(R, M), z(P), dst=z(P)),
    lambda: dsa.compact_pages(z(R, M), z(P), n_live=z(0)),
    lambda: dsa.copy_pages(z(P), z(3), z(3)),
    lambda: dsa.copy_pages(CACHE(), z(3), z(4)),
    lambda: dsa.copy_pages(CACHE(), z(3, t=torch.int64), z(3)),
    lambda: dsa.copy_pages(CACHE()[:, ::2], z(3), z(3)),
])
def test_binding_refuses(lib, call):
    with pytest.raises((ValueError, TypeError)) as e:
        call()
    assert "CUDA" not in str(e.value)  # refused for what is wrong, before the device is looked at


def test_binding_refuses_what_is_no_tensor(lib):
    with pytest.raises(TypeError):
        dsa.quantize_kv4([1.0], CACHE(), z(R, M), z(T), z(T))
    with pytest.raises(TypeError):
        dsa.copy_pages(None, z(3), z(3))
    with pytest.raises(TypeError):
        dsa.reserve_pages(z(R, M), z(P), z(R), z(R), "64")
    with pytest.raises(TypeError):
        dsa.sparse_attn_kv4(z(T, H, D, t=bf16), CACHE(), z(R, M), z(T), z(T, K), scale="1")
