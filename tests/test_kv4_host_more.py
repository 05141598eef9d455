"""The 4-bit cache's calls without a GPU, beyond test_kv4_host.py: refusals of the C ABI and of the binding."""
import ctypes

import pytest
import torch

import kv4_ref as K4
import sparse_attention_indexer_e4m3_gb300 as dsa
from test_kv4_host import CACHE, D, INVALID, M, OK, P, R, T, UNSUPPORTED, bf16, lib, mem, z  # noqa: F401  (lib, mem: fixtures)


def test_reserved_write_refusals(lib, mem):  # noqa: F811
    _, a = mem
    p, i = ctypes.c_void_p, ctypes.c_int
    f = lib.dsa_quantize_kv4_reserved
    f.argtypes = [p, p, p, i, i, p, i, i, p, i, i, p, p]

    def w(kv=a, seq=a, pos=a, N=4, D=128, cache=a, P=2, rows=64, table=a, R=1, M=2, lacking=a):
        return f(kv, seq, pos, N, D, cache, P, rows, table, R, M, lacking, None)

    assert w(lacking=a + 2) == w(kv=None) == w(cache=a + 8) == INVALID and w(D=96) == UNSUPPORTED
    assert w(N=0, kv=None, seq=None, pos=None, lacking=None) == OK


@pytest.mark.parametrize("lacking", [z(2), z(1, 1), z(1, t=torch.int64), 0])
def test_binding_refuses_lacking(lib, lacking):  # noqa: F811
    with pytest.raises((ValueError, TypeError)) as e:
        dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M), z(T), z(T), lacking=lacking)
    assert "CUDA" not in str(e.value)


def test_binding_wants_lacking_on_the_device(lib):  # noqa: F811
    with pytest.raises(ValueError, match="CUDA"):
        dsa.quantize_kv4(z(T, D, t=bf16), CACHE(), z(R, M), z(T), z(T), lacking=z(1))


def test_reserve_refuses_more_entries_than_it_can_count(lib, mem):  # noqa: F811
    """All entries of a table may need pages, and that number has to fit an int: past it the count wrapped."""
    _, a = mem
    f = lambda R, M: lib.dsa_reserve_pages(a, a, a, a, R, M, 3, 16, a, a, a, a, 1 << 10, None)  # noqa: E731
    assert f(1 << 16, 1 << 15) == f(1 << 24, 1 << 24) == f((1 << 30) - 1, 3) == UNSUPPORTED


def test_attention_refuses_longer_lists_than_it_can_scan_in_time(lib, mem):  # noqa: F811
    _, a = mem
    f = lambda K: lib.dsa_sparse_attn_kv4(a, a, 2, 64, a, 1, 2, a, None, None, a, 2, 4, 128, K, 1.0, a, None, None, 0, None)  # noqa: E731
    assert f((1 << 26) + 1) == f(2 ** 31 - 1) == UNSUPPORTED
