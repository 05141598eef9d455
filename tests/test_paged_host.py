"""The bf16 paged cache and the drafts' check without a GPU: the references of their tests against hand-made values, the C ABI's
synchronous refusals, the division by the head count, and the binding's checks of arguments on CPU tensors, which get as far as
the device check."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import paged_ref as PR
import sparse_attention_indexer_e4m3_gb300 as dsa

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_indexer_e4m3_gb300", "csrc")


# ------------------------------------------------------------------------------------ the references


def test_reference_maps_and_slots():
    """Sequences of 5 + 2, 7 + 0, -1 + 1 and 0 + 3 rows; six tokens of eight places."""
    seq, pos, ks, ke = PR.maps([5, 7, -1, 0], [2, 0, 1, 3], 8)
    assert list(seq) == [0, 0, 2, 3, 3, 3, -1, -1] and list(pos) == [5, 6, 0, 0, 1, 2, -1, -1]
    assert list(ks) == [0, 0, 14, 15, 15, 15, 0, 0] and list(ke) == [6, 7, 15, 16, 17, 18, 0, 0]
    table = np.array([[3, -1], [0, 9]])
    got = PR.slots(table, 4, 16, [0, 1, 2], [10, 0, 0], np.array([[9, 10, 25, 26], [-1, 15, 16, 31], [0, 1, 2, 3]]))
    assert got.tolist() == [[-1, 48, 63, -1], [-1, 15, -1, -1], [-1] * 4]


def test_reference_attention():
    """Two rows with scores 0 and ln 3, a sink of ln 4: weights 1/8 and 3/8; a window of one row; nothing to see."""
    q = torch.zeros(4, 1, 2, dtype=torch.float64)
    q[:, 0, 0] = 1
    kv = [torch.tensor([[0.0, 8.0], [math.log(3), 16.0]], dtype=torch.float64)]
    sink = torch.tensor([math.log(4)])
    out, lse, size, err = PR.attn(q, kv, [0, 0, 1, 0], [1, 0, 0, -1], None, 0, sink, 1.0)
    assert torch.allclose(out[0, 0], torch.tensor([3 / 8 * math.log(3), 7.0], dtype=torch.float64))
    assert torch.allclose(lse[:2, 0].exp(), torch.tensor([8.0, 5.0], dtype=torch.float64))
    assert not out[2:].any() and torch.allclose(lse[2:].exp(), torch.full((2, 1), 4.0, dtype=torch.float64))
    out, lse, _, _ = PR.attn(q[:1], kv, [0], [1], 1, 0, None, 1.0)
    assert torch.allclose(out[0, 0], kv[0][1]) and torch.allclose(lse[0], torch.tensor([math.log(3)], dtype=torch.float64))
    out, _, _, _ = PR.attn(q[:1], kv, [0], [1], 1, 1, None, 1.0)
    assert torch.allclose(out[0, 0, 1], torch.tensor((8 + 3 * 16) / 4, dtype=torch.float64))


def test_reference_drafts():
    """p / q = 1/2 at the drafted token: accepted below 1/2; refused, the next token comes from max(p - q, 0)."""
    target = np.array([[[0.25, 0.25, 0.5], [0.0, 1.0, 0.0]]], np.float32)
    draft = np.array([[[0.5, 0.5, 0.0]]], np.float32)
    run = lambda u, n=1, d=0: [int(x[0]) for x in PR.verify(target, draft, np.array([[d]]), [n], np.array([u], np.float32))]  # noqa: E731
    assert run([0.49, 0.3]) == [1, 1] and run([0.5, 0.3]) == [0, 2] and run([0.0, 0.9], d=3) == [0, 2]
    assert run([0.0, 0.24], n=0) == [0, 0] and run([0.0, 0.25], n=0) == [0, 1] and run([0.0, 0.99], n=-1) == [0, -1]
    assert PR.units([1.0, 2.0 ** -55, 2.0 ** -57, 7.0, -1.0, math.nan]) == [2 ** 55, 1, 0, 2 ** 55, 0, 0]


# ------------------------------------------------------------------------------------ C ABI refusals


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_e4m3_gb300 import build

    build.build()
    lib = ctypes.CDLL(dsa.library_path())
    p, i, sz, f, l = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
    lib.dsa_step_maps.argtypes = [p, p, i, i, p, p, p, p, p]
    lib.dsa_page_slots.argtypes = [p, i, i, i, i, p, p, p, i, i, p, p]
    lib.dsa_store_kv.argtypes = [p, l, p, p, i, i, p, i, i, p, i, i, p, p]
    lib.dsa_paged_attn.argtypes = [p, p, i, i, p, i, i, p, p, p, i, i, i, i, i, f, p, p, p, sz, p]
    lib.dsa_paged_attn_workspace_size.argtypes, lib.dsa_paged_attn_workspace_size.restype = [i] * 3, sz
    lib.dsa_verify_drafts.argtypes = [p, p, p, p, p, i, i, i, p, p, p]
    return lib


@pytest.fixture(scope="module")
def a():
    buf = ctypes.create_string_buffer(4096)
    yield (ctypes.addressof(buf) + 63) // 64 * 64
    del buf


OK, INVALID, UNSUPPORTED = 0, 1, 2
TOP = 2 ** 31 - 1


def test_maps_refusals(lib, a):
    at = lambda i: a + (i << 20)  # noqa: E731  (addresses apart; none is read)

    def f(held=a, added=at(1), R=2, T=3, seq=at(2), pos=at(3), ks=at(4), ke=at(5)):
        return lib.dsa_step_maps(held, added, R, T, seq, pos, ks, ke, None)

    assert f(R=-1) == f(T=-1) == INVALID
    for k in ("held", "added", "seq", "pos", "ks", "ke"):
        assert f(**{k: None}) == INVALID and f(**{k: a + 2}) == INVALID, k
    assert f(T=0, held=None, added=None, seq=None, pos=None, ks=None, ke=None) == OK


def test_slots_refusals(lib, a):
    at = lambda i: a + (i << 20)  # noqa: E731  (addresses apart; none is read)

    def f(table=a, R=1, M=2, P=2, rows=64, seq=at(1), start=None, idx=at(2), T=2, K=3, slots=at(3)):
        return lib.dsa_page_slots(table, R, M, P, rows, seq, start, idx, T, K, slots, None)

    assert f(rows=8) == f(rows=48) == f(rows=512) == f(M=1 << 25) == f(P=1 << 25) == UNSUPPORTED
    assert f(R=-1) == f(M=-1) == f(P=-1) == f(T=-1) == f(K=-1) == INVALID
    assert f(start=a + 1) == INVALID
    for k in ("table", "seq", "idx", "slots"):
        assert f(**{k: None}) == INVALID and f(**{k: a + 2}) == INVALID, k
    assert f(T=0, seq=None, idx=None, slots=None) == f(K=0, seq=None, idx=None, slots=None) == OK


def test_store_refusals(lib, a):
    at = lambda i: a + (i << 20)  # noqa: E731  (addresses apart; none is read)

    def f(kv=a, stride=128, seq=at(1), pos=at(2), N=4, D=128, pages=at(3), P=2, rows=64, table=at(4), R=1, M=2, lacking=None):
        return lib.dsa_store_kv(kv, stride, seq, pos, N, D, pages, P, rows, table, R, M, lacking, None)

    assert f(D=96) == f(D=1024) == f(rows=24) == f(M=1 << 25) == UNSUPPORTED
    assert f(N=-1) == f(P=-1) == f(R=-1) == f(M=-1) == f(stride=120) == f(stride=132) == f(stride=-128) == INVALID
    assert f(lacking=a + 2) == f(kv=a + 8) == f(pages=a + 8) == INVALID
    for k in ("kv", "seq", "pos", "pages", "table"):
        assert f(**{k: None}) == INVALID and f(**{k: a + 2}) == INVALID, k
    assert f(N=0, kv=None, seq=None, pos=None) == OK


def test_attention_refusals(lib, a):
    at = lambda i: a + (i << 20)  # noqa: E731  (addresses apart; none is read)

    def f(q=a, pages=at(1), P=2, rows=64, table=at(2), R=1, M=2, seq=at(3), pos=at(4), sink=None, T=2, H=4, D=128, window=0, first=0, out=at(5), lse=None):
        return lib.dsa_paged_attn(q, pages, P, rows, table, R, M, seq, pos, sink, T, H, D, window, first, 1.0, out, lse, None, 0, None)

    assert f(D=96) == f(D=1024) == f(rows=8) == f(M=1 << 25) == f(T=1 << 20, H=1 << 10) == f(P=1 << 25) == UNSUPPORTED
    assert f(T=TOP, H=TOP) == f(T=1, H=TOP) == f(T=TOP, H=1) == UNSUPPORTED
    assert f(T=-1) == f(H=0) == f(H=-5) == f(P=-1) == f(R=-1) == f(M=-1) == f(window=-1) == f(first=-1) == INVALID
    assert f(q=a + 8) == f(pages=a + 8) == f(out=a + 8) == f(sink=a + 2) == f(lse=a + 2) == INVALID
    for k in ("q", "pages", "table", "seq", "pos", "out"):
        assert f(**{k: None}) == INVALID and f(**{k: a + 2}) == INVALID, k
    assert f(T=0, q=None, seq=None, pos=None, out=None) == OK
    for x in ((0, 4, 128), (-1, 4, 128), (4, 0, 128), (4, 4, 96)):
        assert lib.dsa_paged_attn_workspace_size(*x) == 0


def test_drafts_refusals(lib, a):
    at = lambda i: a + (i << 20)  # noqa: E731  (addresses apart; none is read)

    def f(target=a, draft=at(1), tokens=at(2), count=at(3), u=at(4), R=2, G=3, V=5, accepted=at(5), token=at(6)):
        return lib.dsa_verify_drafts(target, draft, tokens, count, u, R, G, V, accepted, token, None)

    assert f(R=-1) == f(G=-1) == f(V=0) == f(V=-1) == INVALID
    assert f(R=1 << 28) == f(G=TOP) == UNSUPPORTED
    for k in ("target", "draft", "tokens", "count", "u", "accepted", "token"):
        assert f(**{k: None}) == INVALID and f(**{k: a + 2}) == INVALID, k
    assert f(R=0, target=None, draft=None, tokens=None, count=None, u=None, accepted=None, token=None) == OK


def test_outputs_that_overlap(lib, a):
    """What would be written while it is read is refused (all other arguments are right)."""
    at = [a + 256 * i for i in range(12)]

    def maps(held=at[0], added=at[1], seq=at[2], pos=at[3], ks=at[4], ke=at[5]):
        return lib.dsa_step_maps(held, added, 4, 6, seq, pos, ks, ke, None)

    assert maps(seq=at[0]) == maps(ke=at[1]) == maps(pos=at[2]) == maps(ks=at[5] + 20) == maps(seq=at[0] + 12) == INVALID

    def slots(table=at[0], seq=at[1], start=at[2], idx=at[3], out=at[4]):
        return lib.dsa_page_slots(table, 2, 2, 8, 16, seq, start, idx, 3, 5, out, None)

    assert slots(out=at[3] + 4) == slots(out=at[3] - 4) == slots(out=at[1]) == slots(out=at[2]) == slots(out=at[0] + 12) == INVALID
    store = lambda kv: lib.dsa_store_kv(kv, 64, at[0], at[0], 2, 64, at[4], 1, 16, at[1], 1, 1, None, None)  # noqa: E731
    assert store(at[4]) == store(at[4] - 128) == store(at[11] + 240) == INVALID  # (pages: 2 KB from at[4] on)
    attn = lambda q, out: lib.dsa_paged_attn(q, at[4], 1, 16, at[0], 1, 1, at[1], at[1], None, 1, 2, 64, 0, 0, 1.0, out, None, None, 0,  # noqa: E731
                                             None)
    assert attn(at[2], at[2] + 16) == attn(at[2] + 16, at[2]) == attn(at[2], at[4] + 16) == INVALID

    def verify(tokens=at[0], count=at[1], u=at[2], accepted=at[3], token=at[4]):
        return lib.dsa_verify_drafts(at[8], at[8], tokens, count, u, 2, 3, 5, accepted, token, None)

    assert verify(accepted=at[1]) == verify(token=at[1]) == verify(token=at[3]) == verify(accepted=at[0] + 20) == verify(token=at[2]) == INVALID


# ------------------------------------------------------------------------------------ what no run shows


def test_division_by_the_head_count():
    """The attention's n / H by a product (its multiplier as set_heads forms it) is the quotient for every n below 2^31."""
    text = open(os.path.join(SRC, "paged.cuh")).read()
    assert "h_mul = static_cast<uint32_t>((((static_cast<uint64_t>(1) << h_shift) - heads) << 32) / heads + 1);" in text
    rng = np.random.default_rng(0)
    for H in list(range(1, 300)) + [1000, 4095, 65535, 65536, 65537, 2 ** 29 + 3, 2 ** 30 - 1]:
        shift = (H - 1).bit_length()
        mul = (((1 << shift) - H) << 32) // H + 1
        assert mul < 2 ** 32
        k = rng.integers(0, 2 ** 30 // H + 1, 200)
        n = np.unique(np.concatenate([k * H - 1, k * H, k * H + H - 1, [0, 1, 2 ** 30 - 1]]))
        n = n[(n >= 0) & (n < 2 ** 31)].astype(object)
        for v in n:  # (the kernel's sum is a 32-bit one)
            s = ((int(v) * mul) >> 32) + int(v)
            assert s < 2 ** 32 and s >> shift == int(v) // H


def test_waits_have_a_limit():
    """No loop of the attention's waits for a barrier but through the wait that gives up; softmax warps pass hardware barriers at a
    unit's ends only where they have rows of q of their own."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(SRC, "paged_attn_kernel.cuh")).read())
    kernel = text[text.index("paged_attn_kernel("):text.index("paged_join_kernel(")]
    assert not re.search(r"(?<![\w_])mbar_wait\(|mbar_try_wait\(", kernel)
    at = [kernel.index(m) for m in ("if (warp == 2) {", "} else if (warp >= kPgFirstLoad) {", "} else if (warp < 2) {",
                                    "} else if constexpr (L::kByRow) {", "float x[kC];")]
    assert at == sorted(at)
    for part in (kernel[a:b] for a, b in zip(at[:3], at[1:4])):
        assert not any(h in part for h in ("named_bar_sync(", "bar_or(", "__syncthreads("))
    by_row = kernel[at[3]:at[4]]
    blocks = by_row[by_row.index("for (int b = static_cast<int>"):by_row.index("gb0 += nb;")]
    assert not any(h in blocks for h in ("named_bar_sync(", "bar_or(", "__syncthreads(", "break;", "return;"))


# ------------------------------------------------------------------------------------ the binding

T, H, D, K, P, B, R, M, G, V = 6, 5, 128, 7, 9, 32, 3, 4, 2, 11
i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32


def z(*shape, t=i32):
    return torch.zeros(shape, dtype=t)


POOL = lambda: z(P, B, D, t=bf16)  # noqa: E731
Q = lambda: z(T, H, D, t=bf16)  # noqa: E731
DRAFTS = lambda **k: dsa.verify_drafts(**{**dict(target=z(R, G + 1, V, t=f32), draft=z(R, G, V, t=f32), tokens=z(R, G), count=z(R),  # noqa: E731
                                                 u=z(R, G + 1, t=f32)), **k})


@pytest.mark.parametrize("call", [
    lambda: dsa.step_maps(z(R), z(R), T, seq=z(T), pos=z(T), ks=z(T), ke=z(T)),
    lambda: dsa.step_maps(z(0), z(0), 0),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T, K), start=z(T), out=z(T, K)),
    lambda: dsa.page_slots(z(P, B, t=torch.uint8), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, t=bf16), POOL(), z(R, M), z(T), z(T), lacking=z(1)),
    lambda: dsa.store_kv(z(T, 2 * D, t=bf16)[:, 16:16 + D], POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), window=3, first=2, attn_sink=z(H, t=f32), scale=1, out=Q(), lse=z(T, H, t=f32),
                           workspace=z(64, t=torch.uint8)),
    lambda: DRAFTS(accepted=z(R), token=z(R)),
    lambda: DRAFTS(target=z(R, 1, V, t=f32), draft=z(R, 0, V, t=f32), tokens=z(R, 0), u=z(R, 1, t=f32)),
])
def test_binding_accepts_shapes_and_wants_cuda(lib, call):
    """Arguments that are right in every other respect get as far as the device check."""
    with pytest.raises(ValueError, match="CUDA"):
        call()


@pytest.mark.parametrize("call", [
    lambda: dsa.step_maps(z(R), z(R + 1), T),
    lambda: dsa.step_maps(z(R, 1), z(R, 1), T),
    lambda: dsa.step_maps(z(R, t=torch.int64), z(R), T),
    lambda: dsa.step_maps(z(R), z(R), -1),
    lambda: dsa.step_maps(z(R), z(R), 1 << 31),
    lambda: dsa.step_maps(z(R), z(R), "4"),
    lambda: dsa.step_maps(z(R), z(R), T, pos=z(T + 1)),
    lambda: dsa.step_maps(z(R), z(R), T, ke=z(2 * T)[::2]),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T - 1, K)),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T, K, 1)),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T, K, t=torch.int64)),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T, K), start=z(T, 1)),
    lambda: dsa.page_slots(POOL(), z(R, M), z(T), z(T, K), out=z(T, K + 1)),
    lambda: dsa.page_slots(z(P, 24, D, t=bf16), z(R, M), z(T), z(T, K)),
    lambda: dsa.page_slots(z(P * B, t=bf16), z(R, M), z(T), z(T, K)),
    lambda: dsa.store_kv(z(T, D, t=torch.float16), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, 1, t=bf16), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, 2 * D, t=bf16)[:, ::2], POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D + 4, t=bf16)[:, :D], POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(1, D, t=bf16).expand(T, D), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, 64, t=bf16), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, t=bf16), z(P, B, D, t=torch.float16), z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, t=bf16), z(P, B, 2 * D, t=bf16)[:, :, :D], z(R, M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, t=bf16), POOL(), z(R * M), z(T), z(T)),
    lambda: dsa.store_kv(z(T, D, t=bf16), POOL(), z(R, M), z(T), z(T + 1)),
    lambda: dsa.store_kv(z(T, D, t=bf16), POOL(), z(R, M), z(T), z(T), lacking=z(2)),
    lambda: dsa.paged_attn(z(T, H, 96, t=bf16), z(P, B, 96, t=bf16), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(z(T, H, D, t=torch.float16), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(z(T, D, t=bf16), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(z(H, T, D, t=bf16).transpose(0, 1), POOL(), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(Q(), z(P, B, 64, t=bf16), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(Q(), z(P, B, D, 1, t=bf16), z(R, M), z(T), z(T)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T + 1), z(T)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T, 1)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), window=0),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), window=-1),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), first=-1),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), first=None),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), scale="1"),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), attn_sink=z(H + 1, t=f32)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), out=z(T, H, D, t=f32)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), lse=z(H, T, t=f32)),
    lambda: dsa.paged_attn(Q(), POOL(), z(R, M), z(T), z(T), workspace=z(64)),
    lambda: DRAFTS(target=z(R, G, V, t=f32)),
    lambda: DRAFTS(target=z(R, G + 1, V, t=bf16)),
    lambda: DRAFTS(target=z(R, G + 1, 0, t=f32), draft=z(R, G, 0, t=f32)),
    lambda: DRAFTS(draft=z(R, G, V + 1, t=f32)),
    lambda: DRAFTS(tokens=z(R, G, t=torch.int64)),
    lambda: DRAFTS(count=z(R + 1)),
    lambda: DRAFTS(u=z(R, G, t=f32)),
    lambda: DRAFTS(accepted=z(R, 1)),
    lambda: DRAFTS(token=z(R + 1)),
])
def test_binding_refuses(lib, call):
    with pytest.raises((ValueError, TypeError, OverflowError)) as e:
        call()
    assert "CUDA" not in str(e.value)  # refused for what is wrong, before the device is looked at


def test_binding_refuses_what_is_no_tensor(lib):
    with pytest.raises(TypeError):
        dsa.step_maps([1], z(1), T)
    with pytest.raises(TypeError):
        dsa.page_slots(None, z(R, M), z(T), z(T, K))
    with pytest.raises(TypeError):
        dsa.page_slots(POOL(), z(R, M), z(T), [0])
    with pytest.raises(TypeError):
        dsa.store_kv([1.0], POOL(), z(R, M), z(T), z(T))
    with pytest.raises(TypeError):
        dsa.paged_attn(None, POOL(), z(R, M), z(T), z(T))
    with pytest.raises(TypeError):
        DRAFTS(u=0.5)
