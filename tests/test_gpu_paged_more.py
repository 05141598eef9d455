"""More of the paged attention on the GPU: what it refuses there, and values, rows of q and steps at which its parts differ."""
import math

import numpy as np
import pytest
import torch

import paged_ref as PR
import sparse_attention_indexer_e4m3_gb300 as dsa
from test_gpu_paged_attn import i32

pytestmark = pytest.mark.gpu

bf16 = torch.bfloat16


def test_workspace_over_other_arrays():
    """A workspace that is part of what the call reads or writes is refused; one right behind it is not."""
    T, H, D = 2, 3, 64
    need = dsa.paged_attn_workspace_size(T, H, D)
    room = torch.zeros(need + 65536, dtype=torch.uint8, device="cuda")
    part = lambda at, n, t: room[at:at + n].view(t)  # noqa: E731
    q, out = (torch.zeros(T, H, D, dtype=bf16, device="cuda") for _ in range(2))
    pages = torch.zeros(2, 16, D, dtype=bf16, device="cuda")
    lse, table, seq = torch.zeros(T, H, device="cuda"), i32([[0], [1]]), i32([0, 1])
    given = dict(q=q, pages=pages, table=table, seq=seq, pos=i32([3, 4]), out=out, lse=lse, attn_sink=torch.zeros(H, device="cuda"))
    for name, x in given.items():
        n = x.numel() * x.element_size()
        for at, refused in ((need + 4096 - need % 4096, False), ((need - 16) // 16 * 16, True)):
            y = part(at, n, x.dtype).view(x.shape).copy_(x)
            call = lambda: dsa.paged_attn(**{**given, name: y}, workspace=room[:need])  # noqa: B023, E731
            if refused:
                with pytest.raises(dsa.DsaError, match="INVALID"):
                    call()
            else:
                call()
    assert dsa.get_device_error() == 0


def best(f, calls=20, times=9):
    """Least device time of a call, of `times` runs of `calls` of them."""
    f()
    t = []
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(calls):
            f()
        b.record()
        torch.cuda.synchronize()
        t.append(a.elapsed_time(b))
    return min(t) / calls


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_places_without_a_token_may_hold_anything(D):
    """q that is no number where no token is, or in another sequence's token of the unit, changes no bit of the others' outputs; in
    places without a token it does not send every row of the sequence through the search for what is no number (2.3 times the time
    at D <= 256)."""
    rng = np.random.default_rng(D)
    H, lens = 8, [20000, 900]
    pages, table, kv = PR.pool(lens, 64, D, rng)
    seq, pos = np.array([0] * 4 + [-1] * 3 + [1]), np.array(list(range(19996, 20000)) + [-1] * 3 + [899])
    q = torch.from_numpy(rng.standard_normal((8, H, D))).to(bf16).cuda()
    out, work = torch.empty_like(q), torch.empty(dsa.paged_attn_workspace_size(8, H, D), dtype=torch.uint8, device="cuda")
    run = lambda x, n=8: dsa.paged_attn(x, pages, table, i32(seq[:n]), i32(pos[:n]))  # noqa: E731
    want = run(q)
    PR.check_attn(want, None, PR.attn(q, kv, seq, pos, None, 0, None, 1 / math.sqrt(D)), D)
    for bad in (math.nan, math.inf):
        x = q.clone()
        x[4:7] = bad
        assert torch.equal(run(x), want)
        x[7] = bad
        assert torch.equal(run(x)[:7], want[:7])
    s, p = i32(seq[:7]), i32(pos[:7])
    time = lambda x: best(lambda: dsa.paged_attn(x, pages, table, s, p, out=out[:7], workspace=work))  # noqa: E731
    assert time(x[:7].contiguous()) < 1.4 * time(q[:7].contiguous())
    assert dsa.get_device_error() == 0
