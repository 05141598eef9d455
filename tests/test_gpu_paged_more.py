"""More of the paged attention on the GPU: what it refuses there, and values, rows of q and steps at which its parts differ."""
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
