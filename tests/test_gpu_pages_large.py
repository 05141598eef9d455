"""The page calls on the largest tables."""
import pytest

from test_gpu_kv4 import dsa  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_fork_of_the_longest_row(dsa):  # noqa: F811
    """One row of 2^31 - 5 entries (8.6 GB), freed: its first, middle and last pages are."""
    import torch

    M = 2 ** 31 - 5
    table = torch.full((1, M), -1, dtype=torch.int32, device="cuda")
    at = [0, 1, 256 << 16, 2 ** 30, M - 2, M - 1]
    for p, j in enumerate(at):
        table[0, j] = p
    ref = torch.ones(len(at) + 1, dtype=torch.int32, device="cuda")
    parent = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dsa.fork_pages(table, parent, ref)
    assert torch.equal(out, table) and bool((ref == 1).all())
    dsa.fork_pages(table, parent - 1, ref, table_out=out)
    assert int(out.max()) == -1 and int(out.min()) == -1
    assert ref.tolist() == [0] * len(at) + [1]
