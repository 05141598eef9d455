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


# Tokens whose sequence is one of 600 rows with a value that is no number in row 70, or one of 40 without; how the block of that row is
# met: seen whole by all of a unit's rows of q, cut by a token's own position, at a window's edge, in a unit of two sequences.
KINDS = {
    "whole": ([0], [599], None, 0),
    "whole, two tokens": ([0, 0], [598, 599], None, 0),
    "own row behind": ([0, 0, 0], [100, 69, 70], None, 0),
    "window's edge": ([0, 0], [169, 170], 100, 0),
    "first rows": ([0, 0], [599, 595], 30, 71),
    "two sequences": ([0, 1, 0], [599, 39, 500], None, 0),
}


def sees(seq, pos, window, first, at):
    return torch.tensor([r == 0 and p >= at and (window is None or at > p - window or at < first) for r, p in zip(seq, pos)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,H", [(64, 16), (128, 40), (256, 9), (512, 30)])
def test_infinite_values(D, H, kind):
    """Whatever the score of a row with infinite values is (infinite of either sign, or no number), all outputs of a token that sees it
    and its lse are no numbers, however its block is met; other tokens' are as without it."""
    rng = np.random.default_rng(D)
    at, dim = 70, D // 3
    seq, pos, window, first = KINDS[kind]
    for values in ([math.inf], [-math.inf], [math.inf, -math.inf]):
        pages, table, kv = PR.pool([600, 40], 32, D, rng)
        for i, v in enumerate(values):
            pages[int(table[0, at // 32]), at % 32, dim + i] = v
        q = torch.from_numpy(rng.standard_normal((len(seq), H, D))).to(bf16)
        q[:, 0, dim] = 0
        lse = torch.empty(len(seq), H, device="cuda")
        out = dsa.paged_attn(q.cuda(), pages, table, i32(seq), i32(pos), window=window, first=first, lse=lse)
        hit = sees(seq, pos, window, first, at)
        assert hit.any() and (q[hit][:, :, dim] > 0).any() and (q[hit][:, :, dim] < 0).any()
        assert torch.isnan(out.cpu()[hit]).all() and torch.isnan(lse.cpu()[hit]).all()
        ref = PR.attn(q, kv, seq, pos, window, first, None, 1 / math.sqrt(D))
        PR.check_attn(out.cpu()[~hit], lse.cpu()[~hit], [x[~hit] for x in ref], D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_infinite_values_of_a_shared_unit(D):
    """The same where many CTAs have a part of the unit, and one of them the row; and in one of two units' tokens."""
    rng = np.random.default_rng(D)
    H, n, at = 6, 20000, 9000
    pages, table, kv = PR.pool([n], 64, D, rng)
    pages[int(table[0, at // 64]), at % 64, 1] = math.inf
    q = torch.from_numpy(rng.standard_normal((2, H, D))).to(bf16)
    for pos in ([n - 1, at - 1], [n - 1, n - 2]):
        lse = torch.empty(2, H, device="cuda")
        out = dsa.paged_attn(q.cuda(), pages, table, i32([0, 0]), i32(pos), lse=lse)
        hit = torch.tensor(pos) >= at
        assert torch.isnan(out.cpu()[hit]).all() and torch.isnan(lse.cpu()[hit]).all()
        ref = PR.attn(q, kv, [0, 0], pos, None, 0, None, 1 / math.sqrt(D))
        PR.check_attn(out.cpu()[~hit], lse.cpu()[~hit], [x[~hit] for x in ref], D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,H", [(64, 16), (128, 40), (256, 9), (512, 30)])
def test_scores_below_fp32(D, H, kind):
    """Finite values whose score overflows to minus infinity weigh 0, however their block is met; beside them a row that begins with
    eight zeros of negative sign counts as any other."""
    rng = np.random.default_rng(D)
    at, dim = 70, D - 2
    seq, pos, window, first = KINDS[kind]
    pages, table, kv = PR.pool([600, 40], 32, D, rng)
    for r, rows in enumerate(kv):
        rows[:, dim] = 0
        if r == 0:
            rows[at + 1, :8] = -0.0
            rows[at, dim] = 2.0 ** 100
        for j in range(len(rows)):
            pages[int(table[r, j // 32]), j % 32] = rows[j].to(bf16)
    q = torch.from_numpy(rng.standard_normal((len(seq), H, D))).to(bf16)
    q[:, :, dim] = -(2.0 ** 100)
    lse = torch.empty(len(seq), H, device="cuda")
    out = dsa.paged_attn(q.cuda(), pages, table, i32(seq), i32(pos), window=window, first=first, lse=lse)
    PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, first, None, 1 / math.sqrt(D), {(0, at)}), D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_scale_of_zero(D):
    """All rows weigh the same, however large their products are (2^126 and less here), in whole and in masked blocks."""
    rng = np.random.default_rng(D)
    n, H = 300, 4
    pages, table, kv = PR.pool([n], 32, D, rng)
    kv[0][:, 3] = torch.from_numpy(2.0 ** rng.integers(0, 64, n))
    for j in range(n):
        pages[int(table[0, j // 32]), j % 32] = kv[0][j].to(bf16)
    q = torch.from_numpy(rng.standard_normal((3, H, D))).to(bf16)
    q[:, :, 3] = 2.0 ** 63
    seq, pos = [0, 0, 0], [299, 100, 0]
    sink = torch.zeros(H, device="cuda")
    for window in (None, 40):
        lse = torch.empty(3, H, device="cuda")
        out = dsa.paged_attn(q.cuda(), pages, table, i32(seq), i32(pos), window=window, attn_sink=sink, scale=0.0, lse=lse)
        PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, 0, sink, 0.0), D)
    assert dsa.get_device_error() == 0


def step(D, H, lens, tokens, rows, places, seed=0):
    """q, pages, a table of `rows` rows, seq and pos of a step: tokens (sequence, how many at its end), -1 in further places."""
    rng = np.random.default_rng(seed)
    M = -(-max(lens) // 64)
    pages = torch.randn(M * len(lens), 64, D, device="cuda").to(bf16)
    table = torch.full((rows, M), -1, dtype=torch.int32, device="cuda")
    table[:len(lens)] = i32(rng.permutation(M * len(lens)).reshape(len(lens), M))
    seq = np.concatenate([np.full(n, r) for r, n in tokens] + [np.full(places, -1)])
    pos = np.concatenate([np.arange(lens[r] - n, lens[r]) for r, n in tokens] + [np.full(places, -1)])
    q = torch.randn(len(seq), H, D, device="cuda").to(bf16)
    return q, pages, table, i32(seq), i32(pos)


@pytest.mark.parametrize("D,H", [(64, 100), (128, 65), (128, 20), (256, 150), (512, 40), (512, 100)])
def test_the_table_s_height_is_no_matter(D, H):
    """The same step, of tokens that share sequences and of some that do not, under a table with many more rows: the same bits, and the
    references' values (200 tokens of one sequence took 1.4 to 1.5 times the time there)."""
    for lens, tokens in (([900], [(0, 200)]), ([300, 700, 40, 333], [(0, 9), (1, 1), (2, 30), (3, 1)]), ([50, 260, 100], [(1, 1), (0, 1), (2, 1)])):
        q, pages, table, seq, pos = step(D, H, lens, tokens, len(lens), 0)
        want = dsa.paged_attn(q, pages, table, seq, pos)
        kv = [pages[t].flatten(0, 1)[:n].double().cpu() for t, n in zip(table.long(), lens)]
        PR.check_attn(want, None, PR.attn(q, kv, seq.cpu(), pos.cpu(), None, 0, None, 1 / math.sqrt(D)), D)
        tall = torch.cat([table, torch.full((400, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        assert torch.equal(want, dsa.paged_attn(q, pages, tall, seq, pos))
    assert dsa.get_device_error() == 0


def test_places_and_pairs_are_no_matter():
    """64 sequences of 4096 rows, a token each, take their time where a place has no token and where a sequence has two, too (1.2 times,
    cut as tokens that share a sequence are); 200 tokens of one sequence take theirs under any table (1.5 times, cut as tokens that
    share none)."""
    D, H = 256, 150
    one = [(r, 1) for r in range(64)]

    def time(lens, tokens, rows, places):
        q, pages, table, seq, pos = step(D, H, lens, tokens, rows, places)
        out, work = torch.empty_like(q), torch.empty(dsa.paged_attn_workspace_size(len(q), H, D), dtype=torch.uint8, device="cuda")
        return best(lambda: dsa.paged_attn(q, pages, table, seq, pos, out=out, workspace=work))

    plain = time([4096] * 64, one, 64, 0)
    assert time([4096] * 64, one, 64, 1) < 1.14 * plain
    assert time([4096] * 64, one[:63] + [(63, 2)], 64, 0) < 1.14 * plain
    assert time([8192], [(0, 200)], 256, 0) < 1.14 * time([8192], [(0, 200)], 1, 0)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,H", [(64, 100), (256, 150), (512, 40)])
def test_cuts_in_one_graph(D, H):
    """The cut follows what the tensors hold when a captured call is replayed: tokens of one sequence, of many, and none."""
    lens = [500] * 40
    q, pages, table, _, _ = step(D, H, lens, [(r, 1) for r in range(40)], 40, 0)
    seq, pos = torch.zeros(40, dtype=torch.int32, device="cuda"), torch.zeros(40, dtype=torch.int32, device="cuda")
    work = torch.empty(dsa.paged_attn_workspace_size(40, H, D), dtype=torch.uint8, device="cuda")
    work.fill_(255)
    dsa.paged_attn(q, pages, table, seq, pos, workspace=work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dsa.paged_attn(q, pages, table, seq, pos, workspace=work)
    kv = [pages[t].flatten(0, 1)[:500].double().cpu() for t in table.long()]
    for s, p in ((np.zeros(40), np.arange(460, 500)), (np.arange(40), np.arange(420, 500, 2)), (np.full(40, -1), np.zeros(40)),
                 (np.repeat(np.arange(8), 5), np.tile(np.arange(495, 500), 8))):
        seq.copy_(i32(s)), pos.copy_(i32(p))
        work.fill_(255)
        g.replay()
        PR.check_attn(out, None, PR.attn(q, kv, s, p, None, 0, None, 1 / math.sqrt(D)), D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,H,rows", [(64, 16, 16), (64, 5, 128), (128, 70, 256), (256, 16, 16), (256, 3, 64), (512, 16, 16), (512, 70, 32), (512, 8, 64),
                                      (512, 8, 256)])
def test_pages_that_are_missing(D, H, rows):
    """Unmapped pages (negative ids, ids past the pool) at a sequence's start, in its middle and at its end, one beside another, are
    skipped; positions behind the table see the rows of its pages."""
    rng = np.random.default_rng(D + rows)
    lens = [5 * rows + 3, 3 * rows, 2 * rows]
    pages, table, kv = PR.pool(lens, rows, D, rng)
    t = table.cpu().numpy().copy()
    gone = [(0, 1), (0, 2), (0, 5), (1, 0), (2, 0), (2, 1)]
    for k, (r, j) in enumerate(gone):
        t[r, j] = (-1, -(2 ** 31), pages.shape[0], 2 ** 31 - 1)[k % 4]
    skip = {(r, i) for r, j in gone for i in range(j * rows, (j + 1) * rows)}
    seq = np.array([0, 0, 0, 1, 1, 1, 2, 3, -7])
    pos = np.array([5 * rows + 2, 5 * rows - 1, 2 * rows, 3 * rows - 1, rows, rows - 1, 2 * rows - 1, 5, 5])
    q = torch.from_numpy(rng.standard_normal((9, H, D))).to(bf16).cuda()
    for window, first in ((None, 0), (rows + 5, rows // 2), (7, 0)):
        for sink in (None, torch.zeros(H, device="cuda")):
            lse = torch.empty(9, H, device="cuda")
            out = dsa.paged_attn(q, pages, i32(t), i32(seq), i32(pos), window=window, first=first, attn_sink=sink, lse=lse)
            PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, first, sink, 1 / math.sqrt(D), skip), D)
    # behind a table of three pages a sequence: all rows of those of 0 and 1, of which 0 has more
    far = np.array([5 * rows + 2, 5 * rows - 1, 2 * rows, 2 ** 31 - 1, 2 ** 31 - 2, 10 ** 6, 2 * rows - 1, 5, 5])
    cut = table[:, :3].contiguous()
    kv = [x[:3 * rows] for x in kv]
    for window, first in ((None, 0), (100, 5)):
        lse = torch.empty(9, H, device="cuda")
        out = dsa.paged_attn(q, pages, cut, i32(seq), i32(far), window=window, first=first, lse=lse)
        PR.check_attn(out, lse, PR.attn(q, kv, seq, far, window, first, None, 1 / math.sqrt(D)), D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,H", [(64, 128), (128, 128), (256, 128)])
def test_infinite_values_found_by_many_warps(D, H):
    """All warps of a block find the same rows, each in its own time and perhaps while another takes them out: no run differs."""
    rng = np.random.default_rng(D)
    n = 2000
    pages, table, kv = PR.pool([n], 64, D, rng)
    for at in (5, 77, 80, 1990, 1500, 640):
        pages[int(table[0, at // 64]), at % 64, int(rng.integers(D))] = (math.inf, -math.inf, math.nan)[at % 3]
    pos = np.array([4, 1999, 100, 1995, 3, 60, 2, 1])
    q = torch.from_numpy(rng.standard_normal((8, H, D))).to(bf16).cuda()
    for window in (None, 90):
        hit = torch.tensor([any(at <= p and (window is None or at > p - window) for at in (5, 77, 80, 1990, 1500, 640)) for p in pos])
        assert hit.any() and not hit.all()
        for _ in range(100):
            lse = torch.empty(8, H, device="cuda")
            out = dsa.paged_attn(q, pages, table, i32(np.zeros(8)), i32(pos), window=window, lse=lse)
            assert torch.equal(torch.isnan(out).all(2).all(1).cpu(), hit) and torch.equal(torch.isnan(lse).all(1).cpu(), hit)
            assert not torch.isnan(out[~hit.cuda()]).any() and not torch.isnan(lse[~hit.cuda()]).any()
        ref = PR.attn(q, kv, np.zeros(8), pos, window, 0, None, 1 / math.sqrt(D))
        PR.check_attn(out.cpu()[~hit], lse.cpu()[~hit], [x[~hit] for x in ref], D)
    assert dsa.get_device_error() == 0
