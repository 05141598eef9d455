"""Attention over the bf16 paged cache against the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_ref as PR
import sparse_attention_indexer_e4m3_gb300 as dsa

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def case(D, H, rows, lens, tokens, seed, window=None, first=0, sink=True, scale=None, tail=0, shuffle=False):
    """tokens: (sequence, how many at its end); -1: tokens without a sequence."""
    rng = np.random.default_rng(seed)
    pages, table, kv = PR.pool(lens, rows, D, rng)
    seq, pos = [], []
    for r, n in tokens:
        seq += [r] * n
        pos += list(range(lens[r] - n, lens[r])) if r >= 0 else [-1] * n
    seq, pos = np.array(seq + [-1] * tail), np.array(pos + [-1] * tail)
    if shuffle:
        at = rng.permutation(len(seq))
        seq, pos = seq[at], pos[at]
    q = torch.from_numpy(rng.standard_normal((len(seq), H, D))).to(torch.bfloat16).cuda()
    s = torch.from_numpy(rng.standard_normal(H).astype(np.float32)).cuda() if sink else None
    lse = torch.full((len(seq), H), 7.0, device="cuda")
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=window, first=first, attn_sink=s, scale=scale, lse=lse)
    assert dsa.get_device_error() == 0
    PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, first, s, scale), D)
    again = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=window, first=first, attn_sink=s, scale=scale)
    assert torch.equal(out, again)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 64])
def test_one_token(D, H):
    """Lengths around a block and a page, one and many blocks; fewer and more CTAs than blocks."""
    for i, n in enumerate((1, 2, 127, 128, 129, 1000)):
        case(D, H, 64, [n], [(0, 1)], 10 + i, sink=i % 2 == 0)


@pytest.mark.parametrize("D,H,rows", [(64, 20, 16), (128, 128, 32), (256, 64, 128), (512, 64, 64), (512, 100, 256), (256, 150, 16), (128, 3, 256)])
def test_batch(D, H, rows):
    """Sequences of very different lengths, one token each, and tokens without a sequence."""
    case(D, H, rows, [1, 700, 33, 128, 5, 1290, 64], [(0, 1), (1, 1), (2, 1), (3, 1), (4, 1), (5, 1), (6, 1)], D + H, tail=3)


@pytest.mark.parametrize("D,H,rows", [(64, 16, 32), (128, 40, 64), (256, 64, 16), (512, 64, 128), (512, 7, 64), (256, 129, 64)])
@pytest.mark.parametrize("window,first", [(None, 0), (1, 0), (60, 0), (60, 4), (130, 200), (500, 1)])
def test_chunks(D, H, rows, window, first):
    """Several tokens of a sequence, windows, first rows that stay visible; units that hold tokens of two sequences."""
    case(D, H, rows, [300, 17, 420], [(0, 9), (1, 5), (2, 12)], D + H + first, window=window, first=first, tail=1)


@pytest.mark.parametrize("D,H", [(64, 2), (128, 33), (256, 10), (512, 16)])
def test_order_and_repeats(D, H):
    """Tokens in any order, a sequence again and again: runs of one token, of several sequences in one unit."""
    case(D, H, 32, [100, 260, 31, 150], [(0, 6), (1, 8), (2, 3), (3, 9), (1, 4)], D, window=70, first=2, shuffle=True, tail=2)


@pytest.mark.parametrize("D,H,rows", [(64, 4, 64), (128, 64, 64), (256, 32, 32), (512, 64, 64)])
def test_prompt(D, H, rows):
    """A prompt from its first row on: more units than CTAs, pieces cut inside units."""
    case(D, H, rows, [400], [(0, 400)], D, sink=False)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_bounds_move(D):
    """Scores that grow along the sequence raise the bound in many blocks; small and large scales, 0 and negative ones."""
    for k, scale in enumerate((0.0, -0.3, 1.0, 3.0)):
        rng = np.random.default_rng(k)
        n, H = 700, 9
        pages, table, kv = PR.pool([n], 64, D, rng)
        q = torch.from_numpy(rng.standard_normal((1, H, D))).to(torch.bfloat16)
        grow = (torch.arange(n, dtype=torch.float64)[:, None] / n * q[0, 0].double()[None, :] * 0.5).to(torch.bfloat16)
        page = table[0, torch.arange(n, device="cuda") // 64].long()
        pages[page, torch.arange(n, device="cuda") % 64] = grow.cuda()
        kv = [grow.double()]
        for sink in (None, torch.full((H,), 300.0).cuda(), torch.full((H,), -300.0).cuda(), torch.full((H,), -math.inf).cuda()):
            lse = torch.empty(1, H, device="cuda")
            out = dsa.paged_attn(q.cuda(), pages, table, i32([0]), i32([n - 1]), attn_sink=sink, scale=scale, lse=lse)
            PR.check_attn(out, lse, PR.attn(q, kv, [0], [n - 1], None, 0, sink, scale), D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,H", [(64, 16), (128, 64), (256, 20), (512, 8)])
def test_values_that_are_no_numbers(D, H):
    """A row that holds one makes the outputs of the tokens that see it no numbers, and no others: not those of other
    tokens of its unit, whose weight of that row is 0."""
    for bad, at in ((math.nan, 290), (math.inf, 293), (-math.inf, 0), (math.nan, 3)):
        rng = np.random.default_rng(5)
        lens, rows, window, first = [300, 40], 32, 200, 2
        pages, table, kv = PR.pool(lens, rows, D, rng)
        pages[int(table[0, at // rows]), at % rows, D // 3] = bad
        seq, pos = np.array([0] * 12 + [1] * 4), np.array(list(range(288, 300)) + list(range(36, 40)))
        q = torch.from_numpy(rng.standard_normal((16, H, D))).to(torch.bfloat16).cuda()
        lse = torch.empty(16, H, device="cuda")
        out = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=window, first=first, lse=lse)
        sees = (seq == 0) & (pos >= at) & ((at > pos - window) | (at < first))
        ref = PR.attn(q, kv, seq, pos, window, first, None, 1 / math.sqrt(D))
        ok = torch.from_numpy(~sees)
        assert sees.any() == (at != 3) and not sees.all()
        PR.check_attn(out.cpu()[ok], lse.cpu()[ok], [x[ok] for x in ref], D)
        assert not torch.isfinite(out.float()).cpu()[~ok].all(-1).any()
    assert dsa.get_device_error() == 0


def test_pages_that_are_missing():
    """Unmapped pages (negative ids, ids past the pool) are skipped; a table shorter than the sequence."""
    D, H, rows = 128, 16, 16
    rng = np.random.default_rng(2)
    pages, table, kv = PR.pool([500, 300], rows, D, rng)
    t = table.cpu().numpy().copy()
    gone = [(0, 3), (0, 4), (0, 30), (1, 0)]
    for k, (r, j) in enumerate(gone):
        t[r, j] = (-1, -(2 ** 31), pages.shape[0], 2 ** 31 - 1)[k]
    skip = {(r, i) for r, j in gone for i in range(j * rows, (j + 1) * rows)}
    seq, pos = np.array([0, 0, 1, 1, 2, -7]), np.array([499, 70, 299, 12, 5, 5])
    q = torch.from_numpy(rng.standard_normal((6, H, D))).to(torch.bfloat16).cuda()
    for window, first in ((None, 0), (50, 70)):
        lse = torch.empty(6, H, device="cuda")
        out = dsa.paged_attn(q, pages, i32(t), i32(seq), i32(pos), window=window, first=first, lse=lse)
        PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, first, None, 1 / math.sqrt(D), skip), D)
    # positions behind the table: the rows of its pages, the last of which nobody wrote
    far = np.array([2 ** 31 - 1, 2 ** 31 - 2, 10 ** 6, 600, 3, 3])
    longer = [torch.cat([x, torch.full((-len(x) % rows, D), math.nan, dtype=torch.float64)]) for x in kv]
    for window, first in ((None, 0), (100, 5)):
        lse = torch.empty(6, H, device="cuda")
        out = dsa.paged_attn(q, pages, table, i32(seq), i32(far), window=window, first=first, lse=lse)
        ref = PR.attn(q, longer, seq, far, window, first, None, 1 / math.sqrt(D))
        ok = ~torch.isnan(ref[1]).any(1)
        assert ok.tolist() == [window is not None] * 4 + [True] * 2
        PR.check_attn(out.cpu()[ok], lse.cpu()[ok], [x[ok] for x in ref], D)
        assert torch.isnan(out.cpu()[~ok]).all() and torch.isnan(lse.cpu()[~ok]).all()
    # no pages, no table, no tokens
    for p, tb in ((pages[:0], table), (pages, table[:, :0]), (pages, table[:0])):
        out = dsa.paged_attn(q, p.contiguous(), tb.contiguous(), i32(seq), i32(pos), lse=lse)
        assert not out.any() and (lse == -math.inf).all()
    assert dsa.paged_attn(q[:0], pages, table, i32([]), i32([])).shape == (0, H, D)
    assert dsa.get_device_error() == 0


def test_large_batch():
    """64 sequences of up to 5000 rows, checked on every eighth; a few heads; every CTA shares units."""
    D, H = 512, 64
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 5000, 64)
    pages, table, kv = PR.pool(list(lens), 64, D, rng)
    q = torch.from_numpy(rng.standard_normal((64, H, D))).to(torch.bfloat16).cuda()
    lse = torch.empty(64, H, device="cuda")
    out = dsa.paged_attn(q, pages, table, i32(np.arange(64)), i32(lens - 1), lse=lse)
    assert dsa.get_device_error() == 0
    pick = np.arange(0, 64, 8)
    PR.check_attn(out[pick], lse[pick], PR.attn(q[pick], kv, pick, lens[pick] - 1, None, 0, None, 1 / math.sqrt(D)), D)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("H", [8, 40, 70, 100])
def test_warps_apart(D, H):
    """Warps whose rows of q are few, or whose bound is raised again and again, beside others: none's weights are taken before they
    are formed, in any of many runs."""
    rng = np.random.default_rng(D + H)
    n, R = 6000, 40
    pages, table, kv = PR.pool([n], 64, D, rng)
    seq, pos = np.zeros(R, int), rng.integers(n // 2, n, R)
    q = torch.from_numpy(rng.standard_normal((R, H, D))).to(torch.bfloat16)
    q[:, H // 3:H // 2] *= 6  # scores that spread: their bounds are raised in many blocks
    q = q.cuda()
    lse = torch.empty(R, H, device="cuda")
    table = table.expand(R, -1).contiguous()
    for window in (None, 900):
        s = np.arange(R)
        out = dsa.paged_attn(q, pages, table, i32(s), i32(pos), window=window, lse=lse)
        PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, window, 0, None, 1 / math.sqrt(D)), D)
        for _ in range(300):
            again = dsa.paged_attn(q, pages, table, i32(s), i32(pos), window=window)
            assert torch.equal(out, again)
    assert dsa.get_device_error() == 0
