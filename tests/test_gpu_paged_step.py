"""The calls of the bf16 paged cache and the drafts' check as a serving program runs them: one after the other, captured and
replayed, on other streams, at once, with arguments of the least alignment and with offsets past 32 bits."""
import math

import numpy as np
import pytest
import torch

import paged_ref as PR
import sparse_attention_indexer_e4m3_gb300 as dsa
from test_gpu_streams import check as check_stream

pytestmark = pytest.mark.gpu

bf16 = torch.bfloat16


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------------------------ a server's steps

R, H, D, B, G, V, M = 4, 16, 128, 16, 3, 500, 24
T = R * (G + 1) + 2  # places of a step (two more than it has tokens)
P = 80


class Server:
    """Sequences that grow by drafted tokens.  A step's drafts, rows and numbers are given; all state stays on the device."""

    def __init__(self, seed, prompts):
        rng = np.random.default_rng(seed)
        self.table = torch.full((R, M), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.pages = torch.full((P, B, D), float("nan"), dtype=bf16, device="cuda")
        self.held = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.sink = torch.from_numpy(rng.standard_normal(H).astype(np.float32)).cuda()
        self.work = torch.empty(dsa.paged_attn_workspace_size(4096, H, D), dtype=torch.uint8, device="cuda")
        self.add(rng, prompts)

    def add(self, rng, prompts):
        """The prompts' rows, in one call each."""
        n = int(sum(prompts))
        self.kv = [torch.from_numpy(rng.standard_normal((int(k), D))).to(bf16) for k in prompts]
        added = i32(prompts)
        lacking = self.reserve(self.held, self.held + added)
        seq, pos, _, _ = dsa.step_maps(self.held, added, n)
        dsa.store_kv(torch.cat(self.kv).cuda(), self.pages, self.table, seq, pos, lacking=lacking)
        self.held += added
        assert lacking.item() == 0

    def reserve(self, begin, end):
        src, dst, lacking = dsa.reserve_pages(self.table, self.ref, begin, end, B)
        dsa.copy_pages(self.pages, src, dst)
        return lacking

    def step(self, x):
        """x: the step's count, q, kv, tokens, target, draft, u.  Returns what it computed."""
        added = torch.where(x["count"] >= 0, x["count"] + 1, 0).to(torch.int32)
        lacking = self.reserve(self.held, self.held + added)
        seq, pos, ks, ke = dsa.step_maps(self.held, added, T)
        dsa.store_kv(x["kv"], self.pages, self.table, seq, pos, lacking=lacking)
        lse = torch.empty(T, H, device="cuda")
        out = dsa.paged_attn(x["q"], self.pages, self.table, seq, pos, attn_sink=self.sink, lse=lse, workspace=self.work)
        near = dsa.paged_attn(x["q"], self.pages, self.table, seq, pos, window=9, first=3, attn_sink=self.sink, workspace=self.work)
        # all keys of each token, as a list over keys packed sequence by sequence
        j = torch.arange(M * B, dtype=torch.int32, device="cuda")[None, :] + ks[:, None]
        idx = torch.where(j < ke[:, None], j, -1).to(torch.int32)
        slots = dsa.page_slots(self.pages, self.table, seq, idx, start=ks)
        listed = dsa.sparse_attn(x["q"], self.pages.flatten(0, 1), slots, attn_sink=self.sink)
        accepted, token = dsa.verify_drafts(x["target"], x["draft"], x["tokens"], x["count"], x["u"])
        self.held += torch.where(x["count"] >= 0, accepted + 1, 0).to(torch.int32)
        return dict(seq=seq, pos=pos, ks=ks, ke=ke, out=out, lse=lse, near=near, listed=listed, accepted=accepted, token=token,
                    lacking=lacking, held=self.held)


def draw(rng):
    """A step's inputs (numpy)."""
    def probs(shape):
        e = np.exp(2 * rng.standard_normal(shape))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    target, draft = probs((R, G + 1, V)), probs((R, G, V))
    same = rng.random((R, G)) < 0.7
    draft[same] = target[:, :G][same]
    return dict(count=rng.integers(-1, G + 1, R).astype(np.int32), q=rng.standard_normal((T, H, D)), kv=rng.standard_normal((T, D)),
                tokens=rng.integers(0, V, (R, G)).astype(np.int32), target=target, draft=draft, u=rng.random((R, G + 1)).astype(np.float32))


def put(x):
    return {k: torch.from_numpy(v).to(bf16 if v.dtype == np.float64 else torch.from_numpy(v).dtype).cuda() for k, v in x.items()}


def test_steps_together():
    """Five steps of drafted tokens behind prompts, against the references; a drafted token that was refused is overwritten."""
    rng = np.random.default_rng(3)
    prompts = [40, 1, 129, 77]
    s = Server(1, prompts)
    kv, held = [x.double() for x in s.kv], list(prompts)
    for _ in range(5):
        x = draw(rng)
        at = put(x)
        got = {k: v.cpu() for k, v in s.step(at).items()}
        added = np.where(x["count"] >= 0, x["count"] + 1, 0)
        for name, want in zip(("seq", "pos", "ks", "ke"), PR.maps(held, added, T)):
            assert np.array_equal(got[name].numpy(), want)
        rows, n = at["kv"].double().cpu(), 0
        for r in range(R):
            kv[r] = torch.cat([kv[r][:held[r]], rows[n:n + added[r]]])
            n += added[r]
        seq, pos = got["seq"].numpy(), got["pos"].numpy()
        ref = PR.attn(at["q"], kv, seq, pos, None, 0, s.sink, 1 / math.sqrt(D))
        PR.check_attn(got["out"], got["lse"], ref, D)
        PR.check_attn(got["listed"], None, ref, D)
        PR.check_attn(got["near"], None, PR.attn(at["q"], kv, seq, pos, 9, 3, s.sink, 1 / math.sqrt(D)), D)
        accepted, token = PR.verify(x["target"], x["draft"], x["tokens"], x["count"], x["u"])
        assert np.array_equal(got["accepted"].numpy(), accepted) and np.array_equal(got["token"].numpy(), token)
        held = [h + (int(a) + 1 if c >= 0 else 0) for h, a, c in zip(held, accepted, x["count"])]
        assert got["held"].tolist() == held and got["lacking"].item() == 0
    assert dsa.get_device_error() == 0


def test_steps_captured():
    """The whole step as a graph, replayed with new inputs and the state it left, gives what the calls give one by one; beside a
    second graph that uses the same workspace in between."""
    rng = np.random.default_rng(4)
    prompts = [3, 100, 16, 60]
    xs = [put(draw(rng)) for _ in range(4)]
    eager = Server(2, prompts)
    want = [{k: v.clone() for k, v in eager.step(x).items()} for x in xs]
    s = Server(2, prompts)
    keep = {k: getattr(s, k).clone() for k in ("table", "ref", "pages", "held")}
    x = {k: v.clone() for k, v in xs[0].items()}
    s.step(x)  # (once before the capture)
    other_seq, other_pos = i32([1, 2, 3]), i32([90, 10, 50])
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step(x)
    with torch.cuda.graph(other):
        alone = dsa.paged_attn(x["q"][:3], s.pages, s.table, other_seq, other_pos, workspace=s.work)
    for k, v in keep.items():
        getattr(s, k).copy_(v)
    for y, w in zip(xs, want):
        for k, v in y.items():
            x[k].copy_(v)
        graph.replay()
        other.replay()
        for k, v in w.items():
            assert torch.equal(got[k], v), k
        assert torch.equal(alone, dsa.paged_attn(x["q"][:3], s.pages, s.table, other_seq, other_pos))
    assert dsa.get_device_error() == 0


# ------------------------------------------------------------------------------------ streams


@pytest.fixture(scope="module")
def world():
    rng = np.random.default_rng(7)
    lens = [900, 65, 400]
    pages, table, kv = PR.pool(lens, 32, 256, rng)
    seq, pos = np.array([0, 1, 2, 0]), np.array([899, 64, 399, 5])
    return dict(pages=pages, table=table, seq=i32(seq), pos=i32(pos), idx=i32(rng.integers(-1, 1000, (4, 600))),
                q=torch.from_numpy(rng.standard_normal((4, 20, 256))).to(bf16).cuda(), held=i32(lens), added=i32([2, 1, 1]),
                x=put(draw(rng)))


def calls(w):
    """Every call that allocates: itself, and the shape and type of what it allocates to return."""
    x = w["x"]
    return {
        "step_maps": (lambda s: dsa.step_maps(w["held"], w["added"], 300, stream=s)[0], (1200,), "int32"),
        "page_slots": (lambda s: dsa.page_slots(w["pages"], w["table"], w["seq"], w["idx"], stream=s), (4, 600), "int32"),
        "paged_attn": (lambda s: dsa.paged_attn(w["q"], w["pages"], w["table"], w["seq"], w["pos"], stream=s), (4, 20, 256), "bfloat16"),
        "verify_drafts": (lambda s: dsa.verify_drafts(x["target"], x["draft"], x["tokens"], x["count"], x["u"], stream=s)[1], (R,), "int32"),
    }


@pytest.mark.parametrize("name", ["step_maps", "page_slots", "paged_attn", "verify_drafts"])
def test_allocations(world, name):
    check_stream(*calls(world)[name])


def test_captured_call_on_a_side_stream(world):
    for f, _, _ in calls(world).values():
        want = f(None).clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            out = f(side)
            torch.cuda.current_stream().wait_stream(side)
        out.zero_()
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_two_at_once(D):
    """Calls of different sizes on two streams, each with a workspace of its own, beside the other calls."""
    rng = np.random.default_rng(D)
    lens = [3000, 200, 1500]
    pages, table, _ = PR.pool(lens, 64, D, rng)
    pick = ([0], [2999]), ([0, 1, 2] + [2] * 40, [2999, 199, 700] + list(range(1460, 1500)))
    work = []
    for seq, pos in pick:
        q = torch.from_numpy(rng.standard_normal((len(seq), 24, D))).to(bf16).cuda()
        work.append((q, i32(seq), i32(pos), torch.empty(dsa.paged_attn_workspace_size(len(seq), 24, D), dtype=torch.uint8, device="cuda"),
                     torch.empty_like(q), torch.cuda.Stream()))
    want = [dsa.paged_attn(q, pages, table, seq, pos) for q, seq, pos, _, _, _ in work]
    x = put(draw(rng))
    drafts = dsa.verify_drafts(x["target"], x["draft"], x["tokens"], x["count"], x["u"])
    torch.cuda.synchronize()
    for _ in range(20):
        found = []
        for q, seq, pos, ws, out, s in work:
            out.zero_()
            s.wait_stream(torch.cuda.current_stream())
            dsa.paged_attn(q, pages, table, seq, pos, out=out, workspace=ws, stream=s)
            with torch.cuda.stream(s):
                found.append(dsa.verify_drafts(x["target"], x["draft"], x["tokens"], x["count"], x["u"]))
        torch.cuda.synchronize()
        for w, (_, _, _, _, out, _) in zip(want, work):
            assert torch.equal(out, w)
        assert all(torch.equal(a, b) for f in found for a, b in zip(f, drafts))
    assert dsa.get_device_error() == 0


# ------------------------------------------------------------------------------------ alignment, refusals, values


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_least_alignment(D):
    """Everything 16 bytes (int32 and fp32: 4) behind an aligned place."""
    rng = np.random.default_rng(D)
    lens = [333, 40]
    pages, table, kv = PR.pool(lens, 32, D, rng)
    shift = lambda x, k: torch.empty(x.numel() + k, dtype=x.dtype, device="cuda")[k:].view(x.shape).copy_(x)  # noqa: E731
    q = torch.from_numpy(rng.standard_normal((6, 5, D))).to(bf16).cuda()
    seq, pos = np.array([0, 0, 1, 1, 1, 0]), np.array([332, 60, 39, 0, 5, 100])
    out, lse = shift(torch.zeros_like(q), 8), shift(torch.zeros(6, 5, device="cuda"), 1)
    ws = torch.empty(dsa.paged_attn_workspace_size(6, 5, D) + 16, dtype=torch.uint8, device="cuda")[16:]
    sink = shift(torch.randn(5, device="cuda"), 1)
    p, t, s, o = shift(pages, 8), shift(table, 1), shift(i32(seq), 1), shift(i32(pos), 1)
    assert dsa.paged_attn(shift(q, 8), p, t, s, o, attn_sink=sink, out=out, lse=lse, workspace=ws) is out
    PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, None, 0, sink, 1 / math.sqrt(D)), D)
    # a row for itself, so that one CTA writes it whole
    dsa.paged_attn(shift(q, 8)[3:4], p, t, s[3:4], o[3:4], attn_sink=sink, out=out[3:4], workspace=ws)
    PR.check_attn(out, lse, PR.attn(q, kv, seq, pos, None, 0, sink, 1 / math.sqrt(D)), D)
    rows = shift(torch.randn(6, D + 8, device="cuda").to(bf16), 8)[:, :D]
    at = i32([300, 301, 7, 8, 9, 302])
    dsa.store_kv(rows, p, t, s, shift(at, 1))
    for i in range(6):
        page = int(table[seq[i], int(at[i]) // 32])
        assert torch.equal(p[page, int(at[i]) % 32], rows[i])
    assert dsa.get_device_error() == 0


def test_workspace_is_checked(world):
    w = world
    need = dsa.paged_attn_workspace_size(4, 20, 256)
    full = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    run = lambda ws: dsa.paged_attn(w["q"], w["pages"], w["table"], w["seq"], w["pos"], workspace=ws)  # noqa: E731
    for ws in (full[:need - 1], full[8:8 + need], full[:0]):
        with pytest.raises(dsa.DsaError, match="WORKSPACE"):
            run(ws)
    full.fill_(255)
    assert torch.equal(run(full[16:]), run(None))


@pytest.mark.parametrize("D,H", [(64, 16), (128, 64), (256, 20), (512, 8), (512, 130)])
def test_queries_that_are_no_numbers(D, H):
    """A token whose q or sink holds one has no numbers; its unit's other tokens and heads do."""
    rng = np.random.default_rng(D + H)
    lens = [290, 40]
    pages, table, kv = PR.pool(lens, 32, D, rng)
    seq, pos = np.array([0] * 6 + [1] * 3), np.array(list(range(284, 290)) + [37, 38, 39])
    sink = torch.zeros(H, device="cuda")
    for bad in (math.nan, math.inf):
        q = torch.from_numpy(rng.standard_normal((9, H, D))).to(bf16).cuda()
        clean = q.clone()
        q[2, 1, 5] = q[7, H - 1, D - 1] = bad
        lse = torch.empty(9, H, device="cuda")
        for window in (None, 100):
            out = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=window, attn_sink=sink, lse=lse)
            ref = PR.attn(clean, kv, seq, pos, window, 0, sink, 1 / math.sqrt(D))
            hit = torch.zeros(9, H, dtype=torch.bool)
            hit[2, 1] = hit[7, H - 1] = True
            PR.check_attn(out.cpu()[~hit], lse.cpu()[~hit], [x[~hit] for x in ref], D)
            assert torch.isnan(out.cpu()[hit]).all() and torch.isnan(lse.cpu()[hit]).all()
    q = torch.from_numpy(rng.standard_normal((9, H, D))).to(bf16).cuda()
    sink[2], sink[3] = math.inf, math.nan
    lse = torch.empty(9, H, device="cuda")
    out = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), attn_sink=sink, lse=lse)
    keep = [h for h in range(H) if h not in (2, 3)]
    ref = PR.attn(q[:, keep], kv, seq, pos, None, 0, sink[keep], 1 / math.sqrt(D))
    PR.check_attn(out[:, keep], lse[:, keep], ref, D)
    assert not out[:, 2].any() and (lse[:, 2] == math.inf).all() and torch.isnan(out[:, 3]).all() and torch.isnan(lse[:, 3]).all()
    assert dsa.get_device_error() == 0


# ------------------------------------------------------------------------------------ sizes


def test_pool_past_32_bits():
    """Pages whose rows lie more than 2^32 bytes and 2^31 values behind the first."""
    D, B, P = 512, 256, 18000  # 4.7 GB
    pages = torch.zeros(P, B, D, dtype=bf16, device="cuda")
    rng = np.random.default_rng(0)
    n = 600
    table = i32([[P - 1, 17000, P - 3], [3, 16385, 0]])  # (row 16385 * 256 * 512 is the first past 2^31 values)
    kv = [torch.from_numpy(rng.standard_normal((n, D))).to(bf16) for _ in range(2)]
    seq, pos = np.repeat([0, 1], n), np.tile(np.arange(n), 2)
    dsa.store_kv(torch.cat(kv).cuda(), pages, table, i32(seq), i32(pos))
    slots = dsa.page_slots(pages, table, i32([0, 1]), i32([[0, 299, 599]] * 2))
    assert slots.tolist() == [[(P - 1) * B, 17000 * B + 43, (P - 3) * B + 87], [3 * B, 16385 * B + 43, 87]]
    for r in range(2):
        assert torch.equal(pages.view(-1, D)[slots[r].long()].cpu(), kv[r][[0, 299, 599]])
    q = torch.from_numpy(rng.standard_normal((2, 7, D))).to(bf16).cuda()
    out = dsa.paged_attn(q, pages, table, i32([0, 1]), i32([n - 1, n - 1]))
    PR.check_attn(out, None, PR.attn(q, [x.double() for x in kv], [0, 1], [n - 1] * 2, None, 0, None, 1 / math.sqrt(D)), D)
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,T,H", [(512, 33000, 128), (64, 70000, 64)])
def test_many_tokens(D, T, H):
    """More units than a CTA keeps the blocks of, and (at 512) outputs past 2^31 values: a window of a few rows over sequences of one page."""
    rng = np.random.default_rng(1)
    lens = [16] * 8
    pages, table, kv = PR.pool(lens, 16, D, rng)
    part = torch.from_numpy(rng.standard_normal((1000, H, D))).to(bf16).cuda()
    q = part.repeat(T // 1000, 1, 1)
    seq, pos = np.arange(T) // 5000 % 9 - 1, np.arange(T) % 17 - 1
    out = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=3)
    assert dsa.get_device_error() == 0
    pick = np.unique(np.concatenate([np.arange(0, T, 997), np.arange(T - 40, T)]))
    PR.check_attn(out[pick], None, PR.attn(q[pick], kv, seq[pick], pos[pick], 3, 0, None, 1 / math.sqrt(D)), D)


def test_counts_near_the_largest_int():
    """As many lists and as many sequences as an int counts: the indexes of the last ones do not wrap."""
    n = 2 ** 31 - 1
    pages = torch.empty(64, 16, 1, device="cuda")
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    idx = torch.zeros(n, dtype=torch.int32, device="cuda")
    idx[-3:] = i32([17, -5, 40])
    dsa.page_slots(pages, i32([[3, 60, -1]]), seq, idx, out=idx)
    assert idx[-4:].tolist() == [48, 60 * 16 + 1, -1, -1] and bool((idx[:-3] == 48).all())
    del idx
    seq[-1], seq[5] = 2, 1  # now the added rows of each sequence; those held are as many
    got = [x.tolist() for x in dsa.step_maps(seq, seq, 4)]
    assert got == [[5, n - 1, n - 1, -1], [1, 2, 3, -1], [0, 2, 2, 0], [2, 5, 6, 0]]
    assert dsa.get_device_error() == 0


@pytest.mark.parametrize("D,H", [(64, 7), (128, 33), (256, 150), (512, 20)])
def test_output_over_the_queries(D, H):
    """out = q, with units that many CTAs share and units of several tokens."""
    rng = np.random.default_rng(D)
    pages, table, _ = PR.pool([2000, 300], 64, D, rng)
    for seq, pos in (([0, 1], [1999, 299]), ([0] * 300 + [1] * 20, list(range(1700, 2000)) + list(range(280, 300)))):
        q = torch.from_numpy(rng.standard_normal((len(seq), H, D))).to(bf16).cuda()
        want = dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=700)
        assert dsa.paged_attn(q, pages, table, i32(seq), i32(pos), window=700, out=q) is q and torch.equal(q, want)
    assert dsa.get_device_error() == 0
