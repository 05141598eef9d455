"""Cases and plain forms of a serving step over a paged bf16 cache, and of the drafts it checks.

A cache holds kv rows (each both key and value) as bf16 pages [P, page_rows, D]; row `pos` of sequence r
is row pos % page_rows of page table[r, pos // page_rows].

  rows     a step's tokens from the sequences' lengths: for each token its sequence, its position and its
           window of packed index keys; then the tokens' kv rows written into their pages;
  slots    lists of keys as the indexer packs them, turned into rows of the pages seen as one matrix (what
           sparse attention over them takes);
  attend   attention of each token over the rows of its sequence up to its own: all of them, or a sliding
           window and a few first rows that stay visible;
  verify   drafted tokens accepted or refused by the target's probabilities with given random numbers, and
           the token that follows the accepted ones.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step of a batch, one row per request; the smallest call
        dict(name="rows_step", op="rows", R=61, T=64, new=1, ragged=False, held=2500, D=512, page_rows=64),
        # a long prompt's chunk beside requests of a few tokens
        dict(name="rows_prompt", op="rows", R=33, T=65536, new=4000, ragged=True, held=1500, D=512, page_rows=64),
        # the indexer's lists of a decoding batch
        dict(name="slots_step", op="slots", R=61, T=61, K=2048, ctx=16384, page_rows=64),
        # the indexer's lists of a long prompt
        dict(name="slots_prompt", op="slots", R=4, T=8192, K=2048, ctx=8192, page_rows=32),
        # one request's next token over a long context: latency counts
        dict(name="attend_one", op="attend", R=1, new=1, ragged=False, ctx=32768, H=64, D=512, page_rows=64, window=0,
             first=0, sink=True),
        # the packed decoding batch: 64 requests whose lengths lie far apart
        dict(name="attend_batch", op="attend", R=64, new=1, ragged=False, ctx=65536, H=64, D=512, page_rows=64,
             window=0, first=0, sink=False),
        # a token and its drafts per request, more heads than one group, ragged with rows that hold no token
        dict(name="attend_drafts", op="attend", R=19, new=4, ragged=True, ctx=9001, H=150, D=256, page_rows=32,
             window=0, first=0, sink=True),
        # decoding with a sliding window and first rows that stay visible, small pages, few heads
        dict(name="attend_window", op="attend", R=128, new=1, ragged=False, ctx=16384, H=20, D=128, page_rows=16,
             window=500, first=4, sink=True),
        # prompts with a sliding window
        dict(name="attend_slide", op="attend", R=3, new=2700, ragged=False, ctx=4001, H=32, D=128, page_rows=64,
             window=1024, first=16, sink=False),
        # a chunk of a long prompt at the widest head dimension; the largest call
        dict(name="attend_prompt", op="attend", R=1, new=4096, ragged=False, ctx=8192, H=64, D=512, page_rows=64,
             window=0, first=0, sink=False),
        # one request's drafts
        dict(name="verify_one", op="verify", R=1, G=4, V=131072),
        # a batch's drafts; a vocabulary whose rows start at odd places
        dict(name="verify_batch", op="verify", R=128, G=3, V=50257),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "slots", "attend", "attend", "attend", "verify"])
    B = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128, 256, 512])
    if op == "rows":
        T = _log(rng, 1, 65536)
        R = min(T, _log(rng, 1, 256))
        return dict(op=op, R=R, T=T, new=max(1, T // R), ragged=rng.random() < 0.5, held=_log(rng, 1, 4000), D=D, page_rows=B)
    if op == "slots":
        T = _log(rng, 1, 8192)
        return dict(op=op, R=min(T, _log(rng, 1, 64)), T=T, K=_log(rng, 1, 2048), ctx=_log(rng, 64, 16384), page_rows=B)
    if op == "verify":
        V = _log(rng, 1000, 131072)
        return dict(op=op, R=min(128, _log(rng, 1, 256)), G=rng.randint(1, 7 if V < 60000 else 3), V=V)
    H = _log(rng, 1, 150)
    window = 0 if rng.random() < 0.5 else _log(rng, 16, 4096)
    first = rng.choice([0, 0, 4, 130])
    while True:
        if rng.random() < 0.5:
            R, new, ctx = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 5]), _log(rng, 16, 65536)
        else:
            R, new, ctx = rng.randint(1, 4), _log(rng, 16, 4096), _log(rng, 64, 8192)
        ctx = max(ctx, new)
        case = dict(op=op, R=R, new=new, ragged=rng.random() < 0.5, ctx=ctx, H=H, D=D, page_rows=B, window=window,
                    first=first, sink=rng.random() < 0.5)
        w = work(case)
        if w["flops"] <= 3.0e12 and w["bytes"] <= 2.0e9 and R * ctx * D * 2 <= 4e9:
            return case


def _lengths(case, rng=None):
    """Held rows and new tokens of each sequence (without a generator: as far as the case fixes them)."""
    R, new = case["R"], case["new"]
    if case["op"] == "rows":
        T = case["T"]
        if rng is None:
            return np.full(R, case["held"]), np.full(R, min(new, T // R))
        held = rng.integers(0, case["held"] + 1, R)
        added = rng.integers(0, new + 1, R) if case["ragged"] else np.full(R, new)
        if case["ragged"] and R > 2:  # one long prompt takes what the others leave, up to a few rows that hold no token
            added[R // 2] = max(0, T - 3 - int(added.sum() - added[R // 2]))
        while added.sum() > T:
            added[np.argmax(added)] = max(0, added.max() - (added.sum() - T))
        return held, added
    ctx = case["ctx"]
    if rng is None:
        return np.full(R, (ctx if R < 2 else 3 * ctx // 5) - new).clip(min=0), np.full(R, new if not case["ragged"] else (new + 1) // 2)
    total = rng.integers(max(new, ctx // 16), ctx + 1, R)
    total[0] = ctx
    added = rng.integers(1, new + 1, R) if case["ragged"] else np.full(R, new)
    added[0] = new
    return total - added, added


def _seen(case, pos):
    """Visible rows of a token at each position."""
    pos = np.asarray(pos, np.int64)
    W, F = case["window"], case["first"]
    if W == 0:
        return pos + 1
    return np.where(pos + 1 <= W, pos + 1, W + np.minimum(F, np.maximum(0, pos + 1 - W)))


def work(case):
    op = case["op"]
    if op == "rows":  # two lengths a sequence and the table in, four numbers a token out, rows in and out
        held, added = _lengths(case)
        n, M = int(added.sum()), _table_width(case)
        return {"bytes": 8 * case["R"] + 16 * case["T"] + min(4 * case["R"] * M, 4 * n) + 4 * n * case["D"], "flops": 0}
    if op == "slots":
        T, K = case["T"], case["K"]
        return {"bytes": 8 * T * K + 8 * T + 4 * case["R"] * -(-case["ctx"] // case["page_rows"]), "flops": 0}
    if op == "verify":  # the row of the target and of the draft that decide, and the drafted tokens' entries
        R, G, V = case["R"], case["G"], case["V"]
        return {"bytes": 8 * R * V + 20 * R * G, "flops": 4 * R * V}
    held, added = _lengths(case)
    H, D, W, F = case["H"], case["D"], case["window"], case["first"]
    pairs = rows = 0
    for h, a in zip(held, added):
        pairs += int(_seen(case, h + np.arange(a)).sum())
        lo = max(0, h + 1 - W) if W else 0
        rows += h + a - lo + min(F, lo)
    T = int(added.sum())
    return {"bytes": int(2 * rows * D + 4 * T * H * D + 4 * T * H + 8 * T), "flops": int(4 * pairs * H * D)}


# ----------------------------------------------------------------------------------- the inputs

def _table_width(case):
    if case["op"] == "rows":
        return -(-(case["held"] + (case["T"] if case["ragged"] else case["new"])) // case["page_rows"])
    return -(-case["ctx"] // case["page_rows"])


def _table(lens, M, B, rng, P=None):
    """A page table [R, M] for sequences of the given lengths, pages drawn from a shuffled pool (of P, or a few more than it takes)."""
    need = -(-np.asarray(lens) // B)
    P = P or int(need.sum()) + 3
    ids = rng.permutation(P)
    table = np.full((len(lens), M), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, P


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dev = "cuda"
    put = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).to(dev)  # noqa: E731
    st = {"case": case}
    op = case["op"]

    def rows(n, D):  # rows of different size, some larger values among ordinary ones
        x = torch.randn(n, D, generator=gen, device=dev)
        x *= torch.exp2(torch.randint(-2, 3, (n, 1), generator=gen, device=dev).float())
        return x.to(torch.bfloat16)

    if op == "rows":
        D, B, T = case["D"], case["page_rows"], case["T"]
        held, added = _lengths(case, rng)
        table, P = _table(held + added, _table_width(case), B, rng, case["R"] * (case["held"] // B + 2) + T // B)
        st.update(held=put(held), added=put(added), table=put(table), kv=rows(T, D),
                  pages=rows(P * B, D).view(P, B, D))
    elif op == "slots":
        R, T, K, ctx, B = (case[k] for k in ("R", "T", "K", "ctx", "page_rows"))
        lens = rng.integers(max(1, ctx // 2), ctx + 1, R)
        lens[0] = ctx
        table, P = _table(lens, -(-ctx // B), B, rng)
        seq = np.sort(rng.integers(0, R, T))
        start = np.concatenate([[0], np.cumsum(lens)])[seq]
        n = torch.from_numpy(lens[seq]).to(dev)[:, None]
        i = torch.arange(K, device=dev)[None, :]
        m = torch.minimum(n, torch.full_like(n, K))  # entries of each list, ascending, then -1
        idx = torch.where(i < m, i * n // m + put(start)[:, None], -1)
        st.update(pages=torch.zeros(P, B, 64, dtype=torch.bfloat16, device=dev), table=put(table), seq=put(seq),
                  start=put(start), idx=idx.to(torch.int32))
    elif op == "attend":
        R, H, D, B = (case[k] for k in ("R", "H", "D", "page_rows"))
        held, added = _lengths(case, rng)
        lens = held + added
        table, P = _table(lens, -(-case["ctx"] // B), B, rng)
        pages = torch.full((P * B, D), float("nan"), dtype=torch.bfloat16, device=dev)  # rows that nobody wrote
        for r in range(R):
            n = int(lens[r])
            j = np.arange(n)
            pages[put(table[r, j // B].astype(np.int64) * B + j % B, np.int64)] = rows(n, D)
        T = R * case["new"]  # what the step has room for; some of it may hold no token
        seq, pos = np.full(T, -1), np.full(T, -1)
        n = int(added.sum())
        seq[:n] = np.repeat(np.arange(R), added)
        pos[:n] = np.concatenate([held[r] + np.arange(added[r]) for r in range(R)])
        q = torch.randn(T, H, D, generator=gen, device=dev).to(torch.bfloat16)
        sink = torch.randn(H, generator=gen, device=dev) if case["sink"] else None
        st.update(q=q, pages=pages.view(P, B, D), table=put(table), seq=put(seq), pos=put(pos), sink=sink,
                  scale=0.25 / math.sqrt(D), held=held, added=added)
    else:
        R, G, V = case["R"], case["G"], case["V"]
        target = torch.empty(R, G + 1, V, device=dev)
        draft = torch.empty(R, G, V, device=dev)
        tokens = torch.empty(R, G, dtype=torch.int32, device=dev)
        for r0 in range(0, R, 16):
            n = min(16, R - r0)
            x = 3.0 * torch.randn(n, G + 1, V, generator=gen, device=dev)
            target[r0:r0 + n] = torch.softmax(x, 2)
            d = torch.softmax(x[:, :G] + 0.7 * torch.randn(n, G, V, generator=gen, device=dev), 2)
            draft[r0:r0 + n] = d
            c = torch.cumsum(d.double(), 2)
            u = torch.rand(n, G, 1, generator=gen, device=dev, dtype=torch.float64) * c[..., -1:]
            tokens[r0:r0 + n] = torch.searchsorted(c, u, right=True).squeeze(2).clamp(max=V - 1).int()
        count = rng.integers(max(0, G - 2), G + 1, R)
        count[0] = G
        st.update(target=target, draft=draft, tokens=tokens, count=put(count),
                  u=torch.rand(R, G + 1, generator=gen, device=dev))
    return st


# ------------------------------------------------------------------------------- the plain forms

def _maps(held, added, T):
    ends = torch.cumsum(added, 0)
    total = torch.cumsum(held + added, 0)
    t = torch.arange(T, device=held.device)
    seq = torch.searchsorted(ends, t, right=True)
    some = seq < held.numel()
    s = torch.where(some, seq, 0)
    pos = t - (ends - added)[s] + held[s]
    ks = (total - held - added)[s]
    pick = lambda x, other: torch.where(some, x, other).int()  # noqa: E731
    return pick(seq, -1), pick(pos, -1), pick(ks, 0), pick(ks + pos + 1, 0)


def _slots(table, seq, pos, B):
    page = table[seq.clamp(min=0).long()].gather(1, (pos.clamp(min=0) // B).long())
    return torch.where((pos >= 0) & (seq >= 0)[:, None] & (page >= 0), page * B + pos % B, -1).int()


def _store(kv, pages, table, seq, pos, B):
    flat = pages.view(-1, pages.shape[2])
    slot = _slots(table, seq, pos[:, None], B)[:, 0].long()
    src = torch.arange(kv.shape[0], device=kv.device)
    lead = torch.argmax((slot >= 0).int())  # a row that has a place; rows without one repeat it
    src = torch.where(slot >= 0, src, lead)
    flat[slot[src]] = kv[src]


def _soft(s, kv, sink):
    """Softmax of scores s [n, H, K] with the sink in its denominator, times kv [n or 1, K, D]; rows of -inf give zeros."""
    m = s.amax(2)
    if sink is not None:
        m = torch.maximum(m, sink[None, :])
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(s - m[..., None])
    z = w.sum(2) if sink is None else w.sum(2) + torch.exp(sink[None, :] - m)
    o = torch.matmul(w, kv) / torch.where(z > 0, z, 1.0)[..., None]
    return o.to(torch.bfloat16), m + torch.log(z)


def _attend(st):
    q, pages, table, seq, pos, sink = (st[k] for k in ("q", "pages", "table", "seq", "pos", "sink"))
    case, B = st["case"], st["case"]["page_rows"]
    W, F = case["window"], case["first"]
    T, H, D = q.shape
    flat = pages.view(-1, D)
    out = torch.zeros_like(q)
    lse = sink.expand(T, H).clone() if sink is not None else torch.full((T, H), -math.inf, device=q.device)
    lens, ends = st["held"] + st["added"], np.cumsum(st["added"])

    def part(t0, t1, keys, ok):  # tokens [t0, t1) over keys [n or 1, K] of which each sees those in ok
        sq = seq[t0:t1] if keys.shape[0] > 1 else seq[t0:t0 + 1]
        slot = _slots(table, sq, keys, B).long().clamp(min=0)
        kv = flat[slot].float()
        kv = torch.where(ok.any(0)[None, :, None] if keys.shape[0] == 1 else ok[..., None], kv, 0.0)
        if keys.shape[0] == 1:
            s = torch.matmul(q[t0:t1].float().view(1, -1, D), kv.transpose(1, 2)).view(t1 - t0, H, -1) * st["scale"]
        else:
            s = torch.matmul(q[t0:t1].float(), kv.transpose(1, 2)) * st["scale"]
        out[t0:t1], lse[t0:t1] = _soft(torch.where(ok[:, None, :], s, -math.inf), kv, sink)

    if case["new"] == 1:  # one token a sequence, some sequences at a time
        n = int(W + F if W else lens.max())
        step = max(1, (1 << 29) // (n * D))
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            p = pos[t0:t1, None].long()
            if W:
                i = torch.arange(F + W, device=q.device)[None, :]
                keys = torch.where(i < F, i, p - W + 1 + i - F)
                ok = (keys >= 0) & (keys <= p) & ((i >= F) | (keys <= p - W))
            else:
                keys = torch.arange(int(lens[t0:t1].max()), device=q.device)[None, :].expand(t1 - t0, -1)
                ok = keys <= p
            keys = torch.where(ok, keys, 0)
            part(t0, t1, keys, ok)
        return {"out": out, "lse": lse}
    for r in range(len(lens)):
        a, b = int(ends[r] - st["added"][r]), int(ends[r])
        step = max(1, (1 << 28) // (H * int(lens[r])))
        for t0 in range(a, b, step):
            t1 = min(b, t0 + step)
            hi = int(st["held"][r]) + t1 - a
            lo = max(0, int(st["held"][r]) + t0 - a + 1 - W) if W else 0
            keys = torch.cat([torch.arange(min(F, lo), device=q.device), torch.arange(lo, hi, device=q.device)])[None, :]
            p = pos[t0:t1, None]
            ok = keys <= p
            if W:
                ok = ok & ((keys > p - W) | (keys < F))
            part(t0, t1, keys, ok)
    return {"out": out, "lse": lse}


def _verify(target, draft, tokens, count, u):
    R, G, V = draft.shape
    at = tokens.long()[..., None]
    p = target[:, :G].gather(2, at).squeeze(2).double()
    q = draft.gather(2, at).squeeze(2).double()
    i = torch.arange(G, device=u.device)[None, :]
    ok = (u[:, :G].double() * q < p) & (i < count[:, None])
    n = torch.cumprod(ok.int(), 1).sum(1)
    r = torch.arange(R, device=u.device)
    t = target[r, n].double()
    d = torch.where((n < count)[:, None], draft[r, n.clamp(max=G - 1)].double(), 0.0)
    left = (t - d).clamp(min=0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, t)
    c = torch.cumsum(left, 1)
    nxt = torch.searchsorted(c, u[:, G:].double() * c[:, -1:], right=True).squeeze(1).clamp(max=V - 1)
    return {"accepted": n.int(), "token": nxt.int()}


def run(st):
    op = st["case"]["op"]
    if own:
        import sparse_attention_indexer_e4m3_gb300 as dsa

        if op == "rows":
            seq, pos, ks, ke = dsa.step_maps(st["held"], st["added"], st["case"]["T"])
            dsa.store_kv(st["kv"], st["pages"], st["table"], seq, pos)
            return {"seq": seq, "pos": pos, "ks": ks, "ke": ke, "pages": st["pages"]}
        if op == "slots":
            return dsa.page_slots(st["pages"], st["table"], st["seq"], st["idx"], start=st["start"])
        if op == "attend":
            q = st["q"]
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
            out = dsa.paged_attn(q, st["pages"], st["table"], st["seq"], st["pos"], window=st["case"]["window"] or None,
                                 first=st["case"]["first"], attn_sink=st["sink"], scale=st["scale"], lse=lse)
            return {"out": out, "lse": lse}
        accepted, token = dsa.verify_drafts(st["target"], st["draft"], st["tokens"], st["count"], st["u"])
        return {"accepted": accepted, "token": token}
    if op == "rows":
        seq, pos, ks, ke = _maps(st["held"], st["added"], st["case"]["T"])
        _store(st["kv"], st["pages"], st["table"], seq, pos, st["case"]["page_rows"])
        return {"seq": seq, "pos": pos, "ks": ks, "ke": ke, "pages": st["pages"]}
    if op == "slots":
        idx, B = st["idx"], st["case"]["page_rows"]
        return _slots(st["table"], st["seq"], torch.where(idx >= 0, idx - st["start"][:, None], -1), B)
    if op == "attend":
        return _attend(st)
    return _verify(st["target"], st["draft"], st["tokens"], st["count"], st["u"])


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "rows":
        held, added, table = (st[k].cpu().numpy() for k in ("held", "added", "table"))
        T, B = case["T"], case["page_rows"]
        m = {"seq": np.full(T, -1, np.int32), "pos": np.full(T, -1, np.int32), "ks": np.zeros(T, np.int32),
             "ke": np.zeros(T, np.int32)}
        pages = st["pages"].cpu()
        kv = st["kv"].cpu()
        t = base = 0
        for r in range(len(held)):
            for i in range(added[r]):
                p = int(held[r]) + i
                m["seq"][t], m["pos"][t], m["ks"][t], m["ke"][t] = r, p, base, base + p + 1
                t += 1
            if added[r]:
                p = held[r] + np.arange(added[r])
                pages[torch.from_numpy(table[r, p // B].astype(np.int64)), torch.from_numpy(p % B)] = kv[t - int(added[r]):t]
            base += int(held[r] + added[r])
        return {**{k: torch.from_numpy(v).cuda() for k, v in m.items()}, "pages": pages.cuda().double()}
    if op == "slots":
        table, seq, start, idx = (st[k].cpu().numpy() for k in ("table", "seq", "start", "idx"))
        B = case["page_rows"]
        out = np.full(idx.shape, -1, np.int32)
        for t in range(len(seq)):
            j = idx[t][idx[t] >= 0] - start[t]
            out[t][idx[t] >= 0] = table[seq[t]][j // B] * B + j % B
        return torch.from_numpy(out).cuda()
    if op == "verify":
        target, draft, u = st["target"].double(), st["draft"].double(), st["u"].double()
        tokens, count = st["tokens"].cpu().tolist(), st["count"].cpu().tolist()
        accepted, token = [], []
        for r in range(case["R"]):
            n = 0
            while n < count[r] and bool(u[r, n] * draft[r, n, tokens[r][n]] < target[r, n, tokens[r][n]]):
                n += 1
            w = target[r, n] - draft[r, n] if n < count[r] else target[r, n]
            w = torch.where(w > 0, w, 0.0)
            if float(w.sum()) == 0.0:
                w = target[r, n]
            c = torch.cumsum(w, 0)
            accepted.append(n)
            token.append(int((c > u[r, case["G"]] * c[-1]).nonzero()[0, 0]))
        return {"accepted": torch.tensor(accepted, dtype=torch.int32, device="cuda"),
                "token": torch.tensor(token, dtype=torch.int32, device="cuda")}
    if work(case)["flops"] > 1e13:
        return None
    q, table, sink = st["q"].double(), st["table"].long(), st["sink"]
    T, H, D = q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    if sink is not None:
        lse[:] = sink.double()
    t = 0
    for r in range(case["R"]):
        n = int(st["held"][r] + st["added"][r])
        kv = st["pages"][table[r]].flatten(0, 1)[:n].double()
        end = t + int(st["added"][r])
        each = max(1, (1 << 27) // (H * n))
        p = int(st["held"][r])
        while t < end:
            k = min(each, end - t)
            at = torch.arange(p, p + k, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")[None, :]
            hidden = j > at
            if case["window"]:
                hidden |= (j <= at - case["window"]) & (j >= case["first"])
            x = (q[t:t + k].reshape(-1, D) @ kv.T).view(k, H, n) * st["scale"]
            x.masked_fill_(hidden[:, None, :], -math.inf)
            if sink is not None:
                x = torch.cat([x, sink.double()[None, :, None].expand(k, H, 1)], 2)
            lse[t:t + k] = torch.logsumexp(x, 2)
            x = torch.exp(x[..., :n] - lse[t:t + k, :, None])
            out[t:t + k] = (x.view(-1, n) @ kv).view(k, H, D)
            t += k
            p += k
    return {"out": out, "lse": lse}
