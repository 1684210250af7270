"""Cases that measure the paged key-value cache of the attention layer.

Five operators, each in a plain form (elementary torch operations) and through
the package's own entry points:

  decode   attention of one new token per sequence over its pages
  extend   causal attention of a ragged batch of new tokens over their pages
  append   keys and values of new tokens into their pages
  turn     one scheduler turn on the pages: finished sequences freed and
           samples forked from their prompts (fork), then pages for the new
           tokens of the turn, copying shared last pages (grow)
  compact  live pages moved to the front of the pool, tables renumbered

Layout: pages [num_pages, kv_heads, page, 128] bf16 for keys and for values
(the pool [planes, num_pages, kv_heads, page, 128] holds them for all layers),
table [seqs, max_pages] int32 page numbers (-1 where none), lengths [seqs]
int32 tokens per sequence, the ones of this call included, refs [num_pages]
int32 table entries that hold a page (0: free).  Lengths come from the case
alone, so that its work is known; which pages hold what comes from the seed.
"""
import math
import random

import torch

own = False

D = 128                       # head width
DEV = "cuda"
BF = torch.bfloat16


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a single chat reply just after a short prompt: latency of one call
        dict(name="decode one short", op="decode", seqs=1, lo=200, hi=200, heads=32, kv=8, page=64, lse=False),
        # the decode batch of the benchmark: 64 sequences of 2048 tokens
        dict(name="decode 64 x 2048", op="decode", seqs=64, lo=2048, hi=2048, heads=32, kv=8, page=64, lse=False),
        # long documents beside short chats, 1 to 131072 tokens, small pages, wider groups, joined with other parts later
        dict(name="decode ragged long", op="decode", seqs=24, lo=1, hi=131072, heads=64, kv=8, page=16, lse=True),
        # five drafted tokens per sequence verified in one call
        dict(name="extend drafts", op="extend", seqs=32, new_lo=5, new_hi=5, lo=300, hi=4096, heads=32, kv=8, page=64,
             lse=False),
        # a prompt's last chunk of 4096 tokens, 12288 cached before it
        dict(name="extend chunk", op="extend", seqs=1, new_lo=4096, new_hi=4096, lo=12288, hi=12288, heads=32, kv=8,
             page=128, lse=False),
        # prompts of all lengths behind shared prefixes, decode rows among them
        dict(name="extend mixed", op="extend", seqs=24, new_lo=1, new_hi=1500, lo=0, hi=6000, heads=32, kv=8, page=32,
             lse=True),
        # one decode step's keys and values
        dict(name="append step", op="append", seqs=64, new_lo=1, new_hi=1, lo=100, hi=8000, heads=32, kv=8, page=64),
        # a prefill batch's keys and values, odd lengths
        dict(name="append prompts", op="append", seqs=33, new_lo=17, new_hi=4001, lo=0, hi=2000, heads=32, kv=8,
             page=32),
        # a small server's turn: 8 slots, one attention layer
        dict(name="turn small", op="turn", seqs=8, lo=50, hi=900, layers=1, kv=8, page=64, spare=40),
        # a full server's turn: 256 slots, the four attention layers of 32
        dict(name="turn large", op="turn", seqs=256, lo=30, hi=1500, layers=4, kv=8, page=64, spare=300),
        # compaction of a small pool
        dict(name="compact small", op="compact", seqs=6, pages=160, live=0.6, layers=1, kv=8, page=64),
        # compaction of a large one, fragmented by finished sequences
        dict(name="compact large", op="compact", seqs=96, pages=2040, live=0.6, layers=4, kv=8, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "extend", "extend", "append", "turn", "compact"])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        seqs = _log(rng, 1, 200)
        hi = max(2, min(_log(rng, 2, 131072), 2_000_000 // (seqs * kv)))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, _log(rng, 1, hi)]), hi=hi, heads=heads, kv=kv, page=page,
                    lse=rng.random() < 0.5)   # slots without tokens (0) among them
    if op == "extend":
        heads = kv * rng.choice([1, 2, 4, 8])
        seqs = _log(rng, 1, 48)
        new = max(1, min(_log(rng, 1, 3000), 12000 // seqs))
        hi = max(1, min(_log(rng, 1, 12000), 200_000 // seqs))
        return dict(op=op, seqs=seqs, new_lo=_log(rng, 1, new), new_hi=new, lo=rng.choice([0, hi // 3]), hi=hi,
                    heads=heads, kv=kv, page=page, lse=rng.random() < 0.5)
    if op == "append":
        seqs = _log(rng, 1, 200)
        new = max(1, min(_log(rng, 1, 4000), 60000 // seqs))
        return dict(op=op, seqs=seqs, new_lo=_log(rng, 1, new), new_hi=new, lo=0, hi=_log(rng, 1, 1000),
                    heads=kv * 4, kv=kv, page=page)
    layers = rng.choice([1, 2, 4])
    if op == "turn":
        lo = _log(rng, 1, 300)
        return dict(op=op, seqs=_log(rng, 4, 256), lo=lo, hi=_log(rng, lo + 1, 1200), layers=layers, kv=kv,
                    page=page, spare=rng.choice([20, 200]))
    return dict(op=op, seqs=_log(rng, 2, 96), pages=_log(rng, 100, 2000 * 64 // page // 2), live=rng.uniform(0.3, 0.9),
                layers=layers, kv=kv, page=page)


# ------------------------------------------------------------- sizes of a case

def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly over their logarithm, in a mixed order."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    v = [int(round(math.exp(a + (b - a) * i / (n - 1)) - 1)) for i in range(n)]
    random.Random(n).shuffle(v)
    return v


def _lengths(c):
    """(new tokens, tokens with them) of each sequence."""
    if c["op"] == "decode":
        return [1] * c["seqs"], _spread(c["seqs"], c["lo"], c["hi"])
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"])
    old = _spread(c["seqs"] + 1, c["lo"], c["hi"])[1:] if c["seqs"] > 1 else [c["hi"]]
    return new, [n + o for n, o in zip(new, old)]


def _turn(c):
    """(lengths before, parent map, tokens to add) of a turn: of each four slots the first two stay as they are, the
    third becomes a sample of the second and the fourth's finished sequence makes room for a new prompt."""
    S = c["seqs"]
    before = _spread(S, c["lo"], c["hi"])
    prompt = _spread(S, c["lo"], c["hi"])[::-1]
    parent = [s - 1 if s % 4 == 2 else -1 if s % 4 == 3 else s for s in range(S)]
    add = [1 if s % 4 == 2 else prompt[s] if s % 4 == 3 else 0 for s in range(S)]
    return before, parent, add


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------- the inputs

def _randn(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _table(g, counts, num_pages, width):
    """A table whose rows hold counts[s] pages of their own, drawn without order from the pool."""
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    first = [0]
    for n in counts:
        first.append(first[-1] + n)
    n, f = (torch.tensor(v, device=DEV) for v in (counts, first[:-1]))
    j = torch.arange(width, device=DEV)
    at = (f[:, None] + j).clamp(max=num_pages - 1)
    return torch.where(j < n[:, None], order[at], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    ints = lambda v: torch.tensor(v, device=DEV, dtype=torch.int32)  # noqa: E731
    P, G = c["page"], c["kv"]
    if c["op"] in ("decode", "extend", "append"):
        new, total = _lengths(c)
        counts = [_pages(n, P) for n in total]
        N = sum(counts) + 5
        width = max(max(counts), 1) + 1
        H, T = c["heads"], sum(new)
        # the fused projection's rows, as the layer holds them: queries, keys, values of each new token
        rows = _randn(g, T, H + 2 * G, D)
        # keys with a few strong channels, values around a mean per channel, as trained layers have them
        scale = 1 + 2 * (torch.rand(G, 1, D, generator=g, device=DEV) < 0.05).to(BF)
        mean = 0.3 * _randn(g, G, 1, D)
        k, v = _randn(g, N, G, P, D).mul_(scale), _randn(g, N, G, P, D).add_(mean)
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        return dict(op=c["op"], lse=c.get("lse"), q=rows[:, :H], k_new=rows[:, H:H + G], v_new=rows[:, H + G:], k=k,
                    v=v, table=_table(g, counts, N, width), lengths=ints(total), q_start=ints(start), new=new,
                    total=total)
    if c["op"] == "turn":
        before, parent, add = _turn(c)
        after = [before[p] if p >= 0 else 0 for p in parent]
        counts = [_pages(n, P) for n in before]
        grown = [_pages(n + a, P) for n, a in zip(after, add)]
        N = sum(max(x, y) for x, y in zip(counts, grown)) + c["spare"]
        table = _table(g, counts, N, max(counts + grown) + 2)
        refs = torch.zeros(N, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        return dict(op="turn", page=P, data=_randn(g, 2 * c["layers"], N, G, P, D), refs=refs, table=table,
                    lengths=ints(before), parent=ints(parent), add=ints(add))
    # compact: the live pages in no order over the sequences, some held by two of them
    N, S = c["pages"], c["seqs"]
    live = max(S, int(N * c["live"]))
    counts = [live // S + (s < live % S) for s in range(S)]
    table = _table(g, counts, N, max(counts) + 3)
    refs = torch.zeros(N, dtype=torch.int32, device=DEV)
    refs[table[table >= 0].long()] = 1
    lengths = [n * P - (7 * s) % P for s, n in enumerate(counts)]
    if S > 2 and counts[1] <= counts[0]:
        refs[table[1][table[1] >= 0].long()] -= 1
        table[1] = table[0]
        refs[table[1][table[1] >= 0].long()] += 1
        lengths[1] = lengths[0]
    return dict(op="compact", page=P, data=_randn(g, 2 * c["layers"], N, G, P, D), refs=refs.clone(),
                table=table.clone(), lengths=ints(lengths), refs0=refs, table0=table)


# -------------------------------------------------------------- the plain forms

def _plain_decode(s):
    q, table, lengths = s["q"].float(), s["table"], s["lengths"]
    B, H, _ = q.shape
    G, P = s["k"].shape[1], s["k"].shape[2]
    at = table.clamp(min=0).long()
    L = at.shape[1] * P
    seen = torch.arange(L, device=DEV) < lengths[:, None]
    # [B, pages, G, P, D] -> [B, G, L, D]; rows behind the last token hold anything, so they become zeros
    k, v = (s[n][at].transpose(1, 2).reshape(B, G, L, D).float().masked_fill_(~seen[:, None, :, None], 0.0)
            for n in ("k", "v"))
    x = torch.matmul(q.view(B, G, H // G, D), k.transpose(2, 3)) / math.sqrt(D)
    x = x.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / total.clamp(min=1e-38)
    lse = (torch.log(total) + top).view(B, H)
    return (o.view(B, H, D).to(BF), lse) if s["lse"] else o.view(B, H, D).to(BF)


def _plain_extend(s):
    q, table = s["q"], s["table"].clamp(min=0).long()
    T, H, _ = q.shape
    G, P = s["k"].shape[1], s["k"].shape[2]
    out, lse, t = torch.empty(T, H, D, dtype=BF, device=DEV), torch.empty(T, H, device=DEV), 0
    for i, (n, length) in enumerate(zip(s["new"], s["total"])):   # each sequence has its own lengths
        pages = table[i, :_pages(length, P)]
        k, v = (s[x][pages].transpose(0, 1).reshape(G, -1, D)[:, :length].float() for x in ("k", "v"))
        x = q[t:t + n].float().view(n, G, H // G, D).permute(1, 2, 0, 3).reshape(G, -1, D)
        x = (torch.matmul(x, k.transpose(1, 2)) / math.sqrt(D)).view(G, H // G, n, length)
        j = torch.arange(length, device=DEV)
        x.masked_fill_(j > (j[length - n:])[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        e = x.sub_(top).exp_()
        total = e.sum(-1, keepdim=True)
        o = torch.matmul(e.view(G, -1, length), v).view(G, H // G, n, D) / total
        out[t:t + n] = o.permute(2, 0, 1, 3).reshape(n, H, D)
        lse[t:t + n] = (torch.log(total) + top).permute(2, 0, 1, 3).reshape(n, H)
        t += n
    return (out, lse) if s["lse"] else out


def _plain_append(s):
    k, v, start = s["k"], s["v"], s["q_start"].long()
    P, T = k.shape[2], s["k_new"].shape[0]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, t, right=True) - 1
    pos = s["lengths"][seq] - start[seq + 1] + t
    page, row = s["table"][seq, pos // P].long(), pos % P
    k[page, :, row] = s["k_new"]
    v[page, :, row] = s["v_new"]
    return k, v


def _plain_turn(s):
    table, lengths, refs, data, parent, P = (s[n] for n in ("table", "lengths", "refs", "data", "parent", "page"))
    S, W = table.shape
    N = refs.shape[0]
    j = torch.arange(W, device=DEV)
    slot = torch.arange(S, device=DEV)
    # fork: rows replaced at once; a page's holders are counted again for the changed rows
    changed = parent != slot
    gone = (parent < 0)[:, None]
    p = parent.clamp(min=0).long()
    old_n = -(-lengths // P)
    new = torch.where(gone, -1, table[p])
    new_len = torch.where(parent < 0, 0, lengths[p])
    hold = lambda t, n: torch.where(changed[:, None] & (j < n[:, None]), t, N).flatten().long()  # noqa: E731
    count = lambda at: torch.zeros(N + 1, dtype=torch.int32, device=DEV).index_add_(  # noqa: E731
        0, at, torch.ones_like(at, dtype=torch.int32))[:N]
    refs += count(hold(new, -(-new_len // P))) - count(hold(table, old_n))
    table.copy_(new)
    lengths.copy_(new_len)
    # grow: the lowest free pages, in the order of the sequences; a shared page that is partly full is copied
    add = s["add"].clamp(min=0)
    n0 = lengths // P
    part = lengths % P
    tail = table.gather(1, n0.clamp(max=W - 1).long()[:, None])[:, 0]
    fresh = -(-(lengths + add) // P) - -(-lengths // P)
    fits = -(-(lengths + add) // P) <= W
    cow = (add > 0) & (part > 0) & (refs[tail.clamp(min=0).long()] > 1)
    want = torch.where(fits, fresh + cow, 0)
    end = torch.cumsum(want, 0)
    free = refs == 0
    granted = fits & ((want == 0) | (end <= free.sum()))
    order = torch.sort(free.to(torch.uint8), stable=True, descending=True).indices.to(torch.int32)
    cow &= granted
    first = torch.where(cow, n0, -(-lengths // P))
    rank = (end - want)[:, None] + j - first[:, None]
    mine = granted[:, None] & (j >= first[:, None]) & (rank < end[:, None])
    pages = torch.where(mine, order[rank.clamp(0, N - 1).long()], table)
    src, dst = (torch.where(cow, t.gather(1, n0.clamp(max=W - 1).long()[:, None])[:, 0], order[-1]).long()
                for t in (table, pages))
    rows = (torch.arange(P, device=DEV) < torch.where(cow, part, 0)[:, None])[None, :, None, :, None]
    data[:, dst] = torch.where(rows, data[:, src], data[:, dst])
    refs.index_add_(0, src, -cow.to(torch.int32))
    refs += count(torch.where(mine, pages, N).flatten().long())
    table.copy_(pages)
    lengths += torch.where(granted, add, 0)
    return table, lengths, refs, granted.to(torch.int32), data


def _plain_compact(s):
    refs, table, data, P = s["refs"], s["table"], s["data"], s["page"]
    N = refs.shape[0]
    live = refs > 0
    n = live.sum()
    i = torch.arange(N, device=DEV)
    hole, mover = ~live & (i < n), live & (i >= n)
    holes = torch.sort(hole.to(torch.uint8), stable=True, descending=True).indices
    rank = (torch.cumsum(mover, 0) - 1).clamp(min=0)
    remap = torch.where(mover, holes[rank], torch.where(live, i, -1))
    held = torch.arange(table.shape[1], device=DEV) < -(-s["lengths"][:, None] // P)
    table.copy_(torch.where(held, remap[table.clamp(min=0).long()].to(torch.int32), table))
    # the page that each one takes its rows from: the mover whose hole it is, or itself (the others write past the end)
    source = torch.arange(N + 1, device=DEV).index_put_((torch.where(mover, remap, N),), i)[:N]
    data.copy_(data[:, source])
    moved = torch.zeros_like(refs).index_add_(0, remap.clamp(min=0), torch.where(live, refs, 0))
    refs.copy_(moved)
    return table, refs, remap.to(torch.int32), data


# ----------------------------------------------------------------------- a pass

def run(state):
    s = state
    op = s["op"]
    if op == "compact":   # the pool as it was before the last pass: its live pages still hold their rows
        s["refs"].copy_(s["refs0"])
        s["table"].copy_(s["table0"])
    if not own:
        return dict(decode=_plain_decode, extend=_plain_extend, append=_plain_append, turn=_plain_turn,
                    compact=_plain_compact)[op](s)
    import mamba_selective_scan_mixer_b200 as J
    if op == "decode":
        return J.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lengths"], want_lse=s["lse"])
    if op == "extend":
        return J.paged_extend(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["q_start"], want_lse=s["lse"])
    if op == "append":
        J.paged_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"], s["q_start"])
        return s["k"], s["v"]
    if op == "turn":
        J.pages_fork(s["parent"], s["refs"], s["table"], s["lengths"], s["page"])
        granted = J.pages_grow(s["add"], s["data"], s["refs"], s["table"], s["lengths"])
        return s["table"], s["lengths"], s["refs"], granted, s["data"]
    remap = J.pages_compact(s["data"], s["refs"], s["table"], s["lengths"])
    return s["table"], s["refs"], remap, s["data"]


def work(case):
    c = case
    P, G = c["page"], c["kv"]
    if c["op"] in ("decode", "extend", "append"):
        new, total = _lengths(c)
        T, H = sum(new), c["heads"]
        index = 4 * (sum(_pages(n, P) for n in total) + 2 * c["seqs"])
        if c["op"] == "append":
            return dict(bytes=2 * T * G * 2 * D * 2 + index, flops=0)
        seen = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total)) if c["op"] == "extend" else sum(total)
        return dict(bytes=sum(total) * G * 2 * D * 2 + 2 * T * H * D * 2 + index, flops=4 * D * H * seen)
    row = G * D * 2 * 2 * c["layers"]      # bytes of a token in all planes
    if c["op"] == "turn":
        before, parent, add = _turn(c)
        copied = sum(before[p] % P for p, a in zip(parent, add) if p >= 0 and a)
        entries = sum(_pages(before[s], P) + _pages((before[p] if p >= 0 else 0) + a, P)
                      for s, (p, a) in enumerate(zip(parent, add)) if p != s)
        N = sum(_pages(n, P) for n in before)
        return dict(bytes=2 * copied * row + 4 * (2 * entries + N + 5 * c["seqs"]), flops=0)
    N = c["pages"]
    live = max(c["seqs"], int(N * c["live"]))
    moved = live * (1 - live / N)          # expected, for live pages in no order
    return dict(bytes=2 * moved * P * row + 4 * (3 * N + 2 * live), flops=0)


# -------------------------------------------------------------------- in 64 bits

def _exact_attention(s):
    out, lse, t = [], [], 0
    q, P = s["q"].double(), s["k"].shape[2]
    G, rep = s["k"].shape[1], q.shape[1] // s["k"].shape[1]
    for i, (n, length) in enumerate(zip(s["new"], s["total"])):
        held = [int(p) for p in s["table"][i, :_pages(length, P)]]
        o, z = (torch.zeros(n, G * rep, w, dtype=torch.float64, device=DEV) for w in (D, 1))
        z -= math.inf
        for g in range(G if held else 0):
            k, v = (torch.cat([s[x][held, g].reshape(-1, D)])[:length].double() for x in ("k", "v"))
            for h in range(g * rep, g * rep + rep):
                x = q[t:t + n, h] @ k.T / math.sqrt(D)
                if s["op"] == "extend":
                    x += torch.full_like(x, -math.inf).triu(length - n + 1)
                z[:, h, 0] = torch.logsumexp(x, 1)
                o[:, h] = torch.softmax(x, 1) @ v
        out.append(o.cpu())
        lse.append(z[..., 0].cpu())
        t += n
    out, lse = torch.cat(out), torch.cat(lse)
    return (out, lse) if s["lse"] else out


def exact(case, seed):
    if case["op"] in ("decode", "extend"):
        if case["op"] == "extend" and case["seqs"] * case["kv"] * (case["heads"] // case["kv"]) > 40000:
            return None
        return _exact_attention(prepare(case, seed))
    return None                            # pages are moved, not computed
