"""The paged key-value cache on the GPU: attention of single tokens and of
ragged chunks, appends, page upkeep and the attention layer over pages, against
the fp64 / integer oracle.

Unused memory of the pools (free pages, rows behind a sequence's last token)
holds NaN, so that anything read from it shows.

Tolerance of attention outputs, per element, in units of spread = sum_j p_j |v_j|
(which bounds |o|): the terms p_j are rounded to bf16 before the product with v (half a
step, 2^-8) and the output once more (2^-8 |o|); scores are fp32 sums of 128
exact products, off by at most 128 * 2^-23 * sum |q k| / sqrt(128) < 2^-12 for the
inputs here (sum |q k| / sqrt(128) < 16), which changes each term by as much, its sum
too: 2 * 2^-12, with ex2 and the fp32 sums (2^-20) covered by the rest of 2^-10.
lse: that bound on the scores, 2^-12, plus fp32 rounding of the result.
"""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import paged as op
from synthetic import AttnShape, attn_input, attn_params
from tests.helpers import TOL_BF16, cuda_or_skip, rel_l2, to_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TOL_O = 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10
NAN = float("nan")


@pytest.fixture(scope="module")
def J():
    cuda_or_skip()
    import mamba_selective_scan_mixer_b200 as J
    J.lib()
    return J


def _cache(rng, lengths, G, P, spare=3, seed=0, width=None):
    """Random pages for sequences of the given lengths; all other memory NaN."""
    counts = [op.held(n, P) for n in lengths]
    N = sum(counts) + spare
    order = rng.permutation(N)
    W = width or max(max(counts), 1) + 1
    table = np.full((len(lengths), W), -1, dtype=np.int32)
    g = torch.Generator()
    g.manual_seed(seed + 17)
    k, v = torch.full((N, G, P, 128), NAN, dtype=BF), torch.full((N, G, P, 128), NAN, dtype=BF)
    at = 0
    for s, n in enumerate(lengths):
        for j in range(counts[s]):
            p = int(order[at])
            at += 1
            table[s, j] = p
            r = min(P, n - j * P)
            k[p, :, :r] = torch.randn(G, r, 128, generator=g).to(BF)
            v[p, :, :r] = (torch.randn(G, r, 128, generator=g) + 0.3).to(BF)
    return k, v, table


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _q(T, H, G, seed):
    """Queries as a slice of fused q|k|v rows (token stride (H + 2G) * 128)."""
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(T, H + 2 * G, 128, generator=g).to(BF).cuda()[:, :H]


def _check(got, lse, want, sel=None):
    o = to_np(got)
    sel = np.isfinite(want["spread"]).all(axis=(1, 2)) if sel is None else sel
    err = np.abs(o[sel] - want["o"][sel])
    bound = TOL_O * want["spread"][sel]
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-30)).max())
    if lse is not None:
        a, b = to_np(lse)[sel], want["lse"][sel]
        assert (np.isinf(a) == np.isinf(b)).all()
        f = np.isfinite(b)
        assert (np.abs(a[f] - b[f]) <= 2.0 ** -12 + 2.0 ** -22 * np.abs(b[f])).all()


# ------------------------------------------------------------------ one token

@pytest.mark.parametrize("lengths,H,G,P", [
    ([1], 4, 1, 16),
    ([0, 1, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 400], 32, 8, 64),
    ([33, 300, 5, 0, 257], 16, 2, 16),            # 8 heads per KV head
    ([100, 1000, 31], 3, 1, 32),                  # 3 heads per KV head
    ([70, 2, 513], 4, 4, 128),                    # one head per KV head
    ([600, 90], 32, 2, 256),                      # 16 heads per KV head
    ([77, 40, 250], 36, 3, 64),                   # 12 heads per KV head
    (list(range(0, 320, 3)), 8, 4, 32),           # many short sequences
])
def test_decode(J, lengths, H, G, P):
    rng = np.random.default_rng(len(lengths) * 100 + H)
    k, v, table = _cache(rng, lengths, G, P)
    S = len(lengths)
    q = _q(S, H, G, H + S)
    got, lse = J.paged_decode(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), np.arange(S + 1))
    _check(got, lse, want)
    assert torch.equal(J.paged_decode(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths)), got)   # bit for bit
    for s, n in enumerate(lengths):
        if n == 0:
            assert (got[s] == 0).all() and torch.isneginf(lse[s]).all()


def test_decode_one_long_among_short(J):
    lengths = [3, 40000, 0, 170, 64]
    rng = np.random.default_rng(9)
    k, v, table = _cache(rng, lengths, 2, 16, width=4000)
    q = _q(5, 8, 2, 9)
    out = torch.full((5, 12, 128), 7.0, dtype=BF, device="cuda")   # heads of a wider row: the rest stays
    got, lse = J.paged_decode(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), out=out[:, 2:10], want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), np.arange(6))
    _check(got, lse, want)
    assert (out[:, :2] == 7).all() and (out[:, 10:] == 7).all()


def test_decode_rising_scores(J):
    """Scores that grow along the sequence up to about 300, k and q exact: the running
    maximum is raised again and again, and the first positions end with no weight."""
    L, G, H, P = 700, 1, 4, 32
    rng = np.random.default_rng(11)
    k, v, table = _cache(rng, [L], G, P)
    q = torch.zeros(1, H, 128, dtype=BF)
    q[:, :, 0] = torch.tensor([1.0, 4.0, -4.0, 0.0])
    for i in range(L):
        row = k[table[0, i // P], :, i % P]
        row.zero_()
        row[:, 0] = float(i + 1)
    got, lse = J.paged_decode(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32([L]), want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array([L]), np.arange(2))
    _check(got, None, want)                        # rows of integers up to 700 round to bf16 before both sides
    # the scores are exact up to the fp32 scale: lse within 2^-20 of its size
    assert (np.abs(to_np(lse) - want["lse"]) <= 2.0 ** -20 * np.abs(want["lse"]) + 2.0 ** -18).all()


def test_bad_device_values_stay_inside(J):
    """Lengths past the table, negative lengths and page numbers that are none: no access
    leaves the pool (rows of such sequences are unspecified), the others are right."""
    import os
    rng = np.random.default_rng(12)
    lengths = [50, 100, 80, 60]
    k, v, table = _cache(rng, lengths, 2, 16)
    k.nan_to_num_(0.0)
    v.nan_to_num_(0.0)
    bad, bad_len = table.copy(), np.array([50, 1000000, -7, 60])
    bad[3, 1] = 99999
    q = _q(4, 8, 2, 3)
    got, lse = J.paged_decode(q, k.cuda(), v.cuda(), _i32(bad), _i32(bad_len), want_lse=True)
    st = _i32([0, 1, 2, 3, 4])
    got2 = J.paged_extend(q, k.cuda(), v.cuda(), _i32(bad), _i32(bad_len), st)
    torch.cuda.synchronize()
    if os.environ.get("JAMBA_CHECKED", "0") == "1":
        with pytest.raises(J.JambaError):
            J.device_status()
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array([50, 0, 0, 0]), np.array([0, 1, 1, 1, 1]))
    only = np.array([True, False, False, False])
    _check(got, lse, want, only)
    _check(got2, None, want, only)
    assert (got[2] == 0).all() and torch.isneginf(lse[2]).all()


# --------------------------------------------------------------- ragged chunks

@pytest.mark.parametrize("new,cached,H,G,P", [
    ([1], [0], 4, 1, 16),
    ([5, 5, 5, 5], [100, 0, 63, 300], 32, 8, 64),
    ([300, 0, 1, 129, 64], [0, 50, 200, 17, 1000], 8, 2, 32),
    ([77, 33], [500, 3], 16, 2, 16),               # 8 heads per KV head
    ([50, 130], [129, 0], 3, 1, 128),              # 3 heads per KV head
    ([200, 260], [30, 0], 4, 4, 256),              # one head per KV head
    ([3, 20], [70, 0], 48, 1, 64),                 # 48 heads per KV head
    ([2, 0, 9], [40, 0, 0], 128, 1, 16),           # 128 heads per KV head
    ([1] * 40 + [90], list(range(0, 400, 10)) + [10], 8, 4, 32),
    ([0, 0, 0], [0, 9, 0], 4, 1, 16),              # no new token at all
])
def test_extend(J, new, cached, H, G, P):
    lengths = [a + b for a, b in zip(new, cached)]
    rng = np.random.default_rng(sum(lengths) + H)
    k, v, table = _cache(rng, lengths, G, P)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    rows = T + 3                                    # rows that no sequence counts
    q = _q(rows, H, G, T + H)
    out = torch.full((rows, H, 128), 7.0, dtype=BF, device="cuda")
    got, lse = J.paged_extend(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), _i32(start), out=out, want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    _check(got, lse, want)
    assert (got[T:] == 7).all()
    again = J.paged_extend(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), _i32(start))
    assert torch.equal(again[:T], got[:T])          # bit for bit


def test_extend_long_sequence_in_parts(J):
    """30 new tokens behind 20000 cached ones (the keys are split over the GPU), with a
    sequence whose first tokens stand before position 0: they see nothing."""
    lengths, new = [20030, 12, 500], [30, 20, 200]
    rng = np.random.default_rng(31)
    k, v, table = _cache(rng, lengths, 2, 64)
    start = np.concatenate([[0], np.cumsum(new)])
    q = _q(int(start[-1]), 8, 2, 31)
    got, lse = J.paged_extend(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), _i32(start), want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    _check(got, lse, want)
    assert (got[30:38] == 0).all() and torch.isneginf(lse[30:38]).all()


def test_extend_rising_scores(J):
    """Scores that grow block after block up to about 300: the reference of the softmax is
    raised many times, per row at its own blocks."""
    L, n, P, H = 900, 300, 32, 4
    rng = np.random.default_rng(33)
    k, v, table = _cache(rng, [L], 1, P)
    g = torch.Generator()
    g.manual_seed(5)
    q = torch.zeros(n, H, 128, dtype=BF)
    q[:, :, 0] = torch.randint(-4, 5, (n, H), generator=g).to(BF)
    for i in range(L):
        row = k[table[0, i // P], :, i % P]
        row.zero_()
        row[:, 0] = float(i + 1)
    got = J.paged_extend(q.cuda(), k.cuda(), v.cuda(), _i32(table), _i32([L]), _i32([0, n]))
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array([L]), np.array([0, n]))
    _check(got, None, want)


def test_parts_join_by_lse(J):
    """Attention over two disjoint sets of keys, joined by their lse, is attention over both."""
    lengths = [700, 90]
    rng = np.random.default_rng(35)
    k, v, table = _cache(rng, lengths, 2, 32)
    q = _q(2, 8, 2, 35)
    kc, vc = k.cuda(), v.cuda()
    o1, l1 = J.paged_decode(q, kc, vc, _i32(table), _i32([320, 64]), want_lse=True)
    rest = np.full_like(table, -1)
    rest[0, :table.shape[1] - 10], rest[1, :table.shape[1] - 2] = table[0, 10:], table[1, 2:]
    o2, l2 = J.paged_decode(q, kc, vc, _i32(rest), _i32([380, 26]), want_lse=True)
    w = torch.softmax(torch.stack([l1, l2]).double(), 0)[..., None]
    joined = o1.double() * w[0] + o2.double() * w[1]
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), np.arange(3))
    assert (np.abs(to_np(joined) - want["o"]) <= TOL_O * want["spread"]).all()


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("new,cached,G,P", [([1, 0, 70, 300, 5], [3, 9, 60, 0, 251], 8, 64), ([40, 1], [0, 15], 1, 16),
                                            ([7], [0], 3, 32), ([130, 3], [2, 0], 40, 128)])
def test_append_ragged(J, new, cached, G, P):
    lengths = [a + b for a, b in zip(new, cached)]
    rng = np.random.default_rng(sum(new))
    k, v, table = _cache(rng, lengths, G, P)
    start = np.concatenate([[0], np.cumsum(new)])
    rows = _q(int(start[-1]) + 2, 2 * G, G, 8)           # two rows that no sequence counts
    kn, vn = rows[:, :G], rows[:, G:]
    kc, vc = k.cuda(), v.cuda()
    J.paged_append(kn, vn, kc, vc, _i32(table), _i32(lengths), _i32(start))
    ko, vo = k.float().numpy(), v.float().numpy()
    op.append(kn.float().cpu().numpy(), vn.float().cpu().numpy(), ko, vo, table, lengths, start)
    np.testing.assert_array_equal(kc.float().cpu().numpy(), ko)
    np.testing.assert_array_equal(vc.float().cpu().numpy(), vo)


def test_append_one_each_and_tokens_before_the_start(J):
    lengths = [5, 0, 33, 16]
    rng = np.random.default_rng(41)
    k, v, table = _cache(rng, lengths, 2, 16)
    rows = _q(4, 4, 2, 8)
    kc, vc = k.cuda(), v.cuda()
    J.paged_append(rows[:, :2], rows[:, 2:], kc, vc, _i32(table), _i32(lengths))
    ko, vo = k.float().numpy(), v.float().numpy()
    sel = [0, 2, 3]                                     # the empty slot is left out
    op.append(rows[sel, :2].float().cpu().numpy(), rows[sel, 2:].float().cpu().numpy(), ko, vo, table[sel],
              np.array(lengths)[sel], [0, 1, 2, 3])
    np.testing.assert_array_equal(kc.float().cpu().numpy(), ko)
    np.testing.assert_array_equal(vc.float().cpu().numpy(), vo)
    # three rows for a sequence of length 2: the first stands before position 0
    kc, vc = k.cuda(), v.cuda()
    J.paged_append(rows[:3, :2], rows[:3, 2:], kc, vc, _i32(table[:1]), _i32([2]), _i32([0, 3]))
    ko = k.float().numpy()
    op.append(rows[:3, :2].float().cpu().numpy(), rows[:3, 2:].float().cpu().numpy(), ko, v.float().numpy(),
              table[:1], [2], [0, 3])
    np.testing.assert_array_equal(kc.float().cpu().numpy(), ko)


# --------------------------------------------------------------------- upkeep

@pytest.mark.parametrize("S,W,N,G,P,layers,turns", [(5, 9, 30, 1, 16, 1, 40), (40, 12, 260, 3, 32, 2, 12),
                                                  (1100, 3, 1500, 1, 16, 1, 4), (3, 200, 9000, 1, 16, 1, 5)])
def test_upkeep_follows_the_oracle(J, S, W, N, G, P, layers, turns):
    """Random turns of fork, free, grow and compact: table, counts, lengths, grants and the
    rows in use equal the oracle's exactly.  Pools run dry and sequences reach max_pages;
    more slots than one step of a plan takes, and more pages; odd page counts."""
    rng = np.random.default_rng(S + N)
    planes = 2 * layers
    data = torch.randn(planes, N, G, P, 128, generator=torch.Generator().manual_seed(S)).to(BF)
    d_o = data.float().numpy().copy()
    refs, table, lengths = np.zeros(N, dtype=int), np.full((S, W), -1), np.zeros(S, dtype=int)
    d, r, t, ln = data.cuda(), _i32(refs), _i32(table), _i32(lengths)
    refused = 0
    for turn in range(turns):
        parent = np.arange(S)
        for s in rng.choice(S, max(1, S // 3), replace=False):
            parent[s] = rng.choice([-1, rng.integers(0, S), rng.integers(0, S)])
        J.pages_fork(_i32(parent), r, t, ln, P)
        op.fork(parent, refs, table, lengths, P)
        np.testing.assert_array_equal(t.cpu().numpy(), table)
        np.testing.assert_array_equal(r.cpu().numpy(), refs)
        np.testing.assert_array_equal(ln.cpu().numpy(), lengths)
        most = 2 * N * P // S if turn % 3 == 2 else N * P // (4 * S) + 2
        add = rng.integers(-2, max(2, most), S)
        granted = J.pages_grow(_i32(add), d, r, t, ln)
        want = op.grow(add, d_o, refs, table, lengths)
        refused += want.count(0)
        assert granted.cpu().tolist() == want
        for got, exp in ((t, table), (r, refs), (ln, lengths)):
            np.testing.assert_array_equal(got.cpu().numpy(), exp)
        np.testing.assert_array_equal(d.float().cpu().numpy(), d_o)
        if turn % 2:
            remap = J.pages_compact(d, r, t, ln)
            want = op.compact(d_o, refs, table, lengths)
            np.testing.assert_array_equal(remap.cpu().numpy(), want)
            for got, exp in ((t, table), (r, refs), (ln, lengths)):
                np.testing.assert_array_equal(got.cpu().numpy(), exp)
            np.testing.assert_array_equal(d.float().cpu().numpy(), d_o)
    assert refused > 0


def test_fork_of_slots_that_change_themselves(J):
    """A cycle, a chain and a fan-out in one call: every slot takes what its parent held before."""
    S, W, N, P = 6, 3, 20, 16
    refs, table, lengths = np.zeros(N, dtype=int), np.full((S, W), -1), np.array([40, 16, 0, 17, 5, 33])
    at = 0
    for s in range(S):
        for j in range(op.held(lengths[s], P)):
            table[s, j] = at
            refs[at] += 1
            at += 1
    refs[7] += 1                                        # a holder outside the table
    parent = [1, 0, 0, 3, 3, -1]
    r, t, ln = _i32(refs), _i32(table), _i32(lengths)
    wide = torch.full((S, W + 2), -5, dtype=torch.int32, device="cuda")   # a table with a row stride of its own
    wide[:, :W] = t
    J.pages_fork(_i32(parent), r, wide[:, :W], ln, P)
    op.fork(parent, refs, table, lengths, P)
    np.testing.assert_array_equal(wide[:, :W].cpu().numpy(), table)
    np.testing.assert_array_equal(r.cpu().numpy(), refs)
    np.testing.assert_array_equal(ln.cpu().numpy(), lengths)
    assert (wide[:, W:] == -5).all()


# ---------------------------------------------------------------- the layer

SH = AttnShape(d_model=256, n_heads=8, n_kv_heads=2, head_dim=128)


def _layer(J, seed=3):
    p = attn_params(SH, seed=seed)
    return J.Attention({k: v.cuda() for k, v in p.items()}, SH), {k: to_np(v) for k, v in p.items()}


def test_layer_serves_a_shared_prefix(J):
    """A prompt, three samples forked from it, two of them with chunks of their own, then
    single tokens, a slot freed and the pool compacted half way: each sample's outputs equal
    the oracle's prefill of everything it was given."""
    att, p = _layer(J)
    cache = J.PagedKVCache(layers=2, n_kv_heads=2, num_pages=60, max_seqs=4, max_len=512, page_size=16)
    cache.data.fill_(NAN)
    given = [[] for _ in range(4)]
    x_all = attn_input(SH, 1, 600, seed=5)[0]
    used = 0

    def turn(add, steps):
        nonlocal used
        add = list(add)
        assert cache.grow(_i32(add)).tolist() == [1] * 4
        rows = []
        for s, n in enumerate(add):
            piece = x_all[used:used + n]
            used += n
            given[s] = given[s] + [piece]
            rows.append(piece)
        x = torch.cat(rows).cuda()
        if steps:
            full = torch.zeros(4, SH.d_model, dtype=BF, device="cuda")
            full[[s for s in range(4) if add[s]]] = x
            out = att.paged_step(full, cache, layer=1)
            outs = [out[s:s + 1] for s in range(4)]
        else:
            start = np.concatenate([[0], np.cumsum(add)])
            out = att.paged_prefill(x, _i32(start), cache, layer=1)
            outs = [out[start[s]:start[s + 1]] for s in range(4)]
        for s, n in enumerate(add):
            if n:
                seq = torch.cat(given[s])[None]
                want = oatt.attention_prefill(p, to_np(seq), SH)["out"][0, -n:]
                assert rel_l2(to_np(outs[s]), want) < TOL_BF16, (s, n)

    turn([150, 0, 0, 0], False)
    cache.fork(_i32([0, 0, 0, 3]))
    given[1], given[2] = list(given[0]), list(given[0])
    turn([0, 37, 70, 20], False)
    turn([1, 1, 1, 1], True)
    cache.free(0)
    given[0] = []
    cache.compact()
    live = int((cache.refs > 0).sum())
    assert bool((cache.refs[:live] > 0).all())
    for _ in range(3):
        # slot 0 is empty: its token is not counted
        assert cache.lengths[0] == 0
        turn([0, 1, 1, 1], True)
    turn([44, 1, 9, 0], False)
    J.device_status()


def test_layer_steps_in_a_graph(J):
    """grow and the step of two layers captured once, replayed: lengths, pages and outputs
    advance as in eager calls."""
    att, p = _layer(J)
    S, steps = 3, 20

    def fresh():
        c = J.PagedKVCache(layers=2, n_kv_heads=2, num_pages=40, max_seqs=S, max_len=160, page_size=16)
        pre = attn_input(SH, 1, 60, seed=7)[0].cuda()
        c.grow(_i32([30, 10, 20]))
        for layer in range(2):
            att.paged_prefill(pre, _i32([0, 30, 40, 60]), c, layer)
        return c

    xs = attn_input(SH, S, steps, seed=8).cuda().transpose(0, 1).contiguous()
    one = _i32([1] * S)
    eager_cache, want = fresh(), []
    for t in range(steps):
        eager_cache.grow(one)
        h = att.paged_step(xs[t], eager_cache, 0, residual=xs[t])
        want.append(att.paged_step(h, eager_cache, 1, residual=h).clone())
    cache = fresh()
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        granted = cache.grow(one)
        h = att.paged_step(x, cache, 0, residual=x)
        y = att.paged_step(h, cache, 1, residual=h)
    for t in range(steps):
        x.copy_(xs[t])
        graph.replay()
        assert torch.equal(y, want[t]), t
        assert granted.tolist() == [1] * S
    for a, b in ((cache.table, eager_cache.table), (cache.refs, eager_cache.refs), (cache.lengths, eager_cache.lengths)):
        assert torch.equal(a, b)


def test_rows_that_no_slot_counts_get_the_residual(J):
    att, _ = _layer(J)
    cache = J.PagedKVCache(layers=1, n_kv_heads=2, num_pages=8, max_seqs=2, max_len=64, page_size=16)
    cache.grow(_i32([5, 0]))
    x = attn_input(SH, 1, 9, seed=9)[0].cuda()
    out = att.paged_prefill(x, _i32([0, 5, 5]), cache, residual=x)
    assert torch.equal(out[5:], x[5:]) and not torch.equal(out[:5], x[:5])
    step = att.paged_step(x[:2], cache, residual=x[:2].contiguous())
    assert torch.equal(step[1], x[1])                   # the empty slot


def test_two_streams_at_once(J):
    """The same calls on two streams, unordered: each has its own workspace."""
    rng = np.random.default_rng(51)
    lengths = [3000, 10, 777]
    k, v, table = _cache(rng, lengths, 2, 32)
    k, v, t, ln = k.cuda(), v.cuda(), _i32(table), _i32(lengths)
    qs = [_q(3, 8, 2, 51), _q(3, 8, 2, 52)]
    qe = _q(90, 8, 2, 53)
    st = _i32([0, 60, 60, 90])
    want = [J.paged_decode(q, k, v, t, ln) for q in qs]
    want_e = J.paged_extend(qe, k, v, t, ln, st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append((J.paged_decode(qs[i], k, v, t, ln, stream=streams[i]),
                           J.paged_extend(qe, k, v, t, ln, st, stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for d, e in got[i]:
            assert torch.equal(d, want[i]) and torch.equal(e, want_e)


def test_binding_refusals(J):
    i32 = torch.int32
    k = torch.zeros(4, 2, 16, 128, dtype=BF, device="cuda")
    table, lengths = torch.zeros(2, 3, dtype=i32, device="cuda"), torch.zeros(2, dtype=i32, device="cuda")
    q = torch.zeros(2, 4, 128, dtype=BF, device="cuda")
    refs = torch.zeros(4, dtype=i32, device="cuda")
    st = torch.zeros(3, dtype=i32, device="cuda")
    bad = [lambda: J.paged_decode(q[:1], k, k, table, lengths),                       # one token per slot
           lambda: J.paged_decode(q.float(), k, k, table, lengths),
           lambda: J.paged_decode(q, k, k[:3], table, lengths),
           lambda: J.paged_decode(q, k, k, table.long(), lengths),
           lambda: J.paged_decode(q, k, k, table, lengths[:1]),
           lambda: J.paged_decode(q, k[:, :, ::2], k, table, lengths),
           lambda: J.paged_decode(q.transpose(0, 1), k, k, table, lengths),
           lambda: J.paged_decode(q, k, k, table.t(), lengths),
           lambda: J.paged_decode(q, k, k, table, lengths, out=q[:, :2]),
           lambda: J.paged_extend(q, k, k, table, lengths, None),
           lambda: J.paged_extend(q, k, k, table, lengths, st[:2]),
           lambda: J.paged_append(q, q, k, k, table, lengths),                        # four heads into two
           lambda: J.pages_fork(lengths[:1], refs, table, lengths, 16),
           lambda: J.pages_grow(lengths, k, refs, table, lengths),
           lambda: J.pages_compact(k[None], refs[:3], table, lengths)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    with pytest.raises(J.JambaError):
        J.paged_decode(q, k, k, table, lengths, out=q)
    with pytest.raises(J.JambaError):
        J.pages_fork(lengths, refs, table, lengths, 24)
    cache = J.PagedKVCache(1, 2, 4, 2, 64)
    with pytest.raises(ValueError):
        cache.free(2)
    with pytest.raises(ValueError):
        cache.config(1)
    att, _ = _layer(J)
    x = torch.zeros(3, SH.d_model, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        att.paged_step(x, cache)
    with pytest.raises(ValueError):
        att.paged_prefill(x, st, J.PagedKVCache(1, 4, 4, 2, 64))


# ------------------------------------------------------------------- the rest

def test_extend_rows_before_the_first_sequence_and_empty_sequences_with_tokens(J):
    """q_start that begins at 2 (two rows that no sequence counts), a sequence whose tokens are
    not in its length (0), a table with a row stride of its own."""
    lengths, start = [40, 0, 150], [2, 9, 14, 34]
    rng = np.random.default_rng(61)
    k, v, table = _cache(rng, lengths, 2, 16)
    wide = torch.full((3, table.shape[1] + 4), 77777, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = _i32(table)
    t = wide[:, :table.shape[1]]
    q = _q(36, 8, 2, 61)
    out = torch.full((36, 8, 128), 7.0, dtype=BF, device="cuda")
    got, lse = J.paged_extend(q, k.cuda(), v.cuda(), t, _i32(lengths), _i32(start), out=out, want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    _check(got, lse, want)
    assert (got[:2] == 7).all() and (got[34:] == 7).all()
    assert (got[9:14] == 0).all() and torch.isneginf(lse[9:14]).all()
    d = J.paged_decode(q[:3], k.cuda(), v.cuda(), t, _i32(lengths))
    _check(d, None, op.attention(to_np(q[:3]), to_np(k), to_np(v), table, np.array(lengths), np.arange(4)))


def test_pages_past_four_gigabytes(J):
    """A plane of 9.2 GB: pages whose rows lie past 2^32 bytes (and 2^31 elements)."""
    G, P, N = 8, 64, 70000
    lengths, new = [300, 90], [70, 1]
    kc, vc = (torch.empty(N, G, P, 128, dtype=BF, device="cuda") for _ in range(2))
    rng = np.random.default_rng(62)
    k, v, small = _cache(rng, lengths, G, P, spare=0)
    k.nan_to_num_(0.0)
    v.nan_to_num_(0.0)
    pages = np.concatenate([small[0, :5], small[1, :2]])
    where = {int(p): N - 1 - 3 * i for i, p in enumerate(pages)}
    table = np.full_like(small, -1)
    table[0, :5], table[1, :2] = [where[int(p)] for p in small[0, :5]], [where[int(p)] for p in small[1, :2]]
    at = torch.tensor([where[int(p)] for p in pages], device="cuda")
    kc[at], vc[at] = k[pages].cuda(), v[pages].cuda()
    q = _q(71, 32, G, 62)
    start = [0, 70, 71]
    rows = _q(71, 2 * G, G, 63)
    J.paged_append(rows[:, :G], rows[:, G:], kc, vc, _i32(table), _i32(lengths), _i32(start))
    kn, vn = k.float().numpy(), v.float().numpy()
    op.append(rows[:, :G].float().cpu().numpy(), rows[:, G:].float().cpu().numpy(), kn, vn, small, lengths, start)
    np.testing.assert_array_equal(kc[at].float().cpu().numpy(), kn[pages])
    want = op.attention(to_np(q), kn.astype(np.float64), vn.astype(np.float64), small, np.array(lengths), start)
    got, lse = J.paged_extend(q, kc, vc, _i32(table), _i32(lengths), _i32(start), want_lse=True)
    _check(got, lse, want)
    last = q[[69, 70]]
    d, dl = J.paged_decode(last, kc, vc, _i32(table), _i32(lengths), want_lse=True)
    _check(d, dl, {n: x[[69, 70]] for n, x in want.items()})
    # compaction from the far end to the front, and a copied last page
    data = torch.stack([kc[-64:], vc[-64:]])
    del kc, vc
    big = torch.empty(2, N // 2, G, P, 128, dtype=BF, device="cuda")
    big[:, -64:] = data
    refs = torch.zeros(N // 2, dtype=torch.int32, device="cuda")
    t = _i32(np.where(table >= 0, table - N + N // 2, -1))
    refs[t[t >= 0].long()] = 1
    ln = _i32(lengths)
    remap = J.pages_compact(big, refs, t, ln)
    assert sorted(remap[remap >= 0].tolist()) == list(range(7)) and int(refs.sum()) == 7
    back = torch.stack([big[0][t[0, :5].long()], big[1][t[0, :5].long()]])
    np.testing.assert_array_equal(back.float().cpu().numpy(), np.stack([kn[small[0, :5]], vn[small[0, :5]]]))


def test_upkeep_in_a_graph(J):
    """fork, grow and compact captured once: every replay does the turn on what it finds."""
    S, W, N, P = 4, 6, 40, 16
    data = torch.randn(2, N, 1, P, 128, generator=torch.Generator().manual_seed(3)).to(BF)
    d_o = data.float().numpy().copy()
    refs, table, lengths = np.zeros(N, dtype=int), np.full((S, W), -1), np.zeros(S, dtype=int)
    d, r, t, ln = data.cuda(), _i32(refs), _i32(table), _i32(lengths)
    parent, add = np.array([0, 0, -1, 2]), np.array([5, 20, 33, 1])
    pg, ag = _i32(parent), _i32(add)
    J.device_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        J.pages_fork(pg, r, t, ln, P)
        granted = J.pages_grow(ag, d, r, t, ln)
        remap = J.pages_compact(d, r, t, ln)
    for _ in range(8):
        graph.replay()
        op.fork(parent, refs, table, lengths, P)
        want = op.grow(add, d_o, refs, table, lengths)
        moved = op.compact(d_o, refs, table, lengths)
        assert granted.tolist() == want
        for got, exp in ((t, table), (r, refs), (ln, lengths), (remap, moved)):
            np.testing.assert_array_equal(got.cpu().numpy(), exp)
        np.testing.assert_array_equal(d.float().cpu().numpy(), d_o)


def test_sequences_that_share_pages(J):
    """Two slots that hold the same pages see the same keys; a third its own length of them."""
    lengths = [200, 200, 77]
    rng = np.random.default_rng(64)
    k, v, table = _cache(rng, [200], 2, 32)
    table = np.repeat(table, 3, axis=0)
    q = _q(3, 8, 2, 64)
    q = q[[0, 0, 2]]
    got, lse = J.paged_decode(q, k.cuda(), v.cuda(), _i32(table), _i32(lengths), want_lse=True)
    _check(got, lse, op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), np.arange(4)))
    assert torch.equal(got[0], got[1])


def test_scores_that_are_not_finite(J):
    """A NaN in a key makes exactly the (token, head) pairs that see it NaN, in sequences that one
    CTA takes and in ones that are cut into parts; keys of -inf (scores of -inf, over whole warps' and
    blocks' positions) have no weight, and where every score is -inf the output is 0 and lse -inf."""
    G, H, P = 2, 8, 32
    rng = np.random.default_rng(71)
    lengths = [40, 1500, 90, 700, 300]
    k, v, table = _cache(rng, lengths, G, P)

    def key(s, g, pos):
        return k[table[s, pos // P], g, pos % P]

    new = [3, 300, 1, 2, 300]
    qs = np.concatenate([[0], np.cumsum(new)])
    q = _q(qs[-1], H, G, 71)
    q[:, :, 0] = q[:, :, 0].abs() + 0.25           # against -inf in a key: a score of -inf
    bad = {(0, 0): 5, (1, 1): 1251, (3, 0): 699}   # (sequence, KV head): position
    for (s, g), pos in bad.items():
        key(s, g, pos)[7] = NAN
    for pos in list(range(0, 256)) + list(range(272, 288)) + [1499]:
        key(1, 0, pos)[0] = -float("inf")
    for pos in range(90):
        key(2, 1, pos)[0] = -float("inf")
    for pos in range(300):
        key(4, 0, pos)[0] = -float("inf")
    kc, vc, tab, lens = k.cuda(), v.cuda(), _i32(table), _i32(lengths)
    ko = to_np(k)
    for (s, g), pos in bad.items():                # the oracle's own answer where nothing is NaN
        ko[table[s, pos // P], g, pos % P, 7] = 0.0
    rep = H // G
    for ragged in (False, True):
        start = qs if ragged else np.arange(len(lengths) + 1)
        rows = np.arange(qs[-1]) if ragged else qs[1:] - 1
        qq = q[torch.tensor(rows, device="cuda")] if not ragged else q
        if ragged:
            got, lse = J.paged_extend(qq, kc, vc, tab, lens, _i32(start), want_lse=True)
        else:
            got, lse = J.paged_decode(qq, kc, vc, tab, lens, want_lse=True)
        with np.errstate(invalid="ignore"):
            want = op.attention(to_np(qq), ko, to_np(v), table, np.array(lengths), start)
        o, z = to_np(got), to_np(lse)
        for s, n in enumerate(lengths):
            for t in range(start[s], start[s + 1]):
                pos = n - start[s + 1] + t
                for h in range(H):
                    g = h // rep
                    if bad.get((s, g), n) <= pos:
                        assert np.isnan(o[t, h]).all() and np.isnan(z[t, h]), (ragged, s, t, h)
                    elif (s, g) in ((2, 1), (4, 0)):
                        assert (o[t, h] == 0).all() and np.isneginf(z[t, h]), (ragged, s, t, h)
                    else:
                        err = np.abs(o[t, h] - want["o"][t, h])
                        assert (err <= TOL_O * want["spread"][t, h]).all(), (ragged, s, t, h)
                        assert abs(z[t, h] - want["lse"][t, h]) <= 2.0 ** -12 + 2.0 ** -22 * abs(want["lse"][t, h])


@pytest.mark.parametrize("lengths,new", [([2000, 1300, 130], [3, 300, 130]), ([128], [128]), ([40, 129, 700], [1, 1, 1])])
def test_scores_far_from_zero(J, lengths, new):
    """Heads whose scores all lie near 181, 45, 0, -45 and -181 (times log2 e: 261, 65, ...), within a first block
    and in later ones, keys of the second half further off by as much again: no reference fits both halves.

    Tolerance: the large product is exact, so the scores' error is that of adding 127 small products to at most
    2 * 2048, half a step of 2^-11 each: 127 * 2^-12 / sqrt(128) < 2^-8.4, on a term and on the sum, 2^-7.4 beside
    TOL_O; of the lse once, beside fp32's rounding of it."""
    G, H, P = 2, 16, 64
    rng = np.random.default_rng(81)
    k, v, table = _cache(rng, lengths, G, P)
    q = _q(sum(new), H, G, 81)
    q[:, :, 0] = torch.tensor([8.0, 2.0, 0.0, -2.0, -8.0, 8.0, -8.0, 0.25] * 2, device="cuda", dtype=BF)
    for s, n in enumerate(lengths):
        for pos in range(n):
            k[table[s, pos // P], :, pos % P, 0] = 256.0 if pos < n // 2 else 512.0
    start = np.concatenate([[0], np.cumsum(new)])
    args = (k.cuda(), v.cuda(), _i32(table), _i32(lengths))
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    last = start[1:] - 1
    for got, lse, rows in (J.paged_extend(q, *args, _i32(start), want_lse=True) + (np.arange(sum(new)),),
                           J.paged_decode(q[torch.tensor(last, device="cuda")], *args, want_lse=True) + (last,)):
        err = np.abs(to_np(got) - want["o"][rows])
        assert (err <= (TOL_O + 2.0 ** -7.4) * want["spread"][rows]).all()
        assert (np.abs(to_np(lse) - want["lse"][rows]) <= 2.0 ** -8.4 + 2.0 ** -20 * np.abs(want["lse"][rows])).all()


# ------------------------------------------------ many short items in one CTA

@pytest.mark.parametrize("H", [64, 128])               # one and two tiles of eight heads
@pytest.mark.parametrize("most", [16, 32])             # half the warps, or three quarters, have no position to look at
def test_decode_many_short_sequences(J, H, most):
    """700 sequences of 0 to 32 tokens, 8 KV heads: a CTA walks some 19 items, each joined through the same shared
    memory as the one before while the faster warps are at the next.  Every repeat gives the same bits."""
    G, P, S = 8, 16, 700
    rng = np.random.default_rng(H + most)
    lengths = rng.integers(0, most + 1, S).tolist()
    k, v, table = _cache(rng, lengths, G, P)
    q = _q(S, H, G, H)
    args = (q, k.cuda(), v.cuda(), _i32(table), _i32(lengths))
    got, lse = J.paged_decode(*args, want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), np.arange(S + 1))
    _check(got, lse, want)
    for _ in range(50):
        again, z = J.paged_decode(*args, want_lse=True)
        assert torch.equal(again, got) and torch.equal(z, lse)


# --------------------------------------------------- one key far from the others

@pytest.mark.parametrize("nats", [134, 198, 282])
@pytest.mark.parametrize("cached,at", [(200, 0), (400, 256)])
def test_extend_one_far_key(J, nats, cached, at):
    """One key of a sequence lies 95, 140 or 200 nats above the others for every row, in turn at each of the
    128 columns of a first unmasked block or of a later one: it has all the weight, in units that one CTA takes
    and in ones that are cut into parts, as in the path of single tokens.

    Tolerance: as in test_scores_far_from_zero; the large product, at most 8 * 282 < 4096, is exact."""
    G, H, P, n = 2, 8, 64, 4
    S = 128
    lengths = [cached + n] * S
    rng = np.random.default_rng(nats + at)
    k, v, table = _cache(rng, lengths, G, P)
    q = _q(S * n, H, G, 91)
    q[:, :, 0] = 8.0
    for s in range(S):
        for pos in range(lengths[s]):
            k[table[s, pos // P], :, pos % P, 0] = float(nats) if pos == at + s else 0.0
    start = np.arange(S + 1) * n
    args = (k.cuda(), v.cuda(), _i32(table), _i32(lengths))
    got, lse = J.paged_extend(q, *args, _i32(start), want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    err = np.abs(to_np(got) - want["o"])
    assert (err <= (TOL_O + 2.0 ** -7.4) * want["spread"]).all()
    assert (np.abs(to_np(lse) - want["lse"]) <= 2.0 ** -8.4 + 2.0 ** -20 * np.abs(want["lse"])).all()


@pytest.mark.parametrize("sign", [1, -1])
def test_extend_far_scores_with_values_of_any_size(J, sign):
    """Scores 37 nats above the reference with values around 2^80, and 37 nats below it with values around 2^-80:
    neither the terms nor their products leave fp32's range.

    Tolerance: as in test_scores_far_from_zero; the large product, 8 * 52, is exact and below 512, so the scores'
    error is below 127 * 2^-15 / sqrt(128) < 2^-8.4 all the more."""
    G, H, P, n = 2, 8, 64, 4
    lengths = [300, 1300, 90, 2000]
    S = len(lengths)
    rng = np.random.default_rng(95)
    k, v, table = _cache(rng, lengths, G, P)
    v = v * 2.0 ** (80 * sign)
    q = _q(S * n, H, G, 95)
    q[:, :, 0] = 8.0
    for s in range(S):
        for pos in range(lengths[s]):
            k[table[s, pos // P], :, pos % P, 0] = 52.0 * sign
    start = np.arange(S + 1) * n
    args = (k.cuda(), v.cuda(), _i32(table), _i32(lengths))
    got, lse = J.paged_extend(q, *args, _i32(start), want_lse=True)
    want = op.attention(to_np(q), to_np(k), to_np(v), table, np.array(lengths), start)
    err = np.abs(to_np(got) - want["o"])
    assert (err <= (TOL_O + 2.0 ** -7.4) * want["spread"]).all()
    assert (np.abs(to_np(lse) - want["lse"]) <= 2.0 ** -8.4 + 2.0 ** -20 * np.abs(want["lse"])).all()


# ------------------------------------------------------ slots that take no part

def _full_pool(J, seed):
    """Two slots that share the pages of a prompt of 40, a third of 16 of its own: no page is left, so neither of
    the first two can take a copy of the shared last page."""
    att, p = _layer(J)
    cache = J.PagedKVCache(layers=1, n_kv_heads=2, num_pages=4, max_seqs=4, max_len=64, page_size=16)
    x = attn_input(SH, 1, 64, seed=seed)[0].cuda()
    assert cache.grow(_i32([40, 0, 8, 0])).tolist() == [1] * 4
    att.paged_prefill(x[:48], _i32([0, 40, 40, 48, 48]), cache)
    cache.fork(_i32([0, 0, 2, 3]))
    return att, p, cache, x


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_refused_slots_and_slots_without_a_token_keep_their_rows(J, ragged, captured):
    """A pool that runs dry under two forks, with a slot that grows, an empty one, and then with no slot growing: with
    active = granted * add no row changes but the new one's, eagerly and in a graph; the slots left out get the residual."""
    att, p, cache, x = _full_pool(J, 97)
    add = _i32([1, 1, 1, 0])
    new = x[48:52].contiguous()
    q_start = _i32([0, 1, 2, 3, 4])

    def turn():
        granted = cache.grow(add)
        args = dict(cache=cache, residual=new, active=granted * add)
        return granted, att.paged_prefill(new, q_start, **args) if ragged else att.paged_step(new, **args)

    before = cache.data.clone()
    J.device_status()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            granted, out = turn()
        graph.replay()
    else:
        granted, out = turn()
    assert granted.tolist() == [0, 0, 1, 1] and cache.lengths.tolist() == [40, 40, 9, 0]
    changed = (cache.data != before).any(-1).nonzero().tolist()
    page = int(cache.table[2, 0])
    assert sorted(changed) == [[plane, page, g, 8] for plane in range(2) for g in range(2)]
    assert torch.equal(out[[0, 1, 3]], new[[0, 1, 3]]) and not torch.equal(out[2], new[2])
    want = oatt.attention_prefill(p, to_np(torch.cat([x[40:48], x[50:51]])[None]), SH)["out"][0, -1]
    assert rel_l2(to_np(out[2]), want + to_np(new[2])) < TOL_BF16
    add.zero_()                                          # live slots without a token
    before = cache.data.clone()
    if captured:
        graph.replay()
    else:
        granted, out = turn()
    assert granted.tolist() == [1] * 4 and torch.equal(cache.data, before) and torch.equal(out, new)


def test_active_lengths(J):
    n = 1000
    lengths, active = torch.arange(n, dtype=torch.int32, device="cuda"), _i32(np.arange(n) % 4 - 1)
    want = torch.where(active > 0, lengths, 0)
    assert torch.equal(J.pages_active(active, lengths), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = J.pages_active(active, lengths, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for a, ln in ((active[:5], lengths), (active.long(), lengths), (active[::2], lengths[::2]), (active.cpu(), lengths),
                  (active[None], lengths[None])):
        with pytest.raises(ValueError):
            J.pages_active(a, ln)
    att, _, cache, x = _full_pool(J, 98)
    with pytest.raises(ValueError):
        att.paged_step(x[:4].contiguous(), cache, active=torch.ones(4, dtype=torch.bool, device="cuda"))


def test_free_in_a_graph(J):
    """free captured with grow: each replay frees the same slots and gives their pages to the next prompts."""
    cache = J.PagedKVCache(layers=1, n_kv_heads=2, num_pages=10, max_seqs=3, max_len=64, page_size=16)
    add = _i32([20, 30, 5])
    cache.grow(add)
    cache.free([0, 2])                                    # eagerly
    assert cache.lengths.tolist() == [0, 30, 0] and int((cache.refs > 0).sum()) == 2
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.free(2)
        cache.free([0, 1])
        granted = cache.grow(add)
    for _ in range(3):
        graph.replay()
        assert granted.tolist() == [1, 1, 1] and cache.lengths.tolist() == [20, 30, 5]
        assert int((cache.refs > 0).sum()) == 5 and int(cache.refs.sum()) == 5


def test_grow_where_the_pages_wanted_pass_32_bits(J):
    """65536 slots that want 32769 pages each, more than 2^31 in all, of a pool of 8: every one is refused, whatever
    its rank, and slots that want one page or none are not, before them and after."""
    S, W, P, N = 1 << 16, (1 << 15) + 1, 16, 8
    table = torch.empty(S, W, dtype=torch.int32, device="cuda")      # 8.6 GB; a slot of length 0 holds no entry
    lengths, refs = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    data = torch.zeros(2, N, 1, P, 128, dtype=BF, device="cuda")
    add = torch.full((S,), W * P, dtype=torch.int32, device="cuda")
    add[:3], add[S - 2:] = 10, 0
    granted = J.pages_grow(add, data, refs, table, lengths)
    assert (granted.nonzero()[:, 0].tolist() == [0, 1, 2, S - 2, S - 1]) and refs.tolist() == [1] * 3 + [0] * 5
    assert lengths.nonzero()[:, 0].tolist() == [0, 1, 2] and table[:3, 0].tolist() == [0, 1, 2]
