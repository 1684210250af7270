"""The paged key-value cache without a GPU: pins of its oracle, and what the C
entry points and the binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as op


@pytest.fixture(scope="module")
def lib():
    from mamba_selective_scan_mixer_b200 import build, _abi
    build.build()
    return _abi.lib()


def _holders(table, lengths, n, page):
    c = np.zeros(n, dtype=int)
    for s, length in enumerate(lengths):
        for j in range(op.held(length, page)):
            c[table[s, j]] += 1
    return c


def test_upkeep_counts_holders_and_keeps_contents():
    rng = np.random.default_rng(3)
    N, S, W, P = 40, 6, 8, 4
    data = np.zeros((2, N, 1, P, 2))
    refs, table, lengths = np.zeros(N, dtype=int), np.full((S, W), -1), np.zeros(S, dtype=int)
    said = [[] for _ in range(S)]          # what each sequence was given, token by token
    for turn in range(200):
        parent = np.arange(S)
        for s in rng.choice(S, 2, replace=False):
            parent[s] = rng.integers(-1, S)
        op.fork(parent, refs, table, lengths, P)
        said = [list(said[p]) if p >= 0 else [] for p in parent]
        add = rng.integers(0, 6, S)
        before = lengths.copy()
        granted = op.grow(add, data, refs, table, lengths)
        for s in range(S):
            if granted[s]:
                assert lengths[s] == before[s] + add[s]
                for pos in range(before[s], lengths[s]):
                    value = rng.normal()
                    data[:, table[s, pos // P], 0, pos % P] = value
                    said[s].append(value)
            else:
                assert lengths[s] == before[s]
        if turn % 7 == 0:
            op.compact(data, refs, table, lengths)
            live = int((refs > 0).sum())
            assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
        assert (refs == _holders(table, lengths, N, P)).all()
        for s in range(S):
            assert op.rows(data[0], table[s], lengths[s])[:, 0, 0].tolist() == said[s]


def test_oracle_attention_equals_contiguous_attention():
    rng = np.random.default_rng(4)
    P, G, H, D = 4, 2, 4, 8
    lengths, new = [9, 0, 5, 1], [3, 0, 5, 1]
    table = np.full((4, 3), -1)
    table[0], table[2, :2], table[3, 0] = [5, 1, 7], [0, 3], 2
    k, v = rng.normal(size=(2, 8, G, P, D))
    starts = np.concatenate([[0], np.cumsum(new)])
    q = rng.normal(size=(starts[-1], H, D))
    got = op.attention(q, k, v, table, lengths, starts)
    for s in range(4):
        a, b = starts[s], starts[s + 1]
        if b > a:
            want = op.contiguous(q[a:b], op.rows(k, table[s], lengths[s]), op.rows(v, table[s], lengths[s]))
            np.testing.assert_allclose(got["o"][a:b], want, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(got["lse"][-1], np.einsum("hd,hd->h", q[-1], np.repeat(k[2, :, 0], 2, 0)) / np.sqrt(D))


def test_entry_points_refuse_before_a_launch(lib):
    from mamba_selective_scan_mixer_b200 import _abi
    BF = _abi.JAMBA_BF16
    n = ctypes.c_size_t()
    p, q, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21), ctypes.c_void_p((1 << 20) + 4)
    fields = dict(num_pages=64, page_size=64, n_kv_heads=8, head_dim=128, planes=2, max_seqs=4, max_pages=16,
                  ld_table=16, dtype=BF)
    cfg = lambda **kw: ctypes.byref(_abi.PagesConfig(**dict(fields, **kw)))  # noqa: E731
    good = cfg()
    assert lib.jamba_pages_workspace_size(good, ctypes.byref(n)) == 0 and n.value >= 4 * 16 * 4
    for kw, code in ((dict(num_pages=0), 1), (dict(max_seqs=0), 1), (dict(max_pages=-1), 1), (dict(n_kv_heads=0), 1),
                     (dict(ld_table=15), 1), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
                     (dict(head_dim=64), 2), (dict(dtype=_abi.JAMBA_F32), 2), (dict(max_pages=1 << 28, ld_table=1 << 28), 2),
                     (dict(num_pages=1 << 28), 2), (dict(n_kv_heads=2000), 2)):
        assert lib.jamba_pages_workspace_size(cfg(**kw), ctypes.byref(n)) == code, kw
    assert lib.jamba_pages_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.jamba_pages_workspace_size(good, None) == 1
    big = 1 << 30
    assert lib.jamba_pages_fork(good, None, p, p, p, p, big, None) == 1
    assert lib.jamba_pages_fork(good, p, odd, p, p, p, big, None) == 1          # refs are read 16 bytes at a time
    assert lib.jamba_pages_fork(good, p, p, p, p, p, 16, None) == 3
    assert lib.jamba_pages_grow(good, p, None, p, p, p, p, p, big, None) == 1
    assert lib.jamba_pages_grow(good, p, p, p, p, p, None, p, big, None) == 1
    assert lib.jamba_pages_grow(cfg(planes=0), p, p, p, p, p, p, p, big, None) == 1
    assert lib.jamba_pages_grow(good, p, p, p, p, p, p, p, 16, None) == 3
    assert lib.jamba_pages_compact(good, p, p, p, p, None, p, big, None) == 1
    assert lib.jamba_pages_compact(good, p, p, p, p, p, p, 16, None) == 3
    # append: a stride that does not hold the heads, one that is no multiple of 8, tokens without q_start
    assert lib.jamba_paged_append(good, p, p, 1023, 4, None, p, p, p, p, None) == 1
    assert lib.jamba_paged_append(good, p, p, 1028, 4, None, p, p, p, p, None) == 1
    assert lib.jamba_paged_append(good, p, p, 1024, 5, None, p, p, p, p, None) == 1
    assert lib.jamba_paged_append(good, p, p, 1024, -1, p, p, p, p, p, None) == 1
    assert lib.jamba_paged_append(good, odd, p, 1024, 4, None, p, p, p, p, None) == 1
    # attention
    assert lib.jamba_paged_decode_workspace_size(good, 32, ctypes.byref(n)) == 0
    assert lib.jamba_paged_decode_workspace_size(good, 30, ctypes.byref(n)) == 1
    assert lib.jamba_paged_decode_workspace_size(good, 8 * 17, ctypes.byref(n)) == 2
    assert lib.jamba_paged_extend_workspace_size(good, 8 * 128, 100, ctypes.byref(n)) == 0
    assert lib.jamba_paged_extend_workspace_size(good, 8 * 129, 100, ctypes.byref(n)) == 2
    assert lib.jamba_paged_extend_workspace_size(good, 32, -1, ctypes.byref(n)) == 1
    dec = lambda c=good, h=32, qq=p, ld=4096, k=p, o=q, ldo=4096, ws=p, nb=big: lib.jamba_paged_decode(  # noqa: E731
        c, h, qq, ld, k, p, p, p, o, ldo, None, ws, nb, None)
    assert dec(o=p) == 1                       # o may not be q
    assert dec(ld=4095) == 1 and dec(ldo=4088) == 1 and dec(qq=odd) == 1 and dec(k=None) == 1
    assert dec(nb=8) == 3
    assert lib.jamba_paged_extend(good, 32, p, 4096, 10, None, p, p, p, p, q, 4096, None, p, big, None) == 1
    # the layer: another number of KV heads, too many heads for the step, out aliasing x
    acfg = _abi.AttnConfig(4096, 32, 8, 128, BF)
    a = ctypes.byref(acfg)
    w = ctypes.byref(_abi.AttnWeights(p, p))
    assert lib.jamba_attn_paged_step_workspace_size(a, good, ctypes.byref(n)) == 0
    assert lib.jamba_attn_paged_step_workspace_size(a, cfg(n_kv_heads=4), ctypes.byref(n)) == 1
    assert lib.jamba_attn_paged_step_workspace_size(a, None, ctypes.byref(n)) == 1
    wide = ctypes.byref(_abi.AttnConfig(4096, 136, 8, 128, BF))
    assert lib.jamba_attn_paged_step_workspace_size(wide, good, ctypes.byref(n)) == 2
    assert lib.jamba_attn_paged_prefill_workspace_size(wide, good, 64, ctypes.byref(n)) == 0
    assert lib.jamba_attn_paged_step(a, w, good, p, None, p, p, p, p, p, p, big, None) == 1
    assert lib.jamba_attn_paged_prefill(a, w, good, p, None, q, 0, p, p, p, p, p, p, big, None) == 1
    assert lib.jamba_attn_paged_prefill(a, w, good, p, None, q, 8, None, p, p, p, p, p, big, None) == 1


def test_binding_refuses_host_tensors():
    import mamba_selective_scan_mixer_b200 as J
    bf, i32 = torch.bfloat16, torch.int32
    pages, table, lengths = torch.zeros(4, 2, 16, 128, dtype=bf), torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    q, refs = torch.zeros(2, 4, 128, dtype=bf), torch.zeros(4, dtype=i32)
    for call in (lambda: J.paged_decode(q, pages, pages, table, lengths),
                 lambda: J.paged_extend(q, pages, pages, table, lengths, torch.zeros(3, dtype=i32)),
                 lambda: J.paged_append(q[:, :2], q[:, :2], pages, pages, table, lengths),
                 lambda: J.pages_fork(lengths, refs, table, lengths, 16),
                 lambda: J.pages_grow(lengths, pages[None], refs, table, lengths),
                 lambda: J.pages_compact(pages[None], refs, table, lengths)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_active_lengths_refuse_before_a_launch(lib):
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
    for args in ((0, p, p, p), ((1 << 20) + 1, p, p, p), (4, None, p, p), (4, p, odd, p), (4, p, p, None)):
        assert lib.jamba_pages_active(*args, None) == 1, args


def test_outputs_that_overlap_queries_are_refused(lib):
    """Views of one buffer: every pair of rows is compared by brute force; a call that does not overlap is
    stopped by its workspace, before a launch."""
    from mamba_selective_scan_mixer_b200 import _abi
    base = 1 << 24
    H = 2
    row = H * 128                                        # elements
    rng = np.random.default_rng(7)
    seen = set()
    for _ in range(3000):
        T = int(rng.integers(1, 7))
        ldq = int(rng.choice([row, row + 8, row + 64, 2 * row, 3 * row, 5 * row]))
        ldo = ldq if rng.random() < 0.5 else int(rng.choice([row, row + 8, 2 * row, 4 * row]))
        off = int(rng.integers(-6 * 5 * row // 8, 6 * 5 * row // 8)) * 8
        if rng.random() < 0.5:
            off = off // row * row
        starts_q, starts_o = np.arange(T) * ldq, off + np.arange(T) * ldo
        overlap = bool((np.abs(starts_q[:, None] - starts_o[None]) < row).any())
        cfg = _abi.PagesConfig(64, 64, 2, 128, 2, T, 16, 16, _abi.JAMBA_BF16)
        v = ctypes.c_void_p
        q, o, p = v(base), v(base + 2 * off), v(1 << 20)
        want = 1 if overlap else 3
        st = lib.jamba_paged_decode(ctypes.byref(cfg), H, q, ldq, p, p, p, p, o, ldo, None, p, 0, None)
        assert st == want, (T, ldq, ldo, off)
        st = lib.jamba_paged_extend(ctypes.byref(cfg), H, q, ldq, T, p, p, p, p, p, o, ldo, None, p, 0, None)
        assert st == want, (T, ldq, ldo, off)
        seen.add((overlap, ldq == ldo))
    assert len(seen) == 4
