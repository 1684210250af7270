"""The paged key-value cache: torch-tensor front end of the jamba_pages_* and
jamba_paged_* entry points (marshalling only).

Pages of a plane are [num_pages, n_kv_heads, page_size, 128] bf16; the pool of a
model holds the keys and values of each attention layer as planes of one tensor
[planes, num_pages, n_kv_heads, page_size, 128] under one page numbering.
refs [num_pages], table [max_seqs, max_pages] and lengths [max_seqs] are int32
on the same device.  Calls run on the tensors' device and on `stream` (default:
that device's current stream); outputs and workspaces are allocated on that
stream, per call, so calls on several streams and captured graphs share none.
"""
import ctypes

import torch

from . import _abi
from ._abi import check, lib

HEAD_DIM = 128


class _Call:
    """The device and stream of one call: entered, both are current, so that
    allocations and launches go there."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        self.guards = []
        if torch.cuda.current_device() != self.device.index:
            self.guards.append(torch.cuda.device(self.device))
        if self.stream is not None:
            self.guards.append(torch.cuda.stream(self.stream))
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _same_device(first, named):
    if not first.is_cuda:
        raise ValueError("libjamba works on CUDA tensors only")
    for name, t in named:
        if not t.is_cuda:
            raise ValueError("libjamba works on CUDA tensors only")
        if t.device != first.device:
            raise ValueError("%s is on %s, the pages on %s" % (name, t.device, first.device))


def _ints(t, name, shape):
    if t.dtype != torch.int32:
        raise ValueError("%s must be int32" % name)
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s" % (name, list(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _config(num_pages, n_kv_heads, page_size, planes, table, lengths):
    if table.dim() != 2 or table.dtype != torch.int32 or (table.numel() and table.stride(1) != 1):
        raise ValueError("table must be int32 [max_seqs, max_pages] with unit-stride rows")
    S, W = table.shape
    _ints(lengths, "lengths", (S,))
    return _abi.PagesConfig(num_pages, page_size, n_kv_heads, HEAD_DIM, planes, S, W,
                            table.stride(0) if S > 1 else W, _abi.JAMBA_BF16)


def _planes(k_pages, v_pages):
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.dim() != 4 or t.shape[3] != HEAD_DIM or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("%s must be contiguous bf16 [num_pages, n_kv_heads, page_size, 128]" % name)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")


def _rows(t, name, heads=None):
    """The token stride of t [tokens, heads, 128], its heads next to one another."""
    if t.dim() != 3 or t.shape[2] != HEAD_DIM or t.dtype != torch.bfloat16 or (heads and t.shape[1] != heads):
        raise ValueError("%s must be bf16 [tokens, %s, 128]" % (name, heads or "heads"))
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != HEAD_DIM)):
        raise ValueError("%s must have its heads next to one another" % name)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * HEAD_DIM


def _p(t):
    return None if t is None else t.data_ptr()


def _pool(data, refs, table, lengths):
    if data.dim() != 5 or data.shape[4] != HEAD_DIM or data.dtype != torch.bfloat16 or not data.is_contiguous():
        raise ValueError("data must be contiguous bf16 [planes, num_pages, n_kv_heads, page_size, 128]")
    _same_device(data, (("refs", refs), ("table", table), ("lengths", lengths)))
    planes, N, G, P, _ = data.shape
    _ints(refs, "refs", (N,))
    return _config(N, G, P, planes, table, lengths)


def _upkeep_workspace(cfg, device):
    n = ctypes.c_size_t()
    check(lib().jamba_pages_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def pages_fork(parent, refs, table, lengths, page_size, stream=None):
    """Slot s becomes a fork of slot parent[s] (sharing its pages), stays with
    parent[s] = s, or is freed with parent[s] = -1; all at once, in place."""
    _same_device(table, (("parent", parent), ("refs", refs), ("lengths", lengths)))
    if refs.dim() != 1:
        raise ValueError("refs must have shape [num_pages]")
    _ints(refs, "refs", (refs.shape[0],))
    cfg = _config(refs.shape[0], 1, page_size, 1, table, lengths)
    _ints(parent, "parent", (table.shape[0],))
    with _Call(table.device, stream) as st:
        ws = _upkeep_workspace(cfg, table.device)
        check(lib().jamba_pages_fork(ctypes.byref(cfg), _p(parent), _p(refs), _p(table), _p(lengths), _p(ws),
                                     ws.numel(), st))


def pages_grow(add, data, refs, table, lengths, stream=None):
    """Room for add[s] more tokens in every slot, counted into lengths; a shared
    last page is copied first.  Returns granted [max_seqs] int32 (0: refused,
    the slot is as it was)."""
    cfg = _pool(data, refs, table, lengths)
    _same_device(data, (("add", add),))
    _ints(add, "add", (table.shape[0],))
    with _Call(data.device, stream) as st:
        ws = _upkeep_workspace(cfg, data.device)
        granted = torch.empty(table.shape[0], dtype=torch.int32, device=data.device)
        check(lib().jamba_pages_grow(ctypes.byref(cfg), _p(add), _p(data), _p(refs), _p(table), _p(lengths),
                                     _p(granted), _p(ws), ws.numel(), st))
    return granted


def pages_compact(data, refs, table, lengths, stream=None):
    """Moves the live pages to the front of the pool.  Returns remap [num_pages]
    int32: each live page's new number, -1 for free pages."""
    cfg = _pool(data, refs, table, lengths)
    with _Call(data.device, stream) as st:
        ws = _upkeep_workspace(cfg, data.device)
        remap = torch.empty(data.shape[1], dtype=torch.int32, device=data.device)
        check(lib().jamba_pages_compact(ctypes.byref(cfg), _p(data), _p(refs), _p(table), _p(lengths), _p(remap),
                                        _p(ws), ws.numel(), st))
    return remap


def paged_append(k, v, k_pages, v_pages, table, lengths, q_start=None, stream=None):
    """Keys and values k, v [tokens, n_kv_heads, 128] of the sequences' last
    tokens into their pages: sequence s has rows q_start[s] .. q_start[s+1] - 1
    (q_start [max_seqs + 1] int32), or one row each without q_start."""
    _planes(k_pages, v_pages)
    named = [("k", k), ("v", v), ("v_pages", v_pages), ("table", table), ("lengths", lengths)]
    _same_device(k_pages, named + ([("q_start", q_start)] if q_start is not None else []))
    N, G, P, _ = k_pages.shape
    cfg = _config(N, G, P, 1, table, lengths)
    ld = _rows(k, "k", G)
    if _rows(v, "v", G) != ld or v.shape != k.shape:
        raise ValueError("k and v must have one shape and one token stride")
    if q_start is not None:
        _ints(q_start, "q_start", (table.shape[0] + 1,))
    if k.shape[0] == 0 and q_start is not None:
        return
    with _Call(k_pages.device, stream) as st:
        check(lib().jamba_paged_append(ctypes.byref(cfg), _p(k), _p(v), ld, k.shape[0], _p(q_start), _p(k_pages),
                                       _p(v_pages), _p(table), _p(lengths), st))


def _attend(q, k_pages, v_pages, table, lengths, q_start, out, want_lse, stream):
    _planes(k_pages, v_pages)
    named = [("q", q), ("v_pages", v_pages), ("table", table), ("lengths", lengths)]
    named += [(n, t) for n, t in (("q_start", q_start), ("out", out)) if t is not None]
    _same_device(k_pages, named)
    N, G, P, _ = k_pages.shape
    cfg = _config(N, G, P, 1, table, lengths)
    S = table.shape[0]
    ld = _rows(q, "q")
    T, H, _ = q.shape
    if q_start is not None:
        _ints(q_start, "q_start", (S + 1,))
    elif T != S:
        raise ValueError("q must hold one token for each of the %d slots" % S)
    L = lib()
    n = ctypes.c_size_t()
    with _Call(k_pages.device, stream) as st:
        if out is None:
            out = torch.empty(T, H, HEAD_DIM, dtype=q.dtype, device=q.device)
        elif out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        ld_o = _rows(out, "out")
        lse = torch.empty(T, H, dtype=torch.float32, device=q.device) if want_lse else None
        if T:
            if q_start is None:
                check(L.jamba_paged_decode_workspace_size(ctypes.byref(cfg), H, ctypes.byref(n)))
            else:
                check(L.jamba_paged_extend_workspace_size(ctypes.byref(cfg), H, T, ctypes.byref(n)))
            ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device=q.device)
            if q_start is None:
                check(L.jamba_paged_decode(ctypes.byref(cfg), H, _p(q), ld, _p(k_pages), _p(v_pages), _p(table),
                                           _p(lengths), _p(out), ld_o, _p(lse), _p(ws), ws.numel(), st))
            else:
                check(L.jamba_paged_extend(ctypes.byref(cfg), H, _p(q), ld, T, _p(q_start), _p(k_pages),
                                           _p(v_pages), _p(table), _p(lengths), _p(out), ld_o, _p(lse), _p(ws),
                                           ws.numel(), st))
    return (out, lse) if want_lse else out


def paged_decode(q, k_pages, v_pages, table, lengths, out=None, want_lse=False, stream=None):
    """Attention of one new token per slot, q [max_seqs, heads, 128], over its
    sequence's pages.  Returns out like q, with want_lse (out, lse [max_seqs,
    heads] fp32).  A slot of length 0 gets 0 and -inf."""
    return _attend(q, k_pages, v_pages, table, lengths, None, out, want_lse, stream)


def paged_extend(q, k_pages, v_pages, table, lengths, q_start, out=None, want_lse=False, stream=None):
    """Causal attention of the sequences' last tokens, q [tokens, heads, 128]
    (rows q_start[s] .. q_start[s+1] - 1 are sequence s's), over their pages.
    Returns out like q, with want_lse (out, lse [tokens, heads] fp32)."""
    if q_start is None:
        raise ValueError("paged_extend needs q_start")
    return _attend(q, k_pages, v_pages, table, lengths, q_start, out, want_lse, stream)


class PagedKVCache:
    """Keys and values of `layers` attention layers for up to max_seqs sequences
    of up to max_len tokens, in num_pages pages of page_size tokens.

    A turn of a server: fork / free the slots that change, grow by the tokens
    each slot brings (granted says which could), then Attention.paged_prefill or
    paged_step of every layer, which write the new keys and values and attend.
    """

    def __init__(self, layers, n_kv_heads, num_pages, max_seqs, max_len, page_size=64, device="cuda"):
        self.layers, self.page_size = layers, page_size
        self.data = torch.zeros(2 * layers, num_pages, n_kv_heads, page_size, HEAD_DIM, dtype=torch.bfloat16,
                                device=device)
        dev = self.data.device
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=dev)
        self.table = torch.full((max_seqs, -(-max_len // page_size)), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(max_seqs, dtype=torch.int32, device=dev)

    def keys(self, layer):
        return self.data[2 * layer]

    def values(self, layer):
        return self.data[2 * layer + 1]

    def fork(self, parent, stream=None):
        """See pages_fork."""
        pages_fork(parent, self.refs, self.table, self.lengths, self.page_size, stream=stream)

    def free(self, slots, stream=None):
        """Frees slots (an index or a list of them)."""
        parent = list(range(self.table.shape[0]))
        for s in [slots] if isinstance(slots, int) else slots:
            if not 0 <= s < len(parent):
                raise ValueError("slot %d is outside 0 .. %d" % (s, len(parent) - 1))
            parent[s] = -1
        with _Call(self.table.device, stream):
            self.fork(torch.tensor(parent, dtype=torch.int32, device=self.table.device), stream=stream)

    def grow(self, add, stream=None):
        """See pages_grow."""
        return pages_grow(add, self.data, self.refs, self.table, self.lengths, stream=stream)

    def compact(self, stream=None):
        """See pages_compact."""
        return pages_compact(self.data, self.refs, self.table, self.lengths, stream=stream)

    def config(self, layer):
        """(jamba_pages_config of one layer, its keys, its values)."""
        if not 0 <= layer < self.layers:
            raise ValueError("layer %d is outside 0 .. %d" % (layer, self.layers - 1))
        _, N, G, P, _ = self.data.shape
        return _config(N, G, P, 1, self.table, self.lengths), self.keys(layer), self.values(layer)
