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
import functools

import torch

from . import _abi
from ._abi import check, lib

HEAD_DIM = 128
_BF16 = torch.bfloat16
_raw_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """Makes a device and a stream current, so that allocations and launches go there."""

    def __init__(self, index, stream):
        self.index, self.stream = index, stream

    def __enter__(self):
        self.guards = [torch.cuda.device(self.index)]
        if self.stream is not None:
            self.guards.append(torch.cuda.stream(self.stream))
        for g in self.guards:
            g.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _run(index, stream, body, *args):
    """body(raw stream, *args) on device `index` and `stream` (None: the device's current one)."""
    if stream is None and torch.cuda.current_device() == index:
        return body(_raw_stream(index), *args)
    with _On(index, stream) as raw:
        return body(raw, *args)


def _same_device(first, named):
    """The index of the CUDA device that all are on."""
    index = first.get_device()
    for name, t in named:
        if t.get_device() != index:
            if index < 0 or not t.is_cuda:
                raise ValueError("libjamba works on CUDA tensors only")
            raise ValueError("%s is on %s, the pages on %s" % (name, t.device, first.device))
    if index < 0:
        raise ValueError("libjamba works on CUDA tensors only")
    return index


def _ints(t, name, shape):
    if t.dtype != torch.int32:
        raise ValueError("%s must be int32" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s" % (name, list(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


class _Sizes:
    """A jamba_pages_config, by reference, and the workspace bytes asked for with it."""

    def __init__(self, *fields):
        self.ref = ctypes.byref(_abi.PagesConfig(*fields))
        self.known = {}

    def workspace(self, index, size_of, *args):
        """What entry point `size_of` says for these sizes on the current device, number `index`."""
        key = (index, size_of) + args
        found = self.known.get(key)
        if found is None:
            if len(self.known) >= 256:
                self.known.clear()
            n = ctypes.c_size_t()
            check(getattr(lib(), size_of)(self.ref, *args, ctypes.byref(n)))
            found = self.known[key] = max(n.value, 16)
        return found


_sizes = functools.lru_cache(maxsize=1024)(_Sizes)


def _config(num_pages, n_kv_heads, page_size, planes, table, lengths):
    if table.dim() != 2 or table.dtype != torch.int32:
        raise ValueError("table must be int32 [max_seqs, max_pages] with unit-stride rows")
    S, W = table.shape
    ld, one = table.stride()
    if one != 1 and W > 1:
        raise ValueError("table must be int32 [max_seqs, max_pages] with unit-stride rows")
    _ints(lengths, "lengths", (S,))
    return _sizes(num_pages, page_size, n_kv_heads, HEAD_DIM, planes, S, W, ld if S > 1 else W, _abi.JAMBA_BF16)


def _planes(k_pages, v_pages):
    """Their shape [num_pages, n_kv_heads, page_size, 128]."""
    shape = k_pages.shape
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.dtype != _BF16 or len(shape) != 4 or shape[3] != HEAD_DIM or not t.is_contiguous():
            raise ValueError("%s must be contiguous bf16 [num_pages, n_kv_heads, page_size, 128]" % name)
    if v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must have one shape")
    return shape


def _rows(t, name, heads=None):
    """(tokens, heads, token stride) of t [tokens, heads, 128], its heads next to one another."""
    shape = t.shape
    if t.dtype != _BF16 or len(shape) != 3 or shape[2] != HEAD_DIM or (heads and shape[1] != heads):
        raise ValueError("%s must be bf16 [tokens, %s, 128]" % (name, heads or "heads"))
    T, H, _ = shape
    ld, head, one = t.stride()
    if T and H and (one != 1 or (H > 1 and head != HEAD_DIM)):
        raise ValueError("%s must have its heads next to one another" % name)
    return T, H, ld if T > 1 else H * HEAD_DIM


def _p(t):
    return None if t is None else t.data_ptr()


def _pool(data, refs, table, lengths, *named):
    shape = data.shape
    if data.dtype != _BF16 or len(shape) != 5 or shape[4] != HEAD_DIM or not data.is_contiguous():
        raise ValueError("data must be contiguous bf16 [planes, num_pages, n_kv_heads, page_size, 128]")
    index = _same_device(data, (("refs", refs), ("table", table), ("lengths", lengths)) + named)
    planes, N, G, P, _ = shape
    _ints(refs, "refs", (N,))
    return index, _config(N, G, P, planes, table, lengths)


def _upkeep_workspace(cfg, device):
    return torch.empty(cfg.workspace(device.index, "jamba_pages_workspace_size"), dtype=torch.uint8, device=device)


def pages_fork(parent, refs, table, lengths, page_size, stream=None):
    """Slot s becomes a fork of slot parent[s] (sharing its pages), stays with
    parent[s] = s, or is freed with parent[s] = -1; all at once, in place."""
    index = _same_device(table, (("parent", parent), ("refs", refs), ("lengths", lengths)))
    if refs.dim() != 1:
        raise ValueError("refs must have shape [num_pages]")
    _ints(refs, "refs", refs.shape)
    cfg = _config(refs.shape[0], 1, page_size, 1, table, lengths)
    _ints(parent, "parent", lengths.shape)

    def body(st):
        ws = _upkeep_workspace(cfg, table.device)
        check(lib().jamba_pages_fork(cfg.ref, _p(parent), _p(refs), _p(table), _p(lengths), _p(ws), ws.numel(), st))

    _run(index, stream, body)


def pages_grow(add, data, refs, table, lengths, stream=None):
    """Room for add[s] more tokens in every slot, counted into lengths; a shared
    last page is copied first.  Returns granted [max_seqs] int32 (0: refused,
    the slot is as it was)."""
    index, cfg = _pool(data, refs, table, lengths, ("add", add))
    _ints(add, "add", lengths.shape)

    def body(st):
        ws = _upkeep_workspace(cfg, data.device)
        granted = torch.empty_like(lengths)
        check(lib().jamba_pages_grow(cfg.ref, _p(add), _p(data), _p(refs), _p(table), _p(lengths), _p(granted), _p(ws),
                                     ws.numel(), st))
        return granted

    return _run(index, stream, body)


def pages_active(active, lengths, stream=None):
    """lengths with 0 in place of the slots that take no part in a call (active [max_seqs]
    int32, 0 or below): what paged_append and the attention take then.  A slot that brings no
    token, or that grow refused, must be left out of a call with one token per slot, and a refused one's
    rows out of a ragged call, or its last keys and values are overwritten, for every holder of the
    page; active = granted * add leaves both out."""
    index = _same_device(lengths, (("active", active),))
    if lengths.dim() != 1:
        raise ValueError("lengths must have shape [max_seqs]")
    _ints(lengths, "lengths", lengths.shape)
    _ints(active, "active", lengths.shape)

    def body(st):
        out = torch.empty_like(lengths)
        check(lib().jamba_pages_active(lengths.shape[0], _p(active), _p(lengths), _p(out), st))
        return out

    return _run(index, stream, body)


def pages_compact(data, refs, table, lengths, stream=None):
    """Moves the live pages to the front of the pool.  Returns remap [num_pages]
    int32: each live page's new number, -1 for free pages."""
    index, cfg = _pool(data, refs, table, lengths)

    def body(st):
        ws = _upkeep_workspace(cfg, data.device)
        remap = torch.empty_like(refs)
        check(lib().jamba_pages_compact(cfg.ref, _p(data), _p(refs), _p(table), _p(lengths), _p(remap), _p(ws), ws.numel(),
                                        st))
        return remap

    return _run(index, stream, body)


def paged_append(k, v, k_pages, v_pages, table, lengths, q_start=None, stream=None):
    """Keys and values k, v [tokens, n_kv_heads, 128] of the sequences' last
    tokens into their pages: sequence s has rows q_start[s] .. q_start[s+1] - 1
    (q_start [max_seqs + 1] int32), or one row each without q_start (slots of length 0
    left out; see pages_active)."""
    named = (("k", k), ("v", v), ("v_pages", v_pages), ("table", table), ("lengths", lengths))
    index = _same_device(k_pages, named if q_start is None else named + (("q_start", q_start),))
    N, G, P, _ = _planes(k_pages, v_pages)
    cfg = _config(N, G, P, 1, table, lengths)
    T, _, ld = _rows(k, "k", G)
    if _rows(v, "v", G) != (T, G, ld):
        raise ValueError("k and v must have one shape and one token stride")
    if q_start is not None:
        _ints(q_start, "q_start", (table.shape[0] + 1,))
        if T == 0:
            return

    def body(st):
        check(lib().jamba_paged_append(cfg.ref, _p(k), _p(v), ld, T, _p(q_start), _p(k_pages), _p(v_pages), _p(table),
                                       _p(lengths), st))

    _run(index, stream, body)


def _attend(q, k_pages, v_pages, table, lengths, q_start, out, want_lse, stream):
    named = (("q", q), ("v_pages", v_pages), ("table", table), ("lengths", lengths))
    if q_start is not None:
        named += (("q_start", q_start),)
    if out is not None:
        named += (("out", out),)
    index = _same_device(k_pages, named)
    N, G, P, _ = _planes(k_pages, v_pages)
    cfg = _config(N, G, P, 1, table, lengths)
    T, H, ld = _rows(q, "q")
    if q_start is not None:
        _ints(q_start, "q_start", (table.shape[0] + 1,))
    elif T != table.shape[0]:
        raise ValueError("q must hold one token for each of the %d slots" % table.shape[0])
    if out is not None and out.shape != q.shape:
        raise ValueError("out must have the shape of q")

    def body(st, out):
        L, device = lib(), q.device
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ld_o = _rows(out, "out")[2]
        lse = torch.empty((T, H), dtype=torch.float32, device=device) if want_lse else None
        if T:
            if q_start is None:
                ws = torch.empty(cfg.workspace(index, "jamba_paged_decode_workspace_size", H), dtype=torch.uint8,
                                 device=device)
                check(L.jamba_paged_decode(cfg.ref, H, _p(q), ld, _p(k_pages), _p(v_pages), _p(table), _p(lengths), _p(out),
                                           ld_o, _p(lse), _p(ws), ws.numel(), st))
            else:
                ws = torch.empty(cfg.workspace(index, "jamba_paged_extend_workspace_size", H, T), dtype=torch.uint8,
                                 device=device)
                check(L.jamba_paged_extend(cfg.ref, H, _p(q), ld, T, _p(q_start), _p(k_pages), _p(v_pages), _p(table),
                                           _p(lengths), _p(out), ld_o, _p(lse), _p(ws), ws.numel(), st))
        return (out, lse) if want_lse else out

    return _run(index, stream, body, out)


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
    paged_step of every layer, which write the new keys and values and attend.  Slots that
    could not grow, and in paged_step those that bring no token, are left out with
    active=granted * add (see pages_active).
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
        """Frees slots (an index or a list of them).  The slots are host values: in a captured
        graph every replay frees the same ones; fork with -1 frees by device values."""
        S, device = self.table.shape[0], self.table.device
        slots = [slots] if isinstance(slots, int) else list(slots)
        for s in slots:
            if not 0 <= s < S:
                raise ValueError("slot %d is outside 0 .. %d" % (s, S - 1))

        def body(_):
            if torch.cuda.is_current_stream_capturing():   # no copy of pageable memory there: a fill for each
                parent = torch.arange(S, dtype=torch.int32, device=device)
                for s in slots:
                    parent[s].fill_(-1)
            else:
                gone = set(slots)
                parent = torch.tensor([-1 if s in gone else s for s in range(S)], dtype=torch.int32, device=device)
            self.fork(parent)

        _run(self.table.get_device(), stream, body)

    def grow(self, add, stream=None):
        """See pages_grow."""
        return pages_grow(add, self.data, self.refs, self.table, self.lengths, stream=stream)

    def active_lengths(self, active, stream=None):
        """See pages_active."""
        return pages_active(active, self.lengths, stream=stream)

    def compact(self, stream=None):
        """See pages_compact."""
        return pages_compact(self.data, self.refs, self.table, self.lengths, stream=stream)

    def config(self, layer):
        """(a layer's sizes, its keys, its values)."""
        if not 0 <= layer < self.layers:
            raise ValueError("layer %d is outside 0 .. %d" % (layer, self.layers - 1))
        _, N, G, P, _ = self.data.shape
        return _config(N, G, P, 1, self.table, self.lengths), self.keys(layer), self.values(layer)
