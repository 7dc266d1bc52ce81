"""Attention over a request's keys, and the paged cache that holds them.

`AttentionIndex` says which keys a query attends over; the functions here
attend.  `attend_selected` reads the keys that `route_refine` or
`select_exhaustive` returned, `attend_cached` all keys of a sequence (one new
token each), `attend_prompt` packed prompts that are not in a cache yet.  The
`cache_*` functions keep the pages: they work on plain device tensors, in
stream order; `PagedCache` holds such tensors for a program that has none.

A call checks its tensors on the host, allocates its output and workspace
with torch on the stream it runs on (so captured graphs and streams never
share a workspace) and waits for nothing.  `stream` is a torch stream on the
tensors' device; by default the current one of that device.  The caller orders
it behind what writes the tensors and before what reads the output; all of
them may be dropped right after.  What the device refuses, or an output that
is not valid, shows in the call's `status` word, or without one in
`attend_check()`.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import _capi as C

_INT, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_CODES = (torch.uint8, torch.float8_e4m3fn)
_HERE = contextlib.nullcontext()


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _dense(t: torch.Tensor, dtype, device, what: str, shape=None):
    """The address of a tensor that has to be dense, of this type and shape, and on this device."""
    if t.dtype is dtype and t.device == device and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous {dtype} tensor on {device}"
                     + ("" if shape is None else f" of shape {tuple(shape)}"))


@contextlib.contextmanager
def _entered(device: torch.device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _on(device: torch.device, stream):
    """The handle of the call's stream, and the context in which the call's memory belongs to that stream: None where
    the caller is in it already."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
        return handle, None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
    _need(stream.device == device, "the stream must be on the tensors' device")
    return stream.cuda_stream, _entered(device, stream)


def _kept(stream, out, *tensors):
    """After a call on a stream of the caller's: its tensors may be dropped now, their memory is not given to others
    before the stream has come this far.  The output, which may be new memory of that stream, is used on the current
    one."""
    if stream is not None:
        for t in (out, *tensors):
            if t is not None:
                t.record_stream(stream)
        if out is not None:
            out.record_stream(torch.cuda.current_stream(stream.device))


@functools.lru_cache(maxsize=None)
def _attend_workspace(device: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return C.ai_attend_workspace(n_heads, n_kv_heads, head_dim)


def _gpu(t: torch.Tensor, what: str) -> torch.device:
    _need(t.is_cuda, f"{what} must be on the GPU")
    return t.device


def _view(k, v, tables, lens, refs=None, k_scale=None, v_scale=None, status=None):
    """The ai_cache of these tensors, and their device."""
    dev = tables.device
    shape, kind, rows = k.shape, k.dtype, tables.shape
    fp8 = kind is not _BF16
    if not tables.is_cuda:
        raise ValueError("tables must be on the GPU")
    if len(rows) != 2:
        raise ValueError("tables must be [n_seqs, max_pages]")
    if not 4 <= len(shape) <= 5:
        raise ValueError("k must be [n_layers, n_pages, page_size, n_kv_heads, head_dim] or one layer of it")
    if fp8 and kind not in _CODES:
        raise ValueError("the cache holds bfloat16, or e4m3 codes")
    if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
        raise ValueError("k_scale and v_scale go with e4m3 codes, and only with them")
    n_pages, page, heads, D = shape[-4:]
    return C.AiCache(
        _dense(k, kind, dev, "k"), _dense(v, kind, dev, "v", shape),
        _dense(k_scale, _F32, dev, "k_scale", shape[:-1]) if fp8 else None,
        _dense(v_scale, _F32, dev, "v_scale", shape[:-1]) if fp8 else None,
        _dense(tables, _INT, dev, "tables"), _dense(lens, _INT, dev, "lens", rows[:1]),
        None if refs is None else _dense(refs, _INT, dev, "refs", (n_pages,)),
        None if status is None else _dense(status, _INT, dev, "status", (1,)),
        C.AI_FP8E4M3 if fp8 else C.AI_BF16, shape[0] if len(shape) == 5 else 1, n_pages, page, heads, D, rows[0],
        rows[1]), dev


def _list(t, dev, what: str, n=None):
    _need(t.dim() == 1, f"{what} must be one-dimensional")
    return _dense(t, _INT, dev, what, None if n is None else (n,))


def _refuse(bits: int):
    """Raises for the AI_DEVFLAG_* bits of a status word; a wait that ran out says more than what was refused."""
    if bits & C.AI_DEVFLAG_TIMEOUT:
        raise C.AiError(-5, "a wait inside a kernel ran out: outputs since the last check are not valid")
    if bits & C.AI_DEVFLAG_RANGE:
        raise C.AiError(-4, "an id, sequence or page was out of range, a sequence was listed twice, or a write reached "
                            "a page of several sequences")
    if bits & C.AI_DEVFLAG_CAPACITY:
        raise C.AiError(-2, "pages or table columns ran out")


def attend_check(device=None):
    """Wait for the device's current stream and raise for what calls without a status word refused since the last
    check (ai_status_read)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        _refuse(C.ai_status_read(torch.cuda.current_stream().cuda_stream))


# ---------------------------------------------------------------- attention
def attend_prompt(q, k, v, cu_q, cu_k=None, *, scale=None, out=None, out_lse=None, status=None, stream=None):
    """Causal attention over packed prompts (ai_attend_prompt).

    q [total_q, Hq, D], k and v [total_k, Hkv, D]: bfloat16, the last
    dimension dense (slices of a fused projection are fine).  cu_q, cu_k:
    int32 [n_seqs + 1] row offsets of the sequences; cu_k None: cu_q.  The last
    query of a sequence sees its last key.  scale: D ** -0.5 by default.
    Returns out [total_q, Hq, D]; out_lse: None or float32 [total_q, Hq]."""
    dev = _gpu(q, "q")
    cu_k = cu_q if cu_k is None else cu_k
    for t in (q, k, v):
        if t.dim() != 3 or t.dtype is not _BF16 or t.device != dev or (t.stride(2) != 1 and t.shape[2] != 1):
            raise ValueError(f"q, k and v must be torch.bfloat16 [tokens, heads, head_dim] on {dev}, the last dimension dense")
    T, Hq, D = q.shape
    if v.shape != k.shape or k.shape[2] != D:
        raise ValueError("k and v must be [total_k, n_kv_heads, head_dim of q]")
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be [n_seqs + 1]")
    pq, pk = _dense(cu_q, _INT, dev, "cu_q"), _dense(cu_k, _INT, dev, "cu_k", cu_q.shape)
    st, ctx = _on(dev, stream)
    po = None if out is None else _dense(out, _BF16, dev, "out", (T, Hq, D))
    pl = None if out_lse is None else _dense(out_lse, _F32, dev, "out_lse", (T, Hq))
    ps = None if status is None else _dense(status, _INT, dev, "status", (1,))
    with ctx or _HERE:
        if out is None:
            out = q.new_empty((T, Hq, D))
            po = out.data_ptr()
        Tk, Hkv = k.shape[0], k.shape[1]
        B = cu_q.shape[0] - 1
        n = C.ai_attend_prompt_workspace(B, T, Tk, Hq, Hkv, D) if Tk >= 1024 * B else 0   # (the call costs 1.5 us)
        ws = q.new_empty((n + 1) // 2) if n else None
        C.ai_attend_prompt(q.data_ptr(), q.stride()[:2], k.data_ptr(), k.stride()[:2], v.data_ptr(), v.stride()[:2],
                           pq, pk, B, T, Tk, Hq, Hkv, D, D ** -0.5 if scale is None else scale, po, pl,
                           ps, ws.data_ptr() if n else None, n, st)
    _kept(stream, out, q, k, v, cu_q, cu_k, out_lse, status)
    return out


def _rows(q, ids, cache, dev, seqs, layer, scale, out, out_lse, stream):
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError("q must be [rows, heads, head_dim of the cache]")
    T, Hq, D = shape
    pq = _dense(q, _BF16, dev, "q")
    ps = None if seqs is None else _list(seqs, dev, "seqs", T)
    po = None if out is None else _dense(out, _BF16, dev, "out", shape)
    pl = None if out_lse is None else _dense(out_lse, _F32, dev, "out_lse", shape[:2])
    if ids is not None:
        if ids.dim() != 2 or ids.shape[0] != T:
            raise ValueError("ids must be [rows, k]")
        pi = _dense(ids, _INT, dev, "ids")
    if scale is None:
        scale = D ** -0.5
    st, ctx = _on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if out is None:
            out = torch.empty_like(q)
            po = out.data_ptr()
        n = _attend_workspace(dev.index, Hq, cache.n_kv_heads, D)
        ws = q.new_empty((n + 1) // 2)
        if ids is None:
            C.ai_attend_cached(cache, layer, pq, T, Hq, ps, scale, po, pl, ws.data_ptr(), n, st)
        else:
            C.ai_attend_selected(cache, layer, pq, pi, T, ids.shape[1], Hq, ps, scale, po, pl, ws.data_ptr(), n, st)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    return out


def attend_cached(q, k, v, tables, lens, seqs=None, *, layer: int = 0, k_scale=None, v_scale=None, scale=None,
                  out=None, out_lse=None, status=None, stream=None):
    """One new token per sequence over all its cached tokens (ai_attend_cached).

    q [rows, Hq, D] bfloat16; k, v: pages [n_layers, n_pages, page_size, Hkv,
    D] or of one layer, bfloat16 or e4m3 codes with k_scale / v_scale (the
    shape without D); tables [n_seqs, max_pages], lens [n_seqs] int32.  Row r
    reads sequence seqs[r] (None: r).  Returns out [rows, Hq, D]."""
    c, dev = _view(k, v, tables, lens, None, k_scale, v_scale, status)
    out = _rows(q, None, c, dev, seqs, layer, scale, out, out_lse, stream)
    _kept(stream, out, q, k, v, tables, lens, seqs, k_scale, v_scale, out_lse, status)
    return out


def attend_selected(q, ids, k, v, tables, lens, seqs=None, *, layer: int = 0, k_scale=None, v_scale=None, scale=None,
                    out=None, out_lse=None, status=None, stream=None):
    """Attention of row t over the cached tokens ids[t, :] (ai_attend_selected).

    ids [rows, k] int32 as `AttentionIndex.route_refine` returns them
    (negative: no key); the rest as for attend_cached.  seqs None: every row
    is the only sequence of the tables, or row t is sequence t."""
    c, dev = _view(k, v, tables, lens, None, k_scale, v_scale, status)
    out = _rows(q, ids, c, dev, seqs, layer, scale, out, out_lse, stream)
    _kept(stream, out, q, ids, k, v, tables, lens, seqs, k_scale, v_scale, out_lse, status)
    return out


# -------------------------------------------------------------------- pages
def _workspace(c, n: int, dev):
    need = C.ai_cache_workspace(c, n)
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def cache_extend(k, v, tables, lens, refs, seqs, counts, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Lengthen sequence seqs[i] by counts[i] tokens, taking free pages (ai_cache_extend)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ps, n = _list(seqs, dev, "seqs"), seqs.shape[0]
    pc = _list(counts, dev, "counts", n)
    st, ctx = _on(dev, stream)
    with ctx or _HERE:
        ws, need = _workspace(c, n, dev)
        C.ai_cache_extend(c, ps, pc, n, ws.data_ptr(), need, st)
    _kept(stream, None, k, v, tables, lens, refs, seqs, counts, k_scale, v_scale, status)


def cache_write(k, v, tables, lens, seqs, cu, new_k, new_v, *, refs=None, layer: int = 0, k_scale=None, v_scale=None,
                status=None, stream=None):
    """Rows [cu[i], cu[i+1]) of new_k, new_v become the last tokens of sequence seqs[i] (ai_cache_write).

    refs: as for cache_extend; with it, rows that reach a page of several sequences are refused."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ps, n = _list(seqs, dev, "seqs"), seqs.shape[0]
    pc = _list(cu, dev, "cu", n + 1)
    shape = (new_k.shape[0], c.n_kv_heads, c.head_dim)
    pk, pv = _dense(new_k, _BF16, dev, "new_k", shape), _dense(new_v, _BF16, dev, "new_v", shape)
    st, ctx = _on(dev, stream)
    with ctx or _HERE:
        C.ai_cache_write(c, layer, pk, pv, ps, pc, n, shape[0], st)
    _kept(stream, None, k, v, tables, lens, refs, seqs, cu, new_k, new_v, k_scale, v_scale, status)


def cache_fork(k, v, tables, lens, refs, src, dst, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Make the empty sequence dst[i] a copy of src[i]: full pages shared, a part page copied (ai_cache_fork)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ps, n = _list(src, dev, "src"), src.shape[0]
    pd = _list(dst, dev, "dst", n)
    st, ctx = _on(dev, stream)
    with ctx or _HERE:
        ws, need = _workspace(c, n, dev)
        C.ai_cache_fork(c, ps, pd, n, ws.data_ptr(), need, st)
    _kept(stream, None, k, v, tables, lens, refs, src, dst, k_scale, v_scale, status)


def cache_free(tables, lens, refs, seqs, *, page_size: int, status=None, stream=None):
    """Release sequences (ai_cache_free)."""
    dev = _gpu(tables, "tables")
    _need(tables.dim() == 2 and refs.dim() == 1, "tables must be [n_seqs, max_pages], refs [n_pages]")
    c = C.AiCache(None, None, None, None, _dense(tables, _INT, dev, "tables"),
                  _dense(lens, _INT, dev, "lens", tables.shape[:1]), _dense(refs, _INT, dev, "refs"),
                  None if status is None else _dense(status, _INT, dev, "status", (1,)),
                  0, 0, refs.shape[0], page_size, 0, 0, *tables.shape)
    ps = _list(seqs, dev, "seqs")
    st, ctx = _on(dev, stream)
    with ctx or _HERE:
        C.ai_cache_free(c, ps, seqs.shape[0], st)
    _kept(stream, None, tables, lens, refs, seqs, status)


def cache_compact(k, v, tables, lens, refs, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Move the live pages to the front of the cache (ai_cache_compact)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    st, ctx = _on(dev, stream)
    with ctx or _HERE:
        ws, need = _workspace(c, 0, dev)
        C.ai_cache_compact(c, ws.data_ptr(), need, st)
    _kept(stream, None, k, v, tables, lens, refs, k_scale, v_scale, status)


class PagedCache:
    """The tensors of a paged key-value cache on the current device, and the calls above on them.

    k, v [n_layers, n_pages, page_size, n_kv_heads, head_dim] (k_scale,
    v_scale for dtype "fp8"), tables, lens, refs, status.  Nothing is read
    back: what a call refused shows in `check()`."""

    def __init__(self, *, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, n_seqs: int, max_pages: int,
                 n_layers: int = 1, dtype: str = "bf16"):
        _need(dtype in ("bf16", "fp8"), "dtype must be bf16 or fp8")
        dev = torch.device("cuda", torch.cuda.current_device())
        shape = (n_layers, n_pages, page_size, n_kv_heads, head_dim)
        kind = _BF16 if dtype == "bf16" else torch.uint8
        self.k, self.v = (torch.zeros(shape, dtype=kind, device=dev) for _ in range(2))
        self.k_scale = self.v_scale = None
        if dtype == "fp8":
            self.k_scale, self.v_scale = (torch.ones(shape[:-1], dtype=_F32, device=dev) for _ in range(2))
        self.tables = torch.full((n_seqs, max_pages), -1, dtype=_INT, device=dev)
        self.lens, self.refs = (torch.zeros(n, dtype=_INT, device=dev) for n in (n_seqs, n_pages))
        self.status = torch.zeros(1, dtype=_INT, device=dev)

    def _scales(self):
        return {"k_scale": self.k_scale, "v_scale": self.v_scale, "status": self.status}

    def extend(self, seqs, counts, stream=None):
        cache_extend(self.k, self.v, self.tables, self.lens, self.refs, seqs, counts, stream=stream, **self._scales())

    def write(self, seqs, cu, new_k, new_v, layer: int = 0, stream=None):
        cache_write(self.k, self.v, self.tables, self.lens, seqs, cu, new_k, new_v, refs=self.refs, layer=layer,
                    stream=stream, **self._scales())

    def fork(self, src, dst, stream=None):
        cache_fork(self.k, self.v, self.tables, self.lens, self.refs, src, dst, stream=stream, **self._scales())

    def free(self, seqs, stream=None):
        cache_free(self.tables, self.lens, self.refs, seqs, page_size=self.k.shape[2], status=self.status,
                   stream=stream)

    def compact(self, stream=None):
        cache_compact(self.k, self.v, self.tables, self.lens, self.refs, stream=stream, **self._scales())

    def attend(self, q, seqs=None, *, layer: int = 0, scale=None, out=None, out_lse=None, stream=None):
        return attend_cached(q, self.k, self.v, self.tables, self.lens, seqs, layer=layer, scale=scale, out=out,
                             out_lse=out_lse, stream=stream, **self._scales())

    def attend_selected(self, q, ids, seqs=None, *, layer: int = 0, scale=None, out=None, out_lse=None, stream=None):
        return attend_selected(q, ids, self.k, self.v, self.tables, self.lens, seqs, layer=layer, scale=scale, out=out,
                               out_lse=out_lse, stream=stream, **self._scales())

    def check(self):
        """Wait for the current stream and raise for what the calls refused since the last check."""
        bits = int(self.status.item())
        self.status.zero_()
        _refuse(bits)
