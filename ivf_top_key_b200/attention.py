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
tensors' device; by default the current one of that device.
"""
from __future__ import annotations

import contextlib

import torch

from . import _capi as C

_INT, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _dense(t: torch.Tensor, dtype, device, what: str, shape=None):
    _need(t.dtype == dtype, f"{what} must be {dtype}")
    _need(t.device == device, f"{what} must be on {device}")
    _need(t.is_contiguous(), f"{what} must be contiguous")
    if shape is not None:
        _need(t.shape == shape, f"{what} must have shape {tuple(shape)}")
    return t.data_ptr()


@contextlib.contextmanager
def _entered(device: torch.device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _on(device: torch.device, stream):
    """Context in which the call's memory belongs to its stream, and that stream's handle."""
    if stream is None:
        s = torch.cuda.current_stream(device)
        if device.index == torch.cuda.current_device():
            return contextlib.nullcontext(), s.cuda_stream
        return torch.cuda.device(device), s.cuda_stream
    _need(stream.device == device, f"the stream must be on {device}")
    return _entered(device, stream), stream.cuda_stream


def _gpu(t: torch.Tensor, what: str) -> torch.device:
    _need(t.is_cuda, f"{what} must be on the GPU")
    return t.device


def _view(k, v, tables, lens, refs=None, k_scale=None, v_scale=None, status=None, pages: bool = True):
    """The ai_cache of these tensors and the number of its layers' leading dimensions."""
    dev = _gpu(tables, "tables")
    c = C.AiCache()
    _need(tables.dim() == 2, "tables must be [n_seqs, max_pages]")
    c.tables = _dense(tables, _INT, dev, "tables")
    c.n_seqs, c.max_pages = tables.shape
    c.lens = _dense(lens, _INT, dev, "lens", tables.shape[:1])
    if pages:
        _need(k.dim() in (4, 5), "k must be [n_layers, n_pages, page_size, n_kv_heads, head_dim] or one layer of it")
        _need(k.dtype in (_BF16, torch.uint8, torch.float8_e4m3fn), "the cache holds bfloat16, or e4m3 codes")
        fp8 = k.dtype != _BF16
        c.k = _dense(k, k.dtype, dev, "k")
        c.v = _dense(v, k.dtype, dev, "v", k.shape)
        c.n_layers = k.shape[0] if k.dim() == 5 else 1
        c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = k.shape[-4:]
        c.dtype = C.AI_FP8E4M3 if fp8 else C.AI_BF16
        _need(fp8 == (k_scale is not None) and fp8 == (v_scale is not None),
              "k_scale and v_scale go with e4m3 codes, and only with them")
        if fp8:
            c.k_scale = _dense(k_scale, _F32, dev, "k_scale", k.shape[:-1])
            c.v_scale = _dense(v_scale, _F32, dev, "v_scale", k.shape[:-1])
        if refs is not None:
            c.refs = _dense(refs, _INT, dev, "refs", (c.n_pages,))
    if status is not None:
        c.status = _dense(status, _INT, dev, "status", (1,))
    return c, dev


def _list(t, dev, what: str, n=None):
    _need(t.dim() == 1, f"{what} must be one-dimensional")
    return _dense(t, _INT, dev, what, None if n is None else (n,))


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
    for t, what in ((q, "q"), (k, "k"), (v, "v")):
        _need(t.dim() == 3, f"{what} must be [tokens, heads, head_dim]")
        _need(t.dtype == _BF16, f"{what} must be torch.bfloat16")
        _need(t.device == dev, f"{what} must be on {dev}")
        _need(t.stride(2) == 1 or t.shape[2] == 1, f"the last dimension of {what} must be dense")
    _need(v.shape == k.shape and k.shape[2] == q.shape[2], "k and v must be [total_k, n_kv_heads, head_dim of q]")
    _need(cu_q.dim() == 1 and cu_q.shape[0] >= 1, "cu_q must be [n_seqs + 1]")
    pq, pk = _dense(cu_q, _INT, dev, "cu_q"), _dense(cu_k, _INT, dev, "cu_k", cu_q.shape)
    T, Hq, D = q.shape
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
        C.ai_attend_prompt(q.data_ptr(), q.stride()[:2], k.data_ptr(), k.stride()[:2], v.data_ptr(), v.stride()[:2],
                           pq, pk, cu_q.shape[0] - 1, T, k.shape[0], Hq, k.shape[1], D,
                           D ** -0.5 if scale is None else scale, _dense(out, _BF16, dev, "out", (T, Hq, D)),
                           None if out_lse is None else _dense(out_lse, _F32, dev, "out_lse", (T, Hq)),
                           None if status is None else _dense(status, _INT, dev, "status", (1,)), st)
    return out


def _rows(q, ids, cache, dev, seqs, layer, scale, out, out_lse, stream):
    _need(q.dim() == 3, "q must be [rows, heads, head_dim]")
    pq = _dense(q, _BF16, dev, "q")
    T, Hq, D = q.shape
    _need(D == cache.head_dim, "q and the cache must have the same head_dim")
    ps = None if seqs is None else _list(seqs, dev, "seqs", T)
    if ids is not None:
        _need(ids.dim() == 2 and ids.shape[0] == T, "ids must be [rows, k]")
        pi = _dense(ids, _INT, dev, "ids")
    scale = D ** -0.5 if scale is None else scale
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
        po = _dense(out, _BF16, dev, "out", (T, Hq, D))
        pl = None if out_lse is None else _dense(out_lse, _F32, dev, "out_lse", (T, Hq))
        n = C.ai_attend_workspace(Hq, cache.n_kv_heads, D)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        if ids is None:
            C.ai_attend_cached(cache, layer, pq, T, Hq, ps, scale, po, pl, ws.data_ptr(), n, st)
        else:
            C.ai_attend_selected(cache, layer, pq, pi, T, ids.shape[1], Hq, ps, scale, po, pl, ws.data_ptr(), n, st)
    return out


def attend_cached(q, k, v, tables, lens, seqs=None, *, layer: int = 0, k_scale=None, v_scale=None, scale=None,
                  out=None, out_lse=None, status=None, stream=None):
    """One new token per sequence over all its cached tokens (ai_attend_cached).

    q [rows, Hq, D] bfloat16; k, v: pages [n_layers, n_pages, page_size, Hkv,
    D] or of one layer, bfloat16 or e4m3 codes with k_scale / v_scale (the
    shape without D); tables [n_seqs, max_pages], lens [n_seqs] int32.  Row r
    reads sequence seqs[r] (None: r).  Returns out [rows, Hq, D]."""
    c, dev = _view(k, v, tables, lens, None, k_scale, v_scale, status)
    return _rows(q, None, c, dev, seqs, layer, scale, out, out_lse, stream)


def attend_selected(q, ids, k, v, tables, lens, seqs=None, *, layer: int = 0, k_scale=None, v_scale=None, scale=None,
                    out=None, out_lse=None, status=None, stream=None):
    """Attention of row t over the cached tokens ids[t, :] (ai_attend_selected).

    ids [rows, k] int32 as `AttentionIndex.route_refine` returns them
    (negative: no key); the rest as for attend_cached.  seqs None: every row
    is the only sequence of the tables, or row t is sequence t."""
    c, dev = _view(k, v, tables, lens, None, k_scale, v_scale, status)
    return _rows(q, ids, c, dev, seqs, layer, scale, out, out_lse, stream)


# -------------------------------------------------------------------- pages
def _workspace(c, n: int, dev):
    need = C.ai_cache_workspace(c, n)
    return torch.empty(need, dtype=torch.uint8, device=dev), need


def cache_extend(k, v, tables, lens, refs, seqs, counts, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Lengthen sequence seqs[i] by counts[i] tokens, taking free pages (ai_cache_extend)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ps, n = _list(seqs, dev, "seqs"), seqs.shape[0]
    pc = _list(counts, dev, "counts", n)
    ctx, st = _on(dev, stream)
    with ctx:
        ws, need = _workspace(c, n, dev)
        C.ai_cache_extend(c, ps, pc, n, ws.data_ptr(), need, st)


def cache_write(k, v, tables, lens, seqs, cu, new_k, new_v, *, layer: int = 0, k_scale=None, v_scale=None,
                status=None, stream=None):
    """Rows [cu[i], cu[i+1]) of new_k, new_v become the last tokens of sequence seqs[i] (ai_cache_write)."""
    c, dev = _view(k, v, tables, lens, None, k_scale, v_scale, status)
    ps, n = _list(seqs, dev, "seqs"), seqs.shape[0]
    pc = _list(cu, dev, "cu", n + 1)
    shape = (new_k.shape[0], c.n_kv_heads, c.head_dim)
    pk, pv = _dense(new_k, _BF16, dev, "new_k", shape), _dense(new_v, _BF16, dev, "new_v", shape)
    ctx, st = _on(dev, stream)
    with ctx:
        C.ai_cache_write(c, layer, pk, pv, ps, pc, n, shape[0], st)


def cache_fork(k, v, tables, lens, refs, src, dst, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Make the empty sequence dst[i] a copy of src[i]: full pages shared, a part page copied (ai_cache_fork)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ps, n = _list(src, dev, "src"), src.shape[0]
    pd = _list(dst, dev, "dst", n)
    ctx, st = _on(dev, stream)
    with ctx:
        ws, need = _workspace(c, n, dev)
        C.ai_cache_fork(c, ps, pd, n, ws.data_ptr(), need, st)


def cache_free(tables, lens, refs, seqs, *, page_size: int, status=None, stream=None):
    """Release sequences (ai_cache_free)."""
    c, dev = _view(None, None, tables, lens, status=status, pages=False)
    _need(refs.dim() == 1, "refs must be [n_pages]")
    c.refs, c.n_pages, c.page_size = _dense(refs, _INT, dev, "refs"), refs.shape[0], page_size
    ps = _list(seqs, dev, "seqs")
    ctx, st = _on(dev, stream)
    with ctx:
        C.ai_cache_free(c, ps, seqs.shape[0], st)


def cache_compact(k, v, tables, lens, refs, *, k_scale=None, v_scale=None, status=None, stream=None):
    """Move the live pages to the front of the cache (ai_cache_compact)."""
    c, dev = _view(k, v, tables, lens, refs, k_scale, v_scale, status)
    ctx, st = _on(dev, stream)
    with ctx:
        ws, need = _workspace(c, 0, dev)
        C.ai_cache_compact(c, ws.data_ptr(), need, st)


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
        cache_write(self.k, self.v, self.tables, self.lens, seqs, cu, new_k, new_v, layer=layer, stream=stream,
                    **self._scales())

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
        if bits & 2:
            raise C.AiError(-4, "an id, sequence or page was out of range, or a sequence was listed twice")
        if bits:
            raise C.AiError(-2, "pages or table columns ran out")
