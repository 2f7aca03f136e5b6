"""The paged cache: keys and values of many sequences kept between calls.

A ``PagedCache`` is the tensor relation [pages, heads, page positions, head
dim] with one block per page; a ``PageBatch`` joins it with a batch of
sequences through a table of page numbers (device tensors, so a captured
graph serves every batch copied into them).  ``cache_append`` writes rows of
K and V into the pages, ``cache_read`` reads them back, ``cache_attention``
attends to them.  All run in libea.so on the current torch stream (or
``stream``) and never block the host; a batch that is out of range is left
out on the device and reported by ``check()``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import CACHE_FORMATS, check_status, lib
from .relation import Relation

_CELLS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _on_device(t: torch.Tensor, dtype, shape, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or tuple(t.shape) != tuple(shape) or \
            not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {dtype}, {tuple(shape)}")
    return t


class PagedCache:
    """``pages`` pages of ``page`` positions (16, 32, 64 or 128) for ``heads``
    key-value heads of ``dim`` 64 or 128.

    ``format``: "bf16", or "e4m3" -- 8-bit floats with one power-of-two scale
    byte per page, head and position: value = code * 2^(byte - 127), 255
    marks a vector of NaN.  ``k``, ``v`` ([pages, heads, page, dim]) and, for
    e4m3, ``k_scale``, ``v_scale`` (uint8 [pages, heads, page]): existing
    tensors to use; default: new, zeroed ones."""

    def __init__(self, pages: int, page: int, heads: int, dim: int, format: str = "bf16",
                 k: torch.Tensor | None = None, v: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None, device=None):
        if format not in CACHE_FORMATS:
            raise ValueError(f"unknown cache format {format!r}")
        self.format, self.pages, self.page, self.heads, self.dim = format, int(pages), int(page), int(heads), int(dim)
        shape = (self.pages, self.heads, self.page, self.dim)
        if (k is None) != (v is None) or (format == "e4m3" and (k is None) != (k_scale is None)) or \
                (k_scale is None) != (v_scale is None) or (format == "bf16" and k_scale is not None):
            raise ValueError("give k and v (and, for e4m3 only, k_scale and v_scale) together")
        if k is None:
            device = device or "cuda"
            k, v = (torch.zeros(shape, dtype=torch.uint8 if format == "e4m3" else torch.bfloat16, device=device)
                    .view(_CELLS[format]) for _ in range(2))
            if format == "e4m3":
                k_scale, v_scale = (torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2))
        self.k, self.v = (_on_device(t, _CELLS[format], shape, "k and v") for t in (k, v))
        self.k_scale, self.v_scale = k_scale, v_scale
        if format == "e4m3":
            for t in (k_scale, v_scale):
                _on_device(t, torch.uint8, shape[:3], "k_scale and v_scale")
        self.device = self.k.device
        if any(t is not None and t.device != self.device for t in (v, k_scale, v_scale)):
            raise ValueError("the cache's tensors lie on different devices")
        h = ctypes.c_void_p()
        ptr = [ctypes.c_void_p(t.data_ptr() if t is not None else None) for t in (k, v, k_scale, v_scale)]
        with torch.cuda.device(self.device):
            check_status(lib().ea_cache_create(CACHE_FORMATS[format], self.pages, self.page, self.heads, self.dim, *ptr,
                                               ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _abi._lib is not None:
            _abi._lib.ea_cache_destroy(h)
            self.handle = None


class PageBatch:
    """A batch of sequences: rows ``starts[i] .. starts[i + 1]`` of a dense
    relation are the last positions of sequence i, which is ``lens[i]`` long;
    its position p is in slot p % page of page ``pages[i, p // page]``.

    int32 CUDA tensors: ``pages`` [sequences, most pages] (rows may be
    strided), ``starts`` [sequences + 1], ``lens`` [sequences].  They are kept;
    write into them for the next step.  ``max_new``:
    an upper bound of starts[i + 1] - starts[i], if known (it spares the
    attention the kernel for longer chunks and, over 8-bit pages, the memory
    where it expands theirs); 0: the dense rows."""

    def __init__(self, pages: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor, max_new: int = 0):
        if not isinstance(pages, torch.Tensor) or pages.dim() != 2 or pages.dtype != torch.int32 or not pages.is_cuda or \
                pages.shape[0] < 1 or pages.shape[1] < 1 or (pages.shape[1] > 1 and pages.stride(1) != 1) or \
                (pages.shape[0] > 1 and pages.stride(0) < pages.shape[1]):
            raise ValueError("pages must be an int32 CUDA tensor [sequences, pages], its rows contiguous")
        n = pages.shape[0]
        _on_device(starts, torch.int32, (n + 1,), "starts")
        _on_device(lens, torch.int32, (n,), "lens")
        if starts.device != pages.device or lens.device != pages.device:
            raise ValueError("the batch's tensors lie on different devices")
        self.pages, self.starts, self.lens, self.max_new = pages, starts, lens, int(max_new)
        self.device = pages.device
        self.args = _abi.PageBatchArgs()
        self.ref = ctypes.byref(self.args)
        self._workspace = {}  # bytes of an attention call's workspace, by everything they depend on besides the batch
        self.args.pages, self.args.starts, self.args.lens = pages.data_ptr(), starts.data_ptr(), lens.data_ptr()
        self.args.page_stride = pages.stride(0) if n > 1 else pages.shape[1]
        self.args.n_seqs, self.args.max_pages, self.args.max_new = n, pages.shape[1], self.max_new

    def check(self, cache: PagedCache, rows: int, write: bool = False):
        """Copy the table to the host and raise ``EaError`` if a sequence or a
        page number is out of range (``write``: or if an append with this
        batch would name a slot twice or a negative position)."""
        pages, starts, lens = (t.cpu().contiguous() for t in (self.pages, self.starts, self.lens))
        a = _abi.PageBatchArgs()
        a.pages, a.starts, a.lens = pages.data_ptr(), starts.data_ptr(), lens.data_ptr()
        a.page_stride, a.n_seqs, a.max_pages, a.max_new = pages.shape[1], pages.shape[0], pages.shape[1], self.max_new
        check_status(lib().ea_cache_check_batch(cache.pages, cache.page, ctypes.byref(a), int(rows), 1 if write else 0))


def _raw_stream(device, stream) -> ctypes.c_void_p:
    """The CUDA stream of a call: ``stream``, or the device's current one."""
    return ctypes.c_void_p(stream.cuda_stream if stream is not None else
                           torch._C._cuda_getCurrentRawStream(device.index))


def _same_device(cache: PagedCache, batch: PageBatch, *relations):
    if batch.device != cache.device:
        raise ValueError("the cache and the batch lie on different devices")
    for r in relations:
        if r is not None and r.storage.device != cache.device:
            raise ValueError("the cache and a relation lie on different devices")


def cache_append(cache: PagedCache, batch: PageBatch, k: Relation, v: Relation, stream=None):
    """Write the batch's rows of ``k`` and ``v`` (relations [rows.., heads,
    dim], f32 or bf16) into the pages, rounded to the cache's format."""
    _same_device(cache, batch, k, v)
    check_status(lib().ea_cache_append(cache.handle, batch.ref, k.handle, v.handle,
                                       _raw_stream(cache.device, stream)))


def cache_read(cache: PagedCache, batch: PageBatch, k: Relation | None = None, v: Relation | None = None,
               rows: int | None = None, dtype: str = "bf16", stream=None):
    """Read the batch's positions into the rows of ``k`` and ``v`` (relations
    [rows.., heads, dim], f32 or bf16); without them, into new relations of
    ``rows`` rows.  Rows of no sequence, and rows before position 0, stay as
    they are.  Returns (k, v)."""
    if k is None and v is None:
        if rows is None:
            raise ValueError("give k and v, or the number of rows")
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(cache.device):
            k, v = (Relation(dtype, (rows, cache.heads, cache.dim), [1, 1, 1], device=cache.device) for _ in range(2))
    if k is None or v is None:
        raise ValueError("give both k and v or neither")
    _same_device(cache, batch, k, v)
    check_status(lib().ea_cache_read(cache.handle, batch.ref, k.handle, v.handle,
                                     _raw_stream(cache.device, stream)))
    return k, v


def cache_attention(q: Relation, cache: PagedCache, batch: PageBatch, scale: float = 0.0, causal: bool = True,
                    out: Relation | None = None, m_out: Relation | None = None, l_out: Relation | None = None,
                    stream=None) -> Relation:
    """Softmax attention of the batch's rows of ``q`` (bf16 relation [rows..,
    query heads, dim]) over their sequences' pages, query heads in groups that
    share a key-value head; ``causal``: a row keeps the positions up to its
    own.  ``scale`` 0 means 1/sqrt(dim).  ``m_out``/``l_out`` (f32 over q's
    dimensions without the last) receive the row maximum and the row sum of
    exp.  Rows of no sequence stay as they are (in a new ``out``: undefined).
    The workspace for partial results comes from torch's allocator on the
    call's stream, one per call."""
    _same_device(cache, batch, q, out, m_out, l_out)
    L = lib()
    shape = (cache.format, cache.pages, cache.page, cache.heads, cache.dim, q.dims)
    need = batch._workspace.get(shape)
    if need is None:
        n = ctypes.c_size_t()
        check_status(L.ea_cache_attention_workspace(cache.handle, batch.ref, q.handle, ctypes.byref(n)))
        need = batch._workspace[shape] = n.value
    work = None
    if stream is None:
        if out is None:
            out = Relation("bf16", q.dims, q.bounds, device=cache.device)
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=cache.device)
    else:
        with torch.cuda.stream(stream):
            if out is None:
                out = Relation("bf16", q.dims, q.bounds, device=cache.device)
            if need:
                work = torch.empty(need, dtype=torch.uint8, device=cache.device)
    o = _abi.CacheAttnOpts(scale, 1 if causal else 0, m_out.handle if m_out is not None else None,
                           l_out.handle if l_out is not None else None, work.data_ptr() if work is not None else None, need)
    check_status(L.ea_cache_attention(cache.handle, batch.ref, q.handle, ctypes.byref(o),
                                      _raw_stream(cache.device, stream), out.handle))
    return out
