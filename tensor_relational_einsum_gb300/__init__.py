"""GB300 (sm_103a) join-agg hot path of Einsummable.

Tensor relations, join-agg specs and the exchange ("Every Kernel Is a Join:
Automatic Multi-GPU Parallelism for AI Computations in Einsummable"),
executed on one GPU by libea.so (C ABI in include/ea.h):

* ``Relation``  -- a CUDA tensor stored as blocks of a tiling;
* ``joinagg``   -- one join-agg: join on shared letters, per-tuple kernel,
                   SUM/MAX aggregation fused into the kernel;
* ``exchange``  -- re-block a relation from one tiling to another;
* ``PagedCache``, ``PageBatch`` -- keys and values of many sequences kept in
                   pages (bf16 or 8-bit cells), and a batch of sequences;
* ``cache_append``, ``cache_read``, ``cache_attention`` -- write rows into
                   the pages, read them back, attend to them;
* ``Rotary``, ``rotary``, ``verify_drafts``, ``cache_keep`` -- rotary
                   positions of a batch's rows; which drafted tokens of a
                   chain or tree are accepted; keeping their rows.

The Python layer only marshals arguments.  Importing this package loads
libea.so lazily; calls raise if it is missing (no CPU fallback).
"""
from ._abi import EaError, lib  # noqa: F401

__all__ = ["Relation", "joinagg", "exchange", "check", "EaError", "lib", "plan_cache_clear", "PagedCache", "PageBatch",
           "cache_append", "cache_read", "cache_attention", "cache_keep", "Rotary", "rotary", "verify_drafts"]


def __getattr__(name):
    if name in ("Relation", "joinagg", "exchange", "check", "plan_cache_clear", "output_layout"):
        from . import relation as module
    elif name in ("PagedCache", "PageBatch", "cache_append", "cache_read", "cache_attention", "cache_keep"):
        from . import cache as module
    elif name in ("Rotary", "rotary", "verify_drafts"):
        from . import drafts as module
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(module, name)  # later look-ups find it at once
    return value
