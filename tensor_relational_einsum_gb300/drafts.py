"""Around drafted tokens: rotary positions of a batch's rows, and verification.

A step of generation appends several rows to each sequence of a ``PageBatch``:
a run of a prompt, a chain of drafted tokens, or the nodes of a tree of them
(``parents``).  ``rotary`` rotates q and k by the rows' positions,
``verify_drafts`` says which branch of a tree the target's probabilities
accept; ``cache_attention`` attends along the branches and ``cache_keep``
keeps the accepted rows.  All run in libea.so on the current torch stream (or
``stream``) and never block the host; what is out of range on the device is
reported by ``check()``.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _abi
from ._abi import ROTARY_LAYOUTS, lib
from .cache import PageBatch, _call, _on_device, _raw_stream, _rows_of
from .relation import Relation


class Rotary:
    """A rotation of ``dims`` columns of a head, from column ``offset`` on.

    ``layout``: "interleaved" pairs (2 i, 2 i + 1) or "half" pairs (i, i +
    dims / 2).  Pair i turns by ``theta ** (-2 i / dims)`` radians a position.
    For contexts longer than the trained one: ``factor`` divides all of them
    (``original`` 0), or, with ``original`` the trained length, those with
    less than ``low`` turns in it, none with more than ``high``, and blends in
    between.  ``freqs``: the radians themselves (dims / 2 numbers) instead.
    ``amplitude`` is a factor of cosine and sine."""

    def __init__(self, dims: int, theta: float = 10000.0, layout: str = "interleaved", offset: int = 0,
                 factor: float = 1.0, original: int = 0, low: float = 1.0, high: float = 4.0, amplitude: float = 1.0,
                 freqs=None):
        if layout not in ROTARY_LAYOUTS:
            raise ValueError(f"unknown layout {layout!r}")
        self.dims, self.offset, self.layout = int(dims), int(offset), layout
        if self.dims < 2 or self.dims % 2 or self.offset < 0:
            raise ValueError("dims must be a positive even number, offset not negative")
        if freqs is None:
            if not theta > 0 or not factor > 0 or (original > 0 and not high > low):
                raise ValueError("theta and factor must be positive, high larger than low")
            freqs = []
            for i in range(self.dims // 2):
                f = float(theta) ** (-2.0 * i / self.dims)
                if original > 0:
                    keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
                    f *= keep + (1.0 - keep) / factor
                else:
                    f /= factor
                freqs.append(f)
        self.freqs = [float(f) for f in freqs]
        if len(self.freqs) != self.dims // 2 or not all(math.isfinite(f) for f in self.freqs):
            raise ValueError("freqs must be dims / 2 finite numbers")
        self.amplitude = float(amplitude)
        if not math.isfinite(self.amplitude) or self.amplitude == 0.0:
            raise ValueError("amplitude must be finite and not 0")
        self._freqs = (ctypes.c_double * len(self.freqs))(*self.freqs)
        self._address = ctypes.addressof(self._freqs)


def rotary(q: Relation, k: Relation | None, plan: Rotary, batch: PageBatch | None = None,
           positions: torch.Tensor | None = None, parents: torch.Tensor | None = None, q_out: Relation | None = None,
           k_out: Relation | None = None, backward: bool = False, stream=None):
    """Rotate the rows of ``q`` and ``k`` (relations [rows.., heads, columns],
    f32 or bf16; ``k`` may be None) by their positions: those of ``batch``, its
    rows being the last ones of their sequences, or nodes of trees with
    ``parents`` (as in ``cache_attention``: the position is the depth behind
    the sequence's other positions), or ``positions`` (int32 CUDA tensor, an
    entry a row).  In place, or into ``q_out`` and ``k_out``; rows of no
    sequence and of negative positions stay as they are.  ``backward``: the
    transposed rotation, which takes the gradients of the results to those of
    q and k.  Returns the results."""
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    if k is not None and (q_out is None) != (k_out is None):
        raise ValueError("give both q_out and k_out, or neither")
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    device = q.device
    o = _abi.RotaryOpts(ROTARY_LAYOUTS[plan.layout], plan.dims, plan.offset, 1 if backward else 0, plan.amplitude, 0,
                        plan._address)
    if positions is not None:
        o.positions = _rows_of(positions, torch.int32, q, 2, "positions").data_ptr()
    if parents is not None:
        o.parents = _rows_of(parents, torch.int32, q, 2, "parents").data_ptr()
    if q_out.device != device or (k is not None and (k.device != device or k_out.device != device)) or \
            (batch is not None and batch.device != device):
        raise ValueError("q, k, their results and the batch lie on different devices")
    _call(lib().ea_rotary, device, ctypes.byref(o), batch.ref if batch is not None else None, q.handle,
          k.handle if k is not None else None, q_out.handle, k_out.handle if k is not None else None,
          _raw_stream(device, stream))
    return q_out, k_out


def verify_drafts(target: Relation, batch: PageBatch, tokens: torch.Tensor, accept: torch.Tensor,
                  sample: torch.Tensor, draft: Relation | None = None, parents: torch.Tensor | None = None,
                  path: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                  picked: torch.Tensor | None = None, stream=None):
    """Speculative sampling: which nodes of each sequence's tree of drafted
    tokens the target's probabilities accept, and the token behind the last.

    ``target`` [rows.., vocab] (f32 or bf16): probabilities of the token behind
    each row; ``draft``: those that the row's children were drawn from, each on
    its own (None: the drafts are certain); ``tokens`` (int32), ``accept`` (f32
    random numbers in [0, 1)): an entry a row; ``sample`` (f32): one a
    sequence; ``parents``: as in ``cache_attention`` (None: chains).  A
    sequence's first row is its last certain token and always accepted.
    Returns (``path`` [sequences, width], the accepted rows counted from the
    sequence's first, -1 behind them; ``counts``, their number; ``picked``, the
    token that follows): int32, new ones by default, width then max_new."""
    device = target.device
    _rows_of(tokens, torch.int32, target, 1, "tokens")
    _rows_of(accept, torch.float32, target, 1, "accept")
    if parents is not None:
        _rows_of(parents, torch.int32, target, 1, "parents")
    n = batch.lens.shape[0]
    _on_device(sample, torch.float32, (n,), "sample")
    if path is not None and (not isinstance(path, torch.Tensor) or path.dim() != 2):
        raise ValueError("path must be an int32 CUDA tensor [sequences, width]")
    if path is None or counts is None or picked is None:
        width = path.shape[1] if path is not None else max(1, min(batch.max_new or tokens.shape[0], tokens.shape[0]))
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device):
            path = torch.empty(n, width, dtype=torch.int32, device=device) if path is None else path
            counts = torch.empty(n, dtype=torch.int32, device=device) if counts is None else counts
            picked = torch.empty(n, dtype=torch.int32, device=device) if picked is None else picked
    width = path.shape[1]
    _on_device(path, torch.int32, (n, width), "path")
    _on_device(counts, torch.int32, (n,), "counts")
    _on_device(picked, torch.int32, (n,), "picked")
    at = device.index
    if sample.get_device() != at or path.get_device() != at or counts.get_device() != at or picked.get_device() != at or \
            batch.device != device or (draft is not None and draft.device != device):
        raise ValueError("the operands of verify_drafts lie on different devices")
    o = _abi.VerifyOpts(tokens.data_ptr(), parents.data_ptr() if parents is not None else None, accept.data_ptr(),
                        sample.data_ptr(), path.data_ptr(), counts.data_ptr(), picked.data_ptr(), width)
    _call(lib().ea_verify_drafts, device, ctypes.byref(o), batch.ref, target.handle,
          draft.handle if draft is not None else None, _raw_stream(device, stream))
    return path, counts, picked
