"""The paged cache in 64 bits: what append, read and attention are to give,
written from their definitions in numpy, and the errors that fp32 sums and
the stated roundings allow."""
from __future__ import annotations

import numpy as np

HALF_BF16 = 2.0 ** -8    # half a step of bf16, relative (eps / 2)


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """x (|x| <= 448) to the nearest e4m3 value, ties to the even code: steps
    of 2^(e - 3) in [2^e, 2^(e + 1)) for e >= -6, of 2^-9 below."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    # log2 can round up to an integer just below a power of two
    e = np.where(np.exp2(e) > np.maximum(np.abs(x), 2.0 ** -6), e - 1, e)
    step = np.exp2(e - 3)
    return np.round(x / step) * step   # numpy rounds halves to even


def e4m3_scale(x: np.ndarray) -> np.ndarray:
    """Exponent of the vectors' scale: least e with max|x| <= 448 * 2^e in
    [-126, 120], 0 for a zero vector."""
    a = np.abs(x).max(-1)
    e = np.zeros(a.shape)
    nz = a > 0
    e[nz] = np.ceil(np.log2(a[nz] / 448.0) - 1e-10)
    return np.where(nz, np.clip(e, -126, 120), 0.0)


def softmax_attention(q, k, v, positions, scale, causal):
    """One head: q [n, d], k, v [t, d]; rows at ``positions``.  Returns out,
    m, l and A = SUM p |v| / l, the magnitudes that p's rounding scales with;
    also the largest rounding a score can carry, relative to exp."""
    n, t = q.shape[0], k.shape[0]
    out, big = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    m, l, slack = np.full(n, -np.inf), np.zeros(n), np.zeros(n)
    for i in range(n):
        end = min(t, max(0, positions[i] + 1)) if causal else t
        if end == 0:
            continue
        s = (k[:end] @ q[i]) * scale
        # d products, each exact in fp32, summed in fp32: at most d roundings or truncations of the partial sums
        slack[i] = ((np.abs(k[:end]) @ np.abs(q[i])) * scale).max() * (q.shape[1] + 4) * 2.0 ** -23
        m[i] = s.max()
        p = np.exp(s - m[i])
        l[i] = p.sum()
        out[i] = p @ v[:end] / l[i]
        big[i] = p @ np.abs(v[:end]) / l[i]
    return out, m, l, big, slack


def out_bound(out, big, slack, keys):
    """Elementwise error of a bf16 output: its own rounding, the rounding of
    every probability (both half a bf16 step), the scores' error on both sides
    of the quotient, and fp32 exponentials and sums over ``keys`` keys."""
    soft = 2.0 * np.expm1(slack)[..., None] + 2.0 ** -18 + 4.0 * keys * 2.0 ** -24
    mid = HALF_BF16 * big + soft * (1 + HALF_BF16) * big
    return mid + HALF_BF16 * (np.abs(out) + mid) + 1e-30


class Batch:
    """Sequences (n rows, length) over a shuffled page table; numpy arrays."""

    def __init__(self, seqs, page, spare=3, before=0, behind=0, seed=0, extra_pages=0):
        rng = np.random.default_rng(seed)
        self.seqs, self.page = list(seqs), page
        need = [-(-t // page) for _, t in self.seqs]
        self.pages_total = sum(need) + spare
        order = rng.permutation(self.pages_total)
        self.max_pages = max(1, max(need)) + extra_pages
        self.pages = np.full((len(self.seqs), self.max_pages), -7, dtype=np.int32)   # unlisted entries: no page at all
        at = 0
        for i, c in enumerate(need):
            self.pages[i, :c] = order[at:at + c]
            at += c
        ns = [n for n, _ in self.seqs]
        self.starts = (before + np.concatenate([[0], np.cumsum(ns)])).astype(np.int32)
        self.lens = np.array([t for _, t in self.seqs], dtype=np.int32)
        self.rows = int(self.starts[-1]) + behind

    def places(self, i):
        """(page, slot) of every position of sequence i."""
        p = np.arange(self.lens[i])
        return self.pages[i, p // self.page], p % self.page

    def rows_of(self, i):
        return slice(int(self.starts[i]), int(self.starts[i + 1]))
