"""Drafted tokens in 64 bits: trees, rotary positions, verification, written
from their definitions in numpy."""
from __future__ import annotations

import math

import numpy as np


def tree(kind: str, n: int, rng=None) -> list[int]:
    """Parents of n nodes."""
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    if kind == "pairs":
        return [-1] + [(j - 1) // 2 for j in range(1, n)]
    return [-1] + [int(rng.integers(-1 if kind == "forest" else 0, j)) for j in range(1, n)]


def way(parents, j: int) -> list[int]:
    """Node j and its ancestors."""
    got = []
    while j >= 0:
        got.append(j)
        j = parents[j]
    return got


def depth(parents, j: int) -> int:
    return len(way(parents, j)) - 1


def kept_positions(parents, j: int, n: int, t: int) -> list[int]:
    """Positions that node j of a sequence of t positions, the last n its nodes, keeps."""
    base = t - n
    return list(range(max(0, base))) + sorted(base + b for b in way(parents, j) if base + b >= 0)


def rotate(x, positions, freqs, layout, offset, amplitude=1.0, backward=False):
    """x [rows, heads, columns] float64 at `positions` (negative: unchanged); also the magnitude |x| + |y| of every
    rotated column's pair (0 elsewhere)."""
    half = len(freqs)
    one = offset + (2 * np.arange(half) if layout == "interleaved" else np.arange(half))
    two = one + (1 if layout == "interleaved" else half)
    out, big = x.copy(), np.zeros_like(x)
    for r, t in enumerate(positions):
        if t < 0:
            continue
        # cosines of the angle modulo a turn, which fp64 holds to 1e-10 at the positions that are tested
        a = np.array([math.fmod(t * f, 2 * math.pi) for f in freqs])
        c, s = amplitude * np.cos(a), amplitude * np.sin(a) * (-1 if backward else 1)
        out[r][:, one] = x[r][:, one] * c - x[r][:, two] * s
        out[r][:, two] = x[r][:, one] * s + x[r][:, two] * c
        big[r][:, one] = big[r][:, two] = abs(amplitude) * (np.abs(x[r][:, one]) + np.abs(x[r][:, two]))
    return out, big


def verify(target, draft, tokens, parents, accept, sample):
    """One sequence (target, draft [n, vocab] float64; draft None: certain tokens).  Returns (path, picked, margin):
    margin is how near the nearest decision was to going the other way, relative to what it compares."""
    n, vocab = target.shape
    path, v, near = [0], 0, math.inf
    while True:
        r, z, step = target[v].copy(), 1.0, None
        for c in range(1, n):
            if parents[c] != v:
                continue
            x = tokens[c]
            d = draft[v] if draft is not None else np.eye(1, vocab, x)[0]
            a, b = accept[c] * d[x] * z, r[x]
            near = min(near, abs(a - b) / max(a, b)) if max(a, b) > 0 else near
            if a < b:
                step = c
                break
            r = np.maximum(r - z * d, 0.0)
            z = math.fsum(r)
        if step is None:
            break
        path.append(step)
        v = step
    if math.fsum(r) == 0.0:
        r = target[v].copy()
    sums = np.cumsum(r)
    if sums[-1] == 0.0:
        return path, -1, near
    at = sample * sums[-1]
    picked = int((sums <= at).sum())
    near = min(near, np.abs(sums[r > 0] - at).min() / sums[-1])
    return path, picked, near
