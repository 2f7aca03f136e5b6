"""CPU tests of the operators around drafted tokens: every refusal of their
entry points (arguments are checked before any device is touched), and the
reference arithmetic that the GPU tests rest on."""
import ctypes
import math

import numpy as np
import pytest

import drafts_util as du
from tensor_relational_einsum_gb300 import _abi
from test_cache_host import ARG, BASE, DTYPE, PART, SHAPE, UNSUP, L, batch, cache, rel  # noqa: F401

FAR = 1 << 20


def rotary_opts(**kw):
    o = _abi.RotaryOpts()
    freqs = (ctypes.c_double * 128)(*[1.0 / (i + 1) for i in range(128)])
    o.layout, o.dims, o.freqs = 1, 64, ctypes.addressof(freqs)
    for x, y in kw.items():
        setattr(o, x, y)
    return o, freqs


def test_rotary_refuses(L):  # noqa: F811
    at = [BASE + i * FAR for i in range(8)]
    q, k = rel(L, "bf16", (10, 6, 64), at=at[0]), rel(L, "bf16", (10, 2, 64), at=at[1])
    qo, ko = rel(L, "bf16", (10, 6, 64), at=at[2]), rel(L, "bf16", (10, 2, 64), at=at[3])
    far = dict(pages=BASE << 6, starts=BASE << 7, lens=BASE << 8)

    def run(q=q, k=k, qo=qo, ko=ko, b=True, **kw):
        o, keep = rotary_opts(**kw)
        b = ctypes.byref(batch(**far)) if b is True else ctypes.byref(b) if b else None
        return L.ea_rotary(ctypes.byref(o), b, q, k, qo, ko, None)

    assert L.ea_rotary(None, ctypes.byref(batch()), q, k, qo, ko, None) == ARG
    assert run(q=None) == ARG and run(qo=None) == ARG and run(k=None) == ARG and run(ko=None) == ARG
    assert run(freqs=None) == ARG and run(layout=2) == ARG and run(amplitude=float("nan")) == ARG
    assert run(b=None) == ARG and run(positions=BASE << 9) == ARG           # neither and both
    assert run(b=None, positions=BASE << 9, parents=BASE << 10) == ARG
    for b in (batch(n_seqs=0, **far), batch(n_seqs=65537, **far), batch(max_new=-1, **far), batch(starts=None), batch(lens=None)):
        assert run(b=b) == ARG
    for dims, offset in ((0, 0), (63, 0), (66, 0), (64, 2), (64, -2), (-2, 0)):
        assert run(dims=dims, offset=offset) == SHAPE, (dims, offset)
    wide = [rel(L, "bf16", (10, 2, 512), at=at[i]) for i in range(4)]
    assert run(*wide, dims=258) == UNSUP
    assert run(q=rel(L, "f32", (10, 6, 64), at=at[0])) == DTYPE and run(ko=rel(L, "f32", (10, 2, 64), at=at[3])) == DTYPE
    assert run(k=rel(L, "bf16", (9, 2, 64), at=at[1])) == SHAPE and run(qo=rel(L, "bf16", (10, 5, 64), at=at[2])) == SHAPE
    assert run(k=rel(L, "bf16", (10, 2, 128), at=at[1]), ko=rel(L, "bf16", (10, 2, 128), at=at[3])) == SHAPE
    assert run(q=rel(L, "bf16", (10, 6, 64), [1, 2, 1], at=at[0])) == PART
    assert run(q=rel(L, "bf16", (10, 64), at=at[0])) == SHAPE
    assert run(qo=rel(L, "bf16", (10, 6, 64), at=at[0] + 64)) == ARG        # overlaps q, but is not q
    assert run(qo=k, q=rel(L, "bf16", (10, 2, 64), at=at[0])) == ARG and run(ko=rel(L, "bf16", (10, 2, 64), at=at[0])) == ARG
    assert run(ko=rel(L, "bf16", (10, 2, 64), at=at[2] + 256)) == ARG
    assert run(qo=q) == ARG                                                 # q in place, k not
    for field in ("starts", "lens"):
        for where in (at[2], at[3] + 16):
            assert run(b=batch(**{**far, field: where})) == ARG
    assert run(parents=at[2]) == ARG and run(b=None, positions=at[3]) == ARG
    assert run(parents=(BASE << 10) + 2) == ARG
    long = [rel(L, "bf16", (200, h, 64), at=BASE + i * (1 << 24)) for i, h in enumerate((6, 2, 6, 2))]
    assert run(*long, parents=BASE << 10) == UNSUP                          # up to 200 nodes
    bad, keep = rotary_opts()
    for x in (float("nan"), float("inf")):
        keep[5] = x
        assert L.ea_rotary(ctypes.byref(bad), ctypes.byref(batch(**far)), q, k, qo, ko, None) == ARG


def test_verify_refuses(L):  # noqa: F811
    at = [BASE + i * FAR for i in range(12)]
    target, draft = rel(L, "f32", (10, 100), at=at[0]), rel(L, "f32", (10, 100), at=at[1])
    base = dict(tokens=at[2], accept=at[3], sample=at[4], path=at[5], counts=at[6], picked=at[7], width=10)
    far = dict(pages=None, starts=BASE << 7, lens=BASE << 8)

    def run(t=target, d=draft, b=None, **kw):
        o = _abi.VerifyOpts()
        for x, y in {**base, **kw}.items():
            setattr(o, x, y)
        return L.ea_verify_drafts(ctypes.byref(o), ctypes.byref(b or batch(**far)), t, d, None)

    for x in ("tokens", "accept", "sample", "path", "counts", "picked"):
        assert run(**{x: None}) == ARG
    assert run(t=None) == ARG and L.ea_verify_drafts(None, ctypes.byref(batch()), target, draft, None) == ARG
    assert run(d=rel(L, "bf16", (10, 100), at=at[1])) == DTYPE
    assert run(d=rel(L, "f32", (10, 101), at=at[1])) == SHAPE and run(d=rel(L, "f32", (9, 100), at=at[1])) == SHAPE
    assert run(t=rel(L, "f32", (10, 100), [1, 2], at=at[0])) == PART and run(t=rel(L, "f32", (100,), at=at[0])) == SHAPE
    for b in (batch(n_seqs=0, **far), batch(n_seqs=65537, **far), batch(max_new=-1, **far), batch(starts=None)):
        assert run(b=b) == ARG
    assert run(width=0) == ARG and run(width=9) == ARG and run(width=4, b=batch(max_new=5, **far)) == ARG
    many = [rel(L, "f32", (200, 100), at=BASE + i * (1 << 24)) for i in range(2)]
    assert run(t=many[0], d=many[1], width=200, **{x: (BASE << 12) + i * FAR for i, x in enumerate(base) if x != "width"}) == UNSUP
    for x in ("path", "counts", "picked"):
        for where in (at[0] + 96, at[1], at[2], at[3] + 36, at[4], BASE << 7):
            assert run(**{x: where}) == ARG, (x, where)
    assert run(parents=at[5]) == ARG and run(counts=at[5] + 8) == ARG and run(picked=at[6]) == ARG


def test_keep_refuses(L):  # noqa: F811
    c = cache(L)[1]
    far = dict(pages=BASE << 6, starts=BASE << 7, lens=BASE << 8, max_new=8)

    def run(caches=(c,), n=None, b=None, path=BASE << 9, width=8, counts=BASE << 10, lens_out=BASE << 11):
        arr = (ctypes.c_void_p * max(1, len(caches)))(*[x.value if x is not None else None for x in caches])
        return L.ea_cache_keep(arr, len(caches) if n is None else n, ctypes.byref(b or batch(**far)), path, width, counts,
                               lens_out, None)

    assert run(caches=(None,)) == ARG and run(n=0) == ARG and run(path=None) == ARG and run(counts=None) == ARG
    assert run(width=0) == ARG
    for b in (batch(**{**far, "pages": None}), batch(n_seqs=0, **far), batch(max_pages=4, stride=3, **far)):
        assert run(b=b) == ARG
    assert run(b=batch(**{**far, "max_new": 0})) == UNSUP and run(b=batch(**{**far, "max_new": 129})) == UNSUP
    assert run(caches=(c, cache(L, "e4m3", k=BASE << 12, v=BASE << 13, ks=BASE << 14, vs=BASE << 15)[1])) == DTYPE
    for kw in (dict(pages=9), dict(page=32), dict(heads=3), dict(dim=128)):
        assert run(caches=(c, cache(L, k=BASE << 12, v=BASE << 13, **kw)[1])) == SHAPE
    assert run(caches=(c, c)) == ARG                                        # one cache twice
    for x in (BASE << 1, (BASE << 2) + 64):
        assert run(path=x) == ARG and run(counts=x) == ARG and run(lens_out=x) == ARG
    for x in (BASE << 6, BASE << 7, BASE << 8, BASE << 9, BASE << 10):
        assert run(lens_out=x) == ARG


def test_tree_attention_refuses(L):  # noqa: F811
    c = cache(L)[1]
    q, o = rel(L, "bf16", (10, 6, 64)), rel(L, "bf16", (10, 6, 64), at=BASE + FAR)
    far = dict(pages=BASE << 6, starts=BASE << 7, lens=BASE << 8)

    def run(q=q, o=o, b=None, **kw):
        b = b or batch(**far)
        need = ctypes.c_size_t()
        assert L.ea_cache_attention_workspace(c, ctypes.byref(b), q, ctypes.byref(need)) == 0
        a = _abi.CacheAttnOpts(0.0, 1, None, None, BASE << 9, need.value)
        for x, y in kw.items():
            setattr(a, x, y)
        return L.ea_cache_attention(c, ctypes.byref(b), q, ctypes.byref(a), None, o)

    assert run(parents=BASE + FAR) == ARG and run(parents=(BASE << 10) + 1) == ARG
    long = [rel(L, "bf16", (200, 6, 64), at=BASE + i * (1 << 24)) for i in range(2)]
    assert run(*long, parents=BASE << 10) == UNSUP
    assert run(*long, parents=BASE << 10, b=batch(max_new=129, **far)) == UNSUP


# ------------------------------------------------------------ the references

def test_frequencies_and_their_scaling():
    from tensor_relational_einsum_gb300 import Rotary
    plain = Rotary(8, theta=10000.0).freqs
    assert plain == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    assert Rotary(8, factor=4.0).freqs == pytest.approx([f / 4 for f in plain], rel=1e-14)
    # 1 / (2 pi f) turns in 1000 positions: 159, 15.9, 1.59, 0.159; kept from 4 on, divided below 1, blended between
    got = Rotary(8, factor=4.0, original=1000, low=1.0, high=4.0).freqs
    w = (1000 * 0.01 / (2 * math.pi) - 1.0) / 3.0
    assert got == pytest.approx([1.0, 0.1, 0.01 * (w + (1 - w) / 4), 0.00025], rel=1e-14)
    for kw in (dict(dims=7), dict(dims=0), dict(dims=8, layout="x"), dict(dims=8, offset=-1), dict(dims=8, theta=0.0),
               dict(dims=8, factor=0.0), dict(dims=8, original=10, low=4.0, high=4.0), dict(dims=8, freqs=[1.0]),
               dict(dims=4, freqs=[1.0, float("inf")]), dict(dims=8, amplitude=0.0)):
        with pytest.raises(ValueError):
            Rotary(**kw)


def test_reference_trees_and_rotation():
    p = [-1, 0, 0, 1, 3, -1]
    assert du.way(p, 4) == [4, 3, 1, 0] and du.depth(p, 4) == 3 and du.depth(p, 5) == 0
    assert du.kept_positions(p, 4, 6, 8) == [0, 1, 2, 3, 5, 6] and du.kept_positions(p, 2, 6, 4) == [0]
    assert du.kept_positions(p, 1, 6, 4) == []
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1.0, 2.0, 3.0, 4.0]
    quarter = [math.pi / 2, math.pi]
    out, _ = du.rotate(x, [1], quarter, "interleaved", 0)
    assert np.allclose(out[0, 0], [-2, 1, -3, -4])
    out, _ = du.rotate(x, [1], quarter, "half", 0)
    assert np.allclose(out[0, 0], [-3, -2, 1, -4])
    out, _ = du.rotate(x, [-1], quarter, "half", 0)
    assert np.array_equal(out, x)


def test_reference_verification_keeps_the_targets_distribution():
    """Over a grid of random numbers the first token's frequency is the target's, whatever the draft and however many
    children are asked (three tokens, two children drawn on their own)."""
    target, draft = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    grid = (np.arange(20) + 0.5) / 20
    got = np.zeros(3)
    for a in range(3):
        for b in range(3):
            weight = draft[a] * draft[b] / 20 ** 3
            for ua in grid:
                for ub in grid:
                    for s in grid:
                        t = np.tile(target, (3, 1))
                        path, picked, _ = du.verify(t, np.tile(draft, (3, 1)), [0, a, b], [-1, 0, 0], [0, ua, ub], s)
                        token = [0, a, b][path[1]] if len(path) > 1 else picked
                        got[token] += weight
    assert np.allclose(got, target, atol=0.02)  # the grid's cells: 1 / 20 of the mass at a border, and less at two
