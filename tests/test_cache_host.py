"""CPU tests of the paged cache: every refusal of its entry points (arguments
are checked before any device is touched), the host form of the batch check,
and the reference arithmetic that the GPU tests rest on."""
import ctypes

import numpy as np
import pytest

import cache_util as cu
from tensor_relational_einsum_gb300 import _abi
from tensor_relational_einsum_gb300.build import build

BASE = 1 << 40  # addresses that are never read


@pytest.fixture(scope="module")
def L():
    build()
    return _abi.lib()


def rel(L, dtype, dims, parts=None, at=BASE):
    arr, keep, _ = _abi.dim_parts(dims, parts or [1] * len(dims))
    h = ctypes.c_void_p()
    _abi.check_status(L.ea_relation_create(_abi.DTYPES[dtype], len(dims), _abi.i64(dims), arr, ctypes.c_void_p(at),
                                           ctypes.byref(h)))
    return h


def cache(L, fmt="bf16", pages=8, page=16, heads=2, dim=64, k=BASE << 1, v=BASE << 2, ks=None, vs=None):
    if fmt == "e4m3" and ks is None:
        ks, vs = BASE << 3, BASE << 4
    h = ctypes.c_void_p()
    rc = L.ea_cache_create(_abi.CACHE_FORMATS.get(fmt, fmt), pages, page, heads, dim, ctypes.c_void_p(k), ctypes.c_void_p(v),
                           ctypes.c_void_p(ks), ctypes.c_void_p(vs), ctypes.byref(h))
    return rc, h


def batch(n_seqs=1, max_pages=4, stride=None, max_new=0, pages=BASE, starts=BASE, lens=BASE):
    a = _abi.PageBatchArgs()
    a.pages, a.starts, a.lens = pages, starts, lens
    a.page_stride, a.n_seqs, a.max_pages, a.max_new = stride or max_pages, n_seqs, max_pages, max_new
    return a


ARG, SHAPE, PART, DTYPE, UNSUP, BOUNDS = 7, 2, 3, 4, 8, 10


def test_create_refuses(L):
    assert cache(L)[0] == 0 and cache(L, "e4m3")[0] == 0
    assert cache(L, 5)[0] == DTYPE
    assert cache(L, pages=0)[0] == ARG and cache(L, pages=1 << 31)[0] == ARG
    for page in (0, 8, 24, 256, -16):
        assert cache(L, page=page)[0] == UNSUP
    for dim in (0, 32, 96, 256):
        assert cache(L, dim=dim)[0] == UNSUP
    assert cache(L, heads=0)[0] == ARG
    assert cache(L, k=None)[0] == ARG
    assert cache(L, k=(BASE << 1) + 8)[0] == ARG            # alignment
    assert cache(L, k=BASE, v=BASE + 64)[0] == ARG          # overlap
    assert cache(L, "bf16", ks=BASE << 3, vs=BASE << 4)[0] == ARG
    assert cache(L, "e4m3", ks=BASE << 3, vs=None)[0] == ARG
    assert L.ea_cache_create(0, 1, 16, 1, 64, ctypes.c_void_p(BASE), ctypes.c_void_p(BASE << 1), None, None, None) == ARG


@pytest.mark.parametrize("call", ["ea_cache_append", "ea_cache_read"])
def test_rows_refuse(L, call):
    f = getattr(L, call)
    c = cache(L)[1]
    k, v = rel(L, "bf16", (10, 2, 64)), rel(L, "bf16", (10, 2, 64), at=BASE + (1 << 20))

    def run(b=None, kk=k, vv=v, cc=c):
        return f(cc, ctypes.byref(b or batch()), kk, vv, None)

    assert run(cc=None) == ARG and run(kk=None) == ARG
    assert f(c, None, k, v, None) == ARG
    for b in (batch(pages=None), batch(starts=None), batch(lens=None), batch(n_seqs=0), batch(n_seqs=65537),
              batch(max_pages=0), batch(max_pages=4, stride=3), batch(max_new=-1)):
        assert run(b) == ARG
    assert run(batch(max_pages=1 << 28)) == UNSUP            # positions beyond 2^31 - 1
    assert run(vv=rel(L, "f32", (10, 2, 64))) == DTYPE
    assert run(vv=rel(L, "bf16", (11, 2, 64))) == SHAPE
    assert run(kk=rel(L, "bf16", (10, 128)), vv=rel(L, "bf16", (10, 128))) == SHAPE
    for dims in ((10, 3, 64), (10, 2, 128)):
        assert run(kk=rel(L, "bf16", dims), vv=rel(L, "bf16", dims, at=BASE + (1 << 20))) == SHAPE
    # heads or head dim cut into blocks; rows cut behind a dimension whose blocks hold several indexes
    assert run(kk=rel(L, "bf16", (10, 2, 64), [1, 2, 1])) == PART
    assert run(kk=rel(L, "bf16", (10, 2, 64), [1, 1, 2])) == PART
    assert run(kk=rel(L, "bf16", (4, 10, 2, 64), [1, 2, 1, 1]), vv=rel(L, "bf16", (4, 10, 2, 64), at=BASE + (1 << 20))) == PART
    assert run(kk=rel(L, "bf16", (10, 2, 64), at=(BASE << 1) + 256)) == ARG   # inside the cache
    if call == "ea_cache_read":
        assert run(vv=k) == ARG


def test_attention_refuses(L):
    c = cache(L)[1]
    q, o = rel(L, "bf16", (10, 6, 64)), rel(L, "bf16", (10, 6, 64), at=BASE + (1 << 20))
    m, l = rel(L, "f32", (10, 6), at=BASE + (1 << 21)), rel(L, "f32", (10, 6), at=BASE + (1 << 22))

    def run(q=q, o=o, b=None, cc=c, **kw):
        a = _abi.CacheAttnOpts()
        need = ctypes.c_size_t()
        for x, y in kw.items():
            setattr(a, x, y)
        rc = L.ea_cache_attention_workspace(cc, ctypes.byref(b or batch()), q, ctypes.byref(need))
        if rc:
            return rc
        if "workspace_bytes" not in kw:
            a.workspace, a.workspace_bytes = BASE << 5, need.value
        return L.ea_cache_attention(cc, ctypes.byref(b or batch()), q, ctypes.byref(a), None, o)

    assert run(cc=None) == ARG and run(q=None) == ARG and run(o=None) == ARG
    assert run(q=rel(L, "f32", (10, 6, 64))) == DTYPE
    assert run(o=rel(L, "f32", (10, 6, 64), at=BASE + (1 << 20))) == DTYPE
    assert run(q=rel(L, "bf16", (10, 5, 64))) == SHAPE          # 5 heads over 2
    assert run(q=rel(L, "bf16", (10, 6, 128))) == SHAPE
    assert run(o=rel(L, "bf16", (9, 6, 64), at=BASE + (1 << 20))) == SHAPE
    assert run(q=rel(L, "bf16", (10, 258, 64))) == UNSUP        # 129 heads to a key-value head
    assert run(o=rel(L, "bf16", (10, 6, 64), [1, 2, 1], at=BASE + (1 << 20))) == PART
    assert run(o=q) == ARG and run(o=rel(L, "bf16", (10, 6, 64), at=BASE << 1)) == ARG
    assert run(scale=-1.0) == ARG and run(scale=float("nan")) == ARG and run(scale=float("inf")) == ARG
    assert run(m_out=m.value) == ARG and run(l_out=l.value) == ARG
    assert run(m_out=m.value, l_out=m.value) == ARG
    assert run(m_out=m.value, l_out=rel(L, "bf16", (10, 6)).value) == DTYPE
    assert run(m_out=m.value, l_out=rel(L, "f32", (10, 5)).value) == SHAPE
    assert run(b=batch(n_seqs=0)) == ARG
    assert L.ea_cache_attention_workspace(c, ctypes.byref(batch()), q, None) == ARG


def host_batch(b: cu.Batch, **kw):
    keep = [np.ascontiguousarray(x) for x in (b.pages, b.starts, b.lens)]
    a = batch(n_seqs=len(b.lens), max_pages=b.max_pages, **kw)
    a.pages, a.starts, a.lens = (x.ctypes.data for x in keep)
    return a, keep


def test_batch_check(L):
    def check(b, write=1, rows=None, pages=None, **kw):
        a, keep = host_batch(b, **kw)
        return L.ea_cache_check_batch(b.pages_total if pages is None else pages, b.page, ctypes.byref(a),
                                      b.rows if rows is None else rows, write)

    seqs = [(3, 40), (0, 5), (17, 17), (1, 1)]
    assert check(cu.Batch(seqs, 16, before=2, behind=3)) == 0
    assert check(cu.Batch(seqs, 16), rows=20) == BOUNDS                 # rows beyond the dense relation
    assert check(cu.Batch(seqs, 16), max_new=16) == BOUNDS              # more new rows than promised
    assert check(cu.Batch(seqs, 16), max_new=17) == 0
    assert check(cu.Batch(seqs, 16), pages=3) == BOUNDS                 # page numbers beyond the cache
    for bad in (-1, 1 << 30):
        b = cu.Batch(seqs, 16)
        b.pages[0, 2] = bad
        assert check(b) == BOUNDS
        b = cu.Batch(seqs, 16)
        b.pages[1, 0] = bad                                             # an idle sequence needs no page
        assert check(b) == 0
    b = cu.Batch(seqs, 16)
    b.starts[2] = 1                                                     # decreasing
    assert check(b) == BOUNDS
    b = cu.Batch(seqs, 16)
    b.lens[0] = b.max_pages * 16 + 1
    assert check(b) == BOUNDS
    b = cu.Batch(seqs, 16)
    b.lens[2] = -1
    assert check(b) == BOUNDS
    b = cu.Batch([(5, 3)], 16)                                          # rows before the first position
    assert check(b) == BOUNDS and check(b, write=0) == 0
    b = cu.Batch(seqs, 16)
    b.pages[3, 0] = b.pages[2, 0]                                       # two sequences write one slot
    assert check(b) == BOUNDS and check(b, write=0) == 0
    a, keep = host_batch(cu.Batch(seqs, 16))
    assert L.ea_cache_check_batch(0, 16, ctypes.byref(a), 21, 0) == ARG
    assert L.ea_cache_check_batch(9, 16, None, 21, 0) == ARG


def test_reference_e4m3_grid():
    # every finite value of the format is a fixed point, halves go to the even code, the largest is 448
    grid = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    grid = np.array(grid[:-1])
    assert grid[-1] == 448 and len(grid) == 127
    assert np.array_equal(cu.e4m3_round(grid), grid)
    mid = (grid[1:] + grid[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, grid[:-1], grid[1:])
    assert np.array_equal(cu.e4m3_round(mid), even)
    x = np.array([[448.0, 1.0], [448.1, 0.0], [224.0, 1.0], [0.0, 0.0], [2.0 ** -140, 0.0], [3.0e38, 1.0]])
    assert list(cu.e4m3_scale(x)) == [0, 1, -1, 0, -126, 120]


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = np.ones((7, 4)), rng.normal(size=(7, 4))
    out, m, l, big, _ = cu.softmax_attention(rng.normal(size=(3, 4)), k, v, np.array([4, 5, 6]), 0.5, True)
    for i, end in enumerate((5, 6, 7)):            # equal keys: the mean of what is kept
        assert np.allclose(out[i], v[:end].mean(0)) and np.isclose(l[i], end)
    out, m, l, *_ = cu.softmax_attention(rng.normal(size=(2, 4)), k[:1], v[:1], np.array([-1, 0]), 1.0, True)
    assert not out[0].any() and m[0] == -np.inf and l[0] == 0 and np.allclose(out[1], v[0])


def split(L, b, heads, group, tok, kt, causal, lo, hi, ctas):
    a, keep = host_batch(b)
    sp = (ctypes.c_int32 * 7)(heads, group, tok, kt, causal, lo, hi)
    cap = 1 << 16
    parts, n = np.zeros((cap, 7), dtype=np.int64), ctypes.c_int64()
    _abi.check_status(L.ea_cache_attention_split(ctypes.byref(a), b.page, b.rows, sp, ctas, cap,
                                                 parts.ctypes.data_as(_abi.P64), ctypes.byref(n)))
    return parts[:n.value]


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("group,tok,kt,lo,hi", [(4, 8, 64, 1, 32), (1, 256, 128, 33, 1 << 30), (3, 42, 128, 1, 1 << 30),
                                                (7, 36, 128, 0, 1 << 30), (128, 2, 128, 0, 1 << 30), (16, 16, 512, 1, 256)])
@pytest.mark.parametrize("ctas", [1, 7, 152, 304])
def test_work_list_against_enumeration(L, causal, group, tok, kt, lo, hi, ctas):
    """Every unit of every item exactly once and in order, shares equal to within one unit, whatever the lengths."""
    rng = np.random.default_rng(ctas + 10 * group + causal)
    seqs = [(1, 1), (0, 9), (5, 0), (300, 120), (7, 7), (64, 700), (33, 33), (1, 900), (257, 999), (0, 0), (40, 3)]
    seqs += [(int(rng.integers(0, 60)), int(rng.integers(0, 400))) for _ in range(20)]
    heads = 3
    want = []
    for i, (n, t) in enumerate(seqs):
        if n == 0 or not lo <= n * group <= hi:
            continue
        for h in range(heads):
            for j in range(-(-n // tok)):
                last = min(n, (j + 1) * tok)
                e = max(0, t - n + last) if causal else t
                units = max(1, -(-e // kt))
                want += [(i, h, j, u, units) for u in range(units)]
    parts = split(L, cu.Batch(seqs, 16), heads, group, tok, kt, causal, lo, hi, ctas)
    got = [(s, h, j, u, units) for _, s, h, j, u0, u1, units in parts.tolist() for u in range(u0, u1)]
    assert got == want
    share = np.bincount(parts[:, 0], weights=parts[:, 5] - parts[:, 4])
    assert len(share) == min(ctas, len(want)) and share.max() - share.min() <= 1
    # at most the first and the last part of a CTA are pieces of an item
    for x in range(len(share)):
        mine = parts[parts[:, 0] == x]
        cut = (mine[:, 4] > 0) | (mine[:, 5] < mine[:, 6])
        assert not cut[1:-1].any()


def test_work_list_of_long_sequences(L):
    """Sums in closed form at lengths where an enumeration by unit is out of reach: units add up, items tile the tokens."""
    b = cu.Batch([(1, 1)], 16)
    b.seqs, b.lens = [(1 << 20, 1 << 24)], np.array([1 << 24], dtype=np.int32)
    b.starts, b.rows, b.max_pages = np.array([0, 1 << 20], dtype=np.int32), 1 << 20, 1 << 20
    b.pages = np.zeros((1, 1), dtype=np.int32)
    parts = split(L, b, 1, 3, 84, 128, 1, 0, (1 << 31) - 1, 152)
    items = -(-(1 << 20) // 84)
    ends = (1 << 24) - (1 << 20) + np.minimum(1 << 20, (np.arange(items) + 1) * 84)
    assert (parts[:, 5] - parts[:, 4]).sum() == (-(-ends // 128)).sum()
    for j, (a, z) in zip(parts[:, 3], parts[:, 4:7:2]):
        assert z == -(-ends[j] // 128)
