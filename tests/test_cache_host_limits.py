"""CPU tests of what the paged cache's entry points refuse at the ends of their
ranges (arguments are checked before any device is touched)."""
import ctypes

import numpy as np

import cache_util as cu
from tensor_relational_einsum_gb300 import _abi
from test_cache_host import ARG, BASE, UNSUP, L, batch, cache, host_batch, rel  # noqa: F401


def test_split_refuses_a_negative_capacity(L):  # noqa: F811
    """`parts` holds `capacity` of them: none for a negative one (nothing may be written), nor for negative rows."""
    a, keep = host_batch(cu.Batch([(3, 400), (1, 90)], 16))
    sp = (ctypes.c_int32 * 7)(2, 1, 8, 64, 1, 1, 1 << 30)
    parts, n = np.full((64, 7), -5, dtype=np.int64), ctypes.c_int64()

    def run(capacity, rows=4):
        return L.ea_cache_attention_split(ctypes.byref(a), 16, rows, sp, 4, capacity, parts.ctypes.data_as(_abi.P64), ctypes.byref(n))

    assert run(-1) == ARG and (parts == -5).all()
    assert run(0) == ARG and run(1) == ARG and run(64, rows=-1) == ARG
    assert run(64) == 0 and n.value > 1


def test_positions_and_rows_near_2_to_the_31_are_refused(L):  # noqa: F811
    """The kernels step over a sequence's end by a few thousand positions at most (a warp's pages of a tile) and by a
    tile of rows: what could pass 2^31 - 1 that way is refused."""
    c = cache(L)[1]
    k, v = rel(L, "bf16", (10, 2, 64)), rel(L, "bf16", (10, 2, 64), at=BASE + (1 << 20))
    q, o = rel(L, "bf16", (10, 6, 64)), rel(L, "bf16", (10, 6, 64), at=BASE + (1 << 20))
    need = ctypes.c_size_t()
    for pages in ((1 << 27) - 1, ((1 << 31) - 4096) // 16):
        b = ctypes.byref(batch(max_pages=pages))
        assert L.ea_cache_append(c, b, k, v, None) == UNSUP and L.ea_cache_read(c, b, k, v, None) == UNSUP
        assert L.ea_cache_attention_workspace(c, b, q, ctypes.byref(need)) == UNSUP
        assert L.ea_cache_attention(c, b, q, None, None, o) == UNSUP
        a, keep = host_batch(cu.Batch([(1, 1)], 16))
        a.max_pages = a.page_stride = pages
        assert L.ea_cache_check_batch(8, 16, ctypes.byref(a), 1, 1) == UNSUP
    big = 1 << 40
    one = cache(L, heads=1, k=BASE << 3, v=BASE << 4)[1]
    rows = (1 << 31) - 4096
    k, v = rel(L, "bf16", (rows, 1, 64), at=big), rel(L, "bf16", (rows, 1, 64), at=2 * big)
    assert L.ea_cache_append(one, ctypes.byref(batch(pages=BASE << 6, starts=BASE << 6, lens=BASE << 6)), k, v, None) == UNSUP


def test_what_a_call_writes_may_not_hold_the_batch(L):  # noqa: F811
    """The kernels read the table throughout a call: outputs and (append) the cache lie apart from it.  Only refusals:
    the addresses are never read."""
    at = BASE << 6
    c = cache(L)[1]
    k, v = rel(L, "bf16", (10, 2, 64)), rel(L, "bf16", (10, 2, 64), at=BASE + (1 << 20))
    q, o = rel(L, "bf16", (10, 6, 64)), rel(L, "bf16", (10, 6, 64), at=BASE + (1 << 20))
    m, l = rel(L, "f32", (10, 6), at=BASE + (1 << 21)), rel(L, "f32", (10, 6), at=BASE + (1 << 22))
    size, pool = 10 * 2 * 64 * 2, 8 * 2 * 16 * 64 * 2
    opts = _abi.CacheAttnOpts(0.0, 1, m.value, l.value, None, 0)
    for field, n in (("pages", (2 * 7 + 4) * 4), ("starts", 16), ("lens", 12)):
        def b(where):
            kw = dict(pages=at, starts=at + (1 << 16), lens=at + (1 << 17))
            kw[field] = where
            return ctypes.byref(batch(n_seqs=3, stride=7, **kw))
        for lo in (BASE << 1, BASE << 2):                            # the cache's K and V
            for where in (lo, lo + pool - 4, lo - n + 4):
                assert L.ea_cache_append(c, b(where), k, v, None) == ARG
        for lo in (BASE, BASE + (1 << 20)):                          # what a read writes
            for where in (lo, lo + size - 4, lo - n + 4):
                assert L.ea_cache_read(c, b(where), k, v, None) == ARG
        for lo in (BASE + (1 << 20), BASE + (1 << 21), BASE + (1 << 22)):
            for where in (lo, lo - n + 4):
                assert L.ea_cache_attention(c, b(where), q, ctypes.byref(opts), None, o) == ARG
