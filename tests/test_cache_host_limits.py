"""CPU tests of what the paged cache's entry points refuse at the ends of their
ranges (arguments are checked before any device is touched)."""
import ctypes

import numpy as np

import cache_util as cu
from tensor_relational_einsum_gb300 import _abi
from test_cache_host import ARG, L, host_batch  # noqa: F401


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
