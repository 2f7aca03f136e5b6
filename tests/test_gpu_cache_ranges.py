"""GPU tests of the paged cache at the ends of its ranges.

Results are exact, or within cache_util.out_bound as in test_gpu_cache."""
import numpy as np
import pytest

import cache_util as cu
from test_gpu_cache import MARK, _built, bits, fill, nan_cache, on_gpu, relation  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ------------------------------------------------------------ whole batches

def spoiled(spoil):
    """Batch arrays with a sequence out of range that no row need lead to: (starts, lens, rows)."""
    starts, lens, rows = [0, 3, 5, 20, 21], [40, 40, 40, 40], 24
    if spoil == "last bound lower":
        starts, lens, rows = [0, 10, 4], [40, 40], 12
    elif spoil == "middle bound lower":
        starts = [0, 3, 1, 20, 21]
    elif spoil == "beyond the rows":
        starts, lens, rows = [30, 31, 33], [40, 40], 24
    elif spoil == "idle beyond the rows":
        starts, lens, rows = [0, 3, 20, 30, 30], [40, 40, 0, 40], 24
    elif spoil == "idle, negative length":
        starts, lens = [0, 3, 3, 20, 21], [40, -1, 40, 40]
    elif spoil == "idle, too long":
        starts, lens = [0, 3, 3, 20, 21], [40, 49, 40, 40]
    elif spoil == "negative rows":
        starts = [-5, -2, 5, 20, 21]
    elif spoil == "idle among many":
        starts, lens = list(range(21)) + [20] * 1500, [40] * 20 + [3] * 1499 + [-7]
    return starts, lens, rows


@pytest.mark.parametrize("spoil", ["last bound lower", "middle bound lower", "beyond the rows", "idle beyond the rows",
                                   "idle, negative length", "idle, too long", "negative rows", "idle among many"])
def test_append_and_read_check_every_sequence(spoil):
    """A sequence out of range is reported whether or not a row of the call leads to it, as the attention and the host
    check do; nothing is written but rows and slots of sequences that are in range."""
    from tensor_relational_einsum_gb300 import EaError, PageBatch, PagedCache, cache_append, cache_read
    from tensor_relational_einsum_gb300.relation import check
    starts, lens, rows = spoiled(spoil)
    n, page = len(lens), 16
    own = [i for i in range(n) if lens[i] == 40]                 # pages to the sequences that have positions
    table = np.zeros((n, 3), dtype=np.int32)
    table[own] = np.random.default_rng(30).permutation(3 * len(own)).reshape(-1, 3)
    c = PagedCache(3 * len(own), page, 2, 64)
    before = bits(c.k).copy()
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = PageBatch(torch.from_numpy(table).cuda(), torch.tensor(starts, **i32), torch.tensor(lens, **i32))
    with pytest.raises(EaError):
        batch.check(c, rows)
    x = relation(torch.ones(rows, 2, 64, dtype=torch.bfloat16, device="cuda"))
    y = relation(torch.ones(rows, 2, 64, dtype=torch.bfloat16, device="cuda"))
    cache_append(c, batch, x, y)
    with pytest.raises(EaError) as e:
        check()
    assert e.value.code == 10
    check()                                                      # reported once
    allowed, mine = np.zeros((c.pages, page), dtype=bool), np.zeros(rows, dtype=bool)
    for i, t in enumerate(lens):
        a, z = starts[i], starts[i + 1]
        if 0 <= a <= z <= rows and 0 <= t <= 48:
            pos = np.arange(t - (z - a), t)
            allowed[table[i, pos // page], pos % page] = True
            mine[a:z] = True
    changed = (bits(c.k) != before).any(axis=(1, 3))
    assert not (changed & ~allowed).any()
    outs = [torch.full((rows, 2, 64), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache_read(c, batch, *(relation(t) for t in outs))
    with pytest.raises(EaError) as e:
        check()
    assert e.value.code == 10
    for t in outs:
        assert (t[torch.from_numpy(~mine)] == MARK).all()


# ------------------------------------------------- reads before position 0

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_read_leaves_rows_before_position_0(fmt, dtype):
    """A batch may hold more rows of a sequence than positions (the attention takes it, the host check accepts it): the
    rows before position 0 stay as they were, the others are read, nothing is raised."""
    from tensor_relational_einsum_gb300 import cache_read
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(5, 3), (2, 0), (4, 40), (20, 17), (0, 7)], 16, behind=1)
    c = nan_cache(b, 3, 64, fmt)
    held = fill(c, b, np.random.default_rng(31))
    batch = on_gpu(b)
    batch.check(c, b.rows)
    want = np.full((2, b.rows, 3, 64), MARK)
    for i, (n, t) in enumerate(b.seqs):
        k = min(n, t)
        for w in range(2):
            want[w, int(b.starts[i + 1]) - k:int(b.starts[i + 1])] = held[i][w][t - k:]
    outs = [torch.full((b.rows, 3, 64), MARK, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
            for _ in range(2)]
    cache_read(c, batch, *(relation(t) for t in outs))
    check()
    for t, w in zip(outs, want):
        assert np.array_equal(t.double().cpu().numpy(), w)
