"""GPU tests of the paged cache at the ends of its ranges.

Results are exact, or within cache_util.out_bound as in test_gpu_cache."""
import ctypes

import numpy as np
import pytest

import cache_util as cu
from test_gpu_cache import MARK, _built, attend, bits, fill, nan_cache, on_gpu, relation, values, verify  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def put(c, b, held):
    """Write held[i] = [k, v] (float64 [t, heads, dim]) into the cache by the definitions; held becomes what it holds."""
    e4m3 = c.format == "e4m3"
    cells = [x.view(torch.uint8).cpu() if e4m3 else x.cpu() for x in (c.k, c.v)]
    scales = [x.cpu() for x in (c.k_scale, c.v_scale)] if e4m3 else None
    for i in range(len(b.lens)):
        pg, sl = b.places(i)
        if len(pg) == 0:
            continue
        for w in range(2):
            x = held[i][w]
            if e4m3:
                e = cu.e4m3_scale(x)
                y = cu.e4m3_round(x / np.exp2(e)[..., None])
                cells[w][pg, :, sl] = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[w][pg, :, sl] = torch.from_numpy((e + 127).astype(np.uint8))
                held[i][w] = y * np.exp2(e)[..., None]
            else:
                r = torch.from_numpy(x).to(torch.bfloat16)
                cells[w][pg, :, sl] = r
                held[i][w] = r.double().numpy()
    for x, y in zip((c.k, c.v), cells):
        x.copy_(y.view(torch.float8_e4m3fn) if e4m3 else y)
    if e4m3:
        c.k_scale.copy_(scales[0])
        c.v_scale.copy_(scales[1])
    return held


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


# ------------------------------------------------------- ends of the range

def rising(rng, b, heads, dim, step, size):
    """Keys whose scores with a query of 1 along axis 3 rise by `step` every 128 positions; values of `size`."""
    held = []
    for t in b.lens:
        k = np.zeros((int(t), heads, dim))
        k[:, :, 3] = (np.arange(t) // 128)[:, None] * step
        held.append([k, rng.normal(size=(int(t), heads, dim)) * size])
    return held


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,max_new", [(1, 1), (40, 40), (200, 200), (300, 0)])
def test_large_values_under_rising_scores(n, max_new, dim, fmt):
    """V near 2^80, every key tile's scores 50 (log2) above the one before: the sums that a running maximum leaves
    behind stay in range, in each kernel."""
    b = cu.Batch([(n, 700), (n, 1000)], 16)       # not cut: one running maximum from the first tile to the last
    c = nan_cache(b, 1, dim, fmt)
    rng = np.random.default_rng(32)
    held = put(c, b, rising(rng, b, 1, dim, 1.0, 2.0 ** 80))
    with ones_queries(50 * np.log(2.0), dim):
        attend(b, c, held, 2, rng, scale=1.0, max_new=max_new)


class ones_queries:
    """Within it, test_gpu_cache.values gives queries of `size` along axis 3 and nothing else."""

    def __init__(self, size, dim):
        self.size, self.dim = size, dim

    def __enter__(self):
        import test_gpu_cache as m
        self.module, self.was = m, m.values

        def q(rng, shape, spread=1.0):
            x = np.zeros(shape)
            x[..., 3] = self.size
            return torch.from_numpy(x).to(torch.bfloat16).double().numpy()
        m.values = q

    def __exit__(self, *a):
        self.module.values = self.was


@pytest.mark.parametrize("power", [-118, -112, 105, 110, 118])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 5, 50])
def test_keys_to_the_ends_of_the_scales(n, dim, power):
    """8-bit K at 2^power and Q at 2^-power: ordinary scores, whatever the scales are."""
    b = cu.Batch([(n, 333), (n, 1200)], 16)
    c = nan_cache(b, 1, dim, "e4m3")
    rng = np.random.default_rng(33)
    held = [[rng.normal(size=(int(t), 1, dim)) * s for s in (2.0 ** power, 1.0)] for t in b.lens]
    put(c, b, held)
    for max_new in (n, 0):
        attend(b, c, held, 4, rng, spread=2.0 ** -power, max_new=max_new)


@pytest.mark.parametrize("n", [5, 60])
def test_rows_without_keys_next_to_tiny_scores(n):
    """Rows that keep no key where Q and K are so small that a score's unit is not an fp32 number."""
    b = cu.Batch([(n, n - 4), (n, 2)], 16)
    c = nan_cache(b, 1, 64, "e4m3")
    rng = np.random.default_rng(34)
    held = [[rng.normal(size=(int(t), 1, 64)) * s for s in (2.0 ** -118, 1.0)] for t in b.lens]
    put(c, b, held)
    out = attend(b, c, held, 2, rng, spread=2.0 ** -12, max_new=n)
    assert not out[:4].any() and np.isfinite(out).all()


@pytest.mark.parametrize("kv,n,t,max_new", [(64, 1, 3000, 1), (160, 1, 512, 1), (4, 1, 500, 1), (2, 8, 6000, 8),
                                            (3, 60, 1000, 60), (2, 60, 4000, 60), (2, 300, 1000, 0)])
def test_small_values_keep_their_bits(kv, n, t, max_new):
    """8-bit V near 2^-120: the quotient by the row's sum and the unit of the sums meet far below fp32's normal
    numbers, and must not lose the result's bits."""
    b = cu.Batch([(n, t)] * 4, 16)
    c = nan_cache(b, kv, 64, "e4m3")
    rng = np.random.default_rng(35)
    held = [[rng.normal(size=(t, kv, 64)) * 0.125, (1.0 + rng.random((t, kv, 64))) * 2.0 ** -120] for _ in range(4)]
    put(c, b, held)
    q = values(rng, (b.rows, kv, 64))
    tq = torch.from_numpy(q).to(torch.bfloat16).cuda()
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    out = cache_attention(relation(tq), c, on_gpu(b, max_new=max_new)).to_dense().double().cpu().numpy() * 2.0 ** 120
    check()
    for h in held:
        h[1] = h[1] * 2.0 ** 120
    verify(b, c, held, 1, q, out, None, None, True, 0.0, False, np.ones(b.rows, dtype=bool))


@pytest.mark.parametrize("dim", [64, 128])
def test_read_of_the_smallest_cells(dim):
    """Every code under the least scales: an fp32 read is exact, a bf16 read (whose least step is 2^-133) the nearest
    bf16 value."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, cache_read
    from tensor_relational_einsum_gb300.relation import check
    c = PagedCache(4, 16, 4, dim, "e4m3")
    codes = torch.arange(256, dtype=torch.int64).repeat(16 * 4 * 4 * dim // 256)
    codes[codes % 128 == 127] = 0                                 # no NaN codes
    c.k.copy_(codes.to(torch.uint8).view(torch.float8_e4m3fn).view(4, 4, 16, dim))
    c.v.copy_(c.k)
    byte = (torch.arange(4 * 4 * 16) // 4 % 4).to(torch.uint8).view(4, 4, 16)
    c.k_scale.copy_(byte)
    c.v_scale.copy_(byte)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = PageBatch(torch.arange(4, **i32)[None], torch.tensor([0, 64], **i32), torch.tensor([64], **i32))
    exact = c.k.cpu().double() * torch.exp2(byte.double() - 127)[..., None]
    exact = exact.permute(0, 2, 1, 3).reshape(64, 4, dim)
    k, v = cache_read(c, batch, rows=64, dtype="f32")
    check()
    assert torch.equal(k.to_dense().cpu().double(), exact) and torch.equal(v.to_dense().cpu().double(), exact)
    k, v = cache_read(c, batch, rows=64)
    check()
    # the nearest multiple of 2^-133, ties to even (all values lie below 2^-117: steps of more than 2^-133 hold 4 bits exactly)
    near = np.where(np.abs(exact.numpy()) < 2.0 ** -126, np.round(exact.numpy() * 2.0 ** 133) * 2.0 ** -133, exact.numpy())
    for t in (k, v):
        assert np.array_equal(t.to_dense().cpu().double().numpy(), near)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_finite_rows(dtype):
    """Rows up to the largest finite value: from 1.9375 * 2^127 on the nearest code is 256 under 2^120, infinity in fp32;
    below, the cell is the nearest code's value."""
    from tensor_relational_einsum_gb300 import cache_append, cache_read
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(3, 3)], 16)
    c = nan_cache(b, 1, 64, "e4m3")
    x = torch.ones(3, 1, 64, dtype=torch.float64) * 2.0 ** 120
    x[:, 0, 7] = torch.tensor([1.9375 * 2.0 ** 127, 1.9296875 * 2.0 ** 127, 1.75 * 2.0 ** 127], dtype=torch.float64)
    t = x.to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    cache_append(c, on_gpu(b), relation(t), relation(t.clone()))
    k, v = cache_read(c, on_gpu(b), rows=3, dtype="f32")
    check()
    for g in (k.to_dense().cpu().double(), v.to_dense().cpu().double()):
        assert g[0, 0, 7] == float("inf") and (g[0, 0, 8:] == 2.0 ** 120).all()
        assert g[1, 0, 7] == 1.875 * 2.0 ** 127 and g[2, 0, 7] == 1.75 * 2.0 ** 127


# --------------------------------------------------------- the workspace

def scaled_fill(c, b, rng):
    """Values of every sequence at a size of its own (8-bit scales that differ between the items of a CTA)."""
    held = [[rng.normal(size=(int(t), c.heads, c.dim)), rng.normal(size=(int(t), c.heads, c.dim)) * 2.0 ** rng.integers(-12, 13)]
            for t in b.lens]
    return put(c, b, held)


def workspace(c, batch, rows, heads):
    from tensor_relational_einsum_gb300 import Relation, _abi
    need = ctypes.c_size_t()
    q = Relation("bf16", (rows, heads, c.dim), [1, 1, 1], device="cuda")
    _abi.check_status(_abi.lib().ea_cache_attention_workspace(c.handle, batch.ref, q.handle, ctypes.byref(need)))
    return need.value


def test_workspace_of_a_step_without_a_promise():
    """64 single tokens, 64 heads over 8 of 128, room for 8192 positions, max_new not given: 8-bit pages are expanded for
    at most the 12 sequences that 64 rows can bring above 32 rows of a group, not for all 64."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache
    c = PagedCache(8, 128, 8, 128, "e4m3")
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = PageBatch(torch.zeros(64, 64, **i32), torch.arange(65, **i32), torch.ones(64, **i32))
    wide = 12 * 8192 * 8 * 128 * 4
    assert wide <= workspace(c, batch, 64, 64) <= wide + (100 << 20)
    short = PageBatch(torch.zeros(64, 64, **i32), torch.arange(65, **i32), torch.ones(64, **i32), max_new=1)
    assert workspace(c, short, 64, 64) <= 100 << 20


@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (40, 64)])
def test_chunks_among_many_idle_sequences(group, dim):
    """Far more sequences than rows could serve: the expanded pages are numbered by rows."""
    n = -(-256 // group)
    seqs = [(0, 30)] * 40 + [(n, n + 200)] + [(0, 0)] * 30 + [(2, 50)] * 3 + [(0, 9)] * 5 + [(n + 5, n + 5), (0, 3), (n // 4 + 1, 300)]
    seqs += [(0, 5)] * 600 + [(1, 7)]
    b = cu.Batch(seqs, 16, before=3, behind=5)
    c = nan_cache(b, 2, dim, "e4m3")
    rng = np.random.default_rng(40)
    attend(b, c, scaled_fill(c, b, rng), group, rng)


def test_overlapping_sequences_of_expanded_pages_are_reported():
    """Bounds that go back and forth, so that more sequences seem to have long chunks than the rows allow: the error is
    raised and rows of no sequence stay as they were."""
    from tensor_relational_einsum_gb300 import EaError, PageBatch, PagedCache, cache_attention
    from tensor_relational_einsum_gb300.relation import check
    c = PagedCache(8, 16, 2, 64, "e4m3")
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = PageBatch(torch.zeros(200, 8, **i32), torch.tensor([0, 60] * 100 + [0], **i32), torch.full((200,), 100, **i32))
    q = torch.randn(64, 16, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, MARK)
    cache_attention(relation(q), c, batch, out=relation(out))
    with pytest.raises(EaError) as e:
        check()
    assert e.value.code == 10
    assert (out[60:] == MARK).all()


# -------------------------------------------------- CTAs with many items

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [60, 0])
def test_chunks_many_whole_items_a_cta(max_new, dim, fmt):
    """More than 900 items of up to 1024 positions: a CTA takes six or more, one after the other (max_new 60: 8-bit pages
    are read as they are; 0: they are expanded)."""
    rng = np.random.default_rng(36)
    seqs = [(int(n), int(n + t)) for n, t in zip(rng.integers(33, 61, size=120), rng.integers(0, 300, size=120))]
    seqs[7], seqs[50], seqs[90] = (60, 1000), (40, 0), (60, 37)
    b = cu.Batch(seqs, 16, behind=2)
    c = nan_cache(b, 8, dim, fmt)
    attend(b, c, scaled_fill(c, b, rng), 1, rng, max_new=max_new)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [85, 0])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_tails_wholes_and_heads_a_cta(causal, max_new, dim, fmt):
    """More than 600 units of 128 keys in items of 1 to 12 of them, several items to a head (84 tokens each): a CTA holds
    an item's tail, whole items and another's head."""
    rng = np.random.default_rng(37)
    seqs = [(int(n), int(n + t)) for n, t in zip(rng.integers(70, 86, size=12), rng.integers(0, 700, size=12))]
    seqs[3], seqs[5], seqs[8] = (85, 1500), (85, 60), (20, 900)
    b = cu.Batch(seqs, 32, before=1)
    c = nan_cache(b, 8, dim, fmt)
    attend(b, c, scaled_fill(c, b, rng), 3, rng, max_new=max_new, causal=causal)


@pytest.mark.parametrize("group,n", [(3, 85), (5, 51), (33, 7), (127, 2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_raw_pages_under_several_items(group, n, dim):
    """Fewer than 256 rows of a sequence in two items a head, 8-bit pages read as they are."""
    b = cu.Batch([(n, 400), (n, n), (n - 1, 1300), (n, 3)], 16)
    c = nan_cache(b, 2, dim, "e4m3")
    rng = np.random.default_rng(38)
    attend(b, c, scaled_fill(c, b, rng), group, rng, max_new=n)


@pytest.mark.parametrize("dim", [64, 128])
def test_raw_pages_where_the_expansion_has_no_room(dim):
    """A table so wide that expanded pages could pass 4 GB: long chunks over the 8-bit pages themselves."""
    b = cu.Batch([(600, 900), (1, 50), (300, 2500)], 128, extra_pages=1 << 16)
    c = nan_cache(b, 2, dim, "e4m3")
    rng = np.random.default_rng(39)
    attend(b, c, scaled_fill(c, b, rng), 2, rng)


def test_a_workspace_over_the_batch_is_refused():
    from tensor_relational_einsum_gb300 import PageBatch, _abi
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(1, 2000), (40, 900)], 16)
    c = nan_cache(b, 1, 64, "bf16")
    rng = np.random.default_rng(41)
    held = fill(c, b, rng)
    q = values(rng, (b.rows, 2, 64))
    rq = relation(torch.from_numpy(q).to(torch.bfloat16).cuda())
    out = torch.full((b.rows, 2, 64), MARK, dtype=torch.bfloat16, device="cuda")
    ro, L = relation(out), _abi.lib()
    first = on_gpu(b)
    need = workspace(c, first, b.rows, 2)
    room = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    opts = _abi.CacheAttnOpts(0.0, 1, None, None, room.data_ptr(), need)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for at, want in ((need - 4, 7), (0, 7), (need, 0)):             # the lengths' place in the buffer; beyond the workspace
        lens = room[at:at + 8].view(torch.int32)
        batch = PageBatch(first.pages, first.starts, lens)
        lens.copy_(first.lens)
        assert L.ea_cache_attention(c.handle, batch.ref, rq.handle, ctypes.byref(opts), stream, ro.handle) == want
        if want:
            assert (out == MARK).all()
    check()
    verify(b, c, held, 2, q, out.double().cpu().numpy(), None, None, True, 0.0, False, np.ones(b.rows, dtype=bool))
