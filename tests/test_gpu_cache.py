"""GPU tests of the paged cache (append, read, attention) against the 64-bit
definitions in cache_util.

Every cache starts full of NaN, so that a cell outside the sequences' own
positions (pages of no sequence, slots behind the last position) that reached
a result would show; dense rows of no sequence hold NaN or a mark and must
stay as they are.

Tolerances: append and read are exact (codes, scale bytes and rounded cells
bit for bit).  Attention: cache_util.out_bound, elementwise -- half a bf16
step for the output, half a step for every probability, and the fp32 error of
scores, exponentials and sums; m within the scores' error, l within that
relative to exp plus its sum's.
"""
import numpy as np
import pytest

import cache_util as cu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MARK = -7.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tensor_relational_einsum_gb300.build import build
    build()
    yield
    from tensor_relational_einsum_gb300.relation import check
    check()


def relation(t):
    from tensor_relational_einsum_gb300 import Relation
    return Relation("f32" if t.dtype == torch.float32 else "bf16", t.shape, [1] * t.dim(), storage=t.reshape(-1))


def on_gpu(b: cu.Batch, max_new=0, strided=False):
    from tensor_relational_einsum_gb300 import PageBatch
    pages = torch.from_numpy(b.pages).cuda()
    if strided:
        wide = torch.full((pages.shape[0], pages.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
        wide[:, :pages.shape[1]] = pages
        pages = wide[:, :pages.shape[1]]
    return PageBatch(pages, torch.from_numpy(b.starts).cuda(), torch.from_numpy(b.lens).cuda(), max_new=max_new)


def nan_cache(b, heads, dim, fmt):
    """A cache whose every cell is NaN (e4m3: NaN scales over the largest codes)."""
    from tensor_relational_einsum_gb300 import PagedCache
    shape = (b.pages_total, heads, b.page, dim)
    if fmt == "bf16":
        k, v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return PagedCache(b.pages_total, b.page, heads, dim, fmt, k=k, v=v)
    k, v = (torch.full(shape, 0x7e, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full(shape[:3], 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    return PagedCache(b.pages_total, b.page, heads, dim, fmt, k=k, v=v, k_scale=ks, v_scale=vs)


def values(rng, shape, spread=1.0):
    """bf16 values as float64."""
    t = torch.from_numpy(rng.normal(size=shape) * spread).to(torch.bfloat16)
    return t.double().numpy()


def fill(c, b, rng, spread=1.0):
    """Put values for every position of every sequence into the cache, by the definitions; returns per sequence (k, v)
    float64 [t, heads, dim] as the cache holds them."""
    held = []
    kc, vc = (x.view(torch.uint8).cpu() if c.format == "e4m3" else x.cpu() for x in (c.k, c.v))
    sc = [x.cpu() for x in (c.k_scale, c.v_scale)] if c.format == "e4m3" else [None, None]
    for i in range(len(b.lens)):
        pg, sl = b.places(i)
        pair = []
        for cells, scale in ((kc, sc[0]), (vc, sc[1])):
            x = values(rng, (int(b.lens[i]), c.heads, c.dim), spread)
            if c.format == "e4m3" and len(x):
                e = cu.e4m3_scale(x)
                y = cu.e4m3_round(x / np.exp2(e)[..., None])
                cells[pg, :, sl] = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8)
                scale[pg, :, sl] = torch.from_numpy((e + 127).astype(np.uint8))
                x = y * np.exp2(e)[..., None]
            elif len(x):
                cells[pg, :, sl] = torch.from_numpy(x).to(torch.bfloat16)
            pair.append(x)
        held.append(pair)
    c.k.copy_(kc.view(torch.float8_e4m3fn) if c.format == "e4m3" else kc)
    c.v.copy_(vc.view(torch.float8_e4m3fn) if c.format == "e4m3" else vc)
    if c.format == "e4m3":
        c.k_scale.copy_(sc[0])
        c.v_scale.copy_(sc[1])
    return held


def bits(t):
    t = t.cpu()
    return t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.view(torch.uint8).numpy()


# ------------------------------------------------------------ append, read

ROWS = [
    # heads, dim, page, sequences (rows, positions)
    (1, 64, 16, [(1, 1)]),
    (8, 128, 16, [(1, t) for t in (1, 15, 16, 17, 32, 100, 333)]),
    (5, 64, 32, [(7, 7), (0, 3), (33, 40), (0, 0), (1, 64), (65, 200)]),
    (3, 128, 64, [(200, 200), (64, 128), (63, 129)]),
    (32, 128, 128, [(130, 300)]),
    (2, 64, 16, [(3, 5)] * 300),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page,seqs", ROWS)
def test_append_and_read(heads, dim, page, seqs, fmt, dtype):
    from tensor_relational_einsum_gb300 import cache_append, cache_read
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch(seqs, page, before=2, behind=3, seed=1)
    c = nan_cache(b, heads, dim, fmt)
    rng = np.random.default_rng(2)
    dense = []
    for _ in range(2):
        x = rng.normal(size=(b.rows, heads, dim)) * np.exp(3.0 * rng.normal(size=(b.rows, heads, 1)))
        x[b.rows // 2, heads // 2] = 0.0                                   # a vector of zeros
        x[int(b.starts[0]), 0, :2] = (448.0, -448.0) if dim == 64 else (449.0, 1.0)
        t = torch.from_numpy(x).to(torch.float32 if dtype == "f32" else torch.bfloat16)
        t[:2] = float("nan")
        t[b.rows - 3:] = float("inf")
        dense.append(t)
    before = [bits(x).copy() for x in ((c.k, c.v, c.k_scale, c.v_scale) if fmt == "e4m3" else (c.k, c.v))]
    kr, vr = (relation(t.cuda()) for t in dense)
    batch = on_gpu(b, strided=True)
    cache_append(c, batch, kr, vr)
    check()
    want, exact = before, []
    for w, t in enumerate(dense):
        x = t.double().numpy()
        got_rows = np.zeros((b.rows, heads, dim))
        for i in range(len(seqs)):
            n = seqs[i][0]
            if n == 0:
                continue
            pg, sl = (y[-n:] for y in b.places(i))
            y = x[b.rows_of(i)]
            if fmt == "e4m3":
                e = cu.e4m3_scale(y)
                code = cu.e4m3_round(y / np.exp2(e)[..., None])
                want[w][pg, :, sl] = torch.from_numpy(code).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                want[2 + w][pg, :, sl] = (e + 127).astype(np.uint8)
                y = code * np.exp2(e)[..., None]
            else:
                r = torch.from_numpy(y).float().to(torch.bfloat16)
                want[w][pg, :, sl] = bits(r)
                y = r.double().numpy()
            got_rows[b.rows_of(i)] = y
        exact.append(got_rows)
    after = [bits(x) for x in ((c.k, c.v, c.k_scale, c.v_scale) if fmt == "e4m3" else (c.k, c.v))]
    for g, w in zip(after, want):
        # -0 and 0 are both right where the reference divides a negative zero
        assert np.array_equal(g, w)
    # read back: rows of no sequence keep their mark
    outs = [torch.full((b.rows, heads, dim), MARK, dtype=torch.float32 if dtype == "f32" else torch.bfloat16,
                       device="cuda") for _ in range(2)]
    cache_read(c, batch, *(relation(t) for t in outs))
    check()
    for t, w in zip(outs, exact):
        g = t.double().cpu().numpy()
        assert (g[:2] == MARK).all() and (g[b.rows - 3:] == MARK).all()
        assert np.array_equal(g[2:b.rows - 3], w[2:b.rows - 3])


def test_read_into_new_rows_and_other_dtype():
    from tensor_relational_einsum_gb300 import cache_read
    b = cu.Batch([(20, 50), (9, 9)], 16)
    c = nan_cache(b, 2, 64, "e4m3")
    held = fill(c, b, np.random.default_rng(3))
    k, v = cache_read(c, on_gpu(b), rows=b.rows)
    assert k.dtype == "bf16"
    want = np.concatenate([held[i][0][-n:] for i, (n, _) in enumerate(b.seqs)])
    assert np.array_equal(k.to_dense().double().cpu().numpy(), want)     # every cell is a bf16 value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_vectors_that_are_not_finite(dtype):
    from tensor_relational_einsum_gb300 import cache_append, cache_read
    b = cu.Batch([(6, 6)], 16)
    c = nan_cache(b, 1, 64, "e4m3")
    t = torch.ones(6, 1, 64, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    t[0, 0, 5], t[1, 0, 63], t[2, 0, 0] = float("inf"), float("nan"), -float("inf")
    t[3] *= 2.0 ** -130           # subnormal in fp32 and bf16: the scale stops at 2^-126
    t[4] *= 3.0e38
    cache_append(c, on_gpu(b), relation(t), relation(t.clone()))
    s = c.k_scale.cpu()[b.pages[0, 0], 0, :6].tolist()
    assert s[:3] == [255] * 3 and s[3] == 1 and s[5] == 127 - 8
    k, _ = cache_read(c, on_gpu(b), rows=6, dtype="f32")
    g = k.to_dense().cpu()
    assert torch.isnan(g[:3]).all() and torch.isfinite(g[3:]).all()
    assert (g[3] == 2.0 ** -130).all() and (g[5] == 1).all()
    assert ((g[4].double() / t[4].double().cpu() - 1).abs() <= 2.0 ** -4).all()


def test_rows_of_a_tiled_relation():
    """Rows over (batch, position) dimensions in blocks, as a block's K and V are laid out."""
    from tensor_relational_einsum_gb300 import Relation, cache_append, cache_read
    b = cu.Batch([(64, 64), (64, 70)], 16)
    c = nan_cache(b, 2, 64, "bf16")
    x = torch.randn(2, 64, 2, 64, device="cuda").to(torch.bfloat16)
    r = Relation.from_dense(x, [2, 4, 1, 1])
    cache_append(c, on_gpu(b), r, r)
    k, v = cache_read(c, on_gpu(b), rows=128)
    assert torch.equal(k.to_dense().view(2, 64, 2, 64), x) and torch.equal(v.to_dense().view(2, 64, 2, 64), x)


# --------------------------------------------------------------- attention

def attend(b, c, held, group, rng, causal=True, scale=0.0, stats=True, spread=1.0, max_new=0, rows=None, run=None):
    """Run the attention on random queries and hold every row to its bound."""
    from tensor_relational_einsum_gb300 import _abi, cache_attention
    from tensor_relational_einsum_gb300.relation import check
    heads = c.heads * group
    q = values(rng, (b.rows, heads, c.dim), spread)
    tq = torch.from_numpy(q).to(torch.bfloat16)
    inside = np.zeros(b.rows, dtype=bool)
    for i in range(len(b.lens)):
        inside[b.rows_of(i)] = True
    tq[~torch.from_numpy(inside)] = float("nan")
    tq = tq.cuda()
    out = torch.full((b.rows, heads, c.dim), MARK, dtype=torch.bfloat16, device="cuda")
    m, l = (torch.full((b.rows, heads), MARK, device="cuda") for _ in range(2))
    batch = on_gpu(b, max_new=max_new)
    (run or (lambda f: f()))(lambda: cache_attention(
        relation(tq), c, batch, scale=scale, causal=causal, out=relation(out),
        m_out=relation(m) if stats else None, l_out=relation(l) if stats else None))
    check()
    assert _abi.last_plan()["kernel"] == "cache_attention"
    out, m, l = (t.double().cpu().numpy() for t in (out, m, l))
    verify(b, c, held, group, q, out, m, l, causal, scale, stats, inside)
    return out


def verify(b, c, held, group, q, out, m, l, causal, scale, stats, inside):
    sc = scale or 1.0 / np.sqrt(c.dim)
    sc = float(np.float32(sc))
    for i, (n, t) in enumerate(zip(np.diff(b.starts), b.lens)):
        if n == 0:
            continue
        pos = t - n + np.arange(n)
        for h in range(c.heads * group):
            k, v = (x[:, h // group] for x in held[i])
            wo, wm, wl, big, slack = cu.softmax_attention(q[b.rows_of(i), h], k, v, pos, sc, causal)
            err = np.abs(out[b.rows_of(i), h] - wo)
            assert (err <= cu.out_bound(wo, big, slack, t)).all(), (i, h, err.max())
            if not stats:
                continue
            empty = wl == 0
            gm, gl = m[b.rows_of(i), h], l[b.rows_of(i), h]
            assert (gm[empty] == -np.inf).all() and (gl[empty] == 0).all()
            gm, gl, wm, wl, slack = (x[~empty] for x in (gm, gl, wm, wl, slack))
            assert (np.abs(gm - wm) <= slack + 2.0 ** -23 * np.abs(wm)).all(), (i, h)
            rel = 2.0 * np.expm1(slack) + 2.0 ** -18 + 4.0 * t * 2.0 ** -24
            assert (np.abs(gl - wl) <= rel * wl).all(), (i, h, np.abs(gl / wl - 1).max())
    assert (out[~inside] == MARK).all()
    if stats:
        assert (m[~inside] == MARK).all() and (l[~inside] == MARK).all()


ATTEND = [
    # key-value heads, group, dim, page, sequences (rows, positions)
    (1, 1, 64, 16, [(1, 1)]),
    (2, 4, 128, 16, [(1, t) for t in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000)]),
    (3, 7, 64, 32, [(1, 31), (0, 40), (2, 32), (4, 33), (1, 500)]),
    (1, 16, 128, 64, [(1, 77), (2, 700), (1, 128)]),
    (1, 32, 128, 16, [(1, 300)]),
    (1, 33, 64, 16, [(1, 129)]),
    (1, 128, 64, 128, [(1, 200), (2, 300), (3, 3)]),
    (1, 100, 128, 32, [(3, 290)]),
    (2, 1, 128, 16, [(5, 5), (17, 40), (33, 161), (0, 0), (16, 16), (31, 1025)]),
    (2, 4, 128, 16, [(8, 8), (9, 200), (32, 33), (33, 500), (64, 64), (65, 300)]),
    (1, 4, 64, 64, [(129, 129), (300, 411), (1, 513)]),
    (1, 1, 128, 128, [(128, 128), (129, 300), (257, 700), (256, 256), (1, 128)]),
    (2, 3, 64, 32, [(85, 99), (86, 170), (43, 43)]),
    (1, 5, 128, 16, [(26, 77), (25, 512), (52, 53)]),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kv,group,dim,page,seqs", ATTEND)
def test_attention(kv, group, dim, page, seqs, fmt):
    b = cu.Batch(seqs, page, before=1, behind=2, seed=5)
    c = nan_cache(b, kv, dim, fmt)
    rng = np.random.default_rng(6)
    held = fill(c, b, rng)
    attend(b, c, held, group, rng)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 4])
def test_rows_without_keys_and_no_causality(fmt, group):
    """Causal rows before position 0 and sequences without positions keep no key; without causality rows may outnumber
    positions."""
    seqs = [(3, 1), (5, 0), (40, 33), (1, 0), (200, 130), (2, 300), (0, 5)]
    b = cu.Batch(seqs, 32, behind=1)
    c = nan_cache(b, 2, 64, fmt)
    rng = np.random.default_rng(7)
    held = fill(c, b, rng)
    out = attend(b, c, held, group, rng, causal=True)
    assert not out[0:2].any() and not out[3:8].any()
    attend(b, c, held, group, rng, causal=False)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,t,kv,group,dim", [(1, 20000, 1, 4, 128), (1, 9999, 2, 1, 64), (7, 12000, 1, 4, 128),
                                              (40, 9000, 1, 2, 128), (200, 5000, 1, 1, 64), (300, 6001, 1, 2, 128)])
def test_long_axis_is_split(n, t, kv, group, dim, fmt):
    b = cu.Batch([(n, t), (1, 3)], 64)
    c = nan_cache(b, kv, dim, fmt)
    rng = np.random.default_rng(8)
    held = fill(c, b, rng)
    attend(b, c, held, group, rng)


@pytest.mark.parametrize("n", [1, 60])
def test_peaked_scores_and_wide_values(n):
    """Scores that spread over hundreds of units (the maximum moves late and far), values of very different size."""
    b = cu.Batch([(n, 700), (n, 1500)], 16)
    c = nan_cache(b, 2, 128, "bf16")
    rng = np.random.default_rng(9)
    held = fill(c, b, rng, spread=4.0)
    attend(b, c, held, 2, rng, scale=1.0, spread=4.0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_scores_that_rise_along_the_positions(fmt):
    b = cu.Batch([(1, 900), (50, 950)], 16)
    c = nan_cache(b, 1, 64, fmt)
    rng = np.random.default_rng(10)
    held = fill(c, b, rng)
    for i in range(2):      # key t is t / 20 along one axis: every tile moves the maximum
        pg, sl = b.places(i)
        x = np.zeros((int(b.lens[i]), 1, 64))
        x[:, 0, 3] = np.arange(b.lens[i]) // 20
        if fmt == "e4m3":
            e = cu.e4m3_scale(x)
            code = cu.e4m3_round(x / np.exp2(e)[..., None])
            kc = c.k.view(torch.uint8).cpu()
            kc[pg, :, sl] = torch.from_numpy(code).to(torch.float8_e4m3fn).view(torch.uint8)
            c.k.copy_(kc.cuda().view(torch.float8_e4m3fn))
            ks = c.k_scale.cpu()
            ks[pg, :, sl] = torch.from_numpy((e + 127).astype(np.uint8))
            c.k_scale.copy_(ks)
            x = code * np.exp2(e)[..., None]
        else:
            kc = c.k.cpu()
            kc[pg, :, sl] = torch.from_numpy(x).to(torch.bfloat16)
            c.k.copy_(kc)
        held[i][0] = x
    attend(b, c, held, 1, rng, scale=1.0, spread=3.0)


def test_shared_pages_and_many_sequences():
    """Sequences that share their first pages, more sequences than threads of a block, promised chunk bound."""
    seqs = [(1, 40 + 3 * (i % 50)) for i in range(700)]
    b = cu.Batch(seqs, 16)
    c = nan_cache(b, 1, 64, "bf16")
    rng = np.random.default_rng(11)
    held = fill(c, b, rng)
    for i in range(1, 700, 7):
        b.pages[i, :2] = b.pages[0, :2]
        for w in range(2):
            held[i][w][:32] = held[0][w][:32]
    attend(b, c, held, 2, rng, max_new=1)


def test_mixed_chunks_in_one_batch():
    """Single tokens and long chunks side by side, idle sequences between them."""
    seqs = [(1, 300), (0, 100), (150, 400), (1, 1), (0, 0), (1, 2000), (40, 40), (3, 90), (129, 1000)]
    for fmt in ("bf16", "e4m3"):
        b = cu.Batch(seqs, 32, before=3, behind=4)
        c = nan_cache(b, 2, 64, fmt)
        rng = np.random.default_rng(12)
        held = fill(c, b, rng)
        attend(b, c, held, 4, rng, max_new=150)
        attend(b, c, held, 1, rng, stats=False)


def test_batch_out_of_range_is_reported_and_left_out():
    """Bad pages, rows and lengths (all caught by the kernels' own checks; the host check refuses the same batch):
    ea_check reports them, the other sequences' rows are right."""
    from tensor_relational_einsum_gb300 import EaError, cache_append, cache_attention, cache_read
    from tensor_relational_einsum_gb300.relation import check
    seqs = [(2, 50), (3, 60), (40, 70), (1, 33)]
    for spoil in ("page", "negative", "len", "start", "new"):
        b = cu.Batch(seqs, 16)
        c = nan_cache(b, 1, 64, "bf16")
        rng = np.random.default_rng(13)
        held = fill(c, b, rng)
        max_new = 0
        good = [0, 2, 3]
        if spoil == "page":
            b.pages[1, 3] = b.pages_total
        elif spoil == "negative":
            b.pages[1, 3] = -1
        elif spoil == "len":
            b.lens[1] = b.max_pages * 16 + 1
        elif spoil == "start":
            b.starts[4] = 1 << 20
            good = [0, 1, 2]
        else:
            max_new, good = 3, [0, 1, 3]
        batch = on_gpu(b, max_new=max_new)
        with pytest.raises(EaError):
            batch.check(c, b.rows)
        q = values(rng, (b.rows, 2, 64))
        tq = torch.from_numpy(q).to(torch.bfloat16).cuda()
        out = torch.full_like(tq, MARK)
        cache_attention(relation(tq), c, batch, out=relation(out))
        with pytest.raises(EaError) as e:
            check()
        assert e.value.code == 10
        check()                                            # reported once
        got = out.double().cpu().numpy()
        for i in good:
            n, t = seqs[i]
            for h in range(2):
                k, v = (x[:, 0] for x in held[i])
                wo, _, _, big, slack = cu.softmax_attention(q[b.rows_of(i), h], k, v, t - n + np.arange(n), 0.125, True)
                assert (np.abs(got[b.rows_of(i), h] - wo) <= cu.out_bound(wo, big, slack, t)).all()
        rows = relation(torch.ones(b.rows, 1, 64, dtype=torch.bfloat16, device="cuda"))
        cells = bits(c.k).copy()
        cache_append(c, batch, rows, relation(torch.ones(b.rows, 1, 64, dtype=torch.bfloat16, device="cuda")))
        with pytest.raises(EaError):
            check()
        changed = (bits(c.k) != cells).any(axis=(1, 3))
        allowed = np.zeros_like(changed)
        for i, (n, t) in enumerate(seqs):
            if i == 1 and spoil in ("page", "negative", "len") and spoil == "len":
                continue
            pg, sl = np.array(b.pages[i, np.arange(t - n, t) // 16]), np.arange(t - n, t) % 16
            ok = (pg >= 0) & (pg < b.pages_total)
            allowed[pg[ok], sl[ok]] = True
        assert not (changed & ~allowed).any()
        cache_read(c, batch, rows, relation(torch.ones(b.rows, 1, 64, dtype=torch.bfloat16, device="cuda")))
        with pytest.raises(EaError):
            check()


# --------------------------------------------------- streams, graphs, runs

def test_other_stream_and_captured_graph():
    """A call on another stream than the current one; a captured call replayed on a batch that grew in place."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(1, 200), (2, 900), (40, 300)], 16, extra_pages=4, spare=30)
    c = nan_cache(b, 2, 64, "bf16")
    rng = np.random.default_rng(14)
    held = fill(c, b, rng)
    side = torch.cuda.Stream()

    def on_side(f):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)

    attend(b, c, held, 2, rng, run=on_side)
    q = values(rng, (b.rows, 4, 64))
    tq = torch.from_numpy(q).to(torch.bfloat16).cuda()
    out = torch.full_like(tq, MARK)
    batch = on_gpu(b)
    r, o = relation(tq), relation(out)
    side.wait_stream(torch.cuda.current_stream())
    cache_attention(r, c, batch, out=o, stream=side)         # the stream argument
    side.synchronize()
    inside = np.ones(b.rows, dtype=bool)
    first = out.double().cpu().numpy()
    verify(b, c, held, 2, q, first, None, None, True, 0.0, False, inside)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        cache_attention(r, c, batch, out=o)
    out.fill_(MARK)
    g.replay()
    check()
    assert np.array_equal(out.double().cpu().numpy(), first)  # the same bits: no sum depends on who comes first
    # the same graph on a longer batch: lengths and a page more, written into the same tensors
    b2 = cu.Batch([(1, 216), (2, 916), (40, 316)], 16, extra_pages=3, spare=27, seed=3)
    b2.pages_total = b.pages_total
    held2 = fill(c, b2, rng)
    batch.pages.copy_(torch.from_numpy(np.pad(b2.pages, ((0, 0), (0, b.max_pages - b2.max_pages)), constant_values=-1)))
    batch.lens.copy_(torch.from_numpy(b2.lens))
    g.replay()
    check()
    verify(b2, c, held2, 2, q, out.double().cpu().numpy(), None, None, True, 0.0, False, inside)


def test_two_calls_at_once_and_two_graphs():
    """Calls that overlap on two streams, and two captured graphs replayed at the same time."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(15)
    jobs = []
    for seed, seqs in ((1, [(1, 6000), (1, 4000)]), (2, [(64, 3000), (1, 5000)])):
        b = cu.Batch(seqs, 16, seed=seed)
        c = nan_cache(b, 2, 128, "bf16")
        held = fill(c, b, rng)
        q = values(rng, (b.rows, 8, 128))
        tq = torch.from_numpy(q).to(torch.bfloat16).cuda()
        out = torch.full_like(tq, MARK)
        jobs.append((b, c, held, q, out, relation(tq), relation(out), on_gpu(b), torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for rep in range(5):
        for b, c, held, q, out, r, o, batch, s in jobs:
            with torch.cuda.stream(s):
                cache_attention(r, c, batch, out=o)
    torch.cuda.synchronize()
    ref = [j[4].clone() for j in jobs]
    for b, c, held, q, out, r, o, batch, s in jobs:
        verify(b, c, held, 4, q, out.double().cpu().numpy(), None, None, True, 0.0, False, np.ones(b.rows, dtype=bool))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="thread_local"):
            cache_attention(r, c, batch, out=o)
        graphs.append(g)
        out.fill_(MARK)
    torch.cuda.synchronize()
    for rep in range(10):
        for g, j in zip(graphs, jobs):
            with torch.cuda.stream(j[8]):
                g.replay()
    torch.cuda.synchronize()
    check()
    for j, w in zip(jobs, ref):
        assert torch.equal(j[4], w)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_generation_as_a_run(fmt):
    """A prompt in two chunks, then single tokens: append and attend, step by step, against the definition on all rows
    so far, and against the dense attention join-agg on what cache_read gives back."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Relation, cache_append, cache_attention, cache_read
    from tensor_relational_einsum_gb300.relation import attention, check
    kv, group, d, page = 2, 4, 128, 16
    rng = np.random.default_rng(16)
    c = PagedCache(64, page, kv, d, fmt)
    order = rng.permutation(64).astype(np.int32)
    table = torch.from_numpy(order.reshape(2, 32)).cuda()
    chunks = [(100, 37), (61, 1), (1, 1), (1, 5), (1, 0), (2, 1)]
    lens = np.zeros(2, dtype=np.int64)
    kept = [[np.zeros((0, kv, d)), np.zeros((0, kv, d))] for _ in range(2)]
    qs = [np.zeros((0, kv * group, d)) for _ in range(2)]
    outs = [np.zeros((0, kv * group, d)) for _ in range(2)]
    for n0, n1 in chunks:
        rows = n0 + n1
        lens += (n0, n1)
        k, v = values(rng, (rows, kv, d)), values(rng, (rows, kv, d))
        q = values(rng, (rows, kv * group, d))
        batch = PageBatch(table, torch.tensor([0, n0, rows], dtype=torch.int32).cuda(),
                          torch.tensor(lens, dtype=torch.int32).cuda(), max_new=max(n0, n1))
        dev = [relation(torch.from_numpy(x).to(torch.bfloat16).cuda()) for x in (q, k, v)]
        cache_append(c, batch, dev[1], dev[2])
        o = cache_attention(dev[0], c, batch).to_dense().double().cpu().numpy()
        check()
        for i, sl in enumerate((slice(0, n0), slice(n0, rows))):
            for w, x in enumerate((k, v)):
                y = x[sl]
                if fmt == "e4m3" and len(y):
                    e = np.exp2(cu.e4m3_scale(y))[..., None]
                    y = cu.e4m3_round(y / e) * e
                kept[i][w] = np.concatenate([kept[i][w], y])
            qs[i] = np.concatenate([qs[i], q[sl]])
            outs[i] = np.concatenate([outs[i], o[sl]])
    for i in range(2):
        t = len(qs[i])
        assert t == lens[i]
        for h in range(kv * group):
            wo, _, _, big, slack = cu.softmax_attention(qs[i][:, h], kept[i][0][:, h // group], kept[i][1][:, h // group],
                                                        np.arange(t), float(np.float32(1 / np.sqrt(d))), True)
            assert (np.abs(outs[i][:, h] - wo) <= cu.out_bound(wo, big, slack, t)).all()
    # whole sequences back, through the dense join-agg: the same result within both operators' bounds
    whole = PageBatch(table, torch.tensor([0, lens[0], lens.sum()], dtype=torch.int32).cuda(),
                      torch.tensor(lens, dtype=torch.int32).cuda())
    k, v = cache_read(c, whole, rows=int(lens.sum()))
    qd = torch.from_numpy(np.concatenate(qs)).to(torch.bfloat16).cuda()
    dense = attention("shd,thd,thd->shd", relation(qd), k, v, causal=True, seq_ends=[int(lens[0]), int(lens.sum())])
    got = cache_attention(relation(qd), c, whole)
    check()
    a, w = dense.to_dense().double(), got.to_dense().double()
    assert (a - w).norm() <= 2 * 2.0 ** -8 * 2 * a.norm()


# ------------------------------------------ the rules that choose a variant

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kv,group,dim,page,seqs", ATTEND)
def test_attention_with_a_promised_bound(kv, group, dim, page, seqs, fmt):
    """max_new says how long chunks can be: it rules kernels out, and with fewer than 256 rows to a sequence the chunk
    kernel reads 8-bit pages itself."""
    b = cu.Batch(seqs, page, seed=17)
    c = nan_cache(b, kv, dim, fmt)
    rng = np.random.default_rng(18)
    held = fill(c, b, rng)
    attend(b, c, held, group, rng, max_new=max(n for n, _ in seqs))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [(1, 4), (3, 4), (2, 9), (16, 1)])
def test_many_short_sequences(rows, dim, fmt):
    """At least 608 items of up to 512 positions: a warp an item."""
    n, group = rows
    rng = np.random.default_rng(19)
    seqs = [(int(rng.integers(0, n + 1)), int(t)) for t in rng.integers(0, 80, size=200)] + [(n, 512), (n, 511), (n, 0), (n, 17)] * 2
    b = cu.Batch(seqs, 16, behind=1)
    c = nan_cache(b, 3, dim, fmt)
    held = fill(c, b, rng)
    attend(b, c, held, group, rng, max_new=n)


@pytest.mark.parametrize("n", [1, 5, 30, 100])
def test_scales_far_apart(n):
    """8-bit vectors whose scales spread over 2^16 within a tile and move along the positions: f16 operands brought to a
    common reference must keep every one of them."""
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, 400), (n, 1111)], 16)
    c = nan_cache(b, 2, 128, "e4m3")
    rng = np.random.default_rng(20)
    held = []
    kc, vc = c.k.view(torch.uint8).cpu(), c.v.view(torch.uint8).cpu()
    ks, vs = c.k_scale.cpu(), c.v_scale.cpu()
    for i in range(2):
        pg, sl = b.places(i)
        pair = []
        for cells, scale in ((kc, ks), (vc, vs)):
            t = int(b.lens[i])
            grow = np.exp2(rng.integers(-8, 9, size=(t, 2, 1)) + 4.0 * np.arange(t)[:, None, None] / t)
            x = rng.normal(size=(t, 2, 128)) * (grow if cells is vc else np.exp2(rng.integers(-10, 1, size=(t, 2, 1))))
            e = cu.e4m3_scale(x)
            y = cu.e4m3_round(x / np.exp2(e)[..., None])
            cells[pg, :, sl] = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[pg, :, sl] = torch.from_numpy((e + 127).astype(np.uint8))
            pair.append(y * np.exp2(e)[..., None])
        held.append(pair)
    c.k.copy_(kc.view(torch.float8_e4m3fn))
    c.v.copy_(vc.view(torch.float8_e4m3fn))
    c.k_scale.copy_(ks)
    c.v_scale.copy_(vs)
    check()
    for max_new in (n, 0):
        attend(b, c, held, 2, rng, max_new=max_new)


@pytest.mark.parametrize("spread", [1e-30, 1e-6, 1e6, 1e15])
def test_queries_and_keys_of_any_size(spread):
    """Q far from 1 and K as far the other way: the scores are ordinary."""
    for n in (1, 50):
        b = cu.Batch([(n, 333)], 16)
        c = nan_cache(b, 1, 64, "e4m3")
        rng = np.random.default_rng(21)
        held = fill(c, b, rng)
        pg, sl = b.places(0)
        shift = int(np.round(np.log2(spread)))
        s = c.k_scale.cpu()
        s[pg, :, sl] = (s[pg, :, sl].int() - shift).to(torch.uint8)
        c.k_scale.copy_(s)
        held[0][0] = held[0][0] * 2.0 ** -shift
        attend(b, c, held, 2, rng, spread=2.0 ** shift, max_new=n)


@pytest.mark.parametrize("n,max_new", [(1, 1), (40, 40), (200, 200)])
def test_a_stored_nan_reaches_the_rows_that_keep_it(n, max_new):
    """A NaN vector of an 8-bit cache: rows before it in another tile, and other sequences, stay right."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, 400), (n, 450)], 16)
    c = nan_cache(b, 1, 64, "e4m3")
    rng = np.random.default_rng(22)
    held = fill(c, b, rng)
    c.v_scale[int(b.pages[0, 3]), 0, 5] = 255            # position 53 of sequence 0: all its rows keep it
    q = torch.from_numpy(values(rng, (b.rows, 2, 64))).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    cache_attention(relation(q), c, on_gpu(b, max_new=max_new), out=relation(out))
    check()
    out = out.double().cpu().numpy()
    keeps = 400 - n + np.arange(n) >= 53
    assert np.isnan(out[:n][keeps]).all()
    qd = q.double().cpu().numpy()
    for h in range(2):
        k, v = (x[:, 0] for x in held[1])
        wo, _, _, big, slack = cu.softmax_attention(qd[n:, h], k, v, 450 - n + np.arange(n), 0.125, True)
        assert (np.abs(out[n:, h] - wo) <= cu.out_bound(wo, big, slack, 450)).all()


def test_workspace_is_checked_and_means_nothing():
    """Too small a workspace is refused; whatever it holds, the result is the same."""
    import ctypes
    from tensor_relational_einsum_gb300 import _abi
    from tensor_relational_einsum_gb300.relation import check
    L = _abi.lib()
    b = cu.Batch([(1, 3000), (70, 2000)], 16)
    c = nan_cache(b, 1, 128, "e4m3")
    rng = np.random.default_rng(23)
    fill(c, b, rng)
    q = torch.from_numpy(values(rng, (b.rows, 4, 128))).to(torch.bfloat16).cuda()
    batch, r = on_gpu(b), relation(q)
    need = ctypes.c_size_t()
    assert L.ea_cache_attention_workspace(c.handle, batch.ref, r.handle, ctypes.byref(need)) == 0 and need.value > 0
    got = []
    for fill_byte in (0, 255, 127):
        ws = torch.full((need.value,), fill_byte, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        o = relation(out)
        for size, ptr, want in ((need.value - 1, ws.data_ptr(), 7), (need.value, None, 7), (need.value, ws.data_ptr() + 8, 7),
                                (need.value, ws.data_ptr(), 0)):
            opts = _abi.CacheAttnOpts(0.0, 1, None, None, ptr, size)
            stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
            assert L.ea_cache_attention(c.handle, batch.ref, r.handle, ctypes.byref(opts), stream, o.handle) == want
        check()
        got.append(out)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]) and torch.isfinite(got[0]).all()


def test_large_pool_offsets():
    """A pool of more than 2^31 bytes and 2^32 elements' worth of offsets: pages at its far end."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, cache_append, cache_attention, cache_read
    from tensor_relational_einsum_gb300.relation import check
    pages, page, heads, dim = 70000, 128, 4, 128          # 4.6e9 cells a tensor
    k, v = (torch.empty(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = PagedCache(pages, page, heads, dim, k=k, v=v)
    rng = np.random.default_rng(24)
    n = 300
    table = torch.tensor([[pages - 1, 5, pages - 2], [pages - 3, pages // 2, 0]], dtype=torch.int32, device="cuda")
    batch = PageBatch(table, torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda"),
                      torch.tensor([n, 1], dtype=torch.int32, device="cuda"))
    x = [values(rng, (n + 1, heads, dim)) for _ in range(2)]
    kr, vr = (relation(torch.from_numpy(t).to(torch.bfloat16).cuda()) for t in x)
    cache_append(c, batch, kr, vr)
    got = cache_read(c, batch, rows=n + 1)
    assert all(torch.equal(g.to_dense(), w.to_dense()) for g, w in zip(got, (kr, vr)))
    q = values(rng, (n + 1, heads, dim))
    out = cache_attention(relation(torch.from_numpy(q).to(torch.bfloat16).cuda()), c, batch).to_dense().double().cpu().numpy()
    check()
    sc = float(np.float32(1 / np.sqrt(dim)))
    for h in range(heads):
        for rows, pos in ((slice(0, n), np.arange(n)), (slice(n, n + 1), np.arange(1))):
            wo, _, _, big, slack = cu.softmax_attention(q[rows, h], x[0][rows, h], x[1][rows, h], pos, sc, True)
            assert (np.abs(out[rows, h] - wo) <= cu.out_bound(wo, big, slack, n)).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_cached_attention_as_one_captured_graph(fmt):
    """The step of a generation loop -- append and attend -- captured once and replayed while lengths grow and a page is
    added; an eager pass of other calls lives at the same time."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache
    from tensor_relational_einsum_gb300.graphs import CachedAttention, capture
    from tensor_relational_einsum_gb300.relation import check
    kv, group, d, page, seqs = 2, 4, 64, 16, 3
    rng = np.random.default_rng(25)
    c = PagedCache(32, page, kv, d, fmt)
    table = torch.full((seqs, 4), -1, dtype=torch.int32, device="cuda")
    table[:, :2] = torch.from_numpy(rng.permutation(32)[:6].reshape(3, 2).astype(np.int32))
    starts, lens = torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), torch.tensor([1, 29, 7], dtype=torch.int32, device="cuda")
    batch = PageBatch(table, starts, lens, max_new=1)
    q, k, v = (torch.zeros(seqs, h, d, dtype=torch.bfloat16, device="cuda") for h in (kv * group, kv, kv))
    step = CachedAttention(relation(q), relation(k), relation(v), c, batch)
    old = lens.cpu().numpy()
    held = [[values(rng, (int(t) - 1, kv, d)) for _ in range(2)] for t in old]
    from tensor_relational_einsum_gb300 import cache_append
    for i, t in enumerate(old):       # what was there before
        if t > 1:
            b = PageBatch(table[i:i + 1], torch.tensor([0, t - 1], dtype=torch.int32, device="cuda"),
                          torch.tensor([t - 1], dtype=torch.int32, device="cuda"))
            cache_append(c, b, *(relation(torch.from_numpy(x).to(torch.bfloat16).cuda()) for x in held[i]))
        if fmt == "e4m3":
            for w in range(2):
                e = np.exp2(cu.e4m3_scale(held[i][w]))[..., None]
                held[i][w] = cu.e4m3_round(held[i][w] / e) * e
    graph = capture(step.run)
    for n in range(6):
        x = [values(rng, (seqs, h, d)) for h in (kv * group, kv, kv)]
        for t, y in zip((q, k, v), x):
            t.copy_(torch.from_numpy(y).to(torch.bfloat16))
        if n == 4:
            table[1, 2] = 31 if 31 not in table.cpu().tolist()[0] + table.cpu().tolist()[1] + table.cpu().tolist()[2] else 30
        if fmt == "e4m3":
            for w in (1, 2):
                e = np.exp2(cu.e4m3_scale(x[w]))[..., None]
                x[w] = cu.e4m3_round(x[w] / e) * e
        graph.replay()
        check()
        got = step.O.to_dense().double().cpu().numpy()
        for i in range(seqs):
            held[i] = [np.concatenate([held[i][w], x[w + 1][i:i + 1]]) for w in range(2)]
            t = len(held[i][0])
            assert t == int(lens[i])
            for h in range(kv * group):
                wo, _, _, big, slack = cu.softmax_attention(x[0][i:i + 1, h], held[i][0][:, h // group], held[i][1][:, h // group],
                                                            np.array([t - 1]), 0.125, True)
                assert (np.abs(got[i, h] - wo[0]) <= cu.out_bound(wo, big, slack, t)[0]).all()
        lens += 1
        if n == 2:                    # other calls between replays
            cache_append(c, PageBatch(table[:1, :2], torch.tensor([0, 0], dtype=torch.int32, device="cuda"),
                                      torch.tensor([1], dtype=torch.int32, device="cuda")), step.k, step.v)


def test_empty_relations_and_batches():
    """No rows at all, and a batch whose sequences have none: nothing is written, nothing is raised."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Relation, cache_append, cache_attention, cache_read
    from tensor_relational_einsum_gb300.relation import check
    c = PagedCache(4, 16, 2, 64)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    b = PageBatch(torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), z, z[:1])
    for rows in (0, 5):
        k, v, q = (Relation("bf16", (rows, h, 64), [1, 1, 1], device="cuda") for h in (2, 2, 4))
        k.storage.zero_(), v.storage.zero_(), q.storage.zero_()
        out = Relation("bf16", (rows, 4, 64), [1, 1, 1], device="cuda")
        out.storage.fill_(MARK)
        cache_append(c, b, k, v)
        cache_read(c, b, k, v)
        cache_attention(q, c, b, out=out)
        check()
        assert (out.storage == MARK).all() and not c.k.any()


def test_python_refusals():
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, cache_append, cache_read
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        PagedCache(4, 16, 2, 64, "fp8")
    with pytest.raises(ValueError):
        PagedCache(4, 16, 2, 64, k=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        PagedCache(4, 16, 2, 64, k=x, v=x.float())
    with pytest.raises(ValueError):
        PagedCache(4, 16, 2, 64, k=x, v=x.transpose(0, 1).contiguous().transpose(0, 1))
    c = PagedCache(4, 16, 2, 64)
    good = (torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    PageBatch(*good)
    for spoil in range(3):
        for bad in (good[spoil].long(), good[spoil].cpu(), good[spoil][:1] if spoil else good[0].t()):
            args = list(good)
            args[spoil] = bad
            with pytest.raises(ValueError):
                PageBatch(*args)
    b = PageBatch(*good)
    with pytest.raises(ValueError):
        cache_read(c, b)
    k = relation(torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        cache_read(c, b, k=k)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_relations_off_a_32_byte_boundary(fmt, dtype):
    """Relations promise 16 bytes: inputs, outputs and the workspace at odd multiples of it, through every kernel."""
    import ctypes
    from tensor_relational_einsum_gb300 import _abi, cache_append, cache_read
    from tensor_relational_einsum_gb300.relation import check

    def off(t):
        flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        flat = flat[16 // t.element_size():][:t.numel()]
        assert flat.data_ptr() % 32 == 16
        flat.copy_(t.reshape(-1))
        return flat.view(t.shape)

    seqs = [(1, 3000), (300, 1200), (40, 40), (2, 9)]
    b = cu.Batch(seqs, 32)
    rng = np.random.default_rng(26)
    for dim in (64, 128):
        c = nan_cache(b, 2, dim, fmt)
        held = fill(c, b, rng)
        batch = on_gpu(b)
        outs = [off(torch.full((b.rows, 2, dim), MARK, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda"))
                for _ in range(2)]
        rel_kv = [relation(t) for t in outs]
        cache_read(c, batch, *rel_kv)
        check()
        for w in range(2):
            want = np.concatenate([held[i][w][-n:] for i, (n, _) in enumerate(seqs)])
            assert np.array_equal(outs[w].double().cpu().numpy(), want)
        cache_append(c, batch, *rel_kv)                     # what was read: nothing changes
        q = values(rng, (b.rows, 4, dim))
        tq = off(torch.from_numpy(q).to(torch.bfloat16).cuda())
        out = off(torch.full((b.rows, 4, dim), MARK, dtype=torch.bfloat16, device="cuda"))
        rq, ro = relation(tq), relation(out)
        need = ctypes.c_size_t()
        L = _abi.lib()
        _abi.check_status(L.ea_cache_attention_workspace(c.handle, batch.ref, rq.handle, ctypes.byref(need)))
        ws = off(torch.empty(need.value, dtype=torch.uint8, device="cuda"))
        opts = _abi.CacheAttnOpts(0.0, 1, None, None, ws.data_ptr(), need.value)
        _abi.check_status(L.ea_cache_attention(c.handle, batch.ref, rq.handle, ctypes.byref(opts),
                                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ro.handle))
        check()
        verify(b, c, held, 2, q, out.double().cpu().numpy(), None, None, True, 0.0, False, np.ones(b.rows, dtype=bool))


def test_one_batch_over_two_caches():
    """The same batch object with a bf16 and an 8-bit cache of the same shape, whose workspaces differ."""
    b = cu.Batch([(300, 2000), (1, 700)], 16)
    rng = np.random.default_rng(27)
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    batch = on_gpu(b)
    q = values(rng, (b.rows, 2, 64))
    r = relation(torch.from_numpy(q).to(torch.bfloat16).cuda())
    for fmt in ("bf16", "e4m3", "bf16"):
        c = nan_cache(b, 1, 64, fmt)
        held = fill(c, b, rng)
        out = cache_attention(r, c, batch).to_dense().double().cpu().numpy()
        check()
        verify(b, c, held, 2, q, out, None, None, True, 0.0, False, np.ones(b.rows, dtype=bool))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("n,max_new", [(1, 1), (10, 10), (40, 40), (200, 200)])
def test_a_nan_code_reads_as_nan(n, max_new, which):
    """A NaN code under a finite scale: NaN in a read, and in every row that keeps it, in each kernel."""
    from tensor_relational_einsum_gb300 import cache_attention, cache_read
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, 400), (n, 450)], 16)
    rng = np.random.default_rng(28)
    c = nan_cache(b, 1, 64, "e4m3")
    held = fill(c, b, rng)
    getattr(c, which).view(torch.uint8)[int(b.pages[0, 3]), 0, 5, 7] = 0x7f      # position 53, component 7
    q = torch.from_numpy(values(rng, (b.rows, 2, 64))).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    cache_attention(relation(q), c, on_gpu(b, max_new=max_new), out=relation(out))
    check()
    out = out.double().cpu().numpy()
    assert 400 - n > 53
    assert np.isnan(out[:n, :, 7]).all() and (which == "v" or np.isnan(out[:n]).all())
    qd = q.double().cpu().numpy()
    for h in range(2):
        k, v = (x[:, 0] for x in held[1])
        wo, _, _, big, slack = cu.softmax_attention(qd[n:, h], k, v, 450 - n + np.arange(n), 0.125, True)
        assert (np.abs(out[n:, h] - wo) <= cu.out_bound(wo, big, slack, 450)).all()
    whole = cu.Batch([(400, 400), (450, 450)], 16)
    whole.pages = b.pages
    kv = [torch.zeros(850, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache_read(c, on_gpu(whole), *(relation(t) for t in kv))
    check()
    for w, t in zip("kv", kv):
        g = torch.isnan(t)
        assert int(g.sum()) == (1 if w == which else 0) and (w != which or bool(g[53, 0, 7]))


def test_slots_that_rows_share_spare_the_others():
    """Two rows of one append that name one slot: only that slot is unspecified."""
    from tensor_relational_einsum_gb300 import cache_append
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(4, 20), (4, 20)], 16)
    b.pages[1, 1] = b.pages[0, 1]                           # positions 16..19 of both
    c = nan_cache(b, 1, 64, "bf16")
    before = bits(c.k).copy()
    x = torch.ones(8, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache_append(c, on_gpu(b), relation(x), relation(x.clone()))
    check()
    changed = (bits(c.k) != before).any(axis=(1, 3))
    allowed = np.zeros_like(changed)
    allowed[b.pages[0, 1], :4] = True
    assert np.array_equal(changed, allowed)


def test_a_workspace_over_an_operand_is_refused():
    import ctypes
    from tensor_relational_einsum_gb300 import _abi
    b = cu.Batch([(1, 2000), (40, 900)], 16)
    c = nan_cache(b, 1, 64, "bf16")
    q = torch.zeros(b.rows, 2, 64, dtype=torch.bfloat16, device="cuda")
    rq = relation(q)
    need = ctypes.c_size_t()
    batch = on_gpu(b)
    L = _abi.lib()
    _abi.check_status(L.ea_cache_attention_workspace(c.handle, batch.ref, rq.handle, ctypes.byref(need)))
    room = torch.zeros(need.value + q.numel() * 2, dtype=torch.uint8, device="cuda")
    over = room[need.value - 16:][:q.numel() * 2].view(torch.bfloat16).view(q.shape)    # shares the workspace's last bytes
    beyond = room[need.value:][:q.numel() * 2].view(torch.bfloat16).view(q.shape)
    assert over.data_ptr() % 16 == 0
    opts = _abi.CacheAttnOpts(0.0, 1, None, None, room.data_ptr(), need.value)

    def call(o, rel):
        return L.ea_cache_attention(c.handle, batch.ref, rel.handle, ctypes.byref(o),
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), out.handle)

    out = relation(over)
    assert call(opts, rq) == 7                              # EA_ERR_ARG
    out = relation(torch.zeros_like(q))
    assert call(opts, relation(over)) == 7
    assert call(_abi.CacheAttnOpts(0.0, 1, None, None, c.v.data_ptr(), need.value), rq) == 7
    out = relation(beyond)
    assert call(opts, rq) == 0
    torch.cuda.synchronize()
