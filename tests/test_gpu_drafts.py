"""GPU tests of the operators around drafted tokens against the 64-bit
definitions in drafts_util and cache_util.

Caches start full of NaN and rows of no sequence hold NaN or a mark, so that
what should not be read would show, and what should not be written too.

Tolerances.  Tree attention: cache_util.out_bound, as for the other rows.
Rotary: cosine and sine are off by at most 3.2e-7 (the angle in half turns is
rounded to 2^-24, which is 2^-24 pi of it, sincospi is good to 1.5 steps of
2^-24 at most, and 2^-23 covers that), the two products and their sum round
three times by 2^-24: 6e-7 of |x| + |y| in all; half a step of bf16 on top.
Moves, paths and tokens are exact; a decision that lies within 1e-9 of its
border in 64 bits would be left out, and the test says that none does.
"""
import ctypes
import math

import numpy as np
import pytest

import cache_util as cu
import drafts_util as du

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_cache import MARK, bits, fill, nan_cache, on_gpu, relation, values  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tensor_relational_einsum_gb300.build import build
    build()
    yield
    from tensor_relational_einsum_gb300.relation import check
    check()


def parents_of(b, kind, seed=5):
    """Parents per sequence, and as a device tensor over all rows (rows of no sequence: far out of range)."""
    rng = np.random.default_rng(seed)
    trees = [du.tree(kind, n, rng) for n, _ in b.seqs]
    flat = np.full(b.rows, 10 ** 6, dtype=np.int32)
    for i, p in enumerate(trees):
        flat[b.rows_of(i)] = p
    return trees, torch.from_numpy(flat).cuda()


# ---------------------------------------------------------- tree attention

def tree_attention(b, c, held, group, trees, parents, rng, max_new, stats=True, spread=1.0, scale=0.0, run=None):
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    heads = c.heads * group
    q = values(rng, (b.rows, heads, c.dim), spread)
    inside = np.zeros(b.rows, dtype=bool)
    inside[int(b.starts[0]):int(b.starts[-1])] = True
    qt = torch.from_numpy(q).to(torch.bfloat16)
    qt[~torch.from_numpy(inside)] = float("nan")
    out = torch.full((b.rows, heads, c.dim), MARK, dtype=torch.bfloat16, device="cuda")
    m, l = (torch.full((b.rows, heads), MARK, device="cuda") for _ in range(2))
    batch = on_gpu(b, max_new=max_new, strided=True)
    kw = dict(scale=scale, parents=parents, out=relation(out))
    if stats:
        kw.update(m_out=relation(m), l_out=relation(l))
    call = lambda: cache_attention(relation(qt.cuda()), c, batch, **kw)  # noqa: E731
    (run or (lambda f: f()))(call)
    check()
    verify_tree(b, c, held, group, trees, q, out, m if stats else None, l, scale, inside)
    return out, m, l


def verify_tree(b, c, held, group, trees, q, out, m, l, scale, inside):
    scale = scale or 1.0 / math.sqrt(c.dim)
    got = out.double().cpu().numpy()
    assert np.all(got[~inside] == MARK)
    if m is not None:
        gm, gl = m.double().cpu().numpy(), l.double().cpu().numpy()
        assert np.all(gm[~inside] == MARK) and np.all(gl[~inside] == MARK)
    for i, (n, t) in enumerate(b.seqs):
        r0 = int(b.starts[i])
        for j in range(n):
            keep = du.kept_positions(trees[i], j, n, t)
            for h in range(c.heads * group):
                k, v = (x[keep, h // group] for x in held[i])
                o, wm, wl, big, slack = cu.softmax_attention(q[r0 + j:r0 + j + 1, h], k, v, None, scale, False)
                bound = cu.out_bound(o, big, slack, max(1, len(keep)))
                err = np.abs(got[r0 + j, h] - o[0])
                assert np.all(err <= bound[0]), (i, j, h, float((err - bound[0]).max()))
                if m is None:
                    continue
                if not keep:
                    assert gm[r0 + j, h] == -np.inf and gl[r0 + j, h] == 0.0 and np.all(got[r0 + j, h] == 0.0)
                    continue
                assert abs(gm[r0 + j, h] - wm[0]) <= slack[0] + 2.0 ** -22 * abs(wm[0])
                rel = 2.0 * np.expm1(2 * slack[0]) + 2.0 ** -18 + 4.0 * len(keep) * 2.0 ** -24
                assert abs(gl[r0 + j, h] - wl[0]) <= rel * wl[0]


TREES = [
    # kv, group, dim, page, sequences (nodes, positions)
    (1, 1, 64, 16, [(1, 1)]),
    (1, 4, 128, 16, [(8, 8)]),
    (2, 4, 128, 16, [(1, 5), (3, 3), (4, 40), (0, 9), (2, 70)]),            # 16 rows
    (2, 4, 64, 32, [(8, 611), (7, 64), (5, 3), (8, 71), (1, 1), (6, 130)]),  # 32 rows; n > t
    (1, 1, 128, 16, [(32, 32), (31, 100), (17, 513)]),
    (1, 3, 128, 64, [(33, 33), (12, 200), (64, 65), (40, 39)]),              # chunks
    (2, 8, 64, 16, [(64, 300), (16, 16), (9, 129), (0, 0), (64, 127), (63, 128)]),
    (1, 2, 128, 128, [(128, 128), (128, 400), (100, 1100)]),
    (1, 16, 64, 32, [(2, 9), (1, 600), (11, 12)]),
    (5, 1, 128, 16, [(3, 20)] * 9),
    (1, 128, 64, 16, [(2, 30), (1, 7)]),
]


@pytest.mark.parametrize("kind", ["random", "chain", "forest"])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("kv,group,dim,page,seqs", TREES)
def test_tree_attention(kv, group, dim, page, seqs, fmt, kind):
    b = cu.Batch(seqs, page, before=2, behind=3, seed=3)
    c = nan_cache(b, kv, dim, fmt)
    rng = np.random.default_rng(4)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, kind)
    tree_attention(b, c, held, group, trees, parents, rng, max_new=max(n for n, _ in seqs))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,t,group", [(8, 9000, 4), (24, 5000, 4), (64, 3100, 1), (1, 7000, 8), (128, 2100, 2)])
def test_tree_behind_a_long_axis(n, t, group, fmt):
    """One sequence: its items are cut and merged; the nodes' columns lie in one part or two."""
    for off in (0, 37):
        b = cu.Batch([(n, t + off)], 32, before=1, seed=6)
        c = nan_cache(b, 1, 128, fmt)
        rng = np.random.default_rng(7)
        held = fill(c, b, rng)
        trees, parents = parents_of(b, "random")
        tree_attention(b, c, held, group, trees, parents, rng, max_new=n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_many_trees_in_a_wide_table(fmt, dim):
    """More items than CTAs, of one tile of rows and of two, over tables that allow cutting: whole items, cut ones, and
    items without or with a single key tile, in one call."""
    rng = np.random.default_rng(14)
    seqs = [(int(n), int(t)) for n, t in zip(rng.integers(9, 17, 66), rng.integers(20, 1400, 66))]
    seqs[3:6] = [(40, 300), (64, 900), (33, 33)]       # two tiles of rows
    seqs[10:13] = [(12, 12), (11, 5), (0, 700)]
    b = cu.Batch(seqs, 64, before=1, behind=1, seed=15, extra_pages=4)
    c = nan_cache(b, 4, dim, fmt)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, "random")
    tree_attention(b, c, held, 4, trees, parents, rng, max_new=64)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,n", [(3, 85), (4, 16), (4, 8), (1, 127)])
def test_every_run_gives_the_same_bits(group, n, fmt, dim):
    """Trees and rows in order, many parts a CTA: 40 runs of one call."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(37)
    seqs = [(int(x), int(x + t)) for x, t in zip(rng.integers(max(1, n // 2), n + 1, size=16), rng.integers(0, 1300, size=16))]
    seqs[3] = (n, 2500)
    b = cu.Batch(seqs, 32, before=1)
    c = nan_cache(b, 8, dim, fmt)
    fill(c, b, rng)
    q = relation(torch.from_numpy(values(rng, (b.rows, 8 * group, dim))).to(torch.bfloat16).cuda())
    _, parents = parents_of(b, "random")
    batch = on_gpu(b, max_new=n)
    for tree in (parents, None):
        first = None
        for _ in range(40):
            out = torch.zeros(b.rows, 8 * group, dim, dtype=torch.bfloat16, device="cuda")
            cache_attention(q, c, batch, out=relation(out), parents=tree)
            first = out if first is None else first
            assert torch.equal(out, first)
    check()


@pytest.mark.parametrize("kind", ["star", "roots", "pairs"])
def test_tree_without_a_bound_and_a_scale(kind):
    """max_new 0: the dense rows say how many nodes there can be; peaked scores."""
    b = cu.Batch([(20, 90), (3, 300), (31, 64)], 16, before=0, behind=4, seed=8)
    c = nan_cache(b, 2, 64, "bf16")
    rng = np.random.default_rng(9)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, kind)
    tree_attention(b, c, held, 2, trees, parents, rng, max_new=0, stats=False, scale=1.0)


@pytest.mark.parametrize("n", [3, 30])
def test_dropped_keys_may_hold_anything(n):
    """A dropped node's key of any size reaches no row (its scores are dropped whatever they are)."""
    b = cu.Batch([(n, 100)], 16, seed=10)
    c = nan_cache(b, 1, 128, "bf16")
    rng = np.random.default_rng(11)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, "star")
    pg, sl = b.places(0)
    for j, x in ((n - 1, float("nan")), (n - 2, float("inf"))):  # leaves: kept by their own rows only
        c.k[int(pg[100 - n + j]), :, int(sl[100 - n + j])] = x
    from tensor_relational_einsum_gb300 import cache_attention
    q = values(rng, (n, 4, 128))
    out = cache_attention(relation(torch.from_numpy(q).to(torch.bfloat16).cuda()), c, on_gpu(b, max_new=n), parents=parents)
    got = out.to_dense().double().cpu().numpy()
    for j in range(n - 2):
        keep = du.kept_positions(trees[0], j, n, 100)
        for h in range(4):
            o, _, _, big, slack = cu.softmax_attention(q[j:j + 1, h], held[0][0][keep, 0], held[0][1][keep, 0], None,
                                                       1 / math.sqrt(128), False)
            assert np.all(np.abs(got[j, h] - o[0]) <= cu.out_bound(o, big, slack, 100)[0])


@pytest.mark.parametrize("n,max_new", [(6, 6), (40, 40)])
def test_parents_out_of_range_are_reported(n, max_new):
    """A node that names itself, a later one or -2: the error word, an end, and other sequences as they should be."""
    from tensor_relational_einsum_gb300 import EaError, cache_attention
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, 80), (n, 90)], 16, seed=12)
    c = nan_cache(b, 1, 64, "bf16")
    rng = np.random.default_rng(13)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, "random")
    q = values(rng, (b.rows, 4, 64))
    for bad in (n - 1, n, 10 ** 9, -2, -(2 ** 31)):
        p = parents.clone()
        p[n - 1] = bad
        out = cache_attention(relation(torch.from_numpy(q).to(torch.bfloat16).cuda()), c, on_gpu(b, max_new=max_new), parents=p)
        with pytest.raises(EaError):
            check()
        got = out.to_dense().double().cpu().numpy()
        for j in range(n):
            keep = du.kept_positions(trees[1], j, n, 90)
            o, _, _, big, slack = cu.softmax_attention(q[n + j:n + j + 1, 0], held[1][0][keep, 0], held[1][1][keep, 0], None,
                                                       0.125, False)
            assert np.all(np.abs(got[n + j, 0] - o[0]) <= cu.out_bound(o, big, slack, 90)[0])


# ------------------------------------------------------------------ rotary

def rotary_bound(want, big, dtype):
    got = 6e-7 * big
    return got + (cu.HALF_BF16 * (np.abs(want) + got) if dtype == torch.bfloat16 else 0) + 1e-37


ROTARY = [
    # heads, kv, columns, rotated, offset
    (32, 8, 128, 128, 0),
    (4, 1, 64, 64, 0),
    (5, 5, 80, 40, 40),
    (7, 2, 96, 24, 8),
    (3, 1, 33, 10, 3),      # columns off every boundary
    (2, 2, 30, 30, 0),
    (1, 1, 2, 2, 0),
    (9, 3, 256, 256, 0),
    (2, 1, 100, 66, 34),
    (65, 1, 16, 12, 4),
    (2, 1, 1501, 10, 3),    # more columns to copy than a CTA has threads for
    (1, 2, 2056, 256, 1800),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("heads,kv,dim,dims,offset", ROTARY)
def test_rotary(heads, kv, dim, dims, offset, layout, dtype):
    from tensor_relational_einsum_gb300 import Rotary, rotary
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(20)
    b = cu.Batch([(1, 1), (7, 50), (0, 3), (20, 131071), (5, 2), (1, 2 ** 20)], 128, before=2, behind=3, seed=1)
    plan = Rotary(dims, layout=layout, offset=offset, factor=2.0, original=4096, amplitude=1.25)
    batch = on_gpu(b, max_new=20)
    trees, parents = parents_of(b, "forest")
    for tree in (False, True):
        at = np.full(b.rows, -1)
        for i, (n, t) in enumerate(b.seqs):
            for j in range(n):
                at[int(b.starts[i]) + j] = t - n + (du.depth(trees[i], j) if tree else j)
        for place in ("new", "in place", "k alone", "positions", "backward"):
            x = [torch.from_numpy(rng.normal(size=(b.rows, h, dim))).to(dtype) for h in (heads, kv)]
            d = [t.cuda() for t in x]
            o = d if place == "in place" else [torch.full_like(t, MARK) for t in d]
            kw = dict(batch=batch, parents=parents if tree else None)
            if place == "positions":
                kw = dict(positions=torch.from_numpy(at.astype(np.int32)).cuda())
            r, ro = [relation(t) for t in d], [relation(t) for t in o]
            if place == "k alone":
                rotary(r[1], None, plan, q_out=ro[1], **kw)
            elif place == "in place":
                rotary(r[0], r[1], plan, **kw)
            else:
                rotary(r[0], r[1], plan, q_out=ro[0], k_out=ro[1], backward=place == "backward", **kw)
            check()
            for w in range(2):
                if place == "k alone" and w == 0:
                    continue
                x64, got = x[w].double().numpy(), o[w].double().cpu().numpy()
                want, big = du.rotate(x64, at, plan.freqs, layout, offset, 1.25, place == "backward")
                still = at < 0
                assert np.array_equal(got[still], x64[still] if place == "in place" else np.full_like(got[still], MARK))
                err, bound = np.abs(got - want)[~still], rotary_bound(want, big, dtype)[~still]
                assert np.all(err <= bound), (place, tree, w, float((err / bound).max()))
                whole = (big == 0) & ~still[:, None, None]
                assert np.array_equal(got[whole], x64[whole])


def test_rotary_gradient_and_differences():
    """The result is linear in q: the gradient of <w, rotary(q)> is the transpose's, and differences give it too."""
    from tensor_relational_einsum_gb300 import Rotary, rotary
    rng = np.random.default_rng(21)
    plan = Rotary(32, layout="half", offset=8, amplitude=0.75)
    at = torch.tensor([0, 5, 77777], dtype=torch.int32, device="cuda")
    q, w = (torch.from_numpy(rng.normal(size=(3, 2, 48))).float().cuda() for _ in range(2))

    def f(t):
        o = torch.empty_like(t)
        rotary(relation(t), None, plan, positions=at, q_out=relation(o))
        return o

    g = torch.empty_like(w)
    rotary(relation(w), None, plan, positions=at, q_out=relation(g), backward=True)
    want, big = du.rotate(w.double().cpu().numpy(), at.tolist(), plan.freqs, "half", 8, 0.75, True)
    assert np.all(np.abs(g.double().cpu().numpy() - want) <= rotary_bound(want, big, torch.float32))
    for r, h, c in ((0, 0, 8), (1, 1, 23), (2, 0, 39), (2, 1, 24), (1, 0, 3), (2, 0, 47)):
        step = torch.zeros_like(q)
        step[r, h, c] = 1.0
        a, b = f(q + step), f(q - step)
        slope = ((a.double() - b.double()) * w.double()).sum().item() / 2.0
        # both sides round every value by 2^-24 and carry 6e-7 of |x| + |y| < 16: over two columns, times |w| < 5
        assert abs(slope - g[r, h, c].item()) <= 2 * 5 * 16 * 1e-6


def test_rotary_many_rows_and_sequences():
    """More sequences than are staged, more rows than a CTA takes, every row's position its own."""
    from tensor_relational_einsum_gb300 import Rotary, rotary
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(1 + i % 5, 1 + i % 5 + 3 * i) for i in range(1500)], 16, behind=1, seed=2)
    plan = Rotary(64)
    rng = np.random.default_rng(22)
    x = torch.from_numpy(rng.normal(size=(b.rows, 2, 64))).float()
    d = x.cuda()
    rotary(relation(d), None, plan, on_gpu(b, max_new=5))
    check()
    at = [-1] * b.rows
    for i, (n, t) in enumerate(b.seqs):
        at[int(b.starts[i]):int(b.starts[i + 1])] = range(t - n, t)
    want, big = du.rotate(x.double().numpy(), at, plan.freqs, "interleaved", 0)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= rotary_bound(want, big, torch.float32))


def test_rotary_far_positions_keep_their_accuracy():
    """The angle modulo a turn is exact: a frequency of 2 pi / 2^20 comes round after 2^20 positions, bit for bit."""
    from tensor_relational_einsum_gb300 import Rotary, rotary
    plan = Rotary(2, freqs=[2 * math.pi / 2 ** 20])
    at = torch.tensor([12345, 12345 + 2 ** 20, 12345 + 2 ** 30, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    x = torch.ones(4, 1, 2, device="cuda")
    rotary(relation(x), None, plan, positions=at)
    # the fraction of a turn is that of the double nearest 2 pi / 2^20, within 2^-53 of it a position: 2^-42 turns at most
    assert (x[0] - x[1]).abs().max().item() <= 2.0 ** -22 and (x[0] - x[2]).abs().max().item() <= 2.0 ** -22
    a = 2 * math.pi * ((2 ** 31 - 1) % 2 ** 20) / 2 ** 20
    assert abs(x[3, 0, 0].item() - (math.cos(a) - math.sin(a))) <= 1.2e-6


def test_rotary_batches_out_of_range():
    from tensor_relational_einsum_gb300 import EaError, PageBatch, Rotary, rotary
    from tensor_relational_einsum_gb300.relation import check
    plan = Rotary(64)
    pages = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for starts, lens, parents in (([0, 3, 2], [5, 5], None), ([0, 2, 9], [5, 5], None), ([0, 2, 4], [5, -1], None),
                                  ([-1, 2, 4], [5, 5], None), ([0, 2, 4], [5, 5], [-1, 1, -1, 0]), ([0, 2, 4], [5, 5], [-1, -3, -1, 0])):
        x = torch.ones(4, 3, 64, device="cuda")
        b = PageBatch(pages, *(torch.tensor(t, dtype=torch.int32, device="cuda") for t in (starts, lens)), max_new=3)
        p = torch.tensor(parents, dtype=torch.int32, device="cuda") if parents else None
        rotary(relation(x), None, plan, b, parents=p)
        with pytest.raises(EaError):
            check()
        if parents:
            assert torch.equal(x[1], torch.ones_like(x[1])) and not torch.equal(x[0], torch.ones_like(x[0]))


# ------------------------------------------------------------ verification

def verify_batch(ns, vocab, dtype, drafts, kind, seed, branch_noise=0.5, before=1, behind=2, sharp=2.0):
    rng = np.random.default_rng(seed)
    b = cu.Batch([(n, n + 4) for n in ns], 16, before=before, behind=behind, seed=seed)
    trees, parents = parents_of(b, kind, seed)
    logits = sharp * rng.normal(size=(b.rows, vocab))

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return torch.from_numpy(e / e.sum(-1, keepdims=True)).to(dtype)

    target, draft = soft(logits), soft(logits + branch_noise * rng.normal(size=logits.shape))
    tokens = np.full(b.rows, -9, dtype=np.int32)
    for i, (n, _) in enumerate(b.seqs):
        for j in range(n):
            up = trees[i][j]
            p = (draft if drafts else target)[int(b.starts[i]) + max(0, up)].double().numpy()
            tokens[int(b.starts[i]) + j] = rng.choice(vocab, p=p / p.sum())
    accept, sample = (rng.random(size).astype(np.float32) for size in (b.rows, len(ns)))
    outside = np.ones(b.rows, dtype=bool)
    outside[int(b.starts[0]):int(b.starts[-1])] = False
    target[torch.from_numpy(outside)] = float("nan")
    return b, trees, parents, target, draft if drafts else None, tokens, accept, sample


def run_verify(b, parents, target, draft, tokens, accept, sample, max_new=None, **kw):
    from tensor_relational_einsum_gb300 import verify_drafts
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    max_new = max(n for n, _ in b.seqs) if max_new is None else max_new
    return verify_drafts(relation(target.cuda()), on_gpu(b, max_new=max_new), up(tokens), up(accept), up(sample),
                         draft=relation(draft.cuda()) if draft is not None else None, parents=parents, **kw)


def expect(b, trees, target, draft, tokens, accept, sample, got, least=1e-9):
    path, counts, picked = (t.cpu().numpy() for t in got)
    for i, (n, _) in enumerate(b.seqs):
        if n == 0:
            assert counts[i] == 0 and picked[i] == -1 and np.all(path[i] == -1)
            continue
        r = b.rows_of(i)
        want, token, near = du.verify(target[r].double().numpy(), draft[r].double().numpy() if draft is not None else None,
                                      tokens[r], trees[i], accept[r].astype(np.float64), float(sample[i]))
        assert near > least, (i, near)  # the inputs are fixed: no decision of theirs lies that near its border
        assert list(path[i, :len(want)]) == want and np.all(path[i, len(want):] == -1), (i, path[i], want)
        assert counts[i] == len(want) and picked[i] == token, (i, picked[i], token)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ns,vocab,kind", [
    ([1], 1, "chain"), ([5], 2, "random"), ([3, 0, 1, 8], 17, "random"), ([5] * 3, 2049, "chain"), ([16, 9, 30], 777, "star"),
    ([4, 7], 40001, "random"), ([128, 64], 333, "random"), ([2], 131072, "chain"), ([6, 5, 3] * 70, 301, "random"),
    ([12, 12], 5003, "pairs"),
])
def test_verify(ns, vocab, kind, dtype, drafts):
    from tensor_relational_einsum_gb300.relation import check
    b, trees, parents, target, draft, tokens, accept, sample = verify_batch(ns, vocab, dtype, drafts, kind, seed=30 + len(ns))
    got = run_verify(b, None if kind == "chain" else parents, target, draft, tokens, accept, sample)
    check()
    expect(b, trees, target, draft, tokens, accept, sample, got)


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_with_many_rejections(drafts):
    """Drafts unlike the target: most children are refused, so that several subtractions follow one another."""
    b, trees, parents, target, draft, tokens, accept, sample = verify_batch([24, 17, 30], 3001, torch.float32, drafts, "star", 41,
                                                                            branch_noise=4.0, sharp=0.5)
    got = run_verify(b, parents, target, draft, tokens, accept, sample)
    counts = got[1].cpu().numpy()
    assert counts.min() >= 1
    expect(b, trees, target, draft, tokens, accept, sample, got)


def one(target, draft, tokens, parents, accept, sample, dtype=torch.float32):
    """A single sequence of exactly representable numbers."""
    n = len(tokens)
    b = cu.Batch([(n, n)], 16, spare=0, seed=0)
    d = torch.tensor(draft, dtype=dtype) if draft is not None else None
    path, counts, picked = run_verify(b, torch.tensor(parents, dtype=torch.int32, device="cuda"), torch.tensor(target, dtype=dtype), d,
                                      np.array(tokens, dtype=np.int32), np.array(accept, dtype=np.float32),
                                      np.array([sample], dtype=np.float32))
    return path[0].tolist()[:int(counts[0])], int(picked[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_at_the_borders(dtype):
    """Powers of two: every comparison is exact, so ties go the way that is written."""
    t, d = [[0.25, 0.25, 0.5, 0.0]] * 2, [[0.5, 0.25, 0.25, 0.0]] * 2
    ask = lambda x, u, s, dd=d, tt=t: one(tt, dd, [9, x], [-1, 0], [0.0, u], s, dtype)  # noqa: E731
    assert ask(0, 0.5, 0.0) == ([0], 2)               # u d = r is a rejection; the rest is (0, 0, 0.25, 0)
    assert ask(0, 0.4375, 0.25) == ([0, 1], 1)        # running sums 0.25, 0.5, 1, 1: the first beyond 0.25
    assert ask(0, 0.4375, 0.2421875) == ([0, 1], 0)
    assert ask(0, 0.4375, 0.5) == ([0, 1], 2) and ask(0, 0.4375, 0.99609375) == ([0, 1], 2)
    assert ask(3, 0.0, 0.0) == ([0], 2)               # 0 < 0 does not hold
    assert ask(1, 0.99609375, 0.0) == ([0, 1], 0)
    assert ask(0, 0.25, 0.0, None) == ([0], 1)        # certain: u < r; then the rest is (0, 0.25, 0.5, 0)
    assert ask(0, 0.2421875, 0.0, None) == ([0, 1], 0)
    assert ask(0, 0.5, 0.34375, None) == ([0], 2) and ask(0, 0.5, 0.328125, None) == ([0], 1)
    # the rest is 0 everywhere: the target's row itself
    assert ask(3, 0.5, 0.5, t, t) == ([0], 2)
    assert ask(2, 0.5, 0.75, None, [[0.0, 0.0, 0.0, 0.0]] * 2) == ([0], -1)
    assert ask(2, 0.5, 0.75, None, [[0.0, 0.0, 0.5, 0.0]] * 2) == ([0], 2)
    # two children: (0, 0, 0.25, 0) of mass 0.25 after the first; d Z = (0.125, 0.0625, 0.0625, 0)
    two = lambda x, u, s: one([t[0]] * 3, [d[0]] * 3, [9, 0, x], [-1, 0, 0], [0.0, 0.5, u], s, dtype)  # noqa: E731
    assert two(2, 0.99609375, 0.0) == ([0, 2], 0)     # 0.0625 u < 0.25
    assert two(1, 0.0, 0.5) == ([0], 2)               # 0 < 0 does not hold; the rest (0, 0, 0.1875, 0)
    # a token twice among certain ones leaves the mass once
    assert one([t[0]] * 3, None, [9, 0, 0], [-1, 0, 0], [0.0, 0.5, 0.0], 0.328125, dtype) == ([0], 1)
    # nodes below a rejected one and further roots are not asked
    assert one([t[0]] * 4, None, [9, 3, 2, 2], [-1, 0, 1, -1], [0.0] * 4, 0.0, dtype) == ([0], 0)


def test_verify_values_out_of_range_and_tokens():
    """NaN and negative probabilities count as 0; a token out of range raises the error word and is not accepted."""
    from tensor_relational_einsum_gb300 import EaError
    from tensor_relational_einsum_gb300.relation import check
    nan = float("nan")
    assert one([[nan, -1.0, 0.25, 0.5]], None, [0], [-1], [0.0], 0.0) == ([0], 2)
    check()
    for bad in (4, -1, 2 ** 31 - 1):
        assert one([[0.25] * 4] * 2, None, [0, bad], [-1, 0], [0.0, 0.0], 0.5) == ([0], 2)
        with pytest.raises(EaError):
            check()
    for bad in (1, 7, -2):
        assert one([[0.25] * 4] * 2, None, [0, 1], [-1, bad], [0.0, 0.0], 0.5) == ([0], 2)
        with pytest.raises(EaError):
            check()


def test_verify_batches_out_of_range():
    from tensor_relational_einsum_gb300 import EaError, PageBatch, verify_drafts
    from tensor_relational_einsum_gb300.relation import check
    pages = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    target = relation(torch.full((4, 8), 0.125, device="cuda"))
    tokens, u, s = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(2, device="cuda")
    for starts in ([0, 2, 1], [0, 2, 9], [-1, 2, 4], [0, 4, 4]):
        b = PageBatch(pages, torch.tensor(starts, dtype=torch.int32, device="cuda"), torch.full((2,), 9, dtype=torch.int32, device="cuda"),
                      max_new=3)
        path, counts, picked = verify_drafts(target, b, tokens, u, s)
        with pytest.raises(EaError):
            check()
        bad = 0 if starts in ([-1, 2, 4], [0, 4, 4]) else 1
        assert counts[bad].item() == 0 and picked[bad].item() == -1


# -------------------------------------------------------------------- keep

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page,layers", [(1, 64, 16, 1), (5, 128, 32, 3), (8, 64, 128, 2), (2, 128, 16, 70)])
def test_keep(heads, dim, page, layers, fmt):
    """Bit for bit, places that are read and written in one call among them; the rest of the pools stays."""
    from tensor_relational_einsum_gb300 import PagedCache, cache_keep
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(50)
    seqs = [(9, 30), (1, 1), (0, 0), (128, 200), (20, 20), (5, 100), (40, 64), (0, 12)]
    b = cu.Batch(seqs, page, before=1, behind=2, seed=4)
    paths = [[0, 1, 2, 5, 8], [0], [], sorted(rng.choice(128, 90, replace=False).tolist()), list(range(1, 20)), [3],
             [0, 2, 3, 4, 5, 6, 7, 8, 9, 11, 30, 31, 39], []]
    path = np.full((len(seqs), 128), -5, dtype=np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    counts = np.array([len(p) for p in paths], dtype=np.int32)
    shape = (layers, b.pages_total, heads, page, dim)
    byte = torch.from_numpy(rng.integers(0, 256, size=(2,) + shape[:-1] + (dim * (2 if fmt == "bf16" else 1),), dtype=np.uint8)).cuda()
    scale = torch.from_numpy(rng.integers(0, 256, size=(2,) + shape[:-1], dtype=np.uint8)).cuda()
    was, was_scale = byte.cpu().numpy().copy(), scale.cpu().numpy().copy()
    cells = byte.view(torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn)
    caches = []
    for x in range(layers):
        kw = dict(k_scale=scale[0, x], v_scale=scale[1, x]) if fmt == "e4m3" else {}
        caches.append(PagedCache(b.pages_total, page, heads, dim, fmt, k=cells[0, x], v=cells[1, x], **kw))
    lens = cache_keep(caches if layers > 1 else caches[0], on_gpu(b, max_new=128, strided=True), torch.from_numpy(path).cuda(),
                      torch.from_numpy(counts).cuda())
    check()
    want, want_scale = was.copy(), was_scale.copy()
    for i, (n, t) in enumerate(seqs):
        pg, sl = b.places(i)
        for j, p in enumerate(paths[i]):
            a, o = t - n + p, t - n + j
            want[:, :, pg[o], :, sl[o]] = was[:, :, pg[a], :, sl[a]]
            want_scale[:, :, pg[o], :, sl[o]] = was_scale[:, :, pg[a], :, sl[a]]
    assert np.array_equal(byte.cpu().numpy(), want)
    assert np.array_equal(scale.cpu().numpy(), want_scale if fmt == "e4m3" else was_scale)
    assert lens.tolist() == [t - n + len(p) for (n, t), p in zip(seqs, paths)]


def test_keep_reports_paths_out_of_range():
    from tensor_relational_einsum_gb300 import EaError, PagedCache, cache_keep
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(4, 20), (4, 9)], 16, seed=5)
    k, v = (torch.randn(b.pages_total, 2, 16, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    c = PagedCache(b.pages_total, 16, 2, 64, "bf16", k=k, v=v)
    was = [bits(t).copy() for t in (k, v)]
    for path, count in (([0, 0, 1, 2], 3), ([1, 0, 2, 3], 2), ([0, 4, 5, 6], 2), ([-1, 1, 2, 3], 1), ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1)):
        p = torch.tensor([path, [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
        lens = cache_keep(c, on_gpu(b, max_new=4), p, torch.tensor([count, 2], dtype=torch.int32, device="cuda"))
        with pytest.raises(EaError):
            check()
        assert lens.tolist() == [20, 7] and all(np.array_equal(bits(t), w) for t, w in zip((k, v), was))
    # a page number out of range, and more rows than positions
    wrong = cu.Batch([(4, 20), (6, 5)], 16, seed=5)
    wrong.pages[0, 1] = b.pages_total + 5
    p = torch.tensor([[1, 3, -1, -1], [1, 2, -1, -1]], dtype=torch.int32, device="cuda")
    lens = cache_keep(c, on_gpu(wrong, max_new=6), p, torch.full((2,), 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(EaError):
        check()
    assert lens.tolist() == [20, 5] and all(np.array_equal(bits(t), w) for t, w in zip((k, v), was))


# --------------------------------------------------- streams, graphs, a run

def test_python_refusals():
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Rotary, cache_attention, cache_keep, rotary, verify_drafts
    i32 = dict(dtype=torch.int32, device="cuda")
    b = PageBatch(torch.zeros(1, 1, **i32), torch.tensor([0, 2], **i32), torch.tensor([2], **i32), max_new=2)
    c = PagedCache(2, 16, 1, 64)
    q = relation(torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"))
    for p in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(3, **i32), torch.zeros(2, dtype=torch.int32),
              torch.zeros(4, **i32)[::2]):
        for call in (lambda: cache_attention(q, c, b, parents=p), lambda: rotary(q, None, Rotary(64), b, parents=p),
                     lambda: rotary(q, None, Rotary(64), positions=p)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        rotary(q, q, Rotary(64), b, q_out=q)
    t = relation(torch.zeros(2, 10, device="cuda"))
    tok, u, s = torch.zeros(2, **i32), torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda")
    for args, kw in (((tok.long(), u, s), {}), ((tok, u.double(), s), {}), ((tok, u, u), {}), ((tok, u, s.cpu()), {}),
                     ((tok, u, s), dict(parents=u)), ((tok, u, s), dict(path=tok)), ((tok, u, s), dict(counts=tok))):
        with pytest.raises(ValueError):
            verify_drafts(t, b, *args, **kw)
    path, counts = torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    for args in (([], b, path, counts), (c, b, path[0], counts), (c, b, path, counts.long()), (c, b, path, path[0]),
                 (c, b, path, counts, path[0])):
        with pytest.raises(ValueError):
            cache_keep(*args)


def test_no_rows_and_no_sequences_with_rows():
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Rotary, cache_attention, cache_keep, rotary, verify_drafts
    from tensor_relational_einsum_gb300.relation import check
    i32 = dict(dtype=torch.int32, device="cuda")
    b = PageBatch(torch.zeros(2, 1, **i32), torch.zeros(3, **i32), torch.tensor([3, 0], **i32), max_new=4)
    c = PagedCache(2, 16, 1, 64)
    from tensor_relational_einsum_gb300 import Relation
    none = torch.zeros(0, **i32)
    q = Relation("bf16", (0, 2, 64), [1, 1, 1])
    rotary(q, None, Rotary(64), b)
    cache_attention(q, c, b, parents=none)
    path, counts, picked = verify_drafts(Relation("f32", (0, 9), [1, 1]), b, none, torch.zeros(0, device="cuda"), torch.zeros(2, device="cuda"))
    check()
    assert counts.tolist() == [0, 0] and picked.tolist() == [-1, -1] and (path == -1).all()
    assert cache_keep(c, b, path, counts).tolist() == [3, 0]
    check()


def test_a_step_with_drafts_as_a_captured_run():
    """rotate, append, attend, verify, keep -- three steps of one captured graph on another stream, the batch's tensors
    rewritten in between, against the same steps by definition in 64 bits."""
    from tensor_relational_einsum_gb300 import PageBatch, PagedCache, Rotary, verify_drafts
    from tensor_relational_einsum_gb300.graphs import CachedAttention, capture
    from tensor_relational_einsum_gb300.relation import check
    i32 = dict(dtype=torch.int32, device="cuda")
    heads, kv, dim, page, n, seqs, vocab = 8, 2, 64, 16, 6, 3, 97
    rng = np.random.default_rng(60)
    rows = n * seqs
    pool = 5 * seqs
    table = torch.from_numpy(rng.permutation(pool).astype(np.int32)).cuda().reshape(seqs, 5).contiguous()
    trees = [du.tree("random", n, rng) for _ in range(seqs)]
    lens = np.array([n, n + 9, n + 21])
    t = {x: torch.zeros(rows, h, dim, dtype=torch.bfloat16, device="cuda") for x, h in (("q", heads), ("k", kv), ("v", kv))}
    r = {x: relation(y) for x, y in t.items()}
    batch = PageBatch(table, torch.arange(0, rows + 1, n, **i32), torch.from_numpy(lens.astype(np.int32)).cuda(), max_new=n)
    parents = torch.tensor(sum(trees, []), **i32)
    plan = Rotary(dim, layout="half")
    cache = PagedCache(pool, page, kv, dim)
    step = CachedAttention(r["q"], r["k"], r["v"], cache, batch, rotary=plan, parents=parents)
    target, draft = (torch.zeros(rows, vocab, device="cuda") for _ in range(2))
    tokens, accept, sample = torch.zeros(rows, **i32), torch.zeros(rows, device="cuda"), torch.zeros(seqs, device="cuda")
    path, counts, picked, after = (torch.zeros(s, **i32) for s in ((seqs, n), (seqs,), (seqs,), (seqs,)))
    rt, rd = relation(target), relation(draft)

    def run():
        step.run()
        verify_drafts(rt, batch, tokens, accept, sample, draft=rd, parents=parents, path=path, counts=counts, picked=picked)
        step.keep(path, counts, after)

    # what the cache holds by definition: rows [t, kv, dim] of K and V per sequence
    held = [[np.zeros((0, kv, dim)), np.zeros((0, kv, dim))] for _ in range(seqs)]
    for i in range(seqs):
        old = int(lens[i]) - n
        for w, pool_t in enumerate((cache.k, cache.v)):
            x = values(rng, (old, kv, dim))
            held[i][w] = x
            for p in range(old):
                pool_t[int(table[i, p // page]), :, p % page] = torch.from_numpy(x[p]).to(torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    graph = capture(run)
    for it in range(3):
        new = {x: values(rng, tuple(t[x].shape)) for x in t}
        for x in t:
            t[x].copy_(torch.from_numpy(new[x]).to(torch.bfloat16))
        logits = 2 * rng.normal(size=(rows, vocab))
        soft = lambda x: torch.from_numpy(np.exp(x) / np.exp(x).sum(-1, keepdims=True)).float()  # noqa: E731
        p, d = soft(logits), soft(logits + 0.4 * rng.normal(size=logits.shape))
        tok = np.array([rng.integers(vocab) for _ in range(rows)], dtype=np.int32)
        u, s = rng.random(rows).astype(np.float32) ** 2, rng.random(seqs).astype(np.float32)
        target.copy_(p), draft.copy_(d), tokens.copy_(torch.from_numpy(tok)), accept.copy_(torch.from_numpy(u)), sample.copy_(torch.from_numpy(s))
        batch.lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        check()
        out = step.O.to_dense().double().cpu().numpy()
        now = {x: y.double().cpu().numpy() for x, y in t.items()}
        for i in range(seqs):
            rr = slice(i * n, (i + 1) * n)
            at = [int(lens[i]) - n + du.depth(trees[i], j) for j in range(n)]
            for x in ("q", "k"):  # rotated in place
                want, big = du.rotate(new[x][rr], at, plan.freqs, "half", 0)
                assert np.all(np.abs(now[x][rr] - want) <= rotary_bound(want, big, torch.bfloat16))
            kk, vv = (np.concatenate([held[i][w], now[x][rr]]) for w, x in ((0, "k"), (1, "v")))
            for j in range(n):
                keep = du.kept_positions(trees[i], j, n, int(lens[i]))
                for h in range(heads):
                    o, _, _, big, slack = cu.softmax_attention(now["q"][i * n + j:i * n + j + 1, h], kk[keep, h // 4], vv[keep, h // 4],
                                                               None, 1 / math.sqrt(dim), False)
                    assert np.all(np.abs(out[i * n + j, h] - o[0]) <= cu.out_bound(o, big, slack, len(keep))[0])
            way, token, near = du.verify(p[rr].double().numpy(), d[rr].double().numpy(), tok[rr], trees[i], u[rr].astype(np.float64), float(s[i]))
            assert near > 1e-9
            assert path[i, :len(way)].tolist() == way and counts[i].item() == len(way) and picked[i].item() == token
            base = int(lens[i]) - n
            held[i] = [np.concatenate([x[:base], x[base:][way]]) for x in (kk, vv)]
            assert after[i].item() == base + len(way)
            for w, pool_t in enumerate((cache.k, cache.v)):
                got = np.stack([pool_t[int(table[i, q // page]), :, q % page].double().cpu().numpy() for q in range(base + len(way))])
                assert np.array_equal(got, held[i][w])
        lens = after.cpu().numpy() + n


def test_two_captured_graphs_and_two_streams():
    """Two graphs of the same call over different tensors, replayed on two streams at once, give what each gives alone."""
    from tensor_relational_einsum_gb300 import Rotary, cache_attention, rotary, verify_drafts
    from tensor_relational_einsum_gb300.graphs import capture
    from tensor_relational_einsum_gb300.relation import check
    sets = []
    for seed in (70, 71):
        b = cu.Batch([(16, 1500 + seed), (9, 700), (3, 4000)], 64, seed=seed)
        c = nan_cache(b, 2, 128, "bf16")
        rng = np.random.default_rng(seed)
        fill(c, b, rng)
        _, parents = parents_of(b, "random", seed)
        batch = on_gpu(b, max_new=16)
        q = relation(torch.from_numpy(values(rng, (b.rows, 8, 128))).to(torch.bfloat16).cuda())
        out = relation(torch.zeros(b.rows, 8, 128, dtype=torch.bfloat16, device="cuda"))
        turned = relation(torch.zeros(b.rows, 8, 128, dtype=torch.bfloat16, device="cuda"))
        p = torch.softmax(torch.from_numpy(rng.normal(size=(b.rows, 30011)) * 3).cuda().float(), -1)
        d = torch.softmax(torch.from_numpy(rng.normal(size=(b.rows, 30011)) * 3).cuda().float(), -1)
        tokens = torch.from_numpy(rng.integers(30011, size=b.rows).astype(np.int32)).cuda()
        u, s = (torch.from_numpy(rng.random(k).astype(np.float32)).cuda() for k in (b.rows, 3))
        res = [torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((3, 16), (3,), (3,))]
        rel_p, rel_d = relation(p), relation(d)
        plan = Rotary(128)

        def run(batch=batch, c=c, q=q, out=out, turned=turned, parents=parents, rel_p=rel_p, rel_d=rel_d, tokens=tokens, u=u, s=s,
                res=res, plan=plan):
            rotary(q, None, plan, batch, parents=parents, q_out=turned)
            cache_attention(turned, c, batch, parents=parents, out=out)
            verify_drafts(rel_p, batch, tokens, u, s, draft=rel_d, parents=parents, path=res[0], counts=res[1], picked=res[2])

        run()
        torch.cuda.synchronize()
        want = [out.storage.clone(), *[t.clone() for t in res]]
        sets.append((capture(run), out, res, want, run))  # run: what the graph reads lives on
    streams = [torch.cuda.Stream() for _ in sets]
    for _, out, res, *_ in sets:
        out.storage.zero_()
        for t in res:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, *_), st in zip(sets, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    check()
    for _, out, res, want, _ in sets:
        assert torch.equal(out.storage, want[0]) and all(torch.equal(a, b) for a, b in zip(res, want[1:]))


def test_calls_on_a_given_stream_and_their_new_results():
    from tensor_relational_einsum_gb300 import Rotary, cache_attention, cache_keep, rotary, verify_drafts
    b = cu.Batch([(4, 40)], 16, seed=80)
    c = nan_cache(b, 1, 64, "bf16")
    rng = np.random.default_rng(81)
    fill(c, b, rng)
    _, parents = parents_of(b, "random")
    batch = on_gpu(b, max_new=4)
    x = torch.from_numpy(values(rng, (4, 4, 64))).to(torch.bfloat16).cuda()
    p = relation(torch.full((4, 64), 1.0 / 64, device="cuda"))
    tokens, u, s = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((4,), 0.9, device="cuda"), torch.full((1,), 0.5, device="cuda")

    def all_of(stream):
        q = relation(x.clone())
        torch.cuda.synchronize()
        rotary(q, None, Rotary(64), batch, parents=parents, stream=stream)
        o = cache_attention(q, c, batch, parents=parents, stream=stream)
        path, counts, picked = verify_drafts(p, batch, tokens, u, s, parents=parents, stream=stream)
        lens = cache_keep(c, batch, path, counts, stream=stream)
        torch.cuda.synchronize()
        return [o.storage.clone(), path, counts, picked, lens]

    a, b2 = all_of(None), all_of(torch.cuda.Stream())
    assert all(torch.equal(y, z) for y, z in zip(a, b2)) and a[4].tolist() == [37]


def test_workspace_over_the_parents_is_refused():
    from tensor_relational_einsum_gb300 import _abi
    b = cu.Batch([(8, 3000)], 16, seed=90)
    c = nan_cache(b, 1, 64, "bf16")
    batch = on_gpu(b, max_new=8)
    q, o = (relation(torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")) for _ in range(2))
    L, need = _abi.lib(), ctypes.c_size_t()
    assert L.ea_cache_attention_workspace(c.handle, batch.ref, q.handle, ctypes.byref(need)) == 0 and need.value > 32
    room = torch.zeros(need.value, dtype=torch.uint8, device="cuda")
    a = _abi.CacheAttnOpts(0.0, 1, None, None, room.data_ptr(), need.value, room.data_ptr() + 16)
    assert L.ea_cache_attention(c.handle, batch.ref, q.handle, ctypes.byref(a), None, o.handle) == 7
