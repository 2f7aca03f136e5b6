"""GPU tests of the operators around drafted tokens at the ends of their
ranges: clusters of every size with many rejections at a node, sequences
without rows, sums and scales out of the ordinary.  Definitions and tolerances
as in test_gpu_drafts.
"""
import math

import numpy as np
import pytest

import cache_util as cu
import drafts_util as du

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_gpu_cache import fill, nan_cache, on_gpu, relation, values  # noqa: E402
from test_gpu_cache_ranges import scaled_fill  # noqa: E402
from test_gpu_drafts import expect, parents_of, rotary_bound, run_verify, verify_batch  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tensor_relational_einsum_gb300.build import build
    build()
    yield
    from tensor_relational_einsum_gb300.relation import check
    check()


# ------------------------------------------------------------ verification

@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("vocab", [2048, 4097, 20011, 40000])
def test_verify_sequences_without_rows_in_clusters(vocab, drafts):
    """Empty sequences, whose first CTA has its first order for the others at once, among others: clusters of 1 to 16."""
    from tensor_relational_einsum_gb300.relation import check
    b, trees, parents, target, draft, tokens, accept, sample = verify_batch([0, 0, 3, 0, 1, 0, 0, 5, 0], vocab, torch.float32, drafts,
                                                                            "random", 31)
    for _ in range(5):
        got = run_verify(b, parents, target, draft, tokens, accept, sample)
        check()
        expect(b, trees, target, draft, tokens, accept, sample, got)


def rejections(parents, path):
    """How many children of each accepted node are asked in vain."""
    path = list(path)
    return [sum(p == v and c < after for c, p in enumerate(parents)) for v, after in zip(path, path[1:] + [len(parents)])]


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ns", [[24, 17, 30], [128, 64]])
@pytest.mark.parametrize("vocab", [9000, 20011, 40000])
def test_verify_with_many_rejections_in_clusters(vocab, ns, dtype, drafts):
    """Drafts unlike the target, in clusters of 4, 8 and 16 CTAs: masses of many subtractions go from CTA to CTA."""
    from tensor_relational_einsum_gb300.relation import check
    b, trees, parents, target, draft, tokens, accept, sample = verify_batch(ns, vocab, dtype, drafts, "star", 41, branch_noise=4.0, sharp=0.5)
    got = run_verify(b, parents, target, draft, tokens, accept, sample)
    check()
    expect(b, trees, target, draft, tokens, accept, sample, got)
    path, counts = got[0].cpu().numpy(), got[1].tolist()
    assert max(max(rejections(trees[i], path[i, :counts[i]])) for i in range(len(ns))) >= 16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,value", [(64, 0.5), (300, 1.0), (20011, 1.0), (40000, 2.0 ** -12), (131072, 7.0), (5000, 4.0 / 5000)])
def test_verify_reports_sums_out_of_range(vocab, value, dtype):
    """Rows that add up to 2 and more, to multiples of 4 among them (logits by mistake): the error word, no token, what was
    accepted before stays; the sequence beside it as it should be."""
    from tensor_relational_einsum_gb300 import EaError
    from tensor_relational_einsum_gb300.relation import check
    for kind in ("chain", "star"):
        for drafts in (True, False):
            b, trees, parents, target, draft, tokens, accept, sample = verify_batch([3, 2, 4], vocab, dtype, drafts, kind, 44)
            want, ahead = run_verify(b, parents, target, draft, tokens, accept, sample), int(b.starts[1])
            check()
            accept[ahead + 1] = 1.0
            tokens[ahead + 1] = 5
            if drafts:
                draft[ahead, 5] = 1.0  # u d = 1 >= r: a rejection
            target[ahead:ahead + 2] = value
            target[ahead, 5] = 0.0
            path, counts, picked = run_verify(b, parents, target, draft, tokens, accept, sample)
            with pytest.raises(EaError):
                check()
            assert path[1].tolist() == [0] + [-1] * (path.shape[1] - 1) and counts[1].item() == 1 and picked[1].item() == -1
            for i in (0, 2):
                assert torch.equal(path[i], want[0][i]) and counts[i] == want[1][i] and picked[i] == want[2][i]


def test_verify_sums_just_below_two():
    """1.5 and 1.96875 are in range (two halves more than the distribution that they are scaled from)."""
    from tensor_relational_einsum_gb300.relation import check
    from test_gpu_drafts import one
    for n, x in ((3, 0.5), (63, 0.03125)):
        row = [x] * n + [0.0] * (70 - n)
        for s in (0.0, 0.25, 0.5, 0.99609375):
            assert one([row], None, [0], [-1], [0.0], s) == ([0], int(s * n))
    check()


# ---------------------------------------------------------- tree attention

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,group", [(3, 4), (7, 4), (40, 1), (40, 4), (63, 4), (70, 4)])
@pytest.mark.parametrize("spoil", ["codes", "byte", "large"])
def test_dropped_keys_of_8_bit_cells(spoil, n, group, dim):
    """Leaves whose keys are NaN, or 2^18 times larger than the others: no other row is touched.  12 to 280 rows: both
    kernels, and expanded pages."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, 150), (n, n + 90)], 16, seed=10)
    c = nan_cache(b, 1, dim, "e4m3")
    rng = np.random.default_rng(11)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, "star")
    # the kept keys' scales differ by less than 2^3: 2^20 times the largest would lie beyond the 2^21 that are exact
    large = int(c.k_scale[c.k_scale < 255].max()) + 18
    for i, t in enumerate(b.lens):
        pg, sl = b.places(i)
        for j in (n - 1, n // 2):
            at = (int(pg[t - n + j]), slice(None), int(sl[t - n + j]))
            if spoil == "codes":
                c.k.view(torch.uint8)[at] = 0x7F
            elif spoil == "byte":
                c.k_scale[at] = 255
            else:
                c.k_scale[at] = large
    q = values(rng, (b.rows, group, dim))
    out = cache_attention(relation(torch.from_numpy(q).to(torch.bfloat16).cuda()), c, on_gpu(b, max_new=n), parents=parents)
    check()
    got = out.to_dense().double().cpu().numpy()
    for i, t in enumerate(b.lens):
        for j in range(n):
            if j in (n - 1, n // 2):
                continue
            keep = du.kept_positions(trees[i], j, n, int(t))
            for h in range(group):
                o, _, _, big, slack = cu.softmax_attention(q[i * n + j:i * n + j + 1, h], held[i][0][keep, 0], held[i][1][keep, 0], None,
                                                           1 / math.sqrt(dim), False)
                assert np.all(np.abs(got[i * n + j, h] - o[0]) <= cu.out_bound(o, big, slack, len(keep))[0]), (i, j, h)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,n,kv", [(3, 85, 8), (4, 16, 8), (4, 63, 8), (8, 31, 4), (1, 127, 4)])
def test_8_bit_runs_give_the_same_bits(group, n, kv, dim):
    """Raw 8-bit pages, scales that differ between sequences, items of one and two row tiles: 150 runs of one call, next to
    copies on another stream, give the same outputs, maxima and sums; trees and rows in order."""
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(38)
    seqs = [(int(x), int(x + t)) for x, t in zip(rng.integers(max(1, n // 2), n + 1, size=16), rng.integers(0, 1500, size=16))]
    seqs[3] = (n, 2500)
    b = cu.Batch(seqs, 32, before=1)
    c = nan_cache(b, kv, dim, "e4m3")
    scaled_fill(c, b, rng)
    q = relation(torch.from_numpy(values(rng, (b.rows, kv * group, dim))).to(torch.bfloat16).cuda())
    _, parents = parents_of(b, "random")
    batch, side = on_gpu(b, max_new=n), torch.cuda.Stream()
    other = [torch.zeros(1 << 24, device="cuda") for _ in range(2)]
    for tree in (parents, None):
        out = torch.zeros(b.rows, kv * group, dim, dtype=torch.bfloat16, device="cuda")
        m, l = (torch.zeros(b.rows, kv * group, device="cuda") for _ in range(2))
        got, first, differ = [relation(t) for t in (out, m, l)], None, torch.zeros((), dtype=torch.bool, device="cuda")
        for i in range(150):
            if i % 8 == 0:
                with torch.cuda.stream(side):
                    other[0].copy_(other[1])
            cache_attention(q, c, batch, out=got[0], m_out=got[1], l_out=got[2], parents=tree)
            if first is None:
                first = [t.clone() for t in (out, m, l)]
            for t, w in zip((out, m, l), first):
                differ |= (t != w).any()
        assert not differ.item()
    check()


# ------------------------------------------------------------------ rotary

def test_rotary_refuses_a_result_without_its_operand():
    from tensor_relational_einsum_gb300 import Rotary, rotary
    q, o = (relation(torch.zeros(2, 1, 64, device="cuda")) for _ in range(2))
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rotary(q, None, Rotary(64), positions=at, q_out=q, k_out=o)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("rows,heads,dim,dims,offset", [(3, 65535, 2, 2, 0), (2, 1, 65535, 256, 65279), (300001, 1, 6, 4, 2), (1, 1, 2, 2, 0)])
def test_rotary_largest_and_smallest(rows, heads, dim, dims, offset, layout, dtype):
    """The most heads, columns and many rows, in place and into new rows; positions up to the last one there is."""
    from tensor_relational_einsum_gb300 import PageBatch, Rotary, rotary
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(90)
    plan = Rotary(dims, layout=layout, offset=offset)
    n = min(rows, 128)
    x = torch.from_numpy(rng.normal(size=(rows, heads, dim))).to(dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = PageBatch(torch.zeros(1, 1, **i32), torch.tensor([rows - n, rows], **i32), torch.tensor([2 ** 31 - 1], **i32), max_new=n)
    # at t f = 2^31 half a step of fp64 is 2^-22: t f and 2 pi here, f / 2 pi and its factor there, 4 * 2^-22 of an angle
    at = np.full(rows, -1, dtype=np.int64)
    at[rows - n:] = np.arange(2 ** 31 - 1 - n, 2 ** 31 - 1)
    some = np.unique(np.concatenate([[0], np.arange(max(0, rows - n - 1), rows)]))
    want, big = du.rotate(x[some].double().numpy(), at[some], plan.freqs, layout, offset)
    for place in (True, False):
        d = x.cuda()
        o = d if place else torch.full_like(d, -3.0)
        rotary(relation(d), None, plan, batch, q_out=relation(o))
        check()
        still = at[some] < 0
        got = o[torch.from_numpy(some).cuda()].double().cpu().numpy()
        assert np.array_equal(got[still], x[some].double().numpy()[still] if place else np.full_like(got[still], -3.0))
        assert np.all(np.abs(got - want)[~still] <= (rotary_bound(want, big, dtype) + 1e-6 * big)[~still])


# ------------------------------------------------------------ ends of ranges

def test_a_chain_of_128_accepted_nodes_is_kept_where_it_is():
    """Every node accepted: the longest path; the keep that follows moves nothing."""
    from tensor_relational_einsum_gb300 import cache_keep
    from tensor_relational_einsum_gb300.relation import check
    b, trees, parents, target, draft, tokens, accept, sample = verify_batch([128, 127], 501, torch.float32, True, "chain", 45)
    accept[:] = 0.0
    for p in (None, parents):
        got = run_verify(b, p, target, draft, tokens, accept, sample)
        check()
        expect(b, trees, target, draft, tokens, accept, sample, got)
        assert got[1].tolist() == [128, 127]
    c = nan_cache(b, 1, 64, "bf16")
    fill(c, b, np.random.default_rng(46))
    was = c.k.view(torch.int16).clone()
    lens = cache_keep(c, on_gpu(b, max_new=128), got[0], got[1])
    check()
    assert torch.equal(c.k.view(torch.int16), was) and lens.tolist() == [t for _, t in b.seqs]


@pytest.mark.parametrize("drafts", [True, False])
def test_verify_tokens_twice_and_tiny_vocabularies(drafts):
    """Siblings of one token, and more children than tokens."""
    from tensor_relational_einsum_gb300.relation import check
    for vocab, seed in ((3, 47), (4, 48), (40, 49)):
        b, trees, parents, target, draft, tokens, accept, sample = verify_batch([12, 7, 30, 2], vocab, torch.float32, drafts, "star", seed,
                                                                                branch_noise=1.5)
        accept[:] = np.sqrt(accept)
        got = run_verify(b, parents, target, draft, tokens, accept, sample)
        check()
        expect(b, trees, target, draft, tokens, accept, sample, got)


def test_verify_many_sequences_and_a_wide_vocabulary():
    from tensor_relational_einsum_gb300.relation import check
    for ns, vocab in (([1, 2, 0] * 3000, 5), ([2], (1 << 22) + 5)):
        b, trees, parents, target, draft, tokens, accept, sample = verify_batch(ns, vocab, torch.float32, True, "chain", 51)
        got = run_verify(b, parents, target, draft, tokens, accept, sample)
        check()
        expect(b, trees, target, draft, tokens, accept, sample, got)


def test_keep_many_sequences():
    from tensor_relational_einsum_gb300 import PagedCache, cache_keep
    from tensor_relational_einsum_gb300.relation import check
    rng = np.random.default_rng(52)
    seqs = [(3, 3 + int(t)) for t in rng.integers(0, 14, size=5000)]
    b = cu.Batch(seqs, 16, seed=53)
    pools = [[torch.randint(-9999, 9999, (b.pages_total, 1, 16, 64), dtype=torch.int16, device="cuda") for _ in range(2)] for _ in range(3)]
    was = [[t.clone() for t in p] for p in pools]
    caches = [PagedCache(b.pages_total, 16, 1, 64, "bf16", k=p[0].view(torch.bfloat16), v=p[1].view(torch.bfloat16)) for p in pools]
    path = torch.tensor([0, 2, -1], dtype=torch.int32, device="cuda").repeat(5000, 1)
    lens = cache_keep(caches, on_gpu(b, max_new=3), path, torch.full((5000,), 2, dtype=torch.int32, device="cuda"))
    check()
    assert lens.tolist() == [t - 1 for _, t in seqs]
    t = b.lens.astype(np.int64)
    pages = torch.from_numpy(b.pages).long().cuda()
    i = torch.arange(5000, device="cuda")
    src, dst = torch.from_numpy(t - 1).cuda(), torch.from_numpy(t - 2).cuda()
    for got, old in zip(pools, was):
        for g, w in zip(got, old):
            w[pages[i, dst // 16], :, dst % 16] = w[pages[i, src // 16], :, src % 16]
            assert torch.equal(g, w)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,n", [(128, 128), (31, 77), (7, 128), (5, 6), (33, 1)])
def test_trees_under_wide_groups(group, n, fmt):
    from tensor_relational_einsum_gb300 import cache_attention
    from tensor_relational_einsum_gb300.relation import check
    b = cu.Batch([(n, n + 130), (max(1, n // 2), n)], 32, before=1, seed=54)
    c = nan_cache(b, 1, 64, fmt)
    rng = np.random.default_rng(55)
    held = fill(c, b, rng)
    trees, parents = parents_of(b, "random")
    q = values(rng, (b.rows, group, 64))
    out = cache_attention(relation(torch.from_numpy(q).to(torch.bfloat16).cuda()), c, on_gpu(b, max_new=n), parents=parents)
    check()
    got = out.to_dense().double().cpu().numpy()
    for i, (rows, t) in enumerate(b.seqs):
        k, v = (x[:, 0] for x in held[i])
        for j in range(rows):
            keep = du.kept_positions(trees[i], j, rows, t)
            r = int(b.starts[i]) + j
            o, _, _, big, slack = cu.softmax_attention(q[r], k[keep], v[keep], None, 0.125, False)
            assert np.all(np.abs(got[r] - o) <= cu.out_bound(o, big, slack, len(keep))), (i, j)
