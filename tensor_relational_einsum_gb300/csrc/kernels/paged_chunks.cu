// paged_chunks.cu -- the chunk kernel's plan, and its instances for rows in
// order; paged_chunks_tree.cu has those for trees.
#include "paged_chunks.cuh"

namespace ea {

PgPlan plan_cache_chunks(const PgTable &t, const PgPool &c, int group, int causal, int num_sms, int min_rows) {
    PgPlan pl{};
    if ((int64_t)t.max_new * group < min_rows) return pl;
    const int tpt = kRows / group;
    PgSplit &sp = pl.split;
    sp.heads = c.heads;
    sp.group = group;
    sp.tok = 2 * tpt;
    // Short sequences are not cut: the tiles of an item cost less than the merge (2 x 64 tokens in 600 positions, 32 heads
    // over 8: 30.0 us cut, 24.6 us whole).  As in the token kernel it is the table's width that says so.
    const bool whole = t.cap <= kWhole;
    sp.kt = whole ? kWhole : kKeys;
    sp.causal = causal;
    sp.min_rows = min_rows;
    sp.max_rows = INT32_MAX;
    pl.rows = sp.tok * group;
    const int64_t items = std::min<int64_t>((int64_t)t.n_seqs * ((t.max_new + sp.tok - 1) / sp.tok), t.rows / sp.tok + t.n_seqs);
    const int64_t units = (t.cap + sp.kt - 1) / sp.kt * items * c.heads;
    pl.ctas = (int)std::min<int64_t>(units, num_sms);
    pl.bytes = whole ? 0 : pg_work_bytes(pl.ctas, pl.rows, c.dim);
    return pl;
}

PgExpand plan_cache_expand(const PgTable &t, const PgPool &c, int group, int min_rows) {
    PgExpand x{};
    if (c.fmt != EA_CACHE_E4M3 || (int64_t)t.max_new * group < 2 * kRows) return x;
    const int64_t least = (min_rows + group - 1) / group;  // rows of a sequence served; <= max_new <= t.rows
    const bool by_row = t.rows / least < t.n_seqs;
    const int64_t places = by_row ? t.rows / least : t.n_seqs;
    const int64_t blocks = (t.cap + kKeys - 1) / kKeys, vectors = blocks * kKeys * places * c.heads;
    // Up to 4 GB.  A batch that could need more (many sequences that may have chunks, or a very wide table) keeps to the
    // 8-bit pages.
    if (vectors * c.dim * 4 > (int64_t)1 << 32) return x;
    x.blocks = (int32_t)blocks;
    x.places = (int32_t)places;
    x.place_rows = by_row ? (int32_t)least : 0;
    x.bytes = (size_t)vectors * c.dim * 4;
    return x;
}

cudaError_t launch_cache_chunks(const PgAttn &p, const PgPlan &pl, const PgMaps &maps, const PgWork &w, bool early, cudaStream_t st) {
    return p.parents ? launch_cache_chunks_tree(p, pl, maps, w, early, st) : launch_chunks<false>(p, pl, maps, w, early, st);
}

}  // namespace ea
