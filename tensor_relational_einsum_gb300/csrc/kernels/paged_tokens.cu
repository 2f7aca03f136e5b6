// paged_tokens.cu -- the token kernel's plan, and its instances for rows in
// order; paged_tokens_tree.cu has those for trees.
#include "paged_tokens.cuh"

namespace ea {

PgPlan plan_cache_tokens(const PgTable &t, const PgPool &c, int group, int causal, int num_sms) {
    PgPlan pl{};
    if (group > kPgTokenRows || t.rows == 0) return pl;
    pl.rows = (int64_t)t.max_new * group <= 16 ? 16 : 32;
    PgSplit &sp = pl.split;
    sp.heads = c.heads;
    sp.group = group;
    sp.tok = pl.rows / group;
    sp.causal = causal;
    sp.min_rows = 1;
    sp.max_rows = pl.rows;
    // Short sequences are not cut: another block adds less than the merge's launch.  The table's width says which they
    // are: the lengths are known on the device only.
    const int64_t longest = t.cap;
    sp.kt = longest <= 512 ? 512 : c.fmt == EA_CACHE_E4M3 || c.dim == 64 ? 128 : 64;  // a block
    const int64_t units = (longest + sp.kt - 1) / sp.kt * t.n_seqs * c.heads;
    // Many short sequences: a warp an item, without barriers or a merge between warps.
    sp.solo = sp.kt == 512 && pl.rows == 16 && (int64_t)t.n_seqs * c.heads >= 4 * (int64_t)num_sms;
    pl.ctas = (int)std::min<int64_t>(sp.solo ? (units + 3) / 4 : units, (int64_t)num_sms * 2);
    pl.bytes = units > t.n_seqs * (int64_t)c.heads ? pg_work_bytes(pl.ctas, pl.rows, c.dim) : 0;  // 0: a unit is an item
    return pl;
}

cudaError_t launch_cache_tokens(const PgAttn &p, const PgPlan &pl, const PgWork &w, bool early, cudaStream_t st) {
    return p.parents ? launch_cache_tokens_tree(p, pl, w, early, st) : launch_tokens<false>(p, pl, w, early, st);
}

}  // namespace ea
