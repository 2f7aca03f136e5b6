// cache.cpp -- the paged cache's entry points: handles, checks of arguments,
// and the host form of the batch check.
#include <cmath>
#include <unordered_set>

#include "paged_host.h"

namespace ea {
namespace {

ea_status rows_call(const char *what, bool read, ea_cache cache, const ea_page_batch *batch, ea_relation k,
                    ea_relation v, void *stream) {
    if (!cache || !k || !v) return set_error(EA_ERR_ARG, "%s: NULL argument", what);
    int64_t rows, heads, dim, rows_v, heads_v, dim_v;
    ea_status s = dense_rows(k, what, 2, &rows, &heads, &dim);
    if (s) return s;
    s = dense_rows(v, what, 2, &rows_v, &heads_v, &dim_v);
    if (s) return s;
    if (k->dtype != v->dtype) return set_error(EA_ERR_DTYPE, "%s: K and V have different dtypes", what);
    if (rows != rows_v || heads != heads_v || dim != dim_v)
        return set_error(EA_ERR_SHAPE, "%s: K and V have different extents", what);
    if (heads != cache->heads || dim != cache->dim)
        return set_error(EA_ERR_SHAPE, "%s: rows of %lld x %lld, the cache holds %d x %d", what, (long long)heads,
                         (long long)dim, cache->heads, cache->dim);
    s = batch_args(batch, cache->page, rows);
    if (s) return s;
    if (rows * heads > INT32_MAX) return set_error(EA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 vectors", what);
    if (in_cache(cache, k) || in_cache(cache, v)) return set_error(EA_ERR_ARG, "%s: K or V overlaps the cache", what);
    if (read && overlap(k->arena, k->bytes, v->arena, v->bytes)) return set_error(EA_ERR_ARG, "%s: K and V overlap", what);
    if (read ? in_batch(batch, k->arena, k->bytes) || in_batch(batch, v->arena, v->bytes) : in_batch(batch, cache))
        return set_error(EA_ERR_ARG, "%s: the batch's arrays lie in what the call writes", what);
    std::lock_guard<std::mutex> lk(g_mu);
    DevCtx *c;
    s = here(cache, &c);
    if (s) return s;
    PgRows p{};
    p.t = table_of(batch, cache->page, rows);
    p.c = pool_of(cache);
    p.k = k->arena;
    p.v = v->arena;
    p.f32 = k->dtype == EA_F32;
    p.read = read;
    p.err = c->err;
    int64_t ctas = 0;
    if (rows > 0) {
        cudaError_t e = launch_cache_rows(p, &ctas, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_error(e, what);
    }
    note_launch(kCacheRows, ctas > 0, ctas);
    return EA_OK;
}

}  // namespace
}  // namespace ea

using namespace ea;

extern "C" ea_status ea_cache_create(ea_cache_format format, int64_t pages, int32_t page, int32_t heads, int32_t dim,
                                     void *k, void *v, void *k_scale, void *v_scale, ea_cache *out) {
    return entry([&]() -> ea_status {
        if (!out || !k || !v) return set_error(EA_ERR_ARG, "ea_cache_create: NULL argument");
        if (format != EA_CACHE_BF16 && format != EA_CACHE_E4M3)
            return set_error(EA_ERR_DTYPE, "ea_cache_create: unknown format %d", (int)format);
        if (pages < 1 || pages > INT32_MAX) return set_error(EA_ERR_ARG, "ea_cache_create: %lld pages", (long long)pages);
        if (heads < 1 || heads > 65535) return set_error(EA_ERR_ARG, "ea_cache_create: %d heads", heads);
        int lg = 4;
        while (lg < 7 && (1 << lg) != page) lg++;
        if ((1 << lg) != page) return set_error(EA_ERR_UNSUPPORTED, "ea_cache_create: page of %d positions (16, 32, 64 or 128)", page);
        if (dim != 64 && dim != 128) return set_error(EA_ERR_UNSUPPORTED, "ea_cache_create: head dim %d (64 or 128 only)", dim);
        const bool e4m3 = format == EA_CACHE_E4M3;
        if (e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr))
            return set_error(EA_ERR_ARG, "ea_cache_create: scales belong to the e4m3 format, and only to it");
        for (const void *x : {k, v, k_scale, v_scale})
            if (((uintptr_t)x & 15) != 0) return set_error(EA_ERR_ARG, "ea_cache_create: arrays must be 16-byte aligned");
        if ((double)pages * heads * page > (double)INT32_MAX)
            return set_error(EA_ERR_UNSUPPORTED, "ea_cache_create: more than 2^31 - 1 vectors");
        ea_cache_s c{};
        c.format = format;
        c.n_pages = pages;
        c.page = page;
        c.page_log2 = lg;
        c.heads = heads;
        c.dim = dim;
        c.k = (char *)k;
        c.v = (char *)v;
        c.ks = (uint8_t *)k_scale;
        c.vs = (uint8_t *)v_scale;
        const size_t n = cache_bytes(&c), ns = e4m3 ? n / dim : 0;
        if (overlap(k, n, v, n) || overlap(k_scale, ns, v_scale, ns) || overlap(k, n, k_scale, ns) ||
            overlap(k, n, v_scale, ns) || overlap(v, n, k_scale, ns) || overlap(v, n, v_scale, ns))
            return set_error(EA_ERR_ARG, "ea_cache_create: the arrays overlap");
        cudaError_t e = cudaGetDevice(&c.device);
        if (e != cudaSuccess) {
            cudaGetLastError();  // no device: the handle serves the host checks only
            c.device = -1;
        } else {
            e = cudaDeviceGetAttribute(&c.num_sms, cudaDevAttrMultiProcessorCount, c.device);
            if (e != cudaSuccess) return cuda_error(e, "cudaDeviceGetAttribute");
        }
        *out = new ea_cache_s(c);
        return EA_OK;
    });
}

extern "C" ea_status ea_cache_destroy(ea_cache cache) {
    set_error(EA_OK, "");
    delete cache;
    return EA_OK;
}

extern "C" ea_status ea_cache_append(ea_cache cache, const ea_page_batch *batch, ea_relation k, ea_relation v, void *stream) {
    return entry([&] { return rows_call("ea_cache_append", false, cache, batch, k, v, stream); });
}

extern "C" ea_status ea_cache_read(ea_cache cache, const ea_page_batch *batch, ea_relation k, ea_relation v, void *stream) {
    return entry([&] { return rows_call("ea_cache_read", true, cache, batch, k, v, stream); });
}

namespace ea {
namespace {

// Shape checks of an attention call; fills what the launch needs of q.
ea_status attn_shape(ea_cache cache, const ea_page_batch *batch, ea_relation q, int64_t *rows, int64_t *heads) {
    if (!cache || !q) return set_error(EA_ERR_ARG, "ea_cache_attention: NULL argument");
    int64_t dim;
    ea_status s = dense_rows(q, "ea_cache_attention: Q", 2, rows, heads, &dim);
    if (s) return s;
    if (q->dtype != EA_BF16) return set_error(EA_ERR_DTYPE, "ea_cache_attention: Q must be bf16");
    if (dim != cache->dim)
        return set_error(EA_ERR_SHAPE, "ea_cache_attention: head dim %lld, the cache holds %d", (long long)dim, cache->dim);
    if (*heads < 1 || *heads % cache->heads)
        return set_error(EA_ERR_SHAPE, "ea_cache_attention: %lld query heads over %d key-value heads", (long long)*heads, cache->heads);
    if (*heads / cache->heads > 128)
        return set_error(EA_ERR_UNSUPPORTED, "ea_cache_attention: more than 128 query heads to a key-value head");
    return batch_args(batch, cache->page, *rows);
}

// The kernels of a call.  Sequences with few rows and the others are served
// by kernels of their own, each leaving out the other's sequences; a kernel
// that max_new rules out is not launched.
struct AttnPlans {
    PgPlan tokens;
    PgPlan chunks;
    PgExpand expand;
    size_t bytes;
};

AttnPlans plans_of(const ea_cache_s *cache, const ea_page_batch *batch, int64_t rows, int64_t heads, int causal) {
    AttnPlans a{};
    const PgTable t = table_of(batch, cache->page, rows);
    const int group = (int)(heads / cache->heads);
    a.tokens = plan_cache_tokens(t, pool_of(cache), group, causal, cache->num_sms);
    a.chunks = plan_cache_chunks(t, pool_of(cache), group, causal, cache->num_sms,
                                 a.tokens.ctas ? a.tokens.split.max_rows + 1 : 1);
    if (a.chunks.ctas > 0) a.expand = plan_cache_expand(t, pool_of(cache), group, a.chunks.split.min_rows);
    a.bytes = a.tokens.bytes + a.chunks.bytes + a.expand.bytes;
    return a;
}

ea_status encode(DevCtx *c, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2, CUtensorMap *m) {
    if (!c->encode) return set_error(EA_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
    cuuint64_t gdim[3] = {d0, d1, d2}, gstr[2] = {d0 * 2, d0 * d1 * 2};
    cuuint32_t box[3] = {64, b1, b2}, estr[3] = {1, 1, 1};
    CUresult r = c->encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), gdim, gstr, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EA_OK : set_error(EA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// Tensor maps of a chunk launch: a tile of Q is the group's heads of `tok / 2`
// tokens; a page of K or V is `page` vectors.  `wide`: the pages are the bf16
// ones in the workspace (pages of 128), not the cache's.
ea_status chunk_maps(DevCtx *c, ea_cache_s *cache, const ea_relation_s *q, int64_t heads, int64_t rows, const PgSplit &sp,
                     const PgPool *wide, PgMaps *m) {
    memset(m, 0, sizeof *m);
    ea_status s = encode(c, q->arena, cache->dim, heads, rows, sp.group, sp.tok / 2, &m->q);
    if (s) return s;
    if (wide) {
        const uint64_t vecs = (uint64_t)wide->n_pages * wide->heads << wide->page_log2;
        s = encode(c, wide->k, wide->dim, vecs, 1, 1 << wide->page_log2, 1, &m->k);
        return s ? s : encode(c, wide->v, wide->dim, vecs, 1, 1 << wide->page_log2, 1, &m->v);
    }
    if (cache->format != EA_CACHE_BF16) return EA_OK;
    if (!cache->mapped) {
        const uint64_t vecs = (uint64_t)cache->n_pages * cache->heads * cache->page;
        s = encode(c, cache->k, cache->dim, vecs, 1, cache->page, 1, &cache->k_map);
        if (!s) s = encode(c, cache->v, cache->dim, vecs, 1, cache->page, 1, &cache->v_map);
        if (s) return s;
        cache->mapped = true;
    }
    m->k = cache->k_map;
    m->v = cache->v_map;
    return EA_OK;
}

}  // namespace
}  // namespace ea

extern "C" ea_status ea_cache_attention_workspace(ea_cache cache, const ea_page_batch *batch, ea_relation q, size_t *bytes) {
    return entry([&]() -> ea_status {
        if (!bytes) return set_error(EA_ERR_ARG, "ea_cache_attention_workspace: NULL argument");
        int64_t rows, heads;
        ea_status s = attn_shape(cache, batch, q, &rows, &heads);
        if (s) return s;
        *bytes = plans_of(cache, batch, rows, heads, 1).bytes;
        return EA_OK;
    });
}

extern "C" ea_status ea_cache_attention(ea_cache cache, const ea_page_batch *batch, ea_relation q,
                                        const ea_cache_attn_opts *opts, void *stream, ea_relation out) {
    return entry([&]() -> ea_status {
        if (!out) return set_error(EA_ERR_ARG, "ea_cache_attention: NULL argument");
        ea_cache_attn_opts o{};
        if (opts) o = *opts;
        int64_t rows, heads;
        ea_status s = attn_shape(cache, batch, q, &rows, &heads);
        if (s) return s;
        int64_t rows_o, heads_o, dim_o;
        s = dense_rows(out, "ea_cache_attention: O", 2, &rows_o, &heads_o, &dim_o);
        if (s) return s;
        if (out->dtype != EA_BF16) return set_error(EA_ERR_DTYPE, "ea_cache_attention: O must be bf16");
        if (rows_o != rows || heads_o != heads || dim_o != cache->dim)
            return set_error(EA_ERR_SHAPE, "ea_cache_attention: O must have the extents of Q");
        if (o.scale < 0.0f || !std::isfinite(o.scale)) return set_error(EA_ERR_ARG, "ea_cache_attention: scale must be > 0");
        if ((o.m_out != nullptr) != (o.l_out != nullptr))
            return set_error(EA_ERR_ARG, "ea_cache_attention: give both m_out and l_out or neither");
        for (ea_relation r : {o.m_out, o.l_out}) {
            if (!r) continue;
            int64_t rows_s, heads_s;
            s = dense_rows(r, "ea_cache_attention: m_out / l_out", 1, &rows_s, &heads_s, nullptr);
            if (s) return s;
            if (r->dtype != EA_F32) return set_error(EA_ERR_DTYPE, "ea_cache_attention: m_out and l_out must be f32");
            if (rows_s != rows || heads_s != heads)
                return set_error(EA_ERR_SHAPE, "ea_cache_attention: m_out / l_out have the extents of Q without the head dim");
        }
        const ea_relation_s *outs[3] = {out, o.m_out, o.l_out};
        for (int i = 0; i < 3; i++) {
            if (!outs[i]) continue;
            bool bad = in_cache(cache, outs[i]) || overlap(outs[i]->arena, outs[i]->bytes, q->arena, q->bytes);
            for (int j = 0; j < i; j++) bad |= outs[j] && overlap(outs[i]->arena, outs[i]->bytes, outs[j]->arena, outs[j]->bytes);
            bad |= in_batch(batch, outs[i]->arena, outs[i]->bytes);
            if (bad) return set_error(EA_ERR_ARG, "ea_cache_attention: an output overlaps Q, the cache, the batch or another output");
        }
        if (o.parents) {
            s = tree_args("ea_cache_attention", batch, o.parents, rows);
            if (s) return s;
            for (const ea_relation_s *r : outs)
                if (r && overlap(r->arena, r->bytes, o.parents, rows * 4))
                    return set_error(EA_ERR_ARG, "ea_cache_attention: parents lie in an output");
        }
        std::lock_guard<std::mutex> lk(g_mu);
        DevCtx *c;
        s = here(cache, &c);
        if (s) return s;
        PgAttn p{};
        p.t = table_of(batch, cache->page, rows);
        p.parents = o.parents;
        p.c = pool_of(cache);
        p.q = q->arena;
        p.o = out->arena;
        p.m_out = o.m_out ? (float *)o.m_out->arena : nullptr;
        p.l_out = o.l_out ? (float *)o.l_out->arena : nullptr;
        p.qheads = (int32_t)heads;
        p.group = (int32_t)(heads / cache->heads);
        p.causal = o.causal != 0 && !o.parents;  // a tree's rows: every item has all of the sequence's keys
        p.scale = o.scale == 0.0f ? (float)(1.0 / std::sqrt((double)cache->dim)) : o.scale;
        p.scale_log2 = (float)((double)p.scale * 1.4426950408889634);
        p.err = c->err;
        const AttnPlans a = plans_of(cache, batch, rows, heads, p.causal);
        if (a.bytes > 0 && (!o.workspace || o.workspace_bytes < a.bytes || ((uintptr_t)o.workspace & 15) != 0))
            return set_error(EA_ERR_ARG, "ea_cache_attention: workspace of %zu bytes, 16-byte aligned, needed", a.bytes);
        if (a.bytes > 0) {
            bool bad = in_cache(cache, o.workspace, a.bytes) || overlap(o.workspace, a.bytes, q->arena, q->bytes);
            for (const ea_relation_s *r : outs) bad |= r && overlap(o.workspace, a.bytes, r->arena, r->bytes);
            bad |= in_batch(batch, o.workspace, a.bytes) || (o.parents && overlap(o.workspace, a.bytes, o.parents, rows * 4));
            if (bad) return set_error(EA_ERR_ARG, "ea_cache_attention: the workspace overlaps an operand, the cache or the batch");
        }
        // (expansion,) chunks, tokens, merge: the tokens' CTAs fill the SMs that the chunks' leave
        char *ws = (char *)o.workspace;
        const PgWork wc = pg_work(a.chunks, ws), wt = pg_work(a.tokens, ws + a.chunks.bytes);
        int64_t ctas = 0;
        int launches = 0;
        cudaError_t e = cudaSuccess;
        if (a.chunks.ctas > 0) {
            PgMaps maps;
            PgAttn pc = p;
            if (a.expand.blocks > 0) {
                char *wide = ws + a.chunks.bytes + a.tokens.bytes;
                pc.c = PgPool{wide, wide + a.expand.bytes / 2, nullptr, nullptr, (int64_t)a.expand.places * a.expand.blocks, 7,
                              p.c.heads, p.c.dim, EA_CACHE_BF16};
                pc.t.pages = nullptr;
                pc.t.page_stride = a.expand.blocks;
                pc.t.place_rows = a.expand.place_rows;
            }
            s = chunk_maps(c, cache, q, heads, rows, a.chunks.split, a.expand.blocks > 0 ? &pc.c : nullptr, &maps);
            if (s) return s;
            if (a.expand.blocks > 0) {
                e = launch_cache_expand(p, a.chunks.split, a.expand, pc.c.k, (cudaStream_t)stream);
                if (e != cudaSuccess) return cuda_error(e, "ea_cache_attention");
                ctas += (int64_t)a.expand.places * a.expand.blocks * p.c.heads;
                launches++;
            }
            e = launch_cache_chunks(pc, a.chunks, maps, wc, launches > 0, (cudaStream_t)stream);
            if (e != cudaSuccess) return cuda_error(e, "ea_cache_attention");
            ctas += a.chunks.ctas;
            launches++;
        }
        if (a.tokens.ctas > 0) {
            e = launch_cache_tokens(p, a.tokens, wt, launches > 0, (cudaStream_t)stream);
            if (e != cudaSuccess) return cuda_error(e, "ea_cache_attention");
            ctas += a.tokens.ctas;
            launches++;
        }
        PgMerge m{{wc, wt}, {wc.cut ? a.chunks.ctas - 1 : 0, wt.cut ? a.tokens.ctas - 1 : 0},
                  {a.chunks.rows, a.tokens.rows},
                  {(int32_t)std::min<int64_t>(a.chunks.rows, (int64_t)p.t.max_new * p.group), a.tokens.rows}};
        if (m.cuts[0] + m.cuts[1] > 0) {
            e = launch_cache_merge(p, m, (cudaStream_t)stream);
            if (e != cudaSuccess) return cuda_error(e, "ea_cache_attention");
            ctas += m.cuts[0] + m.cuts[1];
            launches++;
        }
        note_launch(kCacheAttention, launches, ctas);
        return EA_OK;
    });
}

extern "C" ea_status ea_cache_attention_split(const ea_page_batch *batch, int32_t page, int64_t rows, const int32_t *split,
                                              int32_t ctas, int64_t capacity, int64_t *parts, int64_t *n_parts) {
    return entry([&]() -> ea_status {
        if (!split || !parts || !n_parts || ctas < 1 || page < 1 || capacity < 0 || rows < 0)
            return set_error(EA_ERR_ARG, "ea_cache_attention_split: arguments");
        ea_status s = batch_args(batch, page, rows);
        if (s) return s;
        const PgTable t = table_of(batch, page, rows);
        const PgSplit sp{split[0], split[1], split[2], split[3], split[4], split[5], split[6], 0};
        if (sp.heads < 1 || sp.group < 1 || sp.tok < 1 || sp.kt < 1 || ctas > 65535) return set_error(EA_ERR_ARG, "ea_cache_attention_split: split");
        std::vector<PgSeq> seqs(t.n_seqs);
        std::vector<int64_t> first(t.n_seqs + 1, 0);
        for (int i = 0; i < t.n_seqs; i++) {
            pg_seq(t.starts[i], t.starts[i + 1], t.lens[i], rows, t.max_new, (int64_t)t.max_pages * page, &seqs[i]);
            first[i + 1] = first[i] + pg_seq_units(seqs[i], sp);
        }
        struct {
            const std::vector<PgSeq> &v;
            PgSeq operator()(int i) const { return v[i]; }
            int count() const { return (int)v.size(); }
        } get{seqs};
        PgShare sh{};
        sh.total = first[t.n_seqs];
        sh.parts = pg_parts(sh.total, ctas);
        *n_parts = 0;
        for (int x = 0; x < sh.parts; x++) {
            sh.w0 = pg_first(sh.total, sh.parts, x);
            sh.count = pg_first(sh.total, sh.parts, x + 1) - sh.w0;
            sh.seq = (int32_t)(std::upper_bound(first.begin(), first.end(), sh.w0) - first.begin()) - 1;
            sh.off = sh.w0 - first[sh.seq];
            sh.s = seqs[sh.seq];
            PgWalk w;
            for (w.begin(sh, sp); w.left > 0; w.step(w.part(), sp, get)) {
                if (*n_parts == capacity) return set_error(EA_ERR_ARG, "ea_cache_attention_split: capacity");
                const int64_t row[7] = {x, w.seq, w.head, w.item, w.u0, w.u0 + w.part(), w.units};
                std::copy(row, row + 7, parts + 7 * (*n_parts)++);
            }
        }
        return EA_OK;
    });
}

extern "C" ea_status ea_cache_check_batch(int64_t pages, int32_t page, const ea_page_batch *batch, int64_t rows, int write) {
    return entry([&]() -> ea_status {
        if (page < 1 || pages < 1 || rows < 0) return set_error(EA_ERR_ARG, "ea_cache_check_batch: pages, page or rows");
        ea_status s = batch_args(batch, page, rows);
        if (s) return s;
        const PgTable t = table_of(batch, page, rows);
        std::unordered_set<int64_t> slots;
        for (int i = 0; i < t.n_seqs; i++) {
            PgSeq q;
            if (!pg_seq(t.starts[i], t.starts[i + 1], t.lens[i], rows, t.max_new, (int64_t)t.max_pages * page, &q))
                return set_error(EA_ERR_BOUNDS, "sequence %d: rows %d to %d of %lld, %d positions of at most %lld", i,
                                 t.starts[i], t.starts[i + 1], (long long)rows, t.lens[i], (long long)t.max_pages * page);
            if (write && q.n > q.len)
                return set_error(EA_ERR_BOUNDS, "sequence %d: %d rows in %d positions", i, q.n, q.len);
            const int64_t from = write ? q.len - q.n : 0;
            for (int64_t x = from / page; q.n > 0 && x * page < q.len; x++) {
                const int32_t pg = t.pages[i * t.page_stride + x];
                if (pg < 0 || pg >= pages)
                    return set_error(EA_ERR_BOUNDS, "sequence %d: its page %lld is number %d of %lld", i, (long long)x, pg,
                                     (long long)pages);
            }
            for (int64_t p = from; write && q.n > 0 && p < q.len; p++) {
                const int64_t slot = (int64_t)t.pages[i * t.page_stride + p / page] * page + p % page;
                if (!slots.insert(slot).second)
                    return set_error(EA_ERR_BOUNDS, "sequence %d: position %lld shares its slot with another row", i, (long long)p);
            }
        }
        return EA_OK;
    });
}
