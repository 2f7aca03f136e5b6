// paged_host.h -- checks that the entry points over batches of sequences
// share: dense rows, the batch's arguments, overlaps, the device.  Internal.
#pragma once

#include <exception>
#include <initializer_list>

#include "paged.h"
#include "plan.h"

namespace ea {

// Rows, heads and head dim of a dense relation [.., heads, dim] whose arena
// is its rows in row-major order: heads and dim whole, and outside them no
// dimension cut into blocks behind one whose blocks hold several indexes.
inline ea_status dense_rows(const ea_relation_s *r, const char *what, int trailing, int64_t *rows, int64_t *heads, int64_t *dim) {
    if (r->rank < trailing + 1) return set_error(EA_ERR_SHAPE, "%s needs rank >= %d", what, trailing + 1);
    bool wide = false;  // a dimension to the left has blocks of several indexes
    *rows = 1;
    for (int d = 0; d < r->rank; d++) {
        const std::vector<int64_t> &b = r->bounds[d];
        const bool whole = b.size() == 2;
        if (d >= r->rank - trailing ? !whole : (wide && !whole))
            return set_error(EA_ERR_PARTITION, "%s: the blocks do not hold its rows in order; re-block with ea_exchange", what);
        for (size_t i = 0; i + 1 < b.size(); i++) wide |= b[i + 1] - b[i] > 1;
        if (d < r->rank - trailing) *rows *= r->dims[d];
    }
    *heads = r->dims[r->rank - trailing];
    if (dim) *dim = r->dims[r->rank - 1];
    return EA_OK;
}

// Some of the arrays is off a boundary of its 4-byte elements, which a kernel's access would fault on.
inline bool off_4(std::initializer_list<const void *> arrays) {
    for (const void *p : arrays)
        if (((uintptr_t)p & 3) != 0) return true;
    return false;
}

inline ea_status batch_args(const ea_page_batch *b, int32_t page, int64_t rows) {
    if (!b || !b->pages || !b->starts || !b->lens) return set_error(EA_ERR_ARG, "cache: NULL batch or batch array");
    if (off_4({b->pages, b->starts, b->lens})) return set_error(EA_ERR_ARG, "cache: the batch's arrays must be aligned to 4 bytes");
    if (b->n_seqs < 1 || b->n_seqs > 65536) return set_error(EA_ERR_ARG, "cache: n_seqs %d out of [1, 65536]", b->n_seqs);
    if (b->max_pages < 1 || b->page_stride < b->max_pages)
        return set_error(EA_ERR_ARG, "cache: max_pages %d, page_stride %lld", b->max_pages, (long long)b->page_stride);
    // The kernels step over an end by a tile, or a warp's pages of a tile, in 32 bits.
    constexpr int64_t most = INT32_MAX - 8191;
    if ((int64_t)b->max_pages * page > most) return set_error(EA_ERR_UNSUPPORTED, "cache: a sequence of more than %lld positions", (long long)most);
    if (b->max_new < 0) return set_error(EA_ERR_ARG, "cache: max_new %d", b->max_new);
    if (rows > most) return set_error(EA_ERR_UNSUPPORTED, "cache: more than %lld rows", (long long)most);
    return EA_OK;
}

// The parents of a batch's rows (device array of `rows` entries).
inline ea_status tree_args(const char *what, const ea_page_batch *b, const int32_t *parents, int64_t rows) {
    if (off_4({parents})) return set_error(EA_ERR_ARG, "%s: parents must be aligned to 4 bytes", what);
    const int64_t most = b->max_new > 0 && b->max_new < rows ? b->max_new : rows;
    if (most > kPgNodes)
        return set_error(EA_ERR_UNSUPPORTED, "%s: trees of up to %lld nodes (%d at most; give max_new)", what, (long long)most, kPgNodes);
    return EA_OK;
}

inline PgTable table_of(const ea_page_batch *b, int32_t page, int64_t rows) {
    PgTable t{};
    t.cap = (int64_t)b->max_pages * page;
    t.pages = b->pages;
    t.starts = b->starts;
    t.lens = b->lens;
    t.page_stride = b->page_stride;
    t.rows = rows;
    t.n_seqs = b->n_seqs;
    t.max_pages = b->max_pages;
    t.max_new = (int32_t)(b->max_new > 0 && b->max_new < rows ? b->max_new : rows);
    return t;
}

inline PgPool pool_of(const ea_cache_s *c) {
    return PgPool{c->k, c->v, c->ks, c->vs, c->n_pages, c->page_log2, c->heads, c->dim, c->format};
}

inline size_t cache_bytes(const ea_cache_s *c) {
    return (size_t)c->n_pages * c->heads * c->page * c->dim * (c->format == EA_CACHE_BF16 ? 2 : 1);
}

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    return a && b && na && nb && (const char *)a < (const char *)b + nb && (const char *)b < (const char *)a + na;
}

inline bool in_cache(const ea_cache_s *c, const void *p, size_t bytes) {
    const size_t n = cache_bytes(c), ns = (size_t)c->n_pages * c->heads * c->page;
    return overlap(c->k, n, p, bytes) || overlap(c->v, n, p, bytes) || overlap(c->ks, c->ks ? ns : 0, p, bytes) ||
           overlap(c->vs, c->vs ? ns : 0, p, bytes);
}

inline bool in_cache(const ea_cache_s *c, const ea_relation_s *r) { return in_cache(c, r->arena, r->bytes); }

// The batch's arrays share bytes with [p, p + bytes).
inline bool in_batch(const ea_page_batch *b, const void *p, size_t bytes) {
    const size_t n = b->n_seqs;
    return overlap(b->pages, ((n - 1) * b->page_stride + b->max_pages) * 4, p, bytes) || overlap(b->starts, (n + 1) * 4, p, bytes) ||
           overlap(b->lens, n * 4, p, bytes);
}

inline bool in_batch(const ea_page_batch *b, const ea_cache_s *c) {
    const size_t n = cache_bytes(c), ns = (size_t)c->n_pages * c->heads * c->page;
    return in_batch(b, c->k, n) || in_batch(b, c->v, n) || in_batch(b, c->ks, c->ks ? ns : 0) || in_batch(b, c->vs, c->vs ? ns : 0);
}

inline ea_status here(const ea_cache_s *c, DevCtx **ctx) {
    ea_status s = get_ctx(ctx);
    if (s) return s;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    if (dev != c->device)
        return set_error(EA_ERR_ARG, "cache: it lives on device %d, the current device is %d", c->device, dev);
    return EA_OK;
}

inline void note_launch(int kind, int launches, int64_t ctas) {
    t_last = LastPlan{};
    t_last.kind = kind;
    t_last.launches = launches;
    t_last.tiles = ctas;
}

// No exception leaves a C entry.
template <class F>
ea_status entry(F body) {
    set_error(EA_OK, "");
    try {
        return body();
    } catch (const std::bad_alloc &) {
        return set_error(EA_ERR_ALLOC, "out of host memory");
    } catch (const std::exception &e) {
        return set_error(EA_ERR_ARG, "unexpected exception: %s", e.what());
    }
}

}  // namespace ea
