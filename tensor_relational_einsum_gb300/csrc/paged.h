// paged.h -- the paged cache: parameters of its kernels and the index
// arithmetic they share with the host (batch checks, the work list of the
// attention).  Internal.
//
// Attention's work list is made on the device, because the batch lives
// there.  A sequence's query rows (n tokens x g heads of one key-value head,
// token-major) are cut into items of `tok` tokens; an item takes ceil(e / kt)
// units of kt keys, e the keys that its last token keeps (at least one unit,
// so that an item without keys is still written).  Units are numbered
// sequence by sequence, key-value head by key-value head, item by item, and
// CTA x of G takes the units [x W / G, (x + 1) W / G): every CTA has the same
// number of units to within one, however ragged the batch is.  An item whose
// units fall into several CTAs is merged from their partial results.
#pragma once

#include "host.h"

#ifdef __CUDACC__
#define EA_HD __host__ __device__ __forceinline__
#else
#define EA_HD inline
#endif

struct ea_cache_s {
    int format = 0;
    int64_t n_pages = 0;
    int32_t page = 0, page_log2 = 0, heads = 0, dim = 0;
    char *k = nullptr, *v = nullptr;
    uint8_t *ks = nullptr, *vs = nullptr;
    int device = -1;
};

namespace ea {

struct PgPool {
    char *k, *v;         // [pages][heads][page][dim] cells
    uint8_t *ks, *vs;    // [pages][heads][page] scale bytes (e4m3)
    int64_t n_pages;
    int32_t page_log2, heads, dim, fmt;
};

struct PgTable {
    const int32_t *pages, *starts, *lens;
    int64_t page_stride;
    int64_t rows;        // dense rows
    int32_t n_seqs, max_pages, max_new;
};

struct PgRows {          // append and read
    PgTable t;
    PgPool c;
    char *k, *v;         // dense rows [rows][heads][dim]
    int32_t f32;         // dense dtype: 1 fp32, 0 bf16
    int32_t read;        // 0 append, 1 read
    int *err;
};
cudaError_t launch_cache_rows(const PgRows &p, int64_t *ctas, cudaStream_t st);

struct PgAttn {
    PgTable t;
    PgPool c;
    const char *q;       // [rows][qheads][dim] bf16
    char *o;
    float *m_out, *l_out;
    int32_t qheads, group, causal;
    float scale, scale_log2;  // scale * log2(e)
    int *err;
};
cudaError_t launch_cache_attention(const PgAttn &p, int64_t *ctas, cudaStream_t st);

// ------------------------------------------------------------- sequences

struct PgSeq {
    int32_t first, n, len;  // first dense row, rows, positions
};

// Sequence i from its three numbers; false if they are out of range.
EA_HD bool pg_seq(int32_t a, int32_t b, int32_t len, int64_t rows, int32_t max_new, int64_t cap, PgSeq *s) {
    s->first = a;
    s->n = 0;
    s->len = 0;
    if (a < 0 || b < a || b > rows || b - a > max_new || len < 0 || len > cap) return false;
    s->n = b - a;
    s->len = len;
    return true;
}

// Element offset of a vector (page, head, slot) / dim in the pool.
EA_HD int64_t pg_vec(const PgPool &c, int64_t page, int head, int slot) {
    return ((page * c.heads + head) << c.page_log2) + slot;
}

}  // namespace ea
