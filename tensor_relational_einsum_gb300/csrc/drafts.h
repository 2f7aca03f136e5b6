// drafts.h -- parameters of the kernels around drafted tokens: rotary
// positions, verification, keeping the accepted rows.  Internal.
#pragma once

#include "paged.h"

namespace ea {

constexpr int kRoPairs = 128;  // the most pairs of a rotation

struct RoParams {
    const char *x[2];          // q and k: [rows][heads][dim]; k NULL: q alone
    char *y[2];                // results; the same arrays: in place
    int32_t heads[2];
    int32_t dim, dims, offset; // columns of a head; the rotated ones, from `offset` on
    int32_t half;              // pairs (i, i + dims / 2), else (2 i, 2 i + 1)
    int32_t f32;
    int32_t n_seqs, max_new;
    int64_t rows;
    const int32_t *starts, *lens;  // the batch; NULL: positions
    const int32_t *positions;      // [rows]
    const int32_t *parents;        // [rows] or NULL
    float amplitude, sign;         // of cosine and sine; the sine's sign
    int *err;
    uint64_t turn[kRoPairs];   // turns a position, in units of 2^-64
};
cudaError_t launch_rotary(const RoParams &p, int num_sms, int64_t *ctas, cudaStream_t st);

struct VfParams {
    const char *target, *draft;    // [rows][vocab]; draft NULL: tokens that are certain
    const int32_t *tokens, *parents;
    const int32_t *starts;
    const float *accept, *sample;
    int32_t *path, *counts, *picked;
    int64_t rows, vocab;
    int32_t n_seqs, max_new, width; // width: entries of a row of path
    int32_t bf16;
    int *err;
};
cudaError_t launch_verify(const VfParams &p, int num_sms, int64_t *ctas, cudaStream_t st);

constexpr int kKeepCaches = 64;    // caches of one launch
struct KpParams {
    PgTable t;
    int64_t n_pages;
    int32_t page_log2, heads, row_bytes;  // row_bytes: of a vector's cells
    int32_t n_caches, width, each;        // each: caches of a CTA (set by the launch)
    const int32_t *path, *counts;
    int32_t *lens_out;
    int *err;
    char *k[kKeepCaches], *v[kKeepCaches];
    uint8_t *ks[kKeepCaches], *vs[kKeepCaches];
};
cudaError_t launch_cache_keep(const KpParams &p, int num_sms, int64_t *ctas, cudaStream_t st);

}  // namespace ea
