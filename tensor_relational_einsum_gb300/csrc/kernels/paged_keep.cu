// paged_keep.cu -- the accepted rows of a tree of drafted tokens move to the
// first of the sequence's new positions, in all layers' caches at once.
//
// Row path[j] of a sequence's new rows becomes row j.  path increases, so a
// position is read before or by the thread that writes it: a thread takes the
// same 16 bytes of every moved vector, in batches that it reads whole before
// it writes, and path[j] >= j keeps later reads clear of earlier writes.  The
// bytes are few; what takes the time is the chain of look-ups (bounds, path,
// page numbers) before the first vector's address is known, so all layers go
// into one launch, and several into a CTA where they are many.
//
// Measured: 16 sequences of one layer 3.1 us; 64 sequences of 32 layers, 8
// heads of 128, 8-bit cells, 14 MB: 7.2 us (9.5 us with a layer a CTA).
#include "../drafts.h"
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 256;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kThreads) cache_keep_kernel(const __grid_constant__ KpParams p) {
    __shared__ int64_t s_from[kPgNodes], s_to[kPgNodes];  // slots of head 0
    __shared__ int s_moves, s_bad;
    const int seq = blockIdx.x, lg = p.page_log2;
    const int cache0 = blockIdx.y * p.each, caches = min(p.each, p.n_caches - cache0);
    if (threadIdx.x == 0) s_moves = s_bad = 0;
    __syncthreads();
    const PgSeq s = load_seq(p.t, seq, p.err);
    const int count = __ldg(p.counts + seq), base = s.len - s.n;
    bool bad = base < 0 || count < 0 || count > s.n || count > p.width;
    if (bad && threadIdx.x == 0) s_bad = 1;
    const int j = threadIdx.x;
    int from = 0;
    if (!bad && j < count) {
        const int32_t *path = p.path + (int64_t)seq * p.width;
        from = __ldg(path + j);
        const int before = j ? __ldg(path + j - 1) : -1;
        bad = from <= before || from >= s.n;
        if (!bad) {
            const int32_t *pages = p.t.pages + (int64_t)seq * p.t.page_stride;
            const int a = base + from, b = base + j, mask = (1 << lg) - 1;
            const int32_t ga = __ldg(pages + (a >> lg)), gb = __ldg(pages + (b >> lg));
            bad = ga < 0 || ga >= p.n_pages || gb < 0 || gb >= p.n_pages;
            if (!bad) {
                s_from[j] = ((ga * (int64_t)p.heads) << lg) + (a & mask);
                s_to[j] = ((gb * (int64_t)p.heads) << lg) + (b & mask);
                if (from != j) atomicMax(&s_moves, j + 1);
            }
        }
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {
        if (threadIdx.x == 0) {
            batch_fail(p.err);
            if (p.lens_out && cache0 == 0) p.lens_out[seq] = s.len;
        }
        return;
    }
    if (p.lens_out && cache0 == 0 && threadIdx.x == 0) p.lens_out[seq] = base + count;
    const int moves = s_moves;
    if (moves == 0) return;
    // 16 bytes of every moved vector a thread: of a cache's K and V, head after head
    const int chunks = p.row_bytes / 16, cells = 2 * p.heads * chunks;
    for (int c = threadIdx.x; c < caches * cells; c += kThreads) {
        const int x = c / cells, y = c - x * cells, w = y >= cells / 2, hc = w ? y - cells / 2 : y, head = hc / chunks;
        char *pool = w ? p.v[cache0 + x] : p.k[cache0 + x];
        const int64_t off = ((int64_t)head << lg) * p.row_bytes + (hc - head * chunks) * 16;
        for (int j0 = 0; j0 < moves; j0 += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (j0 + i < moves) v[i] = *reinterpret_cast<const uint4 *>(pool + s_from[j0 + i] * p.row_bytes + off);
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (j0 + i < moves && s_from[j0 + i] != s_to[j0 + i])
                    *reinterpret_cast<uint4 *>(pool + s_to[j0 + i] * p.row_bytes + off) = v[i];
        }
    }
    if (!p.ks[0]) return;
    for (int c = threadIdx.x; c < caches * 2 * p.heads; c += kThreads) {
        const int x = c / (2 * p.heads), y = c - x * 2 * p.heads, w = y >= p.heads, head = w ? y - p.heads : y;
        uint8_t *pool = (w ? p.vs[cache0 + x] : p.ks[cache0 + x]) + ((int64_t)head << lg);
        for (int j0 = 0; j0 < moves; j0 += kBatch) {
            uint8_t v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (j0 + i < moves) v[i] = pool[s_from[j0 + i]];
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (j0 + i < moves) pool[s_to[j0 + i]] = v[i];
        }
    }
}

}  // namespace

cudaError_t launch_cache_keep(const KpParams &params, int num_sms, int64_t *ctas, cudaStream_t st) {
    KpParams p = params;
    // one look-up of the positions for several caches, as soon as the CTAs would not all be resident (8 on an SM)
    p.each = 1;
    while (p.each < p.n_caches && (int64_t)p.t.n_seqs * ((p.n_caches + p.each - 1) / p.each) > 8 * num_sms) p.each++;
    const dim3 grid((unsigned)p.t.n_seqs, (unsigned)((p.n_caches + p.each - 1) / p.each));
    *ctas = (int64_t)grid.x * grid.y;
    cache_keep_kernel<<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace ea
