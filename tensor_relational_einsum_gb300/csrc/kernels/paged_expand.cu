// paged_expand.cu -- 8-bit pages of the sequences that the chunk kernel serves
// as bf16 vectors [sequence][128 positions][head][position][dim] in the call's
// workspace, for chunks whose keys are read by many row tiles.
//
// The chunk kernel can rewrite 8-bit tiles itself, but does so once for every
// 256 rows, next to products that take all of shared memory's bandwidth: a
// tile then takes 6000 cycles instead of 3080.  Writing 2 bytes and reading
// them from L2 once for 256 rows is cheaper from about that many rows on
// (2048 tokens after 14336, 32 heads over 8: 610 us there, 412 us with this
// kernel).  Below, the 3 bytes more a cell cost more than the rewriting: 8
// sequences of 8192, 8 heads, 48 / 128 / 240 rows: 118 / 118 / 126 us there,
// 151 / 157 / 166 us expanded; at head dim 64 69 / 71 / 80 against 93 / 96 /
// 106 us.
// Every cell is a bf16 value (but for bits below 2^-133, under scale bytes of
// less than 3), so nothing is lost.  Bound by HBM and L2: one
// byte read and two written a cell, 21 us for 31.6 million of them.
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads)
cache_expand_kernel(const __grid_constant__ PgAttn p, const __grid_constant__ PgSplit sp, char *wk, char *wv, int blocks,
                    int place_rows) {
    constexpr int CPR = D / 16, IT = 128 * CPR / kThreads;  // 16-code chunks of a vector; of a thread and tensor
    let_next_start();
    const int head = blockIdx.x % p.c.heads, at = blockIdx.x / p.c.heads, x = at % blocks, place = at / blocks;
    int i = place;
    if (place_rows > 0) {
        // The last sequence whose first row lies before the next place's.  One that is served has place_rows rows or
        // more, so those behind it start at or beyond the next place.
        const int64_t next = (int64_t)(place + 1) * place_rows;
        int b = p.t.n_seqs - 1;
        for (i = 0; i < b;) {
            const int mid = (i + b + 1) >> 1;
            if (__ldg(p.t.starts + mid) < next) i = mid;
            else b = mid - 1;
        }
    }
    const PgSeq s = load_seq(p.t, i, p.err);
    if (place_rows > 0 && s.first / place_rows != place) return;
    const int key0 = x * 128, lg = p.c.page_log2;
    if (!pg_served(s, sp) || key0 >= s.len) return;
    const int64_t out0 = ((int64_t)at * p.c.heads + head) * 128;  // first vector of the block in the workspace
#pragma unroll 4
    for (int it = 0; it < IT; it++) {
        const int id = it * kThreads + threadIdx.x, r = id / CPR, ch = id % CPR, key = key0 + r;
        if (key >= s.len) break;
        const int32_t g = check_page(__ldg(p.t.pages + (int64_t)i * p.t.page_stride + (key >> lg)), p.c.n_pages, p.err);
        const int64_t vec = pg_vec(p.c, g, head, key & ((1 << lg) - 1));
        const uint4 cells[2] = {__ldg(reinterpret_cast<const uint4 *>(p.c.k + vec * D) + ch),
                                __ldg(reinterpret_cast<const uint4 *>(p.c.v + vec * D) + ch)};
        const float scale[2] = {scale_value(__ldg(p.c.ks + vec)), scale_value(__ldg(p.c.vs + vec))};
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const uint32_t u[4] = {cells[w].x, cells[w].y, cells[w].z, cells[w].w};
            uint32_t o[8];
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[q >> 1] >> (16 * (q & 1))), __NV_E4M3));
                const float2 f = __half22float2(h);
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale[w], f.y * scale[w]);
                o[q] = *reinterpret_cast<const uint32_t *>(&b);
            }
            uint4 *dst = reinterpret_cast<uint4 *>((w ? wv : wk) + (out0 + r) * D * 2) + 2 * ch;
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace

cudaError_t launch_cache_expand(const PgAttn &p, const PgSplit &sp, const PgExpand &x, char *ws, cudaStream_t st) {
    const unsigned grid = (unsigned)((int64_t)x.places * x.blocks * p.c.heads);
    char *wv = ws + x.bytes / 2;
    if (p.c.dim == 64) cache_expand_kernel<64><<<grid, kThreads, 0, st>>>(p, sp, ws, wv, x.blocks, x.place_rows);
    else cache_expand_kernel<128><<<grid, kThreads, 0, st>>>(p, sp, ws, wv, x.blocks, x.place_rows);
    return cudaGetLastError();
}

}  // namespace ea
