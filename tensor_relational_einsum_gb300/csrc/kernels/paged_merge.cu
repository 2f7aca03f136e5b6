// paged_merge.cu -- the partial results of items that were cut between CTAs.
//
// A part holds, per row, the maximum m of its scores, l = SUM e^(scale (s - m))
// and A = SUM e^(scale (s - m)) V.  The parts of an item are merged in the
// order of its positions with
//   M = max m_i,  w_i = e^(scale (m_i - M)),  O = (SUM w_i A_i) / (SUM w_i l_i),
// so the result does not depend on which CTA was done first.  A warp takes a
// row; lanes take D / 32 neighbouring columns.  Bound by the latency of one
// read of the partial results, which are in L2.
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kRowsPerCta = 4;

template <int D>
__global__ void __launch_bounds__(32 * kRowsPerCta)
cache_merge_kernel(const __grid_constant__ PgAttn p, const __grid_constant__ PgSplit sp, const __grid_constant__ PgWork w,
                   int rows) {
    constexpr int C = D / 32;
    const int x = blockIdx.x + 1;
    const PgCut c = w.cut[x];
    if (c.we == 0 || pg_first(c.total, c.parts, x - 1) > c.wi) return;  // not cut here, or merged by an earlier cut
    const PgSeq s = load_seq(p.t, c.seq, p.c.page_log2, p.err);
    const int first = c.item * sp.tok;  // the item's tokens and rows
    const int n = min(sp.tok, s.n - first) * sp.group;
    const int row = blockIdx.y * kRowsPerCta + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (row >= n) return;
    // parts: the last of CTA x - 1 (its only one if the item begins with it), then the first of x, x + 1, ...
    const int slot0 = 2 * (x - 1) + (pg_first(c.total, c.parts, x - 1) < c.wi ? 1 : 0);
    int count = 1;
    while (x - 1 + count < c.parts && pg_first(c.total, c.parts, x - 1 + count) < c.we) count++;
    auto slot = [&](int i) { return i == 0 ? slot0 : 2 * (x - 1 + i); };
    float m = -INFINITY;
    for (int i = lane; i < count; i += 32) m = fmaxf(m, __ldcg(&w.ml[(int64_t)slot(i) * rows + row]).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, a[C] = {};
#pragma unroll 4
    for (int i = 0; i < count; i++) {
        const int64_t at = (int64_t)slot(i) * rows + row;
        const float2 ml = __ldcg(&w.ml[at]);
        const float f = exp2f((ml.x - base) * p.scale_log2);
        float v[C];
        if constexpr (C == 4) {
            const float4 q = __ldcg(reinterpret_cast<const float4 *>(w.acc + at * D) + lane);
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
            const float2 q = __ldcg(reinterpret_cast<const float2 *>(w.acc + at * D) + lane);
            v[0] = q.x; v[1] = q.y;
        }
        l = fmaf(f, ml.y, l);
#pragma unroll
        for (int k = 0; k < C; k++) a[k] = fmaf(f, v[k], a[k]);
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
    const int64_t at = (int64_t)(s.first + first + row / sp.group) * p.qheads + c.head * sp.group + row % sp.group;
    __nv_bfloat162 *out = reinterpret_cast<__nv_bfloat162 *>(p.o + (at * D + lane * C) * 2);
#pragma unroll
    for (int k = 0; k < C / 2; k++) out[k] = __floats2bfloat162_rn(a[2 * k] * inv, a[2 * k + 1] * inv);
    if (p.m_out && lane == 0) {
        p.m_out[at] = m * p.scale;
        p.l_out[at] = l;
    }
}

}  // namespace

cudaError_t launch_cache_merge(const PgAttn &p, const PgPlan &pl, void *ws, cudaStream_t st) {
    if (pl.ctas < 2) return cudaSuccess;
    const PgWork w = pg_work(pl, p.c.dim, ws);
    const dim3 grid(pl.ctas - 1, (pl.rows + kRowsPerCta - 1) / kRowsPerCta);
    if (p.c.dim == 64) cache_merge_kernel<64><<<grid, 32 * kRowsPerCta, 0, st>>>(p, pl.split, w, pl.rows);
    else cache_merge_kernel<128><<<grid, 32 * kRowsPerCta, 0, st>>>(p, pl.split, w, pl.rows);
    return cudaGetLastError();
}

}  // namespace ea
