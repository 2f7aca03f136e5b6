// paged_merge.cu -- the partial results of items that were cut between CTAs.
//
// A part holds, per row, the maximum m of its scores, l = SUM e^(scale (s - m))
// and A = SUM e^(scale (s - m)) V.  The parts of an item are merged in the
// order of its positions with
//   M = max m_i,  w_i = e^(scale (m_i - M)),  O = (SUM w_i A_i) / (SUM w_i l_i),
// so the result does not depend on which CTA was done first.  Bound by the
// latency of reading the partial results, which are in L2, so all that a row
// needs is asked for together: with few parts a warp takes two rows, with many
// one row and eight parts at a time, and rows that leave warps idle are shared.
#include <algorithm>

#include "attn_common.cuh"
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kWarps = 8;
constexpr int kRowsPerCta = 32;  // a CTA without a cut costs too: not too many of them

template <int D>
__device__ __forceinline__ void load_acc(const float *src, int lane, float *v) {
    if constexpr (D == 128) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(src) + lane);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        const float2 q = __ldcg(reinterpret_cast<const float2 *>(src) + lane);
        v[0] = q.x; v[1] = q.y;
    }
}

template <int D>
__device__ __forceinline__ void finish(const PgAttn &p, const PgCut &c, int row, int lane, float m, float l, const float *a) {
    constexpr int C = D / 32;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
    const int64_t at = (int64_t)(c.row0 + row / p.group) * p.qheads + c.head * p.group + row % p.group;
    uint32_t w[C / 2];
#pragma unroll
    for (int k = 0; k < C / 2; k++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a[2 * k] * inv, a[2 * k + 1] * inv);
        w[k] = *reinterpret_cast<const uint32_t *>(&h);
    }
    char *out = p.o + (at * D + lane * C) * 2;
    if constexpr (C == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(out) = w[0];
    if (p.m_out && lane == 0) {
        p.m_out[at] = m * p.scale;
        p.l_out[at] = l;
    }
}

// An item of N parts: a warp two rows at a time, all parts at once.  The first
// row of part 0 is n0, that of part i n1 + (i - 1) step.
template <int D, int N>
__device__ __forceinline__ void merge_few(const PgAttn &p, const PgWork &w, const PgCut &c, int64_t n0, int64_t n1, int64_t step,
                                          int row, int r1, int lane) {
    constexpr int C = D / 32;
    const float2 *ml_at[N];
    const float *acc_at[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int64_t n = i == 0 ? n0 : n1 + (i - 1) * step;
        ml_at[i] = w.ml + n;
        acc_at[i] = w.acc + n * D;
    }
    for (; row < r1; row += 2 * kWarps) {
        float2 ml[2][N];
        float v[2][N][C];
#pragma unroll
        for (int y = 0; y < 2; y++) {
            const int r = min(row + y, r1 - 1);  // a single last row twice: its second result is not stored
#pragma unroll
            for (int i = 0; i < N; i++) {
                ml[y][i] = __ldcg(ml_at[i] + r);
                load_acc<D>(acc_at[i] + r * D, lane, v[y][i]);
            }
        }
#pragma unroll
        for (int y = 0; y < 2; y++) {
            float m = ml[y][0].x;
#pragma unroll
            for (int i = 1; i < N; i++) m = fmaxf(m, ml[y][i].x);
            const float base = m == -INFINITY ? 0.f : m;
            float l = 0.f, a[C] = {};
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float f = attn::ex2((ml[y][i].x - base) * p.scale_log2);
                l = fmaf(f, ml[y][i].y, l);
#pragma unroll
                for (int k = 0; k < C; k++) a[k] = fmaf(f, v[y][i][k], a[k]);
            }
            if (row + y < r1) finish<D>(p, c, row + y, lane, m, l, a);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 4)
cache_merge_kernel(const __grid_constant__ PgAttn p, const __grid_constant__ PgMerge mg) {
    constexpr int C = D / 32;
    __shared__ float s_l[kWarps], s_a[kWarps][D];
    // the cuts of the first kernel by groups of rows, then those of the second
    int at_cut = blockIdx.x, k = 0;
    if (at_cut >= mg.cuts[0] * mg.groups[0]) {
        at_cut -= mg.cuts[0] * mg.groups[0];
        k = 1;
    }
    const int x = at_cut / mg.groups[k] + 1, group = at_cut % mg.groups[k];
    const PgWork &w = mg.w[k];
    const int rows = mg.rows[k];
    wait_for_previous();
    const PgCut c = w.cut[x];
    if (c.we == 0 || pg_first(c.total, c.parts, x - 1) > c.wi) return;  // not cut here, or merged by an earlier cut
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int r0 = group * kRowsPerCta, r1 = min(c.rows, r0 + kRowsPerCta);
    if (r0 >= r1) return;
    // parts: the last of CTA x - 1 (its only one if the item begins with it), then the first of x, x + 1, ...
    const int slot0 = 2 * (x - 1) + (pg_first(c.total, c.parts, x - 1) < c.wi ? 1 : 0);
    const int count = pg_before(c.total, c.parts, c.we) - (x - 1);
    auto at = [&](int i, int row) { return (int64_t)(i == 0 ? slot0 : 2 * (x - 1 + i)) * rows + row; };

    if (count <= 4) {
        const int64_t n0 = (int64_t)slot0 * rows, n1 = (int64_t)2 * x * rows, step = (int64_t)2 * rows;
        if (count == 2) merge_few<D, 2>(p, w, c, n0, n1, step, r0 + 2 * warp, r1, lane);
        else if (count == 3) merge_few<D, 3>(p, w, c, n0, n1, step, r0 + 2 * warp, r1, lane);
        else merge_few<D, 4>(p, w, c, n0, n1, step, r0 + 2 * warp, r1, lane);
        return;
    }
    // many parts, eight at a time; with few rows several warps share a row's parts
    const int left = r1 - r0, share = left <= 1 ? 8 : left <= 2 ? 4 : left <= 4 ? 2 : 1, sub = warp % share;
    for (int row0 = r0; row0 < r1; row0 += kWarps / share) {
        const int row = row0 + warp / share;
        const bool in = row < r1;
        float m = -INFINITY;
        for (int i = lane; in && i < count; i += 32) m = fmaxf(m, __ldcg(&w.ml[at(i, row)]).x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, a[C] = {};
        for (int i0 = sub; in && i0 < count; i0 += 8 * share) {
            float2 ml[8];
            float v[8][C];
#pragma unroll
            for (int y = 0; y < 8; y++) {
                const int i = i0 + y * share;
                ml[y] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < C; k++) v[y][k] = 0.f;
                if (i < count) {
                    ml[y] = __ldcg(&w.ml[at(i, row)]);
                    load_acc<D>(w.acc + at(i, row) * D, lane, v[y]);
                }
            }
#pragma unroll
            for (int y = 0; y < 8; y++) {
                const float f = attn::ex2((ml[y].x - base) * p.scale_log2);
                l = fmaf(f, ml[y].y, l);
#pragma unroll
                for (int k = 0; k < C; k++) a[k] = fmaf(f, v[y][k], a[k]);
            }
        }
        if (share > 1) {  // the same order every time: sub 0, 1, ..
            s_l[warp] = l;
#pragma unroll
            for (int k = 0; k < C; k++) s_a[warp][lane * C + k] = a[k];
            __syncthreads();
            for (int i = 1; sub == 0 && i < share; i++) {
                l += s_l[warp + i];
#pragma unroll
                for (int k = 0; k < C; k++) a[k] += s_a[warp + i][lane * C + k];
            }
        }
        if (in && sub == 0) finish<D>(p, c, row, lane, m, l, a);
        if (share > 1) __syncthreads();
    }
}

}  // namespace

cudaError_t launch_cache_merge(const PgAttn &p, const PgMerge &m, cudaStream_t st) {
    PgMerge g = m;
    for (int k = 0; k < 2; k++) g.groups[k] = std::max(1, (m.rows[k] + kRowsPerCta - 1) / kRowsPerCta);
    const dim3 grid(g.cuts[0] * g.groups[0] + g.cuts[1] * g.groups[1]);
    if (p.c.dim == 64) return launch_after(cache_merge_kernel<64>, grid, 32 * kWarps, 0, st, true, p, g);
    return launch_after(cache_merge_kernel<128>, grid, 32 * kWarps, 0, st, true, p, g);
}

}  // namespace ea
