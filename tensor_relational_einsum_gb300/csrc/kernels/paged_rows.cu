// paged_rows.cu -- append to and read from the paged cache.
//
// One vector (a row's head, 64 or 128 values) is taken by D / 8 lanes, 8
// values a lane: 16-byte loads and stores of bf16, two of them for fp32, 8
// bytes for e4m3 codes.  Both operators move bytes and nothing else: the
// bound is HBM, and for small calls the chain of dependent reads (sequence
// bounds, page number) before a vector's address is known.  So
//   - a CTA takes 16 rows of a few heads, and 16 of its threads look up where
//     the rows live: the sequences' bounds and lengths are staged in shared
//     memory (one round trip for all of them) and searched there, not in
//     global memory, where each of the log2(sequences) steps would wait for
//     the last;
//   - a thread takes the vectors of K and of V at the same place and asks
//     for everything that does not depend on the table first;
//   - the scale bytes of neighbouring positions, which lie next to each other,
//     are stored together (a byte at a time they were a fourth of all writes).
// Quantising: the vector's largest magnitude over its lanes by shuffles on
// the integer bits (an integer maximum orders magnitudes and puts infinities
// and NaN on top), one power-of-two scale, codes rounded once by the hardware
// conversion; the scaling itself is exact.
//
// Measured, 32768 rows of 16 heads of 128, of the measured copy rate: append
// 0.95 (bf16 to bf16, 83 us), 0.89 (to 8 bits, 67 us), 0.97 (fp32 to 8 bits,
// 102 us); read 0.94 (84 us), 0.90 (66 us), 0.93 (8 bits to fp32, 107 us).  A
// step's append takes 4.8 us.
#include <algorithm>

#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 256;
constexpr int kRowsCta = 16;   // rows of a CTA
constexpr int kCheckers = kThreads - 32;  // sequences that a CTA checks
constexpr int kStaged = 1024;  // sequence bounds staged in shared memory; longer batches are searched in global memory

// The sequence that holds dense row r (starts[i] <= r < starts[i + 1]), or -1.
__device__ __forceinline__ int find_seq(const int32_t *starts, int n_seqs, int32_t r) {
    if (r < starts[0] || r >= starts[n_seqs]) return -1;
    int a = 0, b = n_seqs - 1;  // the last i with starts[i] <= r
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (starts[mid] <= r) a = mid;
        else b = mid - 1;
    }
    return r < starts[a + 1] ? a : -1;
}

__device__ __forceinline__ void to_f32(const uint4 *raw, bool f32, float *x) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = __uint_as_float(reinterpret_cast<const uint32_t *>(raw)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(raw)[i];
            x[2 * i] = __uint_as_float(w << 16);
            x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint4 to_bf16(const float *x) {
    uint4 u;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    return u;
}

template <int D, bool F32, bool E4M3, bool READ, int U>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(const __grid_constant__ PgRows p) {
    constexpr int LPV = D / 8;                // lanes of a vector
    constexpr int VPB = kThreads / LPV;       // vectors of a pass
    constexpr int HEADS = U * VPB / kRowsCta; // heads of a CTA
    constexpr int RAW = F32 ? 2 : 1;          // 16-byte words of a lane's dense values
    __shared__ int32_t s_starts[kStaged + 1], s_lens[kStaged];
    __shared__ int64_t s_base[kRowsCta];      // slot of the row's vector of head 0; -1: none
    __shared__ uint8_t s_scale[2][HEADS][kRowsCta];
    const int n_seqs = p.t.n_seqs, heads = p.c.heads, lg = p.c.page_log2;
    const int row0 = blockIdx.x * kRowsCta, head0 = blockIdx.y * HEADS;
    const int lane_v = threadIdx.x % LPV;
    bool on[U];
    int64_t dense[U];                         // the lane's dense element
    uint4 kx[U][RAW], vx[U][RAW];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int v = u * VPB + threadIdx.x / LPV, row = row0 + v % kRowsCta, head = head0 + v / kRowsCta;
        on[u] = row < p.t.rows && head < heads;
        dense[u] = ((int64_t)row * heads + head) * D + lane_v * 8;
        if (!READ && on[u]) {
#pragma unroll
            for (int i = 0; i < RAW; i++) {
                kx[u][i] = __ldg(reinterpret_cast<const uint4 *>(p.k + dense[u] * (F32 ? 4 : 2)) + i);
                vx[u][i] = __ldg(reinterpret_cast<const uint4 *>(p.v + dense[u] * (F32 ? 4 : 2)) + i);
            }
        }
    }
    const bool staged = n_seqs <= kStaged;
    if (staged) {
        for (int i = threadIdx.x; i <= n_seqs; i += kThreads) {
            s_starts[i] = __ldg(p.t.starts + i);
            if (i < n_seqs) s_lens[i] = __ldg(p.t.lens + i);
        }
        __syncthreads();
    }
    if (threadIdx.x < kRowsCta) {
        const int32_t *starts = staged ? s_starts : p.t.starts;
        const int row = row0 + threadIdx.x;
        int64_t base = -1;
        const int i = row < p.t.rows ? find_seq(starts, n_seqs, row) : -1;
        if (i >= 0) {
            PgSeq s;
            const bool ok = pg_seq(starts[i], starts[i + 1], staged ? s_lens[i] : __ldg(p.t.lens + i), p.t.rows, p.t.max_new,
                                   p.t.cap, &s);
            const int pos = s.len - s.n + (row - s.first);
            const bool before = ok && READ && pos < 0;  // a row that no position belongs to: nothing to read
            if (ok && pos >= 0 && (READ || s.n <= s.len)) {
                const int32_t g = __ldg(p.t.pages + (int64_t)i * p.t.page_stride + (pos >> lg));
                if (g >= 0 && g < p.c.n_pages) base = pg_vec(p.c, g, 0, pos & ((1 << lg) - 1));
            }
            if (base < 0 && !before) batch_fail(p.err);
        }
        s_base[threadIdx.x] = base;
    }
    // A sequence out of range is reported whether or not a row led to it (idle ones, those beyond the rows, bounds that
    // decrease, which the search does not expect).  The warps that wait for the first one's look-up check one each.
    const int i = blockIdx.x * kCheckers + (int)threadIdx.x - 32;
    if (blockIdx.y == 0 && threadIdx.x >= 32 && i < n_seqs) {
        PgSeq s;
        const bool ok = staged ? pg_seq(s_starts[i], s_starts[i + 1], s_lens[i], p.t.rows, p.t.max_new, p.t.cap, &s)
                               : pg_seq(__ldg(p.t.starts + i), __ldg(p.t.starts + i + 1), __ldg(p.t.lens + i), p.t.rows,
                                        p.t.max_new, p.t.cap, &s);
        if (!ok || (!READ && s.n > s.len)) batch_fail(p.err);
    }
    __syncthreads();
    int64_t cell[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int v = u * VPB + threadIdx.x / LPV;
        const int64_t base = s_base[v % kRowsCta];
        cell[u] = on[u] && base >= 0 ? base + ((int64_t)(head0 + v / kRowsCta) << lg) : -1;
    }
    if constexpr (!READ) {
#pragma unroll
        for (int u = 0; u < U; u++) {
#pragma unroll
            for (int w = 0; w < 2; w++) {  // K, then V; the shuffles need every lane of the vector
                const uint4 *raw = w ? vx[u] : kx[u];
                char *pool = w ? p.c.v : p.c.k;
                if constexpr (!E4M3) {
                    uint4 out = raw[0];
                    if constexpr (F32) {
                        float x[8];
                        to_f32(raw, true, x);
                        out = to_bf16(x);
                    }
                    if (cell[u] >= 0) *reinterpret_cast<uint4 *>(pool + (cell[u] * D + lane_v * 8) * 2) = out;
                } else {
                    uint32_t amax = 0;  // bits of the largest magnitude, fp32
                    if constexpr (F32) {
#pragma unroll
                        for (int i = 0; i < 8; i++) amax = max(amax, reinterpret_cast<const uint32_t *>(raw)[i] & 0x7fffffffu);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            amax = __vmaxu2(amax, reinterpret_cast<const uint32_t *>(raw)[i] & 0x7fff7fffu);
                        amax = max(amax << 16, amax & 0xffff0000u);
                    }
#pragma unroll
                    for (int o = LPV / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    const uint32_t b = scale_byte(amax);
                    // 2^-(b - 127): normal for every b that scale_byte makes
                    const float inv = __uint_as_float((254u - b) << 23);
                    float x[8];
                    to_f32(raw, F32, x);
                    uint32_t code[2];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv),
                                                                    __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv),
                                                                    __NV_SATFINITE, __NV_E4M3);
                        code[i] = lo | (hi << 16);
                    }
                    if (b == 255u) code[0] = code[1] = 0u;  // NaN
                    if (cell[u] >= 0) *reinterpret_cast<uint2 *>(pool + cell[u] * D + lane_v * 8) = make_uint2(code[0], code[1]);
                    const int v = u * VPB + threadIdx.x / LPV;
                    if (lane_v == 0) s_scale[w][v / kRowsCta][v % kRowsCta] = (uint8_t)b;
                }
            }
        }
        if constexpr (E4M3) {
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * HEADS * kRowsCta; i += kThreads) {
                const int r = i % kRowsCta, h = i / kRowsCta % HEADS, w = i / (kRowsCta * HEADS);
                if (s_base[r] >= 0 && head0 + h < heads)
                    (w ? p.c.vs : p.c.ks)[s_base[r] + ((int64_t)(head0 + h) << lg)] = s_scale[w][h][r];
            }
        }
    } else {
        uint2 kc[U], vc[U];
        uint32_t kb[U], vb[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (cell[u] < 0) continue;
            if constexpr (E4M3) {
                kc[u] = __ldg(reinterpret_cast<const uint2 *>(p.c.k + cell[u] * D + lane_v * 8));
                vc[u] = __ldg(reinterpret_cast<const uint2 *>(p.c.v + cell[u] * D + lane_v * 8));
                kb[u] = __ldg(p.c.ks + cell[u]);
                vb[u] = __ldg(p.c.vs + cell[u]);
            } else {
                kx[u][0] = __ldg(reinterpret_cast<const uint4 *>(p.c.k + (cell[u] * D + lane_v * 8) * 2));
                vx[u][0] = __ldg(reinterpret_cast<const uint4 *>(p.c.v + (cell[u] * D + lane_v * 8) * 2));
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (cell[u] < 0) continue;
#pragma unroll
            for (int w = 0; w < 2; w++) {
                char *dst = (w ? p.v : p.k) + dense[u] * (F32 ? 4 : 2);
                float x[8];
                if constexpr (E4M3) {
                    const uint2 c = w ? vc[u] : kc[u];
                    const float sc = scale_value(w ? vb[u] : kb[u]);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const uint32_t two = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
                        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
                        const float2 f = __half22float2(h);
                        x[2 * i] = f.x * sc;
                        x[2 * i + 1] = f.y * sc;
                    }
                } else {
                    to_f32(w ? vx[u] : kx[u], false, x);
                }
                if constexpr (F32) {
                    st_32(dst, reinterpret_cast<const uint32_t *>(x));
                } else if constexpr (E4M3) {
                    *reinterpret_cast<uint4 *>(dst) = to_bf16(x);
                } else {
                    *reinterpret_cast<uint4 *>(dst) = w ? vx[u][0] : kx[u][0];
                }
            }
        }
    }
}

template <int D, bool F32, bool E4M3, int U>
cudaError_t launch_u(const PgRows &p, int64_t *ctas, cudaStream_t st) {
    constexpr int hc = U * kThreads / (D / 8) / kRowsCta;
    const int64_t by_rows = (p.t.rows + kRowsCta - 1) / kRowsCta, by_seqs = (p.t.n_seqs + kCheckers - 1) / kCheckers;
    const dim3 grid((unsigned)std::max(by_rows, by_seqs), (unsigned)((p.c.heads + hc - 1) / hc));
    *ctas = (int64_t)grid.x * grid.y;
    if (p.read) cache_rows_kernel<D, F32, E4M3, true, U><<<grid, kThreads, 0, st>>>(p);
    else cache_rows_kernel<D, F32, E4M3, false, U><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int D, bool F32, bool E4M3>
cudaError_t launch(const PgRows &p, int64_t *ctas, cudaStream_t st) {
    // two vectors a thread once they make 8 CTAs for each of some 150 SMs
    const int64_t threads = p.t.rows * p.c.heads * (D / 8);
    return threads >= (int64_t)2 * 8 * 150 * kThreads ? launch_u<D, F32, E4M3, 2>(p, ctas, st) : launch_u<D, F32, E4M3, 1>(p, ctas, st);
}

}  // namespace

cudaError_t launch_cache_rows(const PgRows &p, int64_t *ctas, cudaStream_t st) {
    const bool e4m3 = p.c.fmt == EA_CACHE_E4M3;
    if (p.c.dim == 64) {
        if (p.f32) return e4m3 ? launch<64, true, true>(p, ctas, st) : launch<64, true, false>(p, ctas, st);
        return e4m3 ? launch<64, false, true>(p, ctas, st) : launch<64, false, false>(p, ctas, st);
    }
    if (p.f32) return e4m3 ? launch<128, true, true>(p, ctas, st) : launch<128, true, false>(p, ctas, st);
    return e4m3 ? launch<128, false, true>(p, ctas, st) : launch<128, false, false>(p, ctas, st);
}

}  // namespace ea
