// rotary.cu -- rotary positions of q and k.
//
// A pair (x, y) of columns of a head at position t becomes a (x c - y s, x s +
// y c) with c, s the cosine and sine of t f_i.  Every value is read once and
// written once: HBM bounds it, and for a step's few rows the chain of reads
// (bounds, then the positions) before the angle is known.  So
//   - a thread asks for its first values before it looks positions up;
//   - the angle needs no table: f_i in turns a position is a 64-bit fraction
//     of a turn, t f_i mod 1 is that integer's product modulo 2^64, exactly,
//     at any position, and its upper 32 bits are the angle to 2^-33 of a turn;
//   - cosine and sine of a row are computed once, for all of its heads, in
//     shared memory;
//   - a thread keeps to one run of pairs of a head, so that its addresses need
//     no division.
#include <cuda_bf16.h>

#include <algorithm>

#include "../drafts.h"
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;    // rows of a CTA
constexpr int kStaged = 1024;   // sequence bounds staged in shared memory
constexpr int kAhead = 4;       // items in flight of a thread

// Position of dense row r; -1: the row is left as it is.
__device__ __forceinline__ int position_of(const RoParams &p, const int32_t *starts, const int32_t *lens, int64_t r) {
    if (p.positions) return __ldg(p.positions + r);
    if (r < starts[0] || r >= starts[p.n_seqs]) return -1;
    int a = 0, b = p.n_seqs - 1;  // the last i with starts[i] <= r
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (starts[mid] <= r) a = mid;
        else b = mid - 1;
    }
    PgSeq s;
    if (r >= starts[a + 1] || !pg_seq(starts[a], starts[a + 1], lens[a], p.rows, p.max_new, INT32_MAX, &s)) return -1;
    int at = (int)(r - s.first);
    if (p.parents) {
        int depth = 0;
        for (int b = at;; depth++) {  // parents lie before their children: this ends
            const int up = __ldg(p.parents + s.first + b);
            if (up >= b || up < -1) {
                batch_fail(p.err);
                return -1;
            }
            if (up < 0) break;
            b = up;
        }
        at = depth;
    }
    const int64_t pos = (int64_t)s.len - s.n + at;
    return pos < 0 ? -1 : (int)pos;
}

template <int N>
struct alignas(N) Raw {
    uint32_t w[(N + 3) / 4];
};
template <>
struct alignas(2) Raw<2> {
    uint16_t w[1];
};

template <bool F32>
__device__ __forceinline__ float get(const void *raw, int i) {
    if constexpr (F32) return reinterpret_cast<const float *>(raw)[i];
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(raw)[i]);
}
template <bool F32>
__device__ __forceinline__ void put(void *raw, int i, float x) {
    if constexpr (F32) reinterpret_cast<float *>(raw)[i] = x;
    else reinterpret_cast<__nv_bfloat16 *>(raw)[i] = __float2bfloat16_rn(x);
}

// A unit is V pairs: two accesses of V columns (HALF, or a single pair, whose
// columns need not lie on a boundary of two), or one of 2 V.
template <bool F32, bool HALF, int V>
struct Unit {
    static constexpr int ES = F32 ? 4 : 2;
    static constexpr bool TWO = HALF || V == 1;
    static constexpr int COLUMNS = HALF ? V : 2 * V;    // from one unit to the next
    static constexpr int BYTES = (TWO ? V : 2 * V) * ES;
    Raw<BYTES> a[TWO ? 2 : 1];

    __device__ __forceinline__ void load(const char *at, int64_t second) {
        a[0] = *reinterpret_cast<const Raw<BYTES> *>(at);
        if constexpr (TWO) a[1] = *reinterpret_cast<const Raw<BYTES> *>(at + second);
    }
    __device__ __forceinline__ void store(char *at, int64_t second) const {
        *reinterpret_cast<Raw<BYTES> *>(at) = a[0];
        if constexpr (TWO) *reinterpret_cast<Raw<BYTES> *>(at + second) = a[1];
    }
    __device__ __forceinline__ void turn(const float2 *cs) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float2 f = cs[i];
            void *px = &a[0], *py = &a[TWO ? 1 : 0];
            const int ix = TWO ? i : 2 * i, iy = TWO ? i : 2 * i + 1;
            const float x = get<F32>(px, ix), y = get<F32>(py, iy);
            put<F32>(px, ix, x * f.x - y * f.y);
            put<F32>(py, iy, x * f.y + y * f.x);
        }
    }
};

template <bool F32, bool HALF, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RoParams p, const int rows_cta) {
    using U = Unit<F32, HALF, V>;
    extern __shared__ float2 s_cs[];          // [rows][pairs]: cosine and sine
    __shared__ int32_t s_starts[kStaged + 1], s_lens[kStaged];
    __shared__ int32_t s_pos[kMaxRows];
    const int pairs = p.dims / 2, units = pairs / V, heads = p.heads[0] + p.heads[1];
    const int64_t row0 = (int64_t)blockIdx.x * rows_cta;
    const int rows = (int)min((int64_t)rows_cta, p.rows - row0);
    const int unit = threadIdx.x % units, lanes = kThreads / units;  // units <= 128
    const bool works = (int)threadIdx.x < lanes * units;
    const int64_t second = (HALF ? pairs : 1) * U::ES;
    const int column = p.offset + unit * U::COLUMNS;
    int row = 0, head = threadIdx.x / units;  // of the next item to load
    U u[kAhead];
    int r[kAhead], h[kAhead];
    auto place = [&](int rr, int hh) {
        const int w = hh >= p.heads[0];
        return (((row0 + rr) * p.heads[w] + (w ? hh - p.heads[0] : hh)) * p.dim + column) * U::ES;
    };
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            while (head >= heads) {
                head -= heads;
                row++;
            }
            r[i] = works && row < rows ? row : -1;
            h[i] = head;
            if (r[i] >= 0) u[i].load(p.x[head >= p.heads[0]] + place(row, head), second);
            head += lanes;
        }
    };
    fetch();
    const bool staged = !p.positions && p.n_seqs <= kStaged;
    if (staged) {
        for (int i = threadIdx.x; i <= p.n_seqs; i += kThreads) {
            s_starts[i] = __ldg(p.starts + i);
            if (i < p.n_seqs) s_lens[i] = __ldg(p.lens + i);
        }
        __syncthreads();
    }
    if ((int)threadIdx.x < rows)
        s_pos[threadIdx.x] = position_of(p, staged ? s_starts : p.starts, staged ? s_lens : p.lens, row0 + threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int rr = i / pairs, pos = s_pos[rr];
        if (pos < 0) continue;
        const uint64_t turn = (uint64_t)pos * p.turn[i - rr * pairs];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);  // half turns, in [-1, 1]
        s_cs[i] = make_float2(c * p.amplitude, s * p.sign);
    }
    __syncthreads();
    while (r[0] >= 0) {
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            if (r[i] < 0 || s_pos[r[i]] < 0) continue;
            u[i].turn(s_cs + r[i] * pairs + unit * V);
            u[i].store(p.y[h[i] >= p.heads[0]] + place(r[i], h[i]), second);
        }
        fetch();
    }
    // results elsewhere: the columns that are not rotated
    if (p.y[0] != p.x[0] && p.dims < p.dim) {
        const int rest = p.dim - p.dims;
        for (int w = 0; w < 2; w++) {
            if (!p.x[w]) continue;
            for (int i = threadIdx.x; i < rows * p.heads[w] * rest; i += kThreads) {
                const int rh = i / rest, col = i - rh * rest, rr = rh / p.heads[w];
                if (s_pos[rr] < 0) continue;
                const int64_t at = (row0 * p.heads[w] + rh) * p.dim + (col < p.offset ? col : col + p.dims);
                if constexpr (F32) reinterpret_cast<float *>(p.y[w])[at] = reinterpret_cast<const float *>(p.x[w])[at];
                else reinterpret_cast<uint16_t *>(p.y[w])[at] = reinterpret_cast<const uint16_t *>(p.x[w])[at];
            }
        }
    }
    // a sequence out of range is reported whether or not a row led to it
    if (!p.positions) {
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < p.n_seqs; i += (int64_t)gridDim.x * kThreads) {
            PgSeq s;
            if (!pg_seq(__ldg(p.starts + i), __ldg(p.starts + i + 1), __ldg(p.lens + i), p.rows, p.max_new, INT32_MAX, &s))
                batch_fail(p.err);
        }
    }
}

template <bool F32, bool HALF, int V>
cudaError_t launch(const RoParams &p, int64_t *ctas, cudaStream_t st) {
    int rows_cta = kMaxRows;
    while (rows_cta > 1 && (p.rows + rows_cta - 1) / rows_cta < 4 * 152) rows_cta /= 2;
    *ctas = (p.rows + rows_cta - 1) / rows_cta;
    rotary_kernel<F32, HALF, V><<<(unsigned)*ctas, kThreads, (size_t)rows_cta * (p.dims / 2) * sizeof(float2), st>>>(p, rows_cta);
    return cudaGetLastError();
}

template <bool F32, bool HALF>
cudaError_t launch_v(const RoParams &p, int64_t *ctas, cudaStream_t st) {
    // the widest accesses that all units' addresses are aligned to
    constexpr int most = 16 / (F32 ? 4 : 2) / (HALF ? 1 : 2);
    const int run = HALF ? 1 : 2;  // columns of a pair that lie together
    int v = most;
    while (v > 1 && ((p.dims / 2) % v || p.offset % (run * v) || p.dim % (run * v))) v /= 2;
    if constexpr (most >= 8)
        if (v == 8) return launch<F32, HALF, 8>(p, ctas, st);
    if constexpr (most >= 4)
        if (v == 4) return launch<F32, HALF, 4>(p, ctas, st);
    return v == 2 ? launch<F32, HALF, 2>(p, ctas, st) : launch<F32, HALF, 1>(p, ctas, st);
}

}  // namespace

cudaError_t launch_rotary(const RoParams &p, int64_t *ctas, cudaStream_t st) {
    if (p.f32) return p.half ? launch_v<true, true>(p, ctas, st) : launch_v<true, false>(p, ctas, st);
    return p.half ? launch_v<false, true>(p, ctas, st) : launch_v<false, false>(p, ctas, st);
}

}  // namespace ea
