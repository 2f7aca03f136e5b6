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
//   - a thread keeps to one unit of a head, so that its addresses need no
//     division; a CTA takes as many rows as give its threads four units each
//     (more rows leave the last CTAs alone: 46 and 52 us with 8 and 16 units
//     where 4 take 42.5).
//
// Measured: q and k of 12800 rows, 32 + 8 heads of 128, bf16, half layout, 262
// MB: 42.5 us, 0.91 of the measured copy rate (interleaved 0.75; fp32 0.98 and
// 0.91); accesses of 2 bytes (33 pairs in 100 columns) 0.38, of 4 0.6 to 0.76:
// those are bound by instructions; a step of 128 rows 4.1 us.
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
constexpr int kItems = 4;       // units that a thread takes, about

// Position of dense row r; -1: the row is left as it is.  parents: those of rows from `from` on.
__device__ __forceinline__ int position_of(const RoParams &p, const int32_t *starts, const int32_t *lens, const int32_t *parents,
                                           int64_t from, int64_t r) {
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
        if (at >= kPgNodes) {  // more nodes than max_new says: the sequence has been refused above
            batch_fail(p.err);
            return -1;
        }
        for (int b = at;; depth++) {  // parents lie before their children: this ends
            const int up = parents[s.first + b - from];
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

// The widest access that all addresses are aligned to holds V pairs (half
// layout: V first columns, and V second ones; else 2 V columns; a single pair
// is always two accesses, as its columns need not lie on a boundary of two).
// Such a run of V pairs is short where V is, and what a thread does besides
// would weigh more than its values: so a unit is G runs, T apart (T units a
// head, so that neighbouring threads stay neighbours in memory).  Where
// results go elsewhere, other units copy the columns that are not rotated.
template <bool F32, bool HALF, int V>
struct Unit {
    static constexpr int ES = F32 ? 4 : 2;
    static constexpr bool TWO = HALF || V == 1;
    static constexpr int RUN = TWO ? V : 2 * V;         // columns of an access
    static constexpr int BYTES = RUN * ES;
    // 32 bytes a unit; two runs where an access is narrower (four measured the same, eight a half slower)
    static constexpr int G = BYTES >= 8 ? 32 / BYTES / (TWO ? 2 : 1) : 2;
    static constexpr int N = TWO ? 2 * G : G;           // accesses
    Raw<BYTES> a[N];
    int off[N];                                         // byte offsets in a head; -1: none

    __device__ __forceinline__ void load(const char *x) {
#pragma unroll
        for (int n = 0; n < N; n++)
            if (off[n] >= 0) a[n] = *reinterpret_cast<const Raw<BYTES> *>(x + off[n]);
    }
    __device__ __forceinline__ void store(char *y) const {
#pragma unroll
        for (int n = 0; n < N; n++)
            if (off[n] >= 0) *reinterpret_cast<Raw<BYTES> *>(y + off[n]) = a[n];
    }
    // cs: (cosine, sine) of the row's pairs, V > 1: two pairs of every run, then the next two; the unit's runs are
    // run, run + step, ..
    __device__ __forceinline__ void turn(const float2 *cs, int run, int step, int runs) {
#pragma unroll
        for (int g = 0; g < G; g++) {
            if (G > 1 && off[TWO ? 2 * g : g] < 0) break;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                float4 f;
                if constexpr (V == 1) {
                    const float2 c = cs[run + g * step];
                    f = make_float4(c.x, c.y, 0.f, 0.f);
                } else {
                    f = reinterpret_cast<const float4 *>(cs)[(i / 2) * runs + run + g * step];
                }
#pragma unroll
                for (int j = i; j < V && j < i + 2; j++) {
                    const float c = j == i ? f.x : f.z, s = j == i ? f.y : f.w;
                    void *px = &a[TWO ? 2 * g : g], *py = &a[TWO ? 2 * g + 1 : g];
                    const int ix = TWO ? j : 2 * j, iy = TWO ? j : 2 * j + 1;
                    const float x = get<F32>(px, ix), y = get<F32>(py, iy);
                    put<F32>(px, ix, x * c - y * s);
                    put<F32>(py, iy, x * s + y * c);
                }
            }
        }
    }
};

// Units of a head: those that rotate, then those that copy.
template <class U, int V>
__host__ __device__ __forceinline__ void units_of(const RoParams &p, int *turned, int *copied) {
    const int rest = p.y[0] != p.x[0] ? (p.dim - p.dims) / U::RUN : 0;
    *turned = (p.dims / 2 / V + U::G - 1) / U::G;
    *copied = (rest + U::N - 1) / U::N;
}

template <bool F32, bool HALF, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RoParams p, const int rows_cta) {
    using U = Unit<F32, HALF, V>;
    extern __shared__ __align__(16) float2 s_cs[];
    __shared__ int32_t s_starts[kStaged + 1], s_lens[kStaged];
    __shared__ int32_t s_pos[kMaxRows], s_up[kPgNodes + kMaxRows];
    const int pairs = p.dims / 2, runs = pairs / V, heads = p.heads[0] + p.heads[1];
    int turned, copied;
    units_of<U, V>(p, &turned, &copied);
    const int64_t row0 = (int64_t)blockIdx.x * rows_cta;
    const int rows = (int)min((int64_t)rows_cta, p.rows - row0);
    U u;
    char *to;
    // a thread's unit, and where it lies in a head; a head with more units than threads takes several turns
    int unit, lanes, row, head;
    bool works;
    auto take = [&](int unit0) {
        const int n = min(kThreads, turned + copied - unit0);
        unit = unit0 + threadIdx.x % n;
        lanes = kThreads / n;
        works = (int)threadIdx.x < lanes * n;
        row = 0;
        head = threadIdx.x / n;
#pragma unroll
        for (int i = 0; i < U::N; i++) {
            if (unit < turned) {
                const int run = unit + (U::TWO ? i / 2 : i) * turned, col = p.offset + run * (HALF ? V : 2 * V);
                u.off[i] = run < runs ? (col + (U::TWO && (i & 1) ? (HALF ? pairs : 1) : 0)) * U::ES : -1;
            } else {
                const int col = (unit - turned + i * copied) * U::RUN;
                u.off[i] = col < p.dim - p.dims ? (col < p.offset ? col : col + p.dims) * U::ES : -1;
            }
        }
    };
    // The next item of the thread: false if there is none.
    auto fetch = [&]() {
        while (head >= heads) {
            head -= heads;
            row++;
        }
        if (!works || row >= rows) return false;
        const int w = head >= p.heads[0];
        const int64_t at = ((row0 + row) * p.heads[w] + (w ? head - p.heads[0] : head)) * p.dim * U::ES;
        u.load(p.x[w] + at);
        to = p.y[w] + at;
        return true;
    };
    take(0);
    bool any = fetch();
    const bool staged = !p.positions && p.n_seqs <= kStaged;
    const int64_t from = max((int64_t)0, row0 - (kPgNodes - 1));  // a row's tree begins there at the earliest
    if (p.parents && threadIdx.x < row0 + rows - from) s_up[threadIdx.x] = __ldg(p.parents + from + threadIdx.x);
    if (staged) {
        for (int i = threadIdx.x; i <= p.n_seqs; i += kThreads) {
            s_starts[i] = __ldg(p.starts + i);
            if (i < p.n_seqs) s_lens[i] = __ldg(p.lens + i);
        }
    }
    if (staged || p.parents) __syncthreads();
    if ((int)threadIdx.x < rows)
        s_pos[threadIdx.x] = position_of(p, staged ? s_starts : p.starts, staged ? s_lens : p.lens, s_up, from, row0 + threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int rr = i / pairs, pair = i - rr * pairs, pos = s_pos[rr];
        if (pos < 0) continue;
        const uint64_t turn = (uint64_t)pos * p.turn[pair];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);  // half turns, in [-1, 1]
        const int x = V == 1 ? pair : ((pair % V / 2) * runs + pair / V) * 2 + (pair & 1);
        s_cs[rr * pairs + x] = make_float2(c * p.amplitude, s * p.sign);
    }
    __syncthreads();
    for (int unit0 = 0;;) {
        while (any) {
            if (s_pos[row] >= 0) {
                if (unit < turned) u.turn(s_cs + row * pairs, unit, turned, runs);
                u.store(to);
            }
            head += lanes;
            any = fetch();
        }
        unit0 += kThreads;
        if (unit0 >= turned + copied) break;
        take(unit0);
        any = fetch();
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
cudaError_t launch(const RoParams &p, int num_sms, int64_t *ctas, cudaStream_t st) {
    int turned, copied;
    units_of<Unit<F32, HALF, V>, V>(p, &turned, &copied);
    const int64_t items = (int64_t)(p.heads[0] + p.heads[1]) * (turned + copied);  // of a row
    int rows_cta = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRows, kItems * kThreads / items));
    while (rows_cta > 1 && (p.rows + rows_cta - 1) / rows_cta < 2 * num_sms) rows_cta--;
    *ctas = (p.rows + rows_cta - 1) / rows_cta;
    rotary_kernel<F32, HALF, V><<<(unsigned)*ctas, kThreads, (size_t)rows_cta * (p.dims / 2) * sizeof(float2), st>>>(p, rows_cta);
    return cudaGetLastError();
}

template <bool F32, bool HALF>
cudaError_t launch_v(const RoParams &p, int num_sms, int64_t *ctas, cudaStream_t st) {
    // the widest accesses that all units' addresses are aligned to
    constexpr int most = 16 / (F32 ? 4 : 2) / (HALF ? 1 : 2);
    const int run = HALF ? 1 : 2;  // columns of a pair that lie together
    int v = most;
    while (v > 1 && ((p.dims / 2) % v || p.offset % (run * v) || p.dim % (run * v))) v /= 2;
    if constexpr (most >= 8)
        if (v == 8) return launch<F32, HALF, 8>(p, num_sms, ctas, st);
    if constexpr (most >= 4)
        if (v == 4) return launch<F32, HALF, 4>(p, num_sms, ctas, st);
    return v == 2 ? launch<F32, HALF, 2>(p, num_sms, ctas, st) : launch<F32, HALF, 1>(p, num_sms, ctas, st);
}

}  // namespace

cudaError_t launch_rotary(const RoParams &p, int num_sms, int64_t *ctas, cudaStream_t st) {
    if (p.f32) return p.half ? launch_v<true, true>(p, num_sms, ctas, st) : launch_v<true, false>(p, num_sms, ctas, st);
    return p.half ? launch_v<false, true>(p, num_sms, ctas, st) : launch_v<false, false>(p, num_sms, ctas, st);
}

}  // namespace ea
