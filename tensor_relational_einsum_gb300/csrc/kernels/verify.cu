// verify.cu -- which branch of a tree of drafted tokens the target's
// probabilities accept, and the token that follows it.
//
// At node v the rest r begins as the target's row of v with mass Z = 1.  A
// child with token x and random number u is accepted where u d(x) Z < r(x), d
// the draft's row of v; else r becomes max(r - Z d, 0) and Z its sum.  Where
// no child is accepted, the next token is the first x whose running sum of r
// exceeds sample * Z.  A token that is certain has d = 1 at x: then only r(x)
// becomes 0 and Z loses it.
//
// The walk itself needs two numbers a node, which are read at once.  A whole
// row is read only for the sum after a rejection and for the last token, and
// those rows are the kernel's bytes.  What bounds it is the chain: reads, sums,
// the next decision, as often as a sequence has rejections, and the call lasts
// as long as its longest sequence (64 trees: 16% of DRAM's rate, 38% of the
// warps active, which wait at a barrier half of their time).  So
//   - a cluster of CTAs takes a sequence, a warp of it a run of the row; the
//     sums of all runs go to the first CTA, which alone decides (one decision
//     for all: no CTA can wait for one that took another turn);
//   - r is not kept: it follows from the target's and the draft's rows and the
//     masses so far, and is made again where it is needed;
//   - a thread's sum is a pair of floats, each addition's error kept (7
//     instructions where a fixed-point sum takes 13 and the conversion to 64
//     bits is slower still: 69 us that way, 75 with the hardware's conversion,
//     54 with pairs); its total, and all sums of threads, are integers in units
//     of 2^-62, which do not depend on their order.  No fp64: this GPU has
//     little of it.
// Probabilities lie in [0, 1] (others are taken as 0 or 1).  A row's sum has
// room below 2; from 2 on (logits, say) all additions stop at kTop, whatever
// their order, the walk ends and the error word is raised.
//
// Measured, in a graph on the same inputs: one chain of 5 over 32000 tokens,
// fp32: 8.7 us (6.1 us with one node and 1000 tokens: launch, two round trips
// of scalars, a row, the token); 64 trees of up to 16 nodes over 131072, fp32:
// 47 us (56 us with inputs that change, whose rows L2 does not hold); 200
// certain trees of up to 7 over 50021, bf16: 21 us: 8 with one node and 1000
// tokens, 7 more for the row's sum and the search, 7 for the walk over the
// nodes.  The first barrier is 0.3 to 0.8 us of these.
#include <cuda_bf16.h>

#include <type_traits>

#include "../drafts.h"
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 16;           // the most CTAs of a sequence
constexpr int kRuns = kCluster * kWarps;
constexpr int kResident = 4;           // CTAs of an SM
constexpr int kLaneRuns = kRuns / 32;  // runs whose sums a lane holds
constexpr float kUnit = 0x1p-62f;
constexpr uint64_t kTop = ((uint64_t)1 << 63) - 1;  // a sum of 2 or more

// x (|x| < 2) in units of 2^-62, below 2^-39 rounded towards 0.
__device__ __forceinline__ int64_t fixed(float x) {
    const uint32_t b = __float_as_uint(x);
    const int s = (int)(b >> 23 & 255) - 88;
    const uint32_t m = (b & 0x7fffffu) | 0x800000u;
    const int64_t v = s >= 0 ? (int64_t)m << s : (int64_t)(m >> min(31, -s));
    return (int)b < 0 ? -v : v;
}
// The product of two such numbers, rounded down.
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b) { return __umul64hi(a << 1, b << 1); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of a shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t shared_of(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void put_u64(uint32_t at, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}
__device__ __forceinline__ void put_u32(uint32_t at, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// Inclusive sums over the lanes.
__device__ __forceinline__ uint64_t scan(uint64_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// A number as the sum of two floats, the second below half a step of the first.
struct alignas(8) Pair {
    float h, l;
};
__device__ __forceinline__ Pair pair_of(uint64_t x) {  // units of 2^-62
    const float h = __ull2float_rn(x);
    return Pair{h * kUnit, __ll2float_rn((int64_t)(x - __float2ull_rn(h))) * kUnit};
}
// z q, rounded to about 2^-47.
__device__ __forceinline__ Pair times(const Pair &z, float q) {
    const float h = __fmul_rn(z.h, q);
    return Pair{h, fmaf(z.h, q, -h) + __fmul_rn(z.l, q)};
}
// a < b, exactly for the two pairs (differences of neighbouring floats are exact; else the first parts decide).
__device__ __forceinline__ bool less(const Pair &a, const Pair &b) { return __fsub_rn(a.h, b.h) < __fsub_rn(b.l, a.l); }
__device__ __forceinline__ uint64_t fixed(const Pair &x) { return (uint64_t)max((int64_t)0, fixed(x.h) + fixed(x.l)); }
// s += x: the exact error of the first parts' sum goes to the second.
__device__ __forceinline__ void add_to(Pair &s, const Pair &x) {
    const float t = __fadd_rn(s.h, x.h), y = __fsub_rn(t, s.h);
    s.l += __fadd_rn(__fsub_rn(s.h, __fsub_rn(t, y)), __fsub_rn(x.h, y)) + x.l;
    s.h = t;
}

struct Order {                  // what the first CTA asks of all
    int node;                   // -1: nothing more
    int first;                  // the sequence's first dense row
    int rejected;               // subtractions from the target's row (with a draft)
    Pair mass[kPgNodes];        // (8 bytes each, and aligned so) Z before each of them; the first is 1
};

static_assert(sizeof(Pair) == 8 && alignof(Order) == 8 && offsetof(Order, mass) % 8 == 0, "masses go to other CTAs as 64 bits");

// A row of probabilities as 16-byte vectors from the aligned address at or
// before its first element; `skip` elements lie before it.
template <bool BF16>
struct Row {
    static constexpr int VE = BF16 ? 8 : 4;
    const uint4 *at;
    int skip;
    int64_t vectors, end;       // end: skip + vocab
    __device__ __forceinline__ Row(const char *base, int64_t row, int64_t vocab) {
        const char *p = base + row * vocab * (BF16 ? 2 : 4);
        skip = (int)((uintptr_t)p & 15) / (BF16 ? 2 : 4);
        at = reinterpret_cast<const uint4 *>((uintptr_t)p & ~(uintptr_t)15);
        end = skip + vocab;
        vectors = (end + VE - 1) / VE;
    }
    // Whole vectors of the row: [first_whole, last_whole).
    __device__ __forceinline__ int64_t first_whole() const { return skip > 0; }
    __device__ __forceinline__ int64_t last_whole() const { return end / VE; }
    static __device__ __forceinline__ void values(const uint4 &u, float *x) {
        if constexpr (BF16) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            x[0] = __uint_as_float(u.x);
            x[1] = __uint_as_float(u.y);
            x[2] = __uint_as_float(u.z);
            x[3] = __uint_as_float(u.w);
        }
    }
    __device__ __forceinline__ void load(int64_t v, float *x) const {
        if (v >= first_whole() && v < last_whole()) {
            values(__ldg(at + v), x);
        } else {
#pragma unroll
            for (int i = 0; i < VE; i++) {
                const int64_t e = v * VE + i;
                x[i] = 0.f;
                if (e < skip || e >= end) continue;
                if constexpr (BF16) x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(at)[e]);
                else x[i] = __ldg(reinterpret_cast<const float *>(at) + e);
            }
        }
    }
};

// r at one token, from the target's and the draft's probabilities.
__device__ __forceinline__ Pair rest_of(float t, float d, const Order &o) {
    Pair r{__saturatef(t), 0.f};  // NaN: 0
    if (o.rejected > 0) {
        const float q = __saturatef(d);
        const float h = __fsub_rn(r.h, q);
        r = h > 0.f ? Pair{h, __fsub_rn(__fsub_rn(r.h, h), q)} : Pair{0.f, 0.f};  // exact: the larger first
        for (int k = 1; k < o.rejected; k++) {
            const Pair z = o.mass[k];
            const Pair x = times(z, q);
            const float e = __fsub_rn(r.h, x.h);
            if (!(e >= 0.f)) {
                r = Pair{0.f, 0.f};
                continue;
            }
            const float l = __fadd_rn(__fsub_rn(__fsub_rn(r.h, e), x.h), __fsub_rn(r.l, x.l)), g = __fadd_rn(e, l);
            r = g > 0.f ? Pair{g, __fsub_rn(l, __fsub_rn(g, e))} : Pair{0.f, 0.f};
        }
    }
    return r;
}

template <bool BF16, bool DRAFT>
__global__ void __launch_bounds__(kThreads, kResident) verify_kernel(const __grid_constant__ VfParams p) {
    using R = Row<BF16>;
    __shared__ Order s_order;
    __shared__ uint64_t s_runs[kRuns];          // of the first CTA: the runs' sums
    __shared__ int s_up[kPgNodes], s_token[kPgNodes], s_path[kPgNodes], s_out[kPgNodes];
    __shared__ float s_t[kPgNodes], s_d[kPgNodes], s_u[kPgNodes], s_was[kPgNodes];
    constexpr int kAhead = 2;                   // vectors of a lane in flight of two rows; twice as many of one
    cluster_arrive();                           // waited for before the first store to another CTA: that CTA has begun
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int seq = blockIdx.x / ctas, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    PgSeq s{};
    float sample = 0.f;
    if (rank == 0) {
        sample = __ldg(p.sample + seq);
        if (!pg_seq(__ldg(p.starts + seq), __ldg(p.starts + seq + 1), 0, p.rows, p.max_new, 0, &s) && threadIdx.x == 0) batch_fail(p.err);
        const int j = threadIdx.x;
        if (j < s.n) {
            const int64_t row = s.first + j;
            int up = p.parents ? __ldg(p.parents + row) : j - 1;
            const int token = __ldg(p.tokens + row);
            s_u[j] = __ldg(p.accept + row);
            if (up >= j || up < -1 || (j > 0 && (token < 0 || token >= p.vocab))) {
                batch_fail(p.err);
                up = -1;
            }
            if (j == 0) up = -1;
            s_up[j] = up;
            s_token[j] = token;
            s_t[j] = s_d[j] = 0.f;
            if (up >= 0) {
                const int64_t at = (int64_t)(s.first + up) * p.vocab + token;
                s_t[j] = __saturatef(ld_elem(p.target, BF16 ? EA_BF16 : EA_F32, at));
                if constexpr (DRAFT) s_d[j] = __saturatef(ld_elem(p.draft, BF16 ? EA_BF16 : EA_F32, at));
            }
        }
        __syncthreads();
    }
    // the first CTA's first thread: where the walk is
    int node = 0, next = 1, kept = 1, rejected = 0, outs = 0;
    bool have = false;                          // the runs' sums are those of (node, rejected)
    bool over = false;                          // a row's sum was out of range: nothing more
    uint64_t mass = 0, total = 0;
    // Goes on until a row's sums are needed (true) or the next token is to be taken (false).
    auto walk = [&]() {
        for (; next < s.n; next++) {
            if (s_up[next] != node) continue;
            if (rejected > 0 && !have) return true;
            const float u = s_u[next];
            bool yes;
            bool out = false;                   // certain tokens: one that was rejected before
            if constexpr (DRAFT) {
                const Pair d = times(Pair{u, 0.f}, s_d[next]);
                s_order.rejected = rejected;
                const Pair r = rest_of(s_t[next], s_d[next], s_order);
                if (rejected == 0) {
                    yes = less(d, r);
                } else {
                    const Pair z = pair_of(mass), h = times(z, d.h);
                    yes = less(Pair{h.h, h.l + __fmul_rn(z.h, d.l)}, r);
                }
            } else {
                for (int i = 0; i < outs; i++) out |= s_out[i] == s_token[next];
                yes = !out && less(rejected == 0 ? Pair{u, 0.f} : times(pair_of(mass), u), Pair{s_t[next], 0.f});
            }
            if (yes) {
                node = next;
                s_path[kept++] = next;
                rejected = outs = 0;
                have = false;
            } else if constexpr (DRAFT) {
                s_order.mass[rejected++] = pair_of(mass);
                have = false;
            } else {
                rejected++;
                if (!out) {
                    s_was[outs] = s_t[next];
                    s_out[outs++] = s_token[next];
                    if (have) mass -= min(mass, (uint64_t)fixed(s_t[next]));
                }
            }
        }
        if (!have) return true;
        if (mass == 0 && rejected > 0) {        // rounding alone can lead here: the target's row itself
            rejected = outs = 0;
            mass = total;
            have = !DRAFT;
            return !have;
        }
        return false;
    };
    __syncwarp();
    cluster_wait();  // behind the scalars' reads: all CTAs have long arrived
    for (;;) {
        if (rank == 0 && threadIdx.x == 0) {
            s_path[0] = 0;
            const bool more = s.n > 0 && !over && walk();
            s_order.node = more ? node : -1;
            s_order.first = s.first;
            s_order.rejected = rejected;
            for (uint32_t c = 1; c < ctas; c++) {
                put_u32(shared_of(&s_order.node, c), (uint32_t)s_order.node);
                put_u32(shared_of(&s_order.first, c), (uint32_t)s.first);
                put_u32(shared_of(&s_order.rejected, c), (uint32_t)rejected);
                for (int k = 1; more && k < rejected && DRAFT; k++) put_u64(shared_of(&s_order.mass[k], c), *reinterpret_cast<const uint64_t *>(&s_order.mass[k]));
            }
        }
        __syncwarp();
        cluster_sync();
        if (s_order.node < 0) break;
        const R t(p.target, s_order.first + s_order.node, p.vocab), d(DRAFT ? p.draft : p.target, s_order.first + s_order.node, p.vocab);
        const int64_t each = (t.vectors + ctas * kWarps - 1) / (ctas * kWarps);
        const int64_t v0 = (rank * kWarps + warp) * each, v1 = min(v0 + each, t.vectors);
        Pair part{0.f, 0.f};
        const bool both = DRAFT && s_order.rejected > 0;
        auto add = [&](const float *a, const float *b) {
#pragma unroll
            for (int i = 0; i < R::VE; i++) add_to(part, DRAFT ? rest_of(a[i], b[i], s_order) : Pair{__saturatef(a[i]), 0.f});
        };
        // whole vectors, several of a lane in flight
        const int64_t w0 = max(v0, t.first_whole()), w1 = min(v1, t.last_whole());
        auto whole = [&](auto ahead, auto drafts) {
            constexpr int A = decltype(ahead)::value;
            constexpr bool B = decltype(drafts)::value;
            for (int64_t v = w0 + lane; v < w1; v += 32 * A) {
                uint4 a[A], b[B ? A : 1];
#pragma unroll
                for (int k = 0; k < A; k++) {
                    const bool in = v + 32 * k < w1;
                    a[k] = in ? __ldg(t.at + v + 32 * k) : make_uint4(0, 0, 0, 0);
                    if constexpr (B) b[k] = in ? __ldg(d.at + v + 32 * k) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < A; k++) {
                    float x[R::VE], y[R::VE];
                    R::values(a[k], x);
                    if constexpr (B) R::values(b[k], y);
#pragma unroll
                    for (int i = 0; i < R::VE; i++) add_to(part, B ? rest_of(x[i], y[i], s_order) : Pair{__saturatef(x[i]), 0.f});
                }
            }
        };
        if constexpr (DRAFT) {
            if (both) whole(std::integral_constant<int, kAhead>{}, std::true_type{});
            else whole(std::integral_constant<int, 2 * kAhead>{}, std::false_type{});
        } else {
            whole(std::integral_constant<int, 2 * kAhead>{}, std::false_type{});
        }
        // the row's ends: the first vector (lane 0) and the last (lane 1), where they are not whole
        if (lane == 0 || (lane == 1 && t.vectors > 1)) {
            const int64_t v = lane == 0 ? 0 : t.vectors - 1;
            if (v >= v0 && v < v1 && (v < w0 || v >= w1)) {
                float x[R::VE], y[R::VE];
                t.load(v, x);
#pragma unroll
                for (int i = 0; i < R::VE; i++) y[i] = 0.f;
                if (both) d.load(v, y);
                add(x, y);
            }
        }
        __syncwarp();
        uint64_t sum = part.h < 2.f && part.h + part.l < 2.f ? fixed(part) : kTop;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum = min(sum + __shfl_xor_sync(0xffffffffu, sum, o), kTop);
        if (lane == 0) put_u64(shared_of(&s_runs[rank * kWarps + warp], 0), sum);
        __syncwarp();
        cluster_sync();
        if (rank == 0 && warp == 0) {
            const int runs = ctas * kWarps;
            total = 0;
#pragma unroll
            for (int i = 0; i < kLaneRuns; i++) total = min(total + (kLaneRuns * lane + i < runs ? s_runs[kLaneRuns * lane + i] : 0), kTop);
#pragma unroll
            for (int o = 16; o; o >>= 1) total = min(total + __shfl_xor_sync(0xffffffffu, total, o), kTop);
            over = total == kTop;
            if (over && lane == 0) batch_fail(p.err);
            mass = over ? 0 : total;
            if constexpr (!DRAFT) {
                if (lane == 0)  // the tokens that were rejected at this node, each once
                    for (int i = 0; i < outs; i++) mass -= min(mass, (uint64_t)fixed(s_was[i]));
            }
            have = true;
        }
    }
    if (rank != 0) return;
    // ---- the first CTA: the path, and the next token
    __shared__ int s_kept, s_node, s_outs;
    __shared__ uint64_t s_mass, s_warps[kWarps];
    if (threadIdx.x == 0) {
        s_kept = s.n > 0 ? kept : 0;
        s_node = node;
        s_mass = mass;
        s_outs = outs;
        s_order.rejected = rejected;
        p.counts[seq] = s_kept;
        if (s.n == 0 || mass == 0) p.picked[seq] = -1;
        if constexpr (!DRAFT) {  // runs without the tokens that were rejected
            const R t(p.target, s.first + node, p.vocab);
            const int64_t each = (t.vectors + ctas * kWarps - 1) / (ctas * kWarps);
            for (int i = 0; i < outs; i++) {
                uint64_t &run = s_runs[(t.skip + s_out[i]) / R::VE / each];
                run -= min(run, (uint64_t)fixed(s_was[i]));
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.width; j += kThreads) p.path[(int64_t)seq * p.width + j] = j < s_kept ? s_path[j] : -1;
    if (s.n == 0 || s_mass == 0) return;
    const R t(p.target, s.first + s_node, p.vocab), d(DRAFT ? p.draft : p.target, s.first + s_node, p.vocab);
    const int64_t each = (t.vectors + ctas * kWarps - 1) / (ctas * kWarps);
    // the run that holds the running sum to exceed
    uint64_t left;
    int run = 0;
    {
        const int runs = ctas * kWarps;
        uint64_t mine[kLaneRuns], sum = 0;
#pragma unroll
        for (int i = 0; i < kLaneRuns; i++) {
            mine[i] = kLaneRuns * lane + i < runs ? s_runs[kLaneRuns * lane + i] : 0;
            sum += mine[i];
        }
        const uint64_t incl = scan(sum, lane), all = __shfl_sync(0xffffffffu, incl, 31);
        left = min(times((uint64_t)fixed(__saturatef(sample)), all), all - 1);
        const int l = max(0, __ffs((int)__ballot_sync(0xffffffffu, left < incl)) - 1);
        left -= __shfl_sync(0xffffffffu, incl - sum, l);
        run = kLaneRuns * l;
        bool on = true;
#pragma unroll
        for (int i = 0; i < kLaneRuns - 1; i++) {
            const uint64_t one = __shfl_sync(0xffffffffu, mine[i], l);
            on &= left >= one;
            if (on) {
                left -= one;
                run++;
            }
        }
    }
    // a few neighbouring vectors of it a thread, whose sums say which thread has the token
    const int64_t mine = (each + kThreads - 1) / kThreads, v0 = run * each + threadIdx.x * mine, v1 = min(min(v0 + mine, (run + 1) * each), t.vectors);
    // f(r, token) of the thread's tokens in order, until it says so
    auto tokens = [&](auto f) {
        for (int64_t v = v0; v < v1; v++) {
            float a[R::VE], b[R::VE];
            t.load(v, a);
#pragma unroll
            for (int i = 0; i < R::VE; i++) b[i] = 0.f;
            if (DRAFT && s_order.rejected > 0) d.load(v, b);
#pragma unroll
            for (int i = 0; i < R::VE; i++) {
                const int64_t x = v * R::VE + i - t.skip;
                uint64_t r = fixed(DRAFT ? rest_of(a[i], b[i], s_order) : Pair{__saturatef(a[i]), 0.f});
                if constexpr (!DRAFT)
                    for (int k = 0; k < s_outs; k++)
                        if (s_out[k] == x) r = 0;
                if (r > 0 && f(r, (int)x)) return;
            }
        }
    };
    uint64_t sum = 0;
    tokens([&](uint64_t r, int) {
        sum += r;
        return false;
    });
    uint64_t incl = scan(sum, lane);
    if (lane == 31) s_warps[warp] = incl;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) incl += s_warps[w];
        all += s_warps[w];
    }
    // The run's sum was made of pairs of floats, in other groups: it can be larger than this one in the last places.
    left = min(left, all - 1);
    if (all == 0 && threadIdx.x == 0) p.picked[seq] = -1;
    if (left >= incl - sum && left < incl) {
        uint64_t at = incl - sum;
        tokens([&](uint64_t r, int x) {
            at += r;
            if (left < at) p.picked[seq] = x;
            return left < at;
        });
    }
}

template <bool BF16, bool DRAFT>
cudaError_t launch(const VfParams &p, int ctas, cudaStream_t st) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(verify_kernel<BF16, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.n_seqs * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<BF16, DRAFT>, p);
}

}  // namespace

cudaError_t launch_verify(const VfParams &p, int num_sms, int64_t *ctas, cudaStream_t st) {
    // As many CTAs a sequence as are resident at once, with 2048 tokens each at least (figures without the kernel's first
    // barrier, which costs both sides the same): one chain over 32000 tokens takes 8.4
    // us with 8 CTAs, 9.0 with 16; 16 trees of 16 nodes over 131072 25.5 us with 16, 29 with 8.  Trees with a draft's
    // probabilities have several rejections one after the other in some sequences, whose rounds then are the time that the
    // call takes: twice as many CTAs shorten those (64 such trees 46 against 52 us; 64 chains, which mostly end at
    // their first rejection, 36 against 22 us the other way).
    const int waves = p.draft && p.parents ? 2 : 1;
    int c = kCluster;
    while (c > 1 && ((int64_t)p.n_seqs * c > waves * kResident * num_sms || p.vocab < 2048 * c)) c /= 2;
    *ctas = (int64_t)p.n_seqs * c;
    if (p.bf16) return p.draft ? launch<true, true>(p, c, st) : launch<true, false>(p, c, st);
    return p.draft ? launch<false, true>(p, c, st) : launch<false, false>(p, c, st);
}

}  // namespace ea
