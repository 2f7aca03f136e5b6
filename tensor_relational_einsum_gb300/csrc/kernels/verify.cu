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
// those rows are the kernel's bytes: HBM bounds it, and for few sequences the
// chain from reads to sums to the next decision.  So
//   - a cluster of CTAs takes a sequence, a warp of it a run of the row; the
//     sums of all runs go to the first CTA, which alone decides (one decision
//     for all: no CTA can wait for one that took another turn);
//   - r is not kept: it follows from the target's and the draft's rows and the
//     masses so far, and is made again where it is needed;
//   - sums are integers in units of 2^-62: they do not depend on their order,
//     so the running sums agree with the totals exactly, whatever the split.
// Probabilities lie in [0, 1] (others are taken as 0 or 1) and a row's sum
// below 4.
#include <cuda_bf16.h>

#include "../drafts.h"
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;            // the most CTAs of a sequence
constexpr int kRuns = kCluster * kWarps;
constexpr double kUnit = 1.0 / 4611686018427387904.0;  // 2^-62

// x in [0, 1] in units of 2^-62 (below 2^-39: rounded down).
__device__ __forceinline__ uint64_t fixed(float x) {
    const uint32_t b = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));  // NaN: 0
    const int s = (int)(b >> 23) - 88;
    const uint32_t m = (b & 0x7fffffu) | 0x800000u;
    return s >= 0 ? (uint64_t)m << s : (uint64_t)(m >> min(31, -s));
}
// The product of two such numbers, rounded down.
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b) { return __umul64hi(a << 1, b << 1); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

struct Order {                  // what the first CTA asks of all
    int node;                   // -1: nothing more
    int first;                  // the sequence's first dense row
    int rejected;               // subtractions from the target's row (with a draft)
    uint64_t mass[kPgNodes];    // Z before each of them; the first is 1
};

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
    __device__ __forceinline__ void load(int64_t v, float *x) const {
        if ((v > 0 || skip == 0) && (v + 1) * VE <= end) {
            const uint4 u = __ldg(at + v);
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

// r at one token.
__device__ __forceinline__ uint64_t rest_of(float t, float d, const Order &o) {
    uint64_t r = fixed(t);
    if (o.rejected > 0) {
        const uint64_t q = fixed(d);
        r = r > q ? r - q : 0;
        for (int k = 1; k < o.rejected; k++) {
            const uint64_t x = times(o.mass[k], q);
            r = r > x ? r - x : 0;
        }
    }
    return r;
}

template <bool BF16, bool DRAFT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VfParams p) {
    using R = Row<BF16>;
    __shared__ Order s_order;
    __shared__ uint64_t s_runs[kRuns];          // of the first CTA: the runs' sums
    __shared__ int s_up[kPgNodes], s_token[kPgNodes], s_path[kPgNodes], s_out[kPgNodes];
    __shared__ float s_t[kPgNodes], s_d[kPgNodes], s_u[kPgNodes];
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int seq = blockIdx.x / ctas, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    PgSeq s{};
    if (rank == 0) {
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
                s_t[j] = ld_elem(p.target, BF16 ? EA_BF16 : EA_F32, at);
                if constexpr (DRAFT) s_d[j] = ld_elem(p.draft, BF16 ? EA_BF16 : EA_F32, at);
            }
        }
        __syncthreads();
    }
    // the first CTA's first thread: where the walk is
    int node = 0, next = 1, kept = 1, rejected = 0, outs = 0;
    bool have = false;                          // the runs' sums are those of (node, rejected)
    uint64_t mass = 0, total = 0;
    // Goes on until a row's sums are needed (true) or the next token is to be taken (false).
    auto walk = [&]() {
        for (; next < s.n; next++) {
            if (s_up[next] != node) continue;
            if (rejected > 0 && !have) return true;
            const double u = s_u[next];
            bool yes;
            bool out = false;                   // certain tokens: one that was rejected before
            if constexpr (DRAFT) {
                if (rejected == 0) {
                    yes = u * (double)s_d[next] < (double)s_t[next];
                } else {
                    s_order.rejected = rejected;
                    yes = u * (double)s_d[next] * ((double)mass * kUnit) < (double)rest_of(s_t[next], s_d[next], s_order) * kUnit;
                }
            } else {
                for (int i = 0; i < outs; i++) out |= s_out[i] == s_token[next];
                yes = !out && u * (rejected == 0 ? 1.0 : (double)mass * kUnit) < (double)s_t[next];
            }
            if (yes) {
                node = next;
                s_path[kept++] = next;
                rejected = outs = 0;
                have = false;
            } else if constexpr (DRAFT) {
                s_order.mass[rejected++] = mass;
                have = false;
            } else {
                rejected++;
                if (!out) {
                    s_out[outs++] = s_token[next];
                    if (have) mass -= min(mass, fixed(s_t[next]));
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
    for (;;) {
        if (rank == 0 && threadIdx.x == 0) {
            s_path[0] = 0;
            const bool more = s.n > 0 && walk();
            s_order.node = more ? node : -1;
            s_order.first = s.first;
            s_order.rejected = rejected;
            for (uint32_t c = 1; c < ctas; c++) {
                put_u32(shared_of(&s_order.node, c), (uint32_t)s_order.node);
                put_u32(shared_of(&s_order.first, c), (uint32_t)s.first);
                put_u32(shared_of(&s_order.rejected, c), (uint32_t)rejected);
                for (int k = 1; more && k < rejected && DRAFT; k++) put_u64(shared_of(&s_order.mass[k], c), s_order.mass[k]);
            }
        }
        __syncwarp();
        cluster_sync();
        if (s_order.node < 0) break;
        const R t(p.target, s_order.first + s_order.node, p.vocab), d(DRAFT ? p.draft : p.target, s_order.first + s_order.node, p.vocab);
        const int64_t each = (t.vectors + ctas * kWarps - 1) / (ctas * kWarps);
        const int64_t v0 = (rank * kWarps + warp) * each, v1 = min(v0 + each, t.vectors);
        uint64_t sum = 0;
        const bool both = DRAFT && s_order.rejected > 0;
        for (int64_t v = v0 + lane; v < v1; v += 32) {
            float a[R::VE], b[R::VE];
            t.load(v, a);
            if (both) d.load(v, b);
#pragma unroll
            for (int i = 0; i < R::VE; i++) sum += DRAFT ? rest_of(a[i], both ? b[i] : 0.f, s_order) : fixed(a[i]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) put_u64(shared_of(&s_runs[rank * kWarps + warp], 0), sum);
        __syncwarp();
        cluster_sync();
        if (rank == 0 && threadIdx.x == 0) {
            total = 0;
            for (int i = 0; i < (int)ctas * kWarps; i++) total += s_runs[i];
            mass = total;
            if constexpr (!DRAFT) {
                for (int j = 1; j < next; j++) {
                    // the tokens that were rejected at this node, each once
                    if (s_up[j] != node) continue;
                    bool again = false;
                    for (int i = 1; i < j; i++) again |= s_up[i] == node && s_token[i] == s_token[j];
                    if (!again) mass -= min(mass, fixed(s_t[j]));
                }
            }
            have = true;
        }
    }
    if (rank != 0) return;
    // ---- the first CTA: the path, and the next token
    __shared__ int s_kept, s_node, s_outs;
    __shared__ uint64_t s_mass;
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
            for (int i = 0; i < outs; i++)
                s_runs[(t.skip + s_out[i]) / R::VE / each] -= fixed(ld_elem(p.target, BF16 ? EA_BF16 : EA_F32, (int64_t)(s.first + node) * p.vocab + s_out[i]));
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.width; j += kThreads) p.path[(int64_t)seq * p.width + j] = j < s_kept ? s_path[j] : -1;
    if (warp != 0 || s.n == 0 || s_mass == 0) return;
    const R t(p.target, s.first + s_node, p.vocab), d(DRAFT ? p.draft : p.target, s.first + s_node, p.vocab);
    const int64_t each = (t.vectors + ctas * kWarps - 1) / (ctas * kWarps);
    uint64_t left = min(times(fixed(__ldg(p.sample + seq)), s_mass), s_mass - 1);  // the running sum to exceed
    // the run that holds it
    int run = 0;
    {
        const int runs = ctas * kWarps;
        const uint64_t a = 2 * lane < runs ? s_runs[2 * lane] : 0, b = 2 * lane + 1 < runs ? s_runs[2 * lane + 1] : 0;
        uint64_t incl = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int l = max(0, __ffs((int)__ballot_sync(0xffffffffu, left < incl)) - 1);  // incl of the last is the mass
        const uint64_t before = __shfl_sync(0xffffffffu, incl - a - b, l), first = __shfl_sync(0xffffffffu, a, l);
        left -= before;
        run = 2 * l;
        if (left >= first) {
            left -= first;
            run++;
        }
    }
    const int64_t v0 = run * each, v1 = min(v0 + each, t.vectors);
    for (int64_t v = v0; v < v1; v += 32) {
        float a[R::VE], b[R::VE];
        uint64_t r[R::VE], mine = 0;
#pragma unroll
        for (int i = 0; i < R::VE; i++) a[i] = b[i] = 0.f;
        if (v + lane < v1) {
            t.load(v + lane, a);
            if (DRAFT && s_order.rejected > 0) d.load(v + lane, b);
        }
#pragma unroll
        for (int i = 0; i < R::VE; i++) {
            r[i] = DRAFT ? rest_of(a[i], b[i], s_order) : fixed(a[i]);
            if constexpr (!DRAFT) {
                const int64_t x = (v + lane) * R::VE + i - t.skip;
                for (int k = 0; k < s_outs; k++)
                    if (s_out[k] == x) r[i] = 0;
            }
            mine += r[i];
        }
        uint64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const uint32_t found = __ballot_sync(0xffffffffu, left < incl);
        if (found) {
            if (lane == __ffs((int)found) - 1) {
                uint64_t at = incl - mine;
                int i = 0;
#pragma unroll
                for (int k = 0; k < R::VE - 1; k++)
                    if (i == k && left >= at + r[k]) {
                        at += r[k];
                        i = k + 1;
                    }
                p.picked[seq] = (int32_t)((v + lane) * R::VE + i - t.skip);
            }
            return;
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
    }
}

template <bool BF16, bool DRAFT>
cudaError_t launch(const VfParams &p, int ctas, cudaStream_t st) {
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
    int c = kCluster;
    while (c > 1 && ((int64_t)p.n_seqs * c > 4 * num_sms || p.vocab < 2048 * c)) c /= 2;
    *ctas = (int64_t)p.n_seqs * c;
    if (p.bf16) return p.draft ? launch<true, true>(p, c, st) : launch<true, false>(p, c, st);
    return p.draft ? launch<false, true>(p, c, st) : launch<false, false>(p, c, st);
}

}  // namespace ea
