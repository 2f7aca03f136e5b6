// paged_sched.cuh -- a CTA's share of the attention's work list, and the
// walk over it.  The batch's lengths are known on the device only, so every
// CTA sums the units of all sequences (a block-wide scan, a thread a
// sequence), takes its equal share and finds the sequence it begins in.
#pragma once

#include "paged_common.cuh"

namespace ea {
namespace pg {

// NT threads, all of them; scratch: NT / 32 + 1 words of shared memory.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t u, int64_t *incl, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += x;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = u;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w++) {
        const int64_t x = scratch[w];
        if (w < warp) before += x;
        all += x;
    }
    *incl = u + before;
    return all;
}

// Shares blockIdx.x * each .. + each - 1 of gridDim.x * each, into out[].
template <int NT>
__device__ __forceinline__ void take_shares(const PgTable &t, const PgSplit &sp, int *err, int64_t *scratch,
                                            int each, PgShare *out) {
    int64_t u = 0, incl, total = 0, last = 0;
    PgSeq q{};
    for (int base = 0; base < t.n_seqs; base += NT) {
        const int i = base + threadIdx.x;
        if (i < t.n_seqs) q = load_seq(t, i, err);
        u = i < t.n_seqs ? pg_seq_units(q, sp) : 0;
        last = block_scan<NT>(u, &incl, scratch);
        total += last;
    }
    const int parts = pg_parts(total, gridDim.x * each), x0 = blockIdx.x * each;
    if ((int)threadIdx.x < each) {
        const int x = x0 + threadIdx.x;
        const bool any = x < parts;
        PgShare s;
        s.w0 = any ? pg_first(total, parts, x) : 0;
        s.off = 0;
        s.total = total;
        s.count = any ? pg_first(total, parts, x + 1) - s.w0 : 0;
        s.seq = 0;
        s.parts = parts;
        s.s = PgSeq{0, 0, 0};
        out[threadIdx.x] = s;
    }
    __syncthreads();
    int64_t run = 0;
    for (int base = 0; x0 < parts && base < t.n_seqs; base += NT) {
        if (t.n_seqs > NT) {
            const int i = base + threadIdx.x;
            if (i < t.n_seqs) q = load_seq(t, i, err);
            u = i < t.n_seqs ? pg_seq_units(q, sp) : 0;
            last = block_scan<NT>(u, &incl, scratch);
        }
        for (int e = 0; u > 0 && e < each && x0 + e < parts; e++) {
            const int64_t w0 = pg_first(total, parts, x0 + e);
            if (run + incl - u <= w0 && w0 < run + incl) {
                out[e].seq = base + threadIdx.x;
                out[e].off = w0 - (run + incl - u);
                out[e].s = q;
            }
        }
        run += last;
    }
    __syncthreads();
}

// Sequences of the batch for a PgWalk.
struct Seqs {
    const PgTable &t;
    int *err;
    __device__ __forceinline__ PgSeq operator()(int i) const { return load_seq(t, i, err); }
    __device__ __forceinline__ int count() const { return t.n_seqs; }
};

// Say where this CTA's share begins, if that is inside an item (no workspace:
// the plan cuts no item).
__device__ __forceinline__ void note_cut(const PgWork &w, const PgSplit &sp, const PgShare &sh, const PgWalk &k) {
    if (!w.cut) return;
    PgCut c{};
    c.total = sh.total;
    c.parts = sh.parts;
    if (sh.count > 0 && k.u0 > 0) {
        c.wi = sh.w0 - k.u0;
        c.we = c.wi + k.units;
        c.head = k.head;
        c.row0 = k.s.first + k.item * sp.tok;
        c.rows = min(sp.tok, k.s.n - k.item * sp.tok) * sp.group;
    }
    w.cut[blockIdx.x] = c;
}

}  // namespace pg
}  // namespace ea
