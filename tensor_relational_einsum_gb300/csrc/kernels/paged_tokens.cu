// paged_tokens.cu -- attention over the paged cache for sequences with few
// query rows (tokens x grouped heads <= 32 to a key-value head): single
// tokens and short chunks.
//
// Every cached cell is used for at most 32 rows, so reading the pages bounds
// the kernel: 2 bytes (1 byte) of a cell against 64 flops, an eighth of what
// the tensor cores could do meanwhile.  What it needs is bytes in flight on
// every SM all the time, so
//   - the units of all items (a block of 64 or 128 keys of one key-value head)
//     are shared out evenly over the CTAs, whatever the lengths are (paged.h);
//   - a warp owns one or two runs of 16 keys of each block and loads them
//     itself with 16-byte cp.async into its part of a ring of blocks: no
//     barrier between warps inside an item, the next blocks' loads run across
//     items;
//   - 16 keys lie in one page (pages hold a multiple of 16 positions), so a
//     run needs one page number, read one block ahead.
// The products run on mma.sync m16n8k16: its 16-row tile is what a group of
// heads fills (a tcgen05 tile has 128 rows), and the accumulators stay in the
// warp's registers, next to the softmax.  The rows of an item are its tokens
// times its heads, token-major; each warp keeps its own running maximum, sum
// and output over its keys (the merge of (m, l, A) triples is associative),
// and the four are merged through shared memory at the end of a part.
//
// 8-bit cells become f16 in registers, two with one conversion (a code is an
// f16 value exactly), and that is all that is done to them: 4 integer
// instructions a pair, as the way to bf16 takes, bound this kernel at 3.5
// TB/s.  The scales go where there is less to multiply: K's to the columns of
// the scores (relative to the largest of the warp's keys, whose power joins
// that of the row's Q), V's to the probabilities.  What f16 lacks is range, so
//   - Q's rows are brought to [2^14, 2^15) by a power of two (a bf16 value is
//     an f16 value down to 2^-28 of its row's largest, and 2^-39 of it is the
//     step below);
//   - a probability enters as p * 2^7 * 2^(v - vref), v its key's scale and
//     vref the largest that the warp has met: 11 bits down to 2^-21 of the
//     row's largest term, steps of 2^-31 of it below that.
// Powers of two cost nothing in exactness: the f16 products are exact in fp32.
//
// Measured: 64 sequences of 8192 positions, 32 heads over 8 of 128: bf16
// 324-330 us, 6.5-6.6 TB/s (0.96-0.98 of the measured copy rate); 8-bit 185
// us, 5.86 TB/s (0.86; 36% of issue slots, the integer pipe at a third); head
// dim 64 bf16 0.93, 8-bit 0.58, where a block's fixed work weighs twice; four
// tokens each, 64 heads over 8 of 128 (two row tiles): bf16 0.96, 8-bit 0.54.
// A small call takes 6.5 us: a chain of reads (bounds, pages, cells), one
// block and the code itself.
#include "attn_common.cuh"
#include "paged_sched.cuh"

namespace ea {
namespace {

using namespace pg;
using attn::ex2;
using attn::pack_bf16;

constexpr int kThreads = 128;
constexpr float kLazy = 8.f;   // a running maximum moves when it is exceeded by this much (log2): P stays below 2^8

template <int D, bool E4M3, int MT>
struct Cfg {
    static constexpr int CELL = E4M3 ? 1 : 2;
    static constexpr int ROWB = D * CELL;               // bytes of a key's vector
    // A warp takes G runs of 16 keys of a block: two where a run is 4 KB at most, because the waits, votes and
    // shuffles of a block cost the same for both and the products of one run fill the latencies of the other's.
    static constexpr int G = ROWB == 256 ? 1 : 2;
    static constexpr int BLOCK = 64 * G;                // keys of a block
    static constexpr int TILE = 16 * G * ROWB;          // a warp's K (or V) of a block
    static constexpr int STAGE = 4 * 2 * TILE;          // a block
    static constexpr int S = STAGE == 16384 ? 5 : 3;
    static constexpr int SCALES = E4M3 ? 4 * 2 * 16 * G : 0;  // a stage's scale bytes
    static constexpr int Q_OFF = S * (STAGE + SCALES);  // two row tiles: Q's fragments, which registers cannot hold as well
    static constexpr int SMEM = Q_OFF + (MT == 2 ? MT * (D / 16) * 512 : 0);
    static constexpr int CTAS = 2;
};

// n bytes, and zeros up to 16.
__device__ __forceinline__ void cp16n(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a warp's tile.  bf16, and V's
// 8-bit cells: ldmatrix reads one chunk of 8 rows, which must lie in 8
// different 16-byte columns of 128 bytes.  K's 8-bit cells: 8 lanes read 4
// chunks of 2 rows.
template <int ROWB, bool K8>
__device__ __forceinline__ int chunk_at(int r, int c) {
    if constexpr (K8) return r * ROWB + ((ROWB == 128 ? c ^ ((r & 1) << 2) : c) << 4);
    else if constexpr (ROWB >= 128) return r * ROWB + ((c ^ (r & 7)) << 4);
    else return r * ROWB + ((c ^ ((r >> 1) & 3)) << 4);
}

// The loads of a warp's keys, block after block of the CTA's share.
template <int D, bool E4M3, int MT>
struct Loader {
    using C = Cfg<D, E4M3, MT>;
    PgWalk w;
    int keys, off;    // keys of a block; this warp's first one
    int block, last;  // next block of the part, and its first one beyond
    int end;          // keys of the item
    int page[C::G];   // pages of this warp's runs of the next block, not checked yet: nothing waits for them here
    bool more;

    __device__ __forceinline__ void enter(const PgAttn &p, const PgSplit &sp) {
        const int per = sp.kt / keys;
        while (w.left > 0) {
            end = pg_item_end(w.s, sp, w.item);
            block = w.u0 * per;
            last = min((w.u0 + w.part()) * per, (end + keys - 1) / keys);
            if (block < last) break;
            w.step(w.part(), sp, Seqs{p.t, p.err});
        }
        more = w.left > 0;
        look(p);
    }
    __device__ __forceinline__ void look(const PgAttn &p) {
#pragma unroll
        for (int g = 0; g < C::G; g++) {
            const int key0 = block * keys + off + g * 16;
            page[g] = more && key0 < end ? __ldg(p.t.pages + (int64_t)w.seq * p.t.page_stride + (key0 >> p.c.page_log2)) : 0;
        }
    }
    __device__ __forceinline__ void issue(const PgAttn &p, const PgSplit &sp, uint32_t stage, uint32_t scales, int warp,
                                          int lane) {
        if (!more) return;
        constexpr int CPR = C::ROWB / 16, IT = 16 * C::ROWB / 512;  // chunks of a row; copies of a lane and run
        const uint32_t ks = stage + warp * 2 * C::TILE, vs = ks + C::TILE;
#pragma unroll
        for (int g = 0; g < C::G; g++) {
            const int key0 = block * keys + off + g * 16, nv = end - key0;  // valid keys: the rest becomes zero
            if (C::G == 1 && nv <= 0) break;
            const int64_t vec = pg_vec(p.c, check_page(page[g], p.c.n_pages, p.err), w.head, key0 & ((1 << p.c.page_log2) - 1));
            const char *kp = p.c.k + vec * C::ROWB, *vp = p.c.v + vec * C::ROWB;
            if (nv >= 16) {
#pragma unroll
                for (int i = 0; i < IT; i++) {
                    const int x = i * 32 + lane, r = x / CPR, c = x % CPR;
                    cp16(ks + chunk_at<C::ROWB, E4M3>(g * 16 + r, c), kp + x * 16);
                    cp16(vs + chunk_at<C::ROWB, false>(g * 16 + r, c), vp + x * 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < IT; i++) {
                    const int x = i * 32 + lane, r = x / CPR, c = x % CPR, n = r < nv ? 16 : 0;
                    cp16n(ks + chunk_at<C::ROWB, E4M3>(g * 16 + r, c), kp + x * 16, n);
                    cp16n(vs + chunk_at<C::ROWB, false>(g * 16 + r, c), vp + x * 16, n);
                }
            }
            // a warp's scale bytes: K's runs, then V's
            if (E4M3 && lane < 2)
                cp16n(scales + (warp * 2 + lane) * 16 * C::G + g * 16, (lane ? p.c.vs : p.c.ks) + vec, max(0, min(16, nv)));
        }
        if (++block < last) {
            look(p);
        } else {
            w.step(w.part(), sp, Seqs{p.t, p.err});
            enter(p, sp);
        }
    }
};

template <int D, bool E4M3, int MT>
__global__ void __launch_bounds__(kThreads, Cfg<D, E4M3, MT>::CTAS)
cache_tokens_kernel(const __grid_constant__ PgAttn p, const __grid_constant__ PgSplit sp,
                    const __grid_constant__ PgWork ws) {
    using C = Cfg<D, E4M3, MT>;
    constexpr int KS = D / 16, NT = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PgShare shares[4];
    __shared__ int64_t scan[kThreads / 32];
    __shared__ float4 s_ml[4][16 * MT];  // a warp's reference maximum, sum, maximum of its rows; its vref
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    let_next_start();
    const bool solo = MT == 1 && sp.solo != 0;
    take_shares<kThreads>(p.t, sp, p.err, scan, solo ? 4 : 1, shares);
    const PgShare &share = shares[solo ? warp : 0];
    Loader<D, E4M3, MT> ld;
    ld.w.begin(share, sp);
    PgWalk w = ld.w;
    if (threadIdx.x == 0) note_cut(ws, sp, share, w);
    if (share.count == 0) {
        wait_for_previous();
        return;
    }
    const int keys = solo ? C::BLOCK / 4 : C::BLOCK;  // of a block, and this warp's first one
    const int off = solo ? 0 : warp * 16 * C::G;
    ld.keys = keys;
    ld.off = off;
    ld.enter(p, sp);
#pragma unroll 1  // one copy of the code: small calls wait for their instructions
    for (int s = 0; s < C::S - 1; s++) {
        ld.issue(p, sp, base + s * C::STAGE, base + C::S * C::STAGE + s * C::SCALES, warp, lane);
        cp_commit();
    }
    int slot = 0;  // ring slot of the next block to compute
    bool first_part = true;
    const float c = p.scale_log2;
    const int per = sp.kt / keys;

    while (w.left > 0) {
        const int np = w.part();
        const int end = pg_item_end(w.s, sp, w.item);
        const int b0 = w.u0 * per, b1 = min((w.u0 + np) * per, (end + keys - 1) / keys);
        const int tok0 = w.item * sp.tok, nrows = min(sp.tok, w.s.n - tok0) * sp.group;
        // Q's fragments, and the keys that each of the thread's rows keeps
        uint32_t q[MT][KS][4];  // (a row tile alone; else written to shared memory at once)
        int qe[MT][2];    // e4m3: the row's Q is 2^-qe times its f16 values
        int lim[MT][2];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = m * 16 + h * 8 + gid, tok = tok0 + r / sp.group;
                const bool in = r < nrows;
                // rows without a token (Q = 0) keep all: they must not make the others look at every key
                lim[m][h] = !in ? INT32_MAX : sp.causal ? max(0, min(w.s.len, w.s.len - w.s.n + tok + 1)) : w.s.len;
                const char *src = p.q + ((int64_t)(w.s.first + (in ? tok : 0)) * p.qheads + w.head * sp.group +
                                         (in ? r % sp.group : 0)) * D * 2;
                if constexpr (E4M3) {
                    // logical k = (2 t, 2 t + 1, 2 t + 8, 2 t + 9) of step 4 x + s: columns 64 x + 16 t + 4 s + (0, 1, 2, 3)
                    uint32_t u[D / 64][8] = {};
                    uint32_t big = 0;  // the row's largest magnitude: bf16 bits
#pragma unroll
                    for (int x = 0; x < D / 64; x++) {
                        if (in) {
                            const uint4 *g = reinterpret_cast<const uint4 *>(src + (64 * x + 16 * tig) * 2);
                            *reinterpret_cast<uint4 *>(u[x]) = __ldg(g);
                            *reinterpret_cast<uint4 *>(u[x] + 4) = __ldg(g + 1);
                        }
#pragma unroll
                        for (int i = 0; i < 8; i++) big = __vmaxu2(big, u[x][i] & 0x7fff7fffu);
                    }
                    big = max(big >> 16, big & 0xffffu);
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    const int e = big == 0 || big >= 0x7f80u ? 0 : min(126, 14 - ((int)(big >> 7) - 127));
                    const float up = pow2(e);
                    qe[m][h] = e;
#pragma unroll
                    for (int x = 0; x < D / 64; x++)
#pragma unroll
                        for (int s = 0; s < 4; s++)
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const uint32_t w = u[x][2 * s + i];
                                q[m][4 * x + s][h + 2 * i] =
                                    pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                            }
                } else {
#pragma unroll
                    for (int s = 0; s < KS; s++)
#pragma unroll
                        for (int x = 0; x < 2; x++)
                            q[m][s][h + 2 * x] = in ? __ldg(reinterpret_cast<const uint32_t *>(src + (16 * s + 8 * x + 2 * tig) * 2)) : 0u;
                }
            }
        uint4 *q_sm = reinterpret_cast<uint4 *>(smem + C::Q_OFF) + lane;
        if constexpr (MT == 2) {  // every warp has made all fragments; each stores a quarter
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int x = 0; x < KS; x++)
                    if ((x & 3) == warp) q_sm[(m * KS + x) * 32] = make_uint4(q[m][x][0], q[m][x][1], q[m][x][2], q[m][x][3]);
            __syncthreads();
        }
        // A fragment of step x of row tile m
        auto qf = [&](int m, int x, uint32_t *f) {
            if constexpr (MT == 2) {
                const uint4 v = q_sm[(m * KS + x) * 32];
                f[0] = v.x;
                f[1] = v.y;
                f[2] = v.z;
                f[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) f[i] = q[m][x][i];
            }
        };
        float o[MT][NT][4] = {};
        float mref[MT][2], mmax[MT][2], l[MT][2];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                mref[m][h] = mmax[m][h] = -INFINITY;
                l[m][h] = 0.f;
            }
        int least = INT32_MAX;  // keys that all of the thread's rows keep
#pragma unroll
        for (int m = 0; m < MT; m++) least = min(least, min(lim[m][0], lim[m][1]));
        int vref = 0;  // e4m3: the accumulators are in units of 2^(vref - 127 - 7)

        for (int b = b0; b < b1; b++) {
            __syncwarp();  // every lane has read the slot that is filled next
            const int fill = slot == 0 ? C::S - 1 : slot - 1;
            ld.issue(p, sp, base + fill * C::STAGE, base + C::S * C::STAGE + fill * C::SCALES, warp, lane);
            cp_commit();
            cp_wait<C::S - 1>();
            __syncwarp();
            const int key0 = b * keys + off;
            if (key0 < end) {
                constexpr int N = 2 * C::G;  // runs of 8 keys
                const uint32_t kt = base + slot * C::STAGE + warp * 2 * C::TILE, vt = kt + C::TILE;
                float s[MT][N][4] = {};
                if constexpr (E4M3) {
                    const uint8_t *ksm = smem + slot * C::STAGE + warp * 2 * C::TILE;
#pragma unroll
                    for (int x = 0; x < D / 64; x++) {
                        uint4 v[N];
#pragma unroll
                        for (int n = 0; n < N; n++)
                            v[n] = *reinterpret_cast<const uint4 *>(ksm + chunk_at<C::ROWB, true>(n * 8 + gid, 4 * x + tig));
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            uint32_t f[MT][4];
#pragma unroll
                            for (int m = 0; m < MT; m++) qf(m, 4 * x + y, f[m]);
#pragma unroll
                            for (int n = 0; n < N; n++) {
                                uint32_t lo, hi;
                                to_f16(y == 0 ? v[n].x : y == 1 ? v[n].y : y == 2 ? v[n].z : v[n].w, lo, hi);
#pragma unroll
                                for (int m = 0; m < MT; m++) mma16(s[m][n], f[m], lo, hi);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < KS; x++) {
                        uint32_t f[MT][4];
#pragma unroll
                        for (int m = 0; m < MT; m++) qf(m, x, f[m]);
#pragma unroll
                        for (int g = 0; g < C::G; g++) {
                            uint32_t u[4];
                            ldsm4(kt + chunk_at<C::ROWB, false>(g * 16 + (lane >> 4) * 8 + (lane & 7), 2 * x + ((lane >> 3) & 1)), u);
#pragma unroll
                            for (int m = 0; m < MT; m++) {
                                mma(s[m][2 * g], f[m], u[0], u[1]);
                                mma(s[m][2 * g + 1], f[m], u[2], u[3]);
                            }
                        }
                    }
                }
                float vsc[N][2];    // what V's scales make of the probabilities
                float shift = 1.f;  // what a new vref makes of the accumulators
                int kref = 0;       // the largest scale byte of the warp's keys of K: the scores' unit
                if constexpr (E4M3) {
                    // a lane's key: its scale bytes (0 beyond the end), turned into factors once and passed around.  NaN
                    // vectors (255) move neither reference.
                    const uint8_t *sc = smem + C::S * C::STAGE + slot * C::SCALES + warp * 32 * C::G;
                    const int mine = C::G == 2 ? lane : lane & 15;
                    const uint32_t kb = sc[mine], vb = sc[16 * C::G + mine];
                    const int vmax = (int)__reduce_max_sync(0xffffffffu, vb == 255u ? 0u : vb);
                    kref = (int)__reduce_max_sync(0xffffffffu, kb == 255u ? 0u : kb);
                    if (vmax > vref) {
                        shift = pow2(vref - vmax);
                        vref = vmax;
                    }
                    const float kf = kb == 255u ? __uint_as_float(0x7fffffffu) : pow2((int)kb - kref);
                    const float vf = vb == 255u ? __uint_as_float(0x7fffffffu) : pow2((int)vb - vref + 7);
#pragma unroll
                    for (int n = 0; n < N; n++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const float k0 = __shfl_sync(0xffffffffu, kf, n * 8 + 2 * tig + i);
                            vsc[n][i] = __shfl_sync(0xffffffffu, vf, n * 8 + 2 * tig + i);
#pragma unroll
                            for (int m = 0; m < MT; m++)
#pragma unroll
                                for (int h = 0; h < 2; h++) s[m][n][2 * h + i] *= k0;
                        }
                }
                const bool cut = __any_sync(0xffffffffu, least < key0 + 16 * C::G);  // some row drops some key
                uint32_t pf[MT][C::G][4];
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    float mx[2], cr[2];  // cr: what makes exponents (log2) of the products
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (cut) {
                            const int keep = lim[m][h] - key0 - 2 * tig;  // of the thread's keys 0, 1, 8, 9, ..
#pragma unroll
                            for (int n = 0; n < N; n++)
#pragma unroll
                                for (int e = 0; e < 2; e++)
                                    if (n * 8 + e >= keep) s[m][n][2 * h + e] = -INFINITY;
                        }
                        mx[h] = -INFINITY;
#pragma unroll
                        for (int n = 0; n < N; n++) mx[h] = fmaxf(mx[h], fmaxf(s[m][n][2 * h], s[m][n][2 * h + 1]));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                        cr[h] = c;
                        if constexpr (E4M3) {
                            // K's power and Q's in one: each alone may lie beyond fp32's where the other brings it back.
                            // No factor is 0, which would make NaN of a dropped score: below 2^-126 the exponentials take
                            // 2^-126 (scores of less than 2^-95 either way), and the maximum a second factor.
                            const int e = kref - 127 - qe[m][h];
                            const float ft = pow2(min(127, max(e, -126)));
                            mx[h] = mx[h] * ft * pow2(min(0, max(e + 126, -126)));
                            cr[h] = fmaxf(c * ft, 1.2e-38f);
                        }
                        mmax[m][h] = fmaxf(mmax[m][h], mx[h]);
                    }
                    bool move = false;
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        move |= mx[h] != -INFINITY && (mref[m][h] == -INFINITY || (mx[h] - mref[m][h]) * c > kLazy);
                    if constexpr (E4M3) move |= shift != 1.f;
                    if (__any_sync(0xffffffffu, move)) {
                        float f[2];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const float to = mmax[m][h];
                            f[h] = mref[m][h] == -INFINITY ? 0.f : ex2((mref[m][h] - to) * c);
                            mref[m][h] = to;
                            l[m][h] *= f[h];
                            if constexpr (E4M3) f[h] *= shift;
                        }
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            o[m][n][0] *= f[0];
                            o[m][n][1] *= f[0];
                            o[m][n][2] *= f[1];
                            o[m][n][3] *= f[1];
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float nb = mref[m][h] == -INFINITY ? 0.f : -mref[m][h] * c;
#pragma unroll
                        for (int n = 0; n < N; n++) {
                            float e0 = ex2(fmaf(s[m][n][2 * h], cr[h], nb)), e1 = ex2(fmaf(s[m][n][2 * h + 1], cr[h], nb));
                            l[m][h] += e0 + e1;
                            if constexpr (E4M3) {
                                e0 *= vsc[n][0];
                                e1 *= vsc[n][1];
                            }
                            pf[m][n >> 1][h + 2 * (n & 1)] = E4M3 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
                        }
                    }
                }
                if constexpr (E4M3) {
#pragma unroll
                    for (int x = 0; x < D / 32; x++)
#pragma unroll
                        for (int g = 0; g < C::G; g++) {
                            uint32_t u[4];
                            ldsm4_t(vt + chunk_at<C::ROWB, false>(g * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * x + (lane >> 4)), u);
#pragma unroll
                            for (int y = 0; y < 2; y++) {
                                // keys (2 t, 2 t + 1) of two neighbouring columns: by column, then to f16
                                uint32_t e0, e1, d0, d1;
                                to_f16(__byte_perm(u[2 * y], 0, 0x3120), e0, d0);
                                to_f16(__byte_perm(u[2 * y + 1], 0, 0x3120), e1, d1);
#pragma unroll
                                for (int m = 0; m < MT; m++) {
                                    mma16(o[m][4 * x + 2 * y], pf[m][g], e0, e1);
                                    mma16(o[m][4 * x + 2 * y + 1], pf[m][g], d0, d1);
                                }
                            }
                        }
                } else {
#pragma unroll
                    for (int x = 0; x < D / 16; x++)
#pragma unroll
                        for (int g = 0; g < C::G; g++) {
                            uint32_t u[4];
                            ldsm4_t(vt + chunk_at<C::ROWB, false>(g * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * x + (lane >> 4)), u);
#pragma unroll
                            for (int m = 0; m < MT; m++) {
                                mma(o[m][2 * x], pf[m][g], u[0], u[1]);
                                mma(o[m][2 * x + 1], pf[m][g], u[2], u[3]);
                            }
                        }
                }
            }
            slot = slot + 1 == C::S ? 0 : slot + 1;
        }

#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 1);
                l[m][h] += __shfl_xor_sync(0xffffffffu, l[m][h], 2);
            }
        if (solo) {
            const float unit = E4M3 ? ldexpf(1.f, vref - 127 - 7) : 1.f;
            // ---- the warp has the item to itself
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int r = m * 16 + h * 8 + gid;
                    if (r >= nrows) continue;
                    const int64_t at = (int64_t)(w.s.first + tok0 + r / sp.group) * p.qheads + w.head * sp.group + r % sp.group;
                    // 1 / l first, then the unit: their product can lie below fp32's normal numbers where the result does not
                    const float sum = l[m][h], inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
                    if constexpr (E4M3) {
#pragma unroll
                        for (int x = 0; x < D / 16; x++) {
                            const float *a = o[m][2 * x], *d = o[m][2 * x + 1];
                            *reinterpret_cast<uint2 *>(p.o + (at * D + 16 * x + 4 * tig) * 2) = make_uint2(
                                pack_bf16(a[2 * h] * inv * unit, d[2 * h] * inv * unit),
                                pack_bf16(a[2 * h + 1] * inv * unit, d[2 * h + 1] * inv * unit));
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NT; n++)
                            *reinterpret_cast<uint32_t *>(p.o + (at * D + 8 * n + 2 * tig) * 2) =
                                pack_bf16(o[m][n][2 * h] * inv, o[m][n][2 * h + 1] * inv);
                    }
                    if (p.m_out && tig == 0) {
                        const float f = mref[m][h] == -INFINITY ? 0.f : ex2((mref[m][h] - mmax[m][h]) * c);
                        p.m_out[at] = mmax[m][h] * p.scale;
                        p.l_out[at] = sum * f;
                    }
                }
            w.step(np, sp, Seqs{p.t, p.err});
            continue;
        }

        // ---- the four warps' results: scaled to the item's maximum and summed through shared memory.  The scratch is
        // the ring slot that was computed last: it is refilled after this part's barriers.
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                if (tig == 0)
                    s_ml[warp][m * 16 + h * 8 + gid] = make_float4(mref[m][h], l[m][h], mmax[m][h], (float)vref);
        const bool whole = w.u0 == 0 && np == w.units;
        const int64_t part = 2 * (int64_t)blockIdx.x + (first_part ? 0 : 1);
        static_assert(4 * 16 * D * 4 <= C::STAGE, "a slot holds the four warps' rows");
        float *scratch = reinterpret_cast<float *>(smem + (slot == 0 ? C::S - 1 : slot - 1) * C::STAGE);
        const int row = threadIdx.x / 8, col = (threadIdx.x % 8) * 4;
#pragma unroll
        for (int m = 0; m < MT; m++) {
            __syncthreads();  // the slot (or the scratch of the pass before) has been read by every warp
            float *mine = scratch + warp * 16 * D;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = h * 8 + gid, sw = (r << 3) & (D - 8);
                if constexpr (E4M3) {
#pragma unroll
                    for (int x = 0; x < D / 16; x++) {
                        const int n = 2 * x;
                        *reinterpret_cast<float4 *>(mine + r * D + ((16 * x + 4 * tig) ^ sw)) =
                            make_float4(o[m][n][2 * h], o[m][n + 1][2 * h], o[m][n][2 * h + 1], o[m][n + 1][2 * h + 1]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n++)
                        *reinterpret_cast<float2 *>(mine + r * D + ((8 * n + 2 * tig) ^ sw)) =
                            make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
                }
            }
            __syncthreads();
            const int r = m * 16 + row;
            float f[4], top = -INFINITY, sum = 0.f, vtop = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                top = fmaxf(top, s_ml[i][r].z);
                if constexpr (E4M3) vtop = fmaxf(vtop, s_ml[i][r].w);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float4 v = s_ml[i][r];
                f[i] = v.x == -INFINITY ? 0.f : ex2((v.x - top) * c);
                sum = fmaf(f[i], v.y, sum);
                if constexpr (E4M3) f[i] *= pow2((int)(v.w - vtop));  // to the largest of the warps' units
            }
            if (r < nrows) {
                const int64_t at = ((int64_t)(w.s.first + tok0 + r / sp.group) * p.qheads + w.head * sp.group + r % sp.group);
                const float inv = !whole ? 1.f : sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
                const float unit = E4M3 ? ldexpf(1.f, (int)vtop - 127 - 7) : 1.f;
#pragma unroll
                for (int x = 0; x < D / 32; x++) {
                    const int d = 32 * x + col;
                    float a[4] = {};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float4 v = *reinterpret_cast<const float4 *>(scratch + (i * 16 + row) * D + (d ^ ((row << 3) & (D - 8))));
                        a[0] = fmaf(f[i], v.x, a[0]);
                        a[1] = fmaf(f[i], v.y, a[1]);
                        a[2] = fmaf(f[i], v.z, a[2]);
                        a[3] = fmaf(f[i], v.w, a[3]);
                    }
                    if constexpr (E4M3) {
#pragma unroll
                        for (int i = 0; i < 4; i++) a[i] *= unit;
                    }
                    if (whole) {
                        *reinterpret_cast<uint2 *>(p.o + (at * D + d) * 2) =
                            make_uint2(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv));
                    } else {
                        *reinterpret_cast<float4 *>(ws.acc + (part * 16 * MT + r) * D + d) =
                            make_float4(a[0], a[1], a[2], a[3]);
                    }
                }
                if (threadIdx.x % 8 == 0) {
                    if (!whole) ws.ml[part * 16 * MT + r] = make_float2(top, sum);
                    else if (p.m_out) {
                        p.m_out[at] = top * p.scale;
                        p.l_out[at] = sum;
                    }
                }
            }
        }
        __syncthreads();  // the scratch and s_ml are free
        first_part = false;
        w.step(np, sp, Seqs{p.t, p.err});
    }
    cp_wait<0>();
    wait_for_previous();
}

template <int D, bool E4M3, int MT>
cudaError_t launch(const PgAttn &p, const PgPlan &pl, const PgWork &w, cudaStream_t st, bool early) {
    using C = Cfg<D, E4M3, MT>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(cache_tokens_kernel<D, E4M3, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_after(cache_tokens_kernel<D, E4M3, MT>, dim3(pl.ctas), kThreads, C::SMEM, st, early, p, pl.split, w);
}

template <int D, bool E4M3>
cudaError_t launch_m(const PgAttn &p, const PgPlan &pl, const PgWork &w, cudaStream_t st, bool early) {
    return pl.rows == 16 ? launch<D, E4M3, 1>(p, pl, w, st, early) : launch<D, E4M3, 2>(p, pl, w, st, early);
}

}  // namespace

PgPlan plan_cache_tokens(const PgTable &t, const PgPool &c, int group, int causal, int num_sms) {
    PgPlan pl{};
    if (group > kPgTokenRows || t.rows == 0) return pl;
    pl.rows = (int64_t)t.max_new * group <= 16 ? 16 : 32;
    PgSplit &sp = pl.split;
    sp.heads = c.heads;
    sp.group = group;
    sp.tok = pl.rows / group;
    sp.causal = causal;
    sp.min_rows = 1;
    sp.max_rows = pl.rows;
    // Short sequences are not cut: another block adds less than the merge's launch.  The table's width says which they
    // are: the lengths are known on the device only.
    const int64_t longest = t.cap;
    sp.kt = longest <= 512 ? 512 : c.fmt == EA_CACHE_E4M3 || c.dim == 64 ? 128 : 64;  // a block
    const int64_t units = (longest + sp.kt - 1) / sp.kt * t.n_seqs * c.heads;
    // Many short sequences: a warp an item, without barriers or a merge between warps.
    sp.solo = sp.kt == 512 && pl.rows == 16 && (int64_t)t.n_seqs * c.heads >= 4 * (int64_t)num_sms;
    pl.ctas = (int)std::min<int64_t>(sp.solo ? (units + 3) / 4 : units, (int64_t)num_sms * 2);
    pl.bytes = units > t.n_seqs * (int64_t)c.heads ? pg_work_bytes(pl.ctas, pl.rows, c.dim) : 0;  // 0: a unit is an item
    return pl;
}

cudaError_t launch_cache_tokens(const PgAttn &p, const PgPlan &pl, const PgWork &w, bool early, cudaStream_t st) {
    if (p.c.fmt == EA_CACHE_E4M3)
        return p.c.dim == 64 ? launch_m<64, true>(p, pl, w, st, early) : launch_m<128, true>(p, pl, w, st, early);
    return p.c.dim == 64 ? launch_m<64, false>(p, pl, w, st, early) : launch_m<128, false>(p, pl, w, st, early);
}

}  // namespace ea
