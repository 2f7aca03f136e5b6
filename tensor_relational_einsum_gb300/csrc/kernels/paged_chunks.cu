// paged_chunks.cu -- attention over the paged cache on the sm_103a tensor
// cores, for sequences with more query rows than the token kernel takes:
// chunks of a prompt, whole prompts, many grouped heads.
//
// The rows of an item are 2 x `tpt` tokens times the heads of a group,
// token-major, in two tiles of up to 128 rows that share their key tiles
// (128 keys): each K and V tile is read once for 256 rows, which keeps the
// L2 traffic at half of what the products could take in.  The units of all
// items (a key tile of an item) are shared out evenly over the CTAs, one CTA
// per SM, whatever the lengths are; an item that falls into several CTAs is
// merged from its partial (m, l, A) triples.
//
// Key tiles come page by page.  bf16 pages are copied by TMA straight into
// the swizzled operand tiles (a box of up to 128 positions x 64 columns: a
// page is contiguous for a head, so a page is one box per 64 columns).
// 8-bit pages are copied with bulk copies into raw tiles and rewritten as f16
// operands by a warpgroup of their own: a conversion and a product for two
// codes (twice as many integer instructions lead to bf16).  f16's range is
// kept by powers of two, so that the operands are exact: K's vectors are
// brought to the largest scale of their tile, V's to the largest of the part
// so far (exact down to 2^-21 of it), Q's rows to [2^14, 2^15), the
// probabilities to 2^7.  All of these are one number a tile or a row to the
// softmax.  (Scales left to the softmax, a number a key, cost it 64 broadcast
// reads of shared memory a row and tile: 6200 cycles a tile at head dim 64,
// which takes 3800 this way.)  From 256 rows of a sequence on the pages are
// expanded to bf16 first (paged_expand.cu), and this kernel reads those.
//
// What bounds it: shared memory.  The products of 256 rows with a key tile
// take 2048 cycles of the tensor pipe at head dim 128 and read 192 KB of
// operands, to which the copies add 64 KB: 2000 cycles at 128 bytes a cycle.
// They get in each other's way: a tile takes 3080 cycles, 2820 with the
// softmax left out, which itself takes 1220 behind each product.  2048 tokens
// after 14336, 32 heads over 8: 395 us, 1300 TFLOP/s, 0.68 of the measured
// bf16 rate.  At head dim 64 the softmax is as long as the products (317 us
// there, 0.42).  Short items pay for a part's ends, about 5000 cycles: prompts
// of 2048 tokens with 32 heads of their own, 0.39.
//
// Keys at and beyond the sequence's end lie in the last tile only.  Their
// scores are dropped by position whatever they are; the second product stops
// at the next multiple of 16 keys, and the up to 15 rows of V before it are
// cleared in shared memory (a probability of 0 times a stale NaN is NaN).
//
// Roles (one CTA per SM; bf16: 384 threads, e4m3: 512):
//   warps 0-3, 4-7  softmax of tile X = 0, 1: a query row per thread (TMEM
//              lane = row), its 128 scores in registers: mask by position,
//              row maximum, p = 2^(c s - c m), row sum, P as 16 bits over the
//              scores; A is rescaled in TMEM when the reference maximum is
//              exceeded by more than 2^8 (P fits f16 then, and A is at
//              most 2^8 times what it is with the true maximum: the limit on
//              V is that of the token kernel); at the part's end A / l to the
//              output, or (m, l, A) to the workspace.
//   warp 8     copies: Q tiles; K and V pages (or the raw tiles).
//   warp 9     TMEM and MMA issue: per key tile and X, A_X (+)= P_X V, then
//              S_X = Q_X K^T of the next key tile, so that one tile's products
//              run while the other's softmax does.
//   warp 10    hands the CTA's parts of items to the others through a ring.
//   warps 12-15 (e4m3) rewrite the raw tiles and Q as f16, 32 rows a warp.
// Every mbarrier wait is bounded (2 s); on time-out the kernel raises the
// device error word, all roles leave their loops, the copies and MMAs in
// flight are waited for and TMEM is freed before the CTA exits.
#include "attn_common.cuh"
#include "paged_sched.cuh"
#include "tc_common.cuh"

namespace ea {
namespace {

using namespace tc;
using namespace attn;
using namespace pg;

constexpr int kRows = 128;        // rows of a tile (TMEM lanes)
constexpr int kKeys = 128;        // keys of a key tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;   // S_0 [0, 128), S_1 [128, 256), A_0 [256, 256 + D), A_1 [256 + D, ..)
constexpr float kLazy = 8.f;      // a running maximum moves when it is exceeded by this much (log2)
constexpr int kParts = 4;         // ring of parts
constexpr int kMaxStages = 4;
constexpr int kWhole = 1024;      // sequences of up to so many positions are not cut

// Register split (setmaxnreg): the softmax threads keep a row of 128 scores.
// The shares add up to the launch's registers exactly.
template <bool E4M3>
struct Regs {
    static constexpr int THREADS = E4M3 ? 512 : 384;
    static constexpr int LAUNCH = E4M3 ? 128 : 168;
    static constexpr int SOFTMAX = E4M3 ? 176 : 208;
    static constexpr int CTL = E4M3 ? 72 : 88;
    static constexpr int CONV = 88;
    static_assert(128 * (2 * SOFTMAX + CTL + (E4M3 ? CONV : 0)) <= THREADS * LAUNCH, "register split");
};

// The part of an item that a CTA works on, as warp 10 hands it to the others.
struct Part {
    int n[2];       // key tiles of X = 0, 1 (X runs the part's first n[X] tiles)
    int tiles;      // the larger of them; -1: no more parts
    int u0;         // first key tile
    int tok0;       // the item's first token (within the sequence's new tokens)
    int end;        // keys of the item
    int whole, seq, head;
    int row0;       // dense row of token tok0
    int ntok;       // the sequence's tokens from tok0 on
    int pos0, len;  // position of token tok0, length of the sequence
};

__device__ __forceinline__ Part part_of(const PgWalk &w, const PgSplit &sp) {
    Part q;
    const int np = w.part(), half = sp.tok / 2;
    q.u0 = w.u0 * (sp.kt / kKeys);
    q.whole = w.u0 == 0 && np == w.units;
    q.tok0 = w.item * sp.tok;
    q.end = pg_item_end(w.s, sp, w.item);
    q.seq = w.seq;
    q.head = w.head;
    q.row0 = w.s.first + q.tok0;
    q.ntok = w.s.n - q.tok0;
    q.len = w.s.len;
    q.pos0 = w.s.len - w.s.n + q.tok0;
    const int tiles = (q.end + kKeys - 1) / kKeys, u1 = q.u0 + np * (sp.kt / kKeys);
    const bool two = half < q.ntok;
    // keys of tile 0: up to its own last token's
    const int e0 = two && sp.causal ? max(0, q.pos0 + half) : q.end;
    q.n[0] = max(0, min(u1, (e0 + kKeys - 1) / kKeys) - q.u0);
    q.n[1] = two ? max(0, min(u1, tiles) - q.u0) : 0;
    q.tiles = max(q.n[0], q.n[1]);
    return q;
}

struct Ctl {
    uint64_t q_full[2], q_empty[2], q_ready[2];
    uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t raw_full[2][2], raw_empty[2][2];  // of K, of V
    uint64_t s_full[2], p_full[2], o_fin[2];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t top_full[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    PgShare share;
    int64_t scan[16];
    int2 top[2][4];          // e4m3: the largest scale bytes of a tile's K and V, by warp (two tiles' worth)
    Part part[kParts];
};

// e4m3: what a tile's operands were brought to.  K = f16 value * 2^(k - 133),
// V = f16 value * 2^(v - 133).
struct Refs {
    int k, v;
};

template <int D, bool E4M3>
struct Cfg {
    static constexpr int CH = D / 64;                       // 64-column (128-byte) chunks of the head dim
    static constexpr int TILE = kRows * D * 2;
    // Rings of K and of V tiles, each freed by its own product: K of tile t + 2 can arrive from the end of S(t) on and
    // is needed for S(t + 2), more than a tile's time, which is longer than a copy takes.  (With K and V freed
    // together there was half of that, and a tile took 4000 cycles instead of 3000.)  At D = 64 a tile takes half the
    // time, and there is room for four.
    static constexpr int ST = D == 64 ? 4 : 2;
    static constexpr int K_OFF = 2 * TILE;                  // Q_0, Q_1, then K of each stage, V of each stage
    static constexpr int V_OFF = K_OFF + ST * TILE;
    static constexpr int RAW_OFF = V_OFF + ST * TILE;
    static constexpr int NR = D == 64 ? 2 : 1;              // e4m3: raw tiles of K, and of V
    static constexpr int RAW = E4M3 ? kKeys * D : 0;
    static constexpr int RSC_OFF = RAW_OFF + 2 * NR * RAW;  // the scale bytes of a raw K's tile: K's, V's
    // A tile's references are read until its P is written.  K of tile t + 2 ST waits for S(t + ST), which is behind P
    // of tile t + ST - 1, so a ring of 2 ST is safe; Q's scales by part and by the part before.
    static constexpr int SC_OFF = RSC_OFF + (E4M3 ? NR * 2 * kKeys : 0);
    static constexpr int QS_OFF = SC_OFF + (E4M3 ? 2 * ST * (int)sizeof(Refs) : 0);
    static constexpr int CTL_OFF = QS_OFF + (E4M3 ? 2 * 2 * kRows : 0);
    static constexpr int SMEM = 1024 + CTL_OFF + (int)sizeof(Ctl);
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Regs<E4M3>::THREADS, 1)
cache_chunks_kernel(const __grid_constant__ PgAttn p, const __grid_constant__ PgSplit sp,
                    const __grid_constant__ PgWork ws, const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = Cfg<D, E4M3>;
    using R = Regs<E4M3>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::CTL_OFF);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    volatile int *abort = &ctl->abort;
    const Seqs seqs{p.t, p.err};
    const int half_tok = sp.tok / 2;      // tokens of a tile
    const int half_rows = half_tok * sp.group;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; b++) {
            mbar_init(&ctl->q_full[b], 1);
            mbar_init(&ctl->q_empty[b], 1);
            mbar_init(&ctl->q_ready[b], 4);
            mbar_init(&ctl->s_full[b], 1);
            mbar_init(&ctl->p_full[b], 4);
            mbar_init(&ctl->o_fin[b], 1);
        }
        for (int b = 0; b < C::ST; b++) {
            mbar_init(&ctl->k_full[b], E4M3 ? 4 : 1);
            mbar_init(&ctl->k_empty[b], 1);
            mbar_init(&ctl->v_full[b], E4M3 ? 4 : 1);
            mbar_init(&ctl->v_empty[b], 1);
        }
        for (int b = 0; b < 4; b++) {
            mbar_init(&ctl->raw_full[b >> 1][b & 1], 1);
            mbar_init(&ctl->raw_empty[b >> 1][b & 1], 4);
        }
        for (int b = 0; b < kParts; b++) {
            mbar_init(&ctl->part_full[b], 1);
            mbar_init(&ctl->part_empty[b], E4M3 ? 14 : 10);  // the warps that read parts
        }
        for (int b = 0; b < 2; b++) mbar_init(&ctl->top_full[b], 4);
        mbar_init(&ctl->mma_done, 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 9) tmem_alloc(smem_u32(&ctl->tmem_base), kTmemCols);
    tc_fence_before();
    let_next_start();
    take_shares<R::THREADS>(p.t, sp, p.err, ctl->scan, 1, &ctl->share);
    wait_for_previous();  // expanded pages, read through the async proxy
    asm volatile("fence.proxy.async;" ::: "memory");
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    // The next part (whole warp): false when there is none, or a role gave up.
    uint32_t pi = 0;
    auto next_part = [&](Part &P, int code) {
        const int b = pi % kParts;
        if (!warp_wait(&ctl->part_full[b], (pi / kParts) & 1, abort, p.err, code)) return false;
        P = ctl->part[b];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->part_empty[b]);
        pi++;
        return P.tiles >= 0;
    };

    if (warp >= 8 && warp < 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::CTL));
    if (warp == 8) {
        // ------------------------------------------------ copies (the whole warp; a lane looks up and copies a page)
        uint32_t ct = 0, qx0 = 0, qx1 = 0;  // key tiles, items per X
        uint32_t q_armed = 0, q_par = 0, k_armed = 0, k_par = 0, v_armed = 0, v_par = 0, raw_armed = 0, raw_par = 0;
        bool ok = true;
        const int lg = p.c.page_log2, page = 1 << lg;
        Part P;
        while (ok && next_part(P, kDevTimeoutProducer)) {
            // The number of this lane's page of tile j, read a tile ahead: the reads of a tile's pages do not wait for
            // one another, nor the copies for them.
            int place = P.seq;
            if (!E4M3 && p.t.place_rows > 0) place = (P.row0 - P.tok0) / p.t.place_rows;  // expanded pages
            auto look = [&](int j) -> int32_t {
                const int key = (P.u0 + j) * kKeys + (lane << lg);
                if (j >= P.tiles || (lane << lg) >= kKeys || key >= P.end) return 0;
                const int64_t at = (int64_t)place * p.t.page_stride + (key >> lg);
                return p.t.pages ? __ldg(p.t.pages + at) : (int32_t)at;
            };
            int32_t next = look(0);
            // Q, behind the first K and V: its buffers are free only when the part before has done its last scores
            auto load_q = [&]() {
                for (int x = 0; x < 2; x++) {
                    if (P.n[x] == 0) continue;
                    const uint32_t qn = x == 0 ? qx0 : qx1;
                    if (!warp_wait(&ctl->q_empty[x], (qn & 1) ^ 1, abort, p.err, kDevTimeoutProducer)) {
                        return false;
                    }
                    if (lane == 0) {
                        const uint32_t qs = smem_u32(smem + x * C::TILE);
                        mbar_expect_tx(&ctl->q_full[x], half_rows * D * 2);
#pragma unroll
                        for (int c = 0; c < C::CH; c++)
                            tma_load_3d(qs + c * (kRows * 128), &q_map, &ctl->q_full[x], 64 * c, P.head * sp.group,
                                        P.row0 + x * half_tok);
                    }
                    q_armed |= 1u << x;
                    q_par = (q_par & ~(1u << x)) | ((qn & 1) << x);
                    if (x == 0) qx0++;
                    else qx1++;
                }
                return true;
            };
            for (int j = 0; j < P.tiles && ok; j++, ct++) {
                const int key0 = (P.u0 + j) * kKeys, nv = min(kKeys, P.end - key0);
                const int32_t g = check_page(next, p.c.n_pages, p.err);
                next = look(j + 1);
                if constexpr (!E4M3) {
                    const int st = ct % C::ST;
                    const uint32_t ph = (ct / C::ST) & 1;
                    const int np = (nv + page - 1) >> lg;
                    const int row = (int)pg_vec(p.c, g, P.head, 0);
                    auto load = [&](const CUtensorMap *map, uint32_t off, uint64_t *full, uint64_t *empty) {
                        if (!warp_wait(&empty[st], ph ^ 1, abort, p.err, kDevTimeoutProducer)) return false;
                        if (lane == 0) mbar_expect_tx(&full[st], np * page * D * 2);
                        __syncwarp();
                        if (lane < np) {
                            const uint32_t dst = smem_u32(smem + off + st * C::TILE) + lane * page * 128;
#pragma unroll
                            for (int c = 0; c < C::CH; c++) tma_load_3d(dst + c * (kKeys * 128), map, &full[st], 64 * c, row, 0);
                        }
                        return true;
                    };
                    if (!load(&k_map, C::K_OFF, ctl->k_full, ctl->k_empty)) {
                        ok = false;
                        break;
                    }
                    k_armed |= 1u << st;
                    k_par = (k_par & ~(1u << st)) | (ph << st);
                    if (!load(&v_map, C::V_OFF, ctl->v_full, ctl->v_empty)) {
                        ok = false;
                        break;
                    }
                    v_armed |= 1u << st;
                    v_par = (v_par & ~(1u << st)) | (ph << st);
                } else {
                    const int rs = ct % C::NR, np = (nv + page - 1) >> lg;
                    const uint32_t ph = (ct / C::NR) & 1;
                    const int64_t vec = pg_vec(p.c, g, P.head, 0);
#pragma unroll
                    for (int h = 0; h < 2; h++) {  // K with the scales of both, then V
                        if (!warp_wait(&ctl->raw_empty[h][rs], ph ^ 1, abort, p.err, kDevTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_expect_tx(&ctl->raw_full[h][rs], np * page * (h == 0 ? D + 2 : D));
                        __syncwarp();
                        if (lane < np) {
                            bulk_load(smem_u32(smem + C::RAW_OFF + (h * C::NR + rs) * C::RAW) + (lane << lg) * D,
                                      (h ? p.c.v : p.c.k) + vec * D, page * D, &ctl->raw_full[h][rs]);
                            if (h == 0) {
                                const uint32_t sc = smem_u32(smem + C::RSC_OFF + rs * 2 * kKeys) + (lane << lg);
                                bulk_load(sc, p.c.ks + vec, page, &ctl->raw_full[h][rs]);
                                bulk_load(sc + kKeys, p.c.vs + vec, page, &ctl->raw_full[h][rs]);
                            }
                        }
                        raw_armed |= 1u << (2 * h + rs);
                        raw_par = (raw_par & ~(1u << (2 * h + rs))) | (ph << (2 * h + rs));
                    }
                }
                if (ok && j == 0) ok = load_q();
            }
        }
        if (*abort && lane == 0) {
            // Let our own copies land before the CTA can exit.
            for (int s = 0; s < 2; s++)
                if (q_armed & (1u << s)) mbar_wait(&ctl->q_full[s], (q_par >> s) & 1, abort, p.err, 0, kDrainNs, false);
            for (int s = 0; s < C::ST; s++) {
                if (k_armed & (1u << s)) mbar_wait(&ctl->k_full[s], (k_par >> s) & 1, abort, p.err, 0, kDrainNs, false);
                if (v_armed & (1u << s)) mbar_wait(&ctl->v_full[s], (v_par >> s) & 1, abort, p.err, 0, kDrainNs, false);
            }
            for (int s = 0; s < 4; s++)
                if (raw_armed & (1u << s))
                    mbar_wait(&ctl->raw_full[s >> 1][s & 1], (raw_par >> s) & 1, abort, p.err, 0, kDrainNs, false);
        }
    } else if (warp == 9) {
        // ------------------------------------------------ MMA issue (the whole warp; one elected lane issues)
        constexpr uint32_t kBf16 = E4M3 ? (1u << 7) | (1u << 10) : 0u;  // bits that say bf16; f16 is 0
        const uint32_t idesc_s = make_idesc(kRows, kKeys, 0, 0) & ~kBf16;  // Q (K-major) x K (K-major)
        const uint32_t idesc_o = make_idesc(kRows, D, 0, 1) & ~kBf16;      // P (TMEM) x V (MN-major)
        uint32_t ct = 0, qx0 = 0, qx1 = 0, tx0 = 0, tx1 = 0;
        bool ok = true;
        auto mma_s = [&](int x, uint32_t t) {
            const uint64_t qd = sdesc(smem_u32(smem + x * C::TILE), 16, 1024);
            const uint64_t kd = sdesc(smem_u32(smem + C::K_OFF + (t % C::ST) * C::TILE), 16, 1024);
            const uint32_t d = tmem + (uint32_t)(x * kKeys);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; kk++)
                    umma_bf16(d, qd + (uint64_t)sdesc_off((kk >> 2) * (kRows * 128) + (kk & 3) * 32),
                              kd + (uint64_t)sdesc_off((kk >> 2) * (kKeys * 128) + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
                umma_commit(&ctl->s_full[x]);
            }
            __syncwarp();
        };
        // A_x (+)= P_x V_t over the first `steps` runs of 16 keys
        auto mma_o = [&](int x, uint32_t t, bool first, int steps) {
            const uint64_t vd = sdesc(smem_u32(smem + C::V_OFF + (t % C::ST) * C::TILE), kKeys * 128, 1024);
            const uint32_t pa = tmem + (uint32_t)(x * kKeys);
            const uint32_t d = tmem + kOCol + (uint32_t)(x * D);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; kk++)
                    if (kk < steps)
                        umma_bf16_ts(d, pa + kk * 8, vd + (uint64_t)sdesc_off(kk * 2048), idesc_o, (!first || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
        };
        auto commit1 = [&](uint64_t *b) {
            if (elect_one()) umma_commit(b);
            __syncwarp();
        };
        auto k_wait = [&](uint32_t t) { return warp_wait(&ctl->k_full[t % C::ST], (t / C::ST) & 1, abort, p.err, kDevTimeoutMma); };
        // V of tile t is there, with the last rows of a partial tile cleared
        auto v_wait = [&](uint32_t t, int nv) {
            if (!warp_wait(&ctl->v_full[t % C::ST], (t / C::ST) & 1, abort, p.err, kDevTimeoutMma)) return false;
            const int to = (nv + 15) & ~15;
            if (!E4M3 && nv < to) {
                uint8_t *v = smem + C::V_OFF + (t % C::ST) * C::TILE;
                for (int i = lane; i < (to - nv) * 8; i += 32)
#pragma unroll
                    for (int c = 0; c < C::CH; c++)
                        *reinterpret_cast<uint4 *>(v + c * (kKeys * 128) + (nv + i / 8) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
            }
            return true;
        };
        Part P;
        while (ok && next_part(P, kDevTimeoutMma)) {
            const int n = P.tiles, nt0 = P.n[0], nt1 = P.n[1];
            if (n == 0) continue;
            const int last_nv = P.end - (P.u0 + n - 1) * kKeys;  // keys of the part's last tile (may be more than 128)
            if (!k_wait(ct)) break;
            for (int x = 0; x < 2 && ok; x++) {
                const int ntx = x == 0 ? nt0 : nt1;
                if (ntx == 0) continue;
                if (!warp_wait(E4M3 ? &ctl->q_ready[x] : &ctl->q_full[x], (x == 0 ? qx0 : qx1) & 1, abort, p.err, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                if (x == 0) qx0++;
                else qx1++;
                tc_fence_after();
                mma_s(x, ct);
                if (ntx == 1) commit1(&ctl->q_empty[x]);
            }
            if (!ok) break;
            commit1(&ctl->k_empty[ct % C::ST]);
            for (int j = 0; j < n && ok; j++) {
                const uint32_t t = ct + j;
                const int nv = j == n - 1 ? min(kKeys, last_nv) : kKeys;
                bool v_now = false, k_next = false;  // V of tile t, K of tile t + 1 have landed
                for (int x = 0; x < 2; x++) {
                    const int ntx = x == 0 ? nt0 : nt1;
                    if (j >= ntx) continue;  // the rest of the part is beyond what x keeps
                    if (!v_now && !v_wait(t, nv)) {
                        ok = false;
                        break;
                    }
                    v_now = true;
                    if (!warp_wait(&ctl->p_full[x], ((x == 0 ? tx0 : tx1) + j) & 1, abort, p.err, kDevTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_o(x, t, j == 0, (nv + 15) >> 4);
                    if (j == ntx - 1) commit1(&ctl->o_fin[x]);
                    if (x == 1 || j >= nt1) commit1(&ctl->v_empty[t % C::ST]);  // the tile's last product
                    if (j + 1 < ntx) {
                        if (!k_next && !k_wait(t + 1)) {
                            ok = false;
                            break;
                        }
                        k_next = true;
                        mma_s(x, t + 1);
                        if (j + 1 == ntx - 1) commit1(&ctl->q_empty[x]);
                        if (x == 1 || j + 1 >= nt1) commit1(&ctl->k_empty[(t + 1) % C::ST]);
                    }
                }
            }
            ct += n;
            tx0 += nt0;
            tx1 += nt1;
        }
        // Every MMA this thread issued has completed once mma_done flips.
        commit1(&ctl->mma_done);
        if (lane == 0) mbar_wait(&ctl->mma_done, 0, abort, p.err, kDevTimeoutMma, kTimeoutNs, false);
        __syncwarp();
    } else if (warp == 10) {
        if (lane == 0) {
            // ------------------------------------------------ parts
            PgWalk w;
            w.begin(ctl->share, sp);
            note_cut(ws, sp, ctl->share, w);
            for (uint32_t i = 0;; i++) {
                const int b = i % kParts;
                if (!mbar_wait(&ctl->part_empty[b], ((i / kParts) & 1) ^ 1, abort, p.err, kDevTimeoutProducer)) break;
                if (w.left > 0) {
                    ctl->part[b] = part_of(w, sp);
                    w.step(w.part(), sp, seqs);
                } else {
                    ctl->part[b].tiles = -1;
                }
                const bool last = ctl->part[b].tiles < 0;
                mbar_arrive(&ctl->part_full[b]);
                if (last) break;
            }
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::SOFTMAX));
        // ------------------------------------------------ softmax and output
        const int x = warp >> 2;
        const int row = threadIdx.x & (kRows - 1);
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t srow = lane_base + (uint32_t)(x * kKeys);
        const uint32_t orow = lane_base + kOCol + (uint32_t)(x * D);
        const float c = p.scale_log2;
        const int rtok = row / sp.group, rhead = row - rtok * sp.group;  // the row's token and head of the tile
        uint32_t ci = 0, ct = 0;  // parts and key tiles of this X
        uint32_t gt = 0;          // key tiles of both: the ring of scales
        bool ok = true;
        while (ok) {
            int n, u0, slot, whole;  // what the loop over key tiles needs of the part
            int hi;                  // last key the row keeps
            int64_t at;              // the row's place in O; -1: no token of the sequence
            const uint32_t gt0 = gt;
            {
                Part P;
                const bool first_part = pi == 0;
                if (!next_part(P, kDevTimeoutSoftmax)) break;
                gt += P.tiles;
                const int ntok = min(half_tok, P.ntok - x * half_tok);
                if (ntok <= 0) continue;
                n = x == 0 ? P.n[0] : P.n[1];
                u0 = P.u0;
                whole = P.whole;
                slot = 2 * blockIdx.x + (first_part ? 0 : 1);
                // a row without a token goes along with the tile's last one
                const int pos = P.pos0 + x * half_tok + min(rtok, ntok - 1);
                hi = sp.causal ? min(pos, P.len - 1) : P.len - 1;
                at = row < half_rows && rtok < ntok
                         ? (int64_t)(P.row0 + x * half_tok + rtok) * p.qheads + P.head * sp.group + rhead : -1;
            }
            const bool mine = at >= 0;
            float m_ref = -INFINITY, m_max = -INFINITY, l = 0.f;
            int qe = 0;      // e4m3: Q is 2^-qe times its f16 values
            int vref = 0;    // e4m3: A is in units of 2^(vref - 133 - 7), l in units of 2^-7
            for (int j = 0; j < n; j++) {
                if (!warp_wait(&ctl->s_full[x], (ct + j) & 1, abort, p.err, kDevTimeoutSoftmax)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t u[kKeys];
                const int jhi = hi - (u0 + j) * kKeys;
                float hm0, hm1, hm2, hm3;
                tmem_ld32_max(srow, u, hm0);
                tmem_ld32_max(srow + 32, u + 32, hm1);
                tmem_ld32_max(srow + 64, u + 64, hm2);
                tmem_ld32_max(srow + 96, u + 96, hm3);
                float ft = 1.f, ft2 = 1.f, cr = c, shift = 1.f;  // a score is ft * ft2 times what the product gives
                if constexpr (E4M3) {
                    const Refs rf = reinterpret_cast<const Refs *>(smem + C::SC_OFF)[(gt0 + j) % (2 * C::ST)];
                    if (j == 0) {
                        qe = reinterpret_cast<const int8_t *>(smem + C::QS_OFF)[((ci & 1) * 2 + x) * kRows + row];
                        vref = rf.v;
                    }
                    shift = pow2(vref - rf.v);
                    vref = rf.v;
                    // Both powers in one: each alone may lie beyond fp32's where the other brings it back.  Neither factor
                    // is 0, which would make NaN of a dropped score: below 2^-126 the exponentials take 2^-126 (scores of
                    // less than 2^-88 either way), and the maximum a second factor.
                    const int e = rf.k - 133 - qe;
                    ft = pow2(min(127, max(e, -126)));
                    ft2 = pow2(min(0, max(e + 126, -126)));
                    cr = fmaxf(c * ft, 1.2e-38f);
                }
                tmem_wait_ld();
                float mx = fmaxf(max3(hm0, hm1, hm2), hm3);
                if (jhi < kKeys - 1) {
                    mx = -INFINITY;
#pragma unroll
                    for (int q = 0; q < kKeys; q += 32) mx = fmaxf(mx, mask_chunk(u + q, q, 0, jhi));
                }
                if constexpr (E4M3) mx = mx * ft * ft2;
                m_max = fmaxf(m_max, mx);
                float alpha = 1.f;
                if (mx != -INFINITY && (m_ref == -INFINITY || (mx - m_ref) * c > kLazy)) {
                    alpha = m_ref == -INFINITY ? 0.f : ex2((m_ref - mx) * c);
                    m_ref = mx;
                }
                const float base = (m_ref == -INFINITY ? 0.f : m_ref * c) - (E4M3 ? 7.f : 0.f);
                const uint64_t c2 = pack_f32x2(cr, cr), nb2 = pack_f32x2(-base, -base);
                uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < kKeys / 2; q++) {
                    const uint64_t y = fma_f32x2(pack_u32x2(u[2 * q], u[2 * q + 1]), c2, nb2);
                    const float e0 = ex2(lo_f32(y)), e1 = ex2(hi_f32(y));
                    ls[q & 3] = add_f32x2(ls[q & 3], pack_f32x2(e0, e1));
                    u[q] = E4M3 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
                }
                const uint64_t s01 = add_f32x2(add_f32x2(ls[0], ls[1]), add_f32x2(ls[2], ls[3]));
                l = fmaf(l, alpha, lo_f32(s01) + hi_f32(s01));
                if constexpr (E4M3) alpha *= shift;
                tmem_st32(srow, u);
                tmem_st32(srow + 32, u + 32);
                // The previous A += P V of this tile has completed: these scores were computed after it, in order.
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int cc = 0; cc < D / 32; cc++) {
                        uint32_t o[32];
                        tmem_ld32(orow + 32 * cc, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(orow + 32 * cc, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[x]);
            }
            if (!ok) break;
            if (n > 0) {
                if (!warp_wait(&ctl->o_fin[x], ci & 1, abort, p.err, kDevTimeoutSoftmax)) {
                    ok = false;
                    break;
                }
                ct += n;
                ci++;
            }
            tc_fence_after();
            // whole item: A / l as bf16; a part of one: (m, l, A) with the true maximum as reference
            const float to_max = m_max == -INFINITY ? 0.f : ex2((m_ref - m_max) * c);
            const float unit = E4M3 ? ldexpf(1.f, vref - 133 - 7) : 1.f;
            if constexpr (E4M3) l *= 0.0078125f;
            float f = !whole ? to_max : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
            if constexpr (E4M3) {
                if (vref >= 64) {
                    f *= unit;
                } else if (n > 0) {
                    // their product can lie below fp32's normal numbers where the result does not: A takes its unit first
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; cc++) {
                        uint32_t o[32];
                        tmem_ld32(orow + 32 * cc, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * unit);
                        tmem_st32(orow + 32 * cc, o);
                    }
                    tmem_wait_st();
                }
            }
            const int64_t prow = (int64_t)slot * (2 * half_rows) + x * half_rows + row;
#pragma unroll
            for (int cc = 0; cc < D / 32; cc++) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(orow + 32 * cc, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = 0u;
                }
                if (!mine) continue;
                if (whole) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 16; i++) h[i] = pack_bf16(__uint_as_float(o[2 * i]) * f, __uint_as_float(o[2 * i + 1]) * f);
                    char *dst = p.o + (at * D + 32 * cc) * 2;
                    st_32(dst, h);
                    st_32(dst + 32, h + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    float *dst = ws.acc + prow * D + 32 * cc;
#pragma unroll
                    for (int q = 0; q < 4; q++) st_32(dst + 8 * q, o + 8 * q);
                }
            }
            tc_fence_before();
            if (mine) {
                if (!whole) ws.ml[prow] = make_float2(m_max, l * to_max);
                else if (p.m_out) {
                    p.m_out[at] = m_max * p.scale;
                    p.l_out[at] = l * to_max;
                }
            }
        }
    } else if (E4M3 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::CONV));
        // ------------------------------------------------ raw tiles to f16 operands
        const int tid = threadIdx.x - 384;
        constexpr int CPR = D / 16;  // 16-byte chunks (16 codes) of a row
        uint32_t ct = 0, qx0 = 0, qx1 = 0;
        int vref = 0;
        bool ok = true;
        // Q of both tiles, a row a thread, in place: bf16 to f16, brought to [2^14, 2^15) by a power of two
        auto rewrite_q = [&](const Part &P) {
            for (int x = 0; x < 2; x++) {
                if (P.n[x] == 0) continue;
                const uint32_t qn = x == 0 ? qx0 : qx1;
                if (!warp_wait(&ctl->q_full[x], qn & 1, abort, p.err, kDevTimeoutProducer)) return false;
                if (tid < half_rows) {
                    uint8_t *rowp = smem + x * C::TILE + tid * 128;
                    const int s = tid & 7;
                    uint32_t big = 0;
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(rowp + (i / 8) * (kRows * 128) + (((i & 7) ^ s) << 4));
                        big = __vmaxu2(big, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
                        big = __vmaxu2(big, __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    }
                    big = max(big >> 16, big & 0xffffu);
                    const int e = big == 0 || big >= 0x7f80u ? 0 : min(126, 14 - ((int)(big >> 7) - 127));
                    const float up = pow2(e);
                    auto cvt = [&](uint32_t w) { return pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up); };
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        uint4 *at = reinterpret_cast<uint4 *>(rowp + (i / 8) * (kRows * 128) + (((i & 7) ^ s) << 4));
                        const uint4 v = *at;
                        *at = make_uint4(cvt(v.x), cvt(v.y), cvt(v.z), cvt(v.w));
                    }
                    reinterpret_cast<int8_t *>(smem + C::QS_OFF)[((qn & 1) * 2 + x) * kRows + tid] = (int8_t)e;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->q_ready[x]);
                if (x == 0) qx0++;
                else qx1++;
            }
            return true;
        };
        Part P;
        while (ok && next_part(P, kDevTimeoutProducer)) {
            for (int j = 0; j < P.tiles && ok; j++, ct++) {
                const int nv = min(kKeys, P.end - (P.u0 + j) * kKeys);
                const int st = ct % C::ST, rs = ct % C::NR, row0 = (warp - 12) * 32;
                uint32_t fv = 0, fk = 0;  // factors of row row0 + lane of K and V, f16 twice
#pragma unroll
                for (int h = 0; h < 2; h++) {  // K, V
                    if (!warp_wait(h ? &ctl->v_empty[st] : &ctl->k_empty[st], ((ct / C::ST) & 1) ^ 1, abort, p.err, kDevTimeoutProducer) ||
                        !warp_wait(&ctl->raw_full[h][rs], (ct / C::NR) & 1, abort, p.err, kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    // all of the lane's codes first: the raw tile is free, and no load waits behind a store
                    const uint8_t *raw = smem + C::RAW_OFF + (h * C::NR + rs) * C::RAW + row0 * D;
                    uint4 v[CPR];
#pragma unroll
                    for (int i = 0; i < CPR; i++) v[i] = *reinterpret_cast<const uint4 *>(raw + (i * 32 + lane) * 16);
                    uint32_t kb = 0, vb = 0;
                    if (h == 0) {
                        kb = smem[C::RSC_OFF + rs * 2 * kKeys + row0 + lane];
                        vb = smem[C::RSC_OFF + rs * 2 * kKeys + kKeys + row0 + lane];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->raw_empty[h][rs]);
                    if (h == 0) {
                        // NaN vectors (255) and what lies beyond the last key do not move the references
                        const bool in = row0 + lane < nv;
                        const uint32_t tk = __reduce_max_sync(0xffffffffu, in && kb != 255u ? kb : 0u);
                        const uint32_t tv = __reduce_max_sync(0xffffffffu, in && vb != 255u ? vb : 0u);
                        if (lane == 0) {
                            ctl->top[ct & 1][warp - 12] = make_int2((int)tk, (int)tv);
                            mbar_arrive(&ctl->top_full[ct & 1]);
                        }
                        if (!warp_wait(&ctl->top_full[ct & 1], (ct >> 1) & 1, abort, p.err, kDevTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        int kref = 0;
                        if (j == 0) vref = 0;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int2 t = ctl->top[ct & 1][i];
                            kref = max(kref, t.x);
                            vref = max(vref, t.y);
                        }
                        // 2^(byte - reference + 6)
                        auto factor = [&](uint32_t b, int ref) {
                            const float f = !in ? 0.f : b == 255u ? __uint_as_float(0x7fffffffu) : pow2((int)b - ref + 6);
                            return pack_f16(f, f);
                        };
                        fk = factor(kb, kref);
                        fv = factor(vb, vref);
                        if (tid == 0) reinterpret_cast<Refs *>(smem + C::SC_OFF)[ct % (2 * C::ST)] = Refs{kref, vref};
                    }
                    if (nv - row0 < 32) {  // beyond the last key: zeros, whatever is there
#pragma unroll
                        for (int i = 0; i < CPR; i++)
                            if (row0 + (i * 32 + lane) / CPR >= nv) v[i] = make_uint4(0, 0, 0, 0);
                    }
                    uint8_t *dst = smem + (h ? C::V_OFF : C::K_OFF) + st * C::TILE + row0 * 128;
#pragma unroll
                    for (int i = 0; i < CPR; i++) {
                        const int r = (i * 32 + lane) / CPR, ch = lane % CPR;
                        const uint32_t f = __shfl_sync(0xffffffffu, h ? fv : fk, r);
                        uint4 lo, hi;
                        to_f16(v[i].x, lo.x, lo.y);
                        to_f16(v[i].y, lo.z, lo.w);
                        to_f16(v[i].z, hi.x, hi.y);
                        to_f16(v[i].w, hi.z, hi.w);
                        lo = make_uint4(mul_f16x2(lo.x, f), mul_f16x2(lo.y, f), mul_f16x2(lo.z, f), mul_f16x2(lo.w, f));
                        hi = make_uint4(mul_f16x2(hi.x, f), mul_f16x2(hi.y, f), mul_f16x2(hi.z, f), mul_f16x2(hi.w, f));
                        // columns 16 ch .. + 15 of the row: two 16-byte chunks of its 128-byte swizzled piece; the lanes of
                        // the second 64 columns store theirs in the other order (their banks are the same)
                        uint8_t *rowp = dst + (ch / 4) * (kKeys * 128) + r * 128;
                        const int s = r & 7, a = 2 * (ch & 3), flip = ch >> 2;
                        *reinterpret_cast<uint4 *>(rowp + (((a + flip) ^ s) << 4)) = flip ? hi : lo;
                        *reinterpret_cast<uint4 *>(rowp + (((a + 1 - flip) ^ s) << 4)) = flip ? lo : hi;
                    }
                    fence_proxy_async();  // the operand tiles are read by the tensor cores (async proxy)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(h ? &ctl->v_full[st] : &ctl->k_full[st]);
                    // the part's Q between its first K and V: it arrives when the part before has done its last scores
                    if (j == 0 && h == 0 && !rewrite_q(P)) {
                        ok = false;
                        break;
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool E4M3>
cudaError_t launch(const PgAttn &p, const PgPlan &pl, const PgWork &w, const PgMaps &maps, bool early, cudaStream_t st) {
    using C = Cfg<D, E4M3>;
    using R = Regs<E4M3>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        // The register split assumes the block starts with LAUNCH a thread: with fewer, setmaxnreg.inc would wait for
        // registers that never come, so such a build is refused before it can launch.
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, cache_chunks_kernel<D, E4M3>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != R::LAUNCH) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(cache_chunks_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_after(cache_chunks_kernel<D, E4M3>, dim3(pl.ctas), R::THREADS, C::SMEM, st, early, p, pl.split, w, maps.q, maps.k, maps.v);
}

}  // namespace

PgPlan plan_cache_chunks(const PgTable &t, const PgPool &c, int group, int causal, int num_sms, int min_rows) {
    PgPlan pl{};
    if ((int64_t)t.max_new * group < min_rows) return pl;
    const int tpt = kRows / group;
    PgSplit &sp = pl.split;
    sp.heads = c.heads;
    sp.group = group;
    sp.tok = 2 * tpt;
    // Short sequences are not cut: the tiles of an item cost less than the merge (2 x 64 tokens in 600 positions, 32 heads
    // over 8: 30.0 us cut, 24.6 us whole).  As in the token kernel it is the table's width that says so.
    const bool whole = t.cap <= kWhole;
    sp.kt = whole ? kWhole : kKeys;
    sp.causal = causal;
    sp.min_rows = min_rows;
    sp.max_rows = INT32_MAX;
    pl.rows = sp.tok * group;
    const int64_t items = std::min<int64_t>((int64_t)t.n_seqs * ((t.max_new + sp.tok - 1) / sp.tok), t.rows / sp.tok + t.n_seqs);
    const int64_t units = (t.cap + sp.kt - 1) / sp.kt * items * c.heads;
    pl.ctas = (int)std::min<int64_t>(units, num_sms);
    pl.bytes = whole ? 0 : pg_work_bytes(pl.ctas, pl.rows, c.dim);
    return pl;
}

PgExpand plan_cache_expand(const PgTable &t, const PgPool &c, int group, int min_rows) {
    PgExpand x{};
    if (c.fmt != EA_CACHE_E4M3 || (int64_t)t.max_new * group < 2 * kRows) return x;
    const int64_t least = (min_rows + group - 1) / group;  // rows of a sequence served; <= max_new <= t.rows
    const bool by_row = t.rows / least < t.n_seqs;
    const int64_t places = by_row ? t.rows / least : t.n_seqs;
    const int64_t blocks = (t.cap + kKeys - 1) / kKeys, vectors = blocks * kKeys * places * c.heads;
    // Up to 4 GB.  A batch that could need more (many sequences that may have chunks, or a very wide table) keeps to the
    // 8-bit pages.
    if (vectors * c.dim * 4 > (int64_t)1 << 32) return x;
    x.blocks = (int32_t)blocks;
    x.places = (int32_t)places;
    x.place_rows = by_row ? (int32_t)least : 0;
    x.bytes = (size_t)vectors * c.dim * 4;
    return x;
}

cudaError_t launch_cache_chunks(const PgAttn &p, const PgPlan &pl, const PgMaps &maps, const PgWork &w, bool early, cudaStream_t st) {
    if (p.c.fmt == EA_CACHE_E4M3)
        return p.c.dim == 64 ? launch<64, true>(p, pl, w, maps, early, st) : launch<128, true>(p, pl, w, maps, early, st);
    return p.c.dim == 64 ? launch<64, false>(p, pl, w, maps, early, st) : launch<128, false>(p, pl, w, maps, early, st);
}

}  // namespace ea
