// paged.h -- the paged cache: parameters of its kernels and the index
// arithmetic they share with the host (batch checks, the work list of the
// attention).  Internal.
//
// Attention's work list is made on the device, because the batch lives
// there.  A sequence's query rows (n tokens x g heads of one key-value head,
// token-major) are cut into items of `tok` tokens; an item takes ceil(e / kt)
// units of kt keys, e the keys that its last token keeps (at least one unit,
// so that an item without keys is still written).  Units are numbered
// sequence by sequence, key-value head by key-value head, item by item, and
// CTA x of G takes the units [x W / G, (x + 1) W / G): every CTA has the same
// number of units to within one, however ragged the batch is.  An item whose
// units fall into several CTAs is merged from their partial results.
#pragma once

#include <cuda.h>

#include "host.h"

#ifdef __CUDACC__
#define EA_HD __host__ __device__ __forceinline__
#else
#define EA_HD inline
#endif

struct ea_cache_s {
    int format = 0;
    int64_t n_pages = 0;
    int32_t page = 0, page_log2 = 0, heads = 0, dim = 0;
    char *k = nullptr, *v = nullptr;
    uint8_t *ks = nullptr, *vs = nullptr;
    int device = -1, num_sms = 0;
    bool mapped = false;
    CUtensorMap k_map, v_map;  // bf16: the pools for the chunk kernel's copies, made on first use
};

namespace ea {

struct PgPool {
    char *k, *v;         // [pages][heads][page][dim] cells
    uint8_t *ks, *vs;    // [pages][heads][page] scale bytes (e4m3)
    int64_t n_pages;
    int32_t page_log2, heads, dim, fmt;
};

struct PgTable {
    const int32_t *pages, *starts, *lens;  // pages NULL: page x of sequence i is number place(i) * page_stride + x
    int64_t page_stride;
    int64_t rows;        // dense rows
    int64_t cap;         // positions that a sequence can have
    int32_t n_seqs, max_pages, max_new;
    int32_t place_rows;  // pages NULL: the place of sequence i; 0: i; else first row / place_rows
};

struct PgRows {          // append and read
    PgTable t;
    PgPool c;
    char *k, *v;         // dense rows [rows][heads][dim]
    int32_t f32;         // dense dtype: 1 fp32, 0 bf16
    int32_t read;        // 0 append, 1 read
    int *err;
};
cudaError_t launch_cache_rows(const PgRows &p, int64_t *ctas, cudaStream_t st);

struct PgAttn {
    PgTable t;
    PgPool c;
    const char *q;       // [rows][qheads][dim] bf16
    char *o;
    float *m_out, *l_out;
    int32_t qheads, group, causal;
    float scale, scale_log2;  // scale * log2(e)
    int *err;
};

// Where a batch's attention is cut, and the partial results of the cuts.
struct PgSplit {
    int32_t heads, group;        // key-value heads, query heads of one
    int32_t tok;                 // tokens of an item
    int32_t kt;                  // keys of a unit
    int32_t causal;
    int32_t min_rows, max_rows;  // the sequences served: min_rows <= n * group <= max_rows
    int32_t solo;                // token kernel: a warp, not a CTA, takes a share
};

// What a CTA whose range begins inside an item says to the merge.
struct PgCut {
    int64_t wi, we;              // the item's units [wi, we); we = 0: the range begins with an item, or is empty
    int64_t total;               // units of the batch
    int32_t parts;               // CTAs with units
    int32_t head;
    int32_t row0;                // the item's first dense row, and its rows (tokens x group)
    int32_t rows;
};

struct PgWork {                  // the call's workspace
    PgCut *cut;                  // [ctas]
    float2 *ml;                  // [2 * ctas][rows]: maximum score and sum of a partial result
    float *acc;                  // [2 * ctas][rows][dim]: its unnormalised output
};

struct PgPlan {                  // a kernel of the call and its grid
    PgSplit split;
    int32_t ctas;                // 0: not launched
    int32_t rows;                // rows of an item
    size_t bytes;                // workspace; 0: no item is cut
};

// Workspace of a plan, and its parts in it.
inline size_t pg_work_bytes(int ctas, int rows, int dim) {
    const size_t n = (size_t)2 * ctas * rows;
    return ((size_t)ctas * sizeof(PgCut) + 255) / 256 * 256 + (n * sizeof(float2) + 255) / 256 * 256 +
           (n * dim * sizeof(float) + 255) / 256 * 256;
}
inline PgWork pg_work(const PgPlan &pl, char *b) {
    if (pl.bytes == 0) return PgWork{};
    const size_t cut = ((size_t)pl.ctas * sizeof(PgCut) + 255) / 256 * 256;
    const size_t ml = ((size_t)2 * pl.ctas * pl.rows * sizeof(float2) + 255) / 256 * 256;
    return PgWork{(PgCut *)b, (float2 *)(b + cut), (float *)(b + cut + ml)};
}

// Token kernel: few rows a sequence, bound by reading the pages.
constexpr int kPgTokenRows = 32;     // the most rows of a sequence (tokens x group) that it takes
PgPlan plan_cache_tokens(const PgTable &t, const PgPool &c, int group, int causal, int num_sms);
cudaError_t launch_cache_tokens(const PgAttn &p, const PgPlan &pl, const PgWork &w, bool early, cudaStream_t st);

// 8-bit pages as bf16 vectors in the workspace, in blocks of 128 positions.
// There are places for as many sequences as the chunk kernel can serve: one
// has at least `least` rows, so `rows / least` of them at most.  Where the
// batch has more sequences than that, a sequence's place is its first row
// divided by `least`: the first rows of two that are served lie at least so
// far apart.
struct PgExpand {
    int32_t blocks;              // of a sequence; 0: the chunk kernel reads the 8-bit pages itself
    int32_t places;
    int32_t place_rows;          // 0: a sequence's place is its number
    size_t bytes;                // K's vectors and V's
};
PgExpand plan_cache_expand(const PgTable &t, const PgPool &c, int group, int min_rows);
cudaError_t launch_cache_expand(const PgAttn &p, const PgSplit &sp, const PgExpand &x, char *ws, cudaStream_t st);

// Chunk kernel: tiles of 128 rows on the tensor cores.
struct PgMaps {                  // tensor maps: Q's rows; the pools as [vectors][dim] (bf16)
    CUtensorMap q, k, v;
};
PgPlan plan_cache_chunks(const PgTable &t, const PgPool &c, int group, int causal, int num_sms, int min_rows);
cudaError_t launch_cache_chunks(const PgAttn &p, const PgPlan &pl, const PgMaps &maps, const PgWork &w, bool early,
                                cudaStream_t st);

// The merge of both kernels' cut items.
struct PgMerge {
    PgWork w[2];
    int32_t cuts[2];             // CTAs - 1; 0: none
    int32_t rows[2];
    int32_t groups[2];           // CTAs of a cut (set by the launch)
};
cudaError_t launch_cache_merge(const PgAttn &p, const PgMerge &m, cudaStream_t st);

// ------------------------------------------------------------- sequences

struct PgSeq {
    int32_t first, n, len;  // first dense row, rows, positions
};

// Sequence i from its three numbers; false if they are out of range.
EA_HD bool pg_seq(int32_t a, int32_t b, int32_t len, int64_t rows, int32_t max_new, int64_t cap, PgSeq *s) {
    s->first = a;
    s->n = 0;
    s->len = 0;
    if (a < 0 || b < a || b > rows || b - a > max_new || len < 0 || len > cap) return false;
    s->n = b - a;
    s->len = len;
    return true;
}

// ------------------------------------------------------------- work list

// SUM_{i < n} floor((a i + b) / m) for a, b >= 0, m > 0: the published way of
// counting the lattice points under a line with Euclid's algorithm (whole
// parts of a / m and b / m are summed in closed form, then i and the value
// change places).
template <class T>
EA_HD int64_t pg_floor_sum_t(T n, T m, T a, T b) {
    int64_t s = 0;
    while (n > 0) {
        if (a >= m) {
            const T q = a / m;
            s += (int64_t)n * (n - 1) / 2 * q;
            a -= q * m;
        }
        if (b >= m) {
            const T q = b / m;
            s += (int64_t)n * q;
            b -= q * m;
        }
        const T y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y - n * m;
        const T t = m;
        m = a;
        a = t;
    }
    return s;
}
// The values only shrink: what fits 32 bits at the start stays there, and
// takes a GPU thread a fifth of the time.
EA_HD int64_t pg_floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    if (n <= INT32_MAX && a * n + b <= INT32_MAX && m <= INT32_MAX)
        return pg_floor_sum_t<uint32_t>((uint32_t)n, (uint32_t)m, (uint32_t)a, (uint32_t)b);
    return pg_floor_sum_t<int64_t>(n, m, a, b);
}

EA_HD bool pg_served(const PgSeq &s, const PgSplit &sp) {
    const int64_t r = (int64_t)s.n * sp.group;
    return s.n > 0 && r >= sp.min_rows && r <= sp.max_rows;
}

// ceil(a / b) for 0 <= a < 2^31, 0 < b < 2^31 (32 bits: a 64-bit division takes
// a GPU thread a hundred cycles, and these are on the way to the first load).
EA_HD int pg_ceil(int a, int b) { return (int)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b); }

EA_HD int pg_items(const PgSeq &s, const PgSplit &sp) { return pg_ceil(s.n, sp.tok); }

// Keys [0, e) that item j's last token keeps.
EA_HD int pg_item_end(const PgSeq &s, const PgSplit &sp, int j) {
    if (!sp.causal) return s.len;
    const int64_t last = (int64_t)(j + 1) * sp.tok;
    const int64_t e = (int64_t)s.len - s.n + (last < s.n ? last : s.n);
    return e > 0 ? (int)e : 0;
}

EA_HD int pg_item_units(const PgSeq &s, const PgSplit &sp, int j) {
    const int u = pg_ceil(pg_item_end(s, sp, j), sp.kt);
    return u > 0 ? u : 1;
}

// Units of the items before item j of one key-value head (j < items).
EA_HD int64_t pg_units_before(const PgSeq &s, const PgSplit &sp, int j) {
    if (j <= 0) return 0;
    if (!sp.causal) return (int64_t)j * pg_item_units(s, sp, 0);
    const int64_t c = (int64_t)s.len - s.n;
    int64_t none = c < 0 ? (int64_t)((uint32_t)-c / (uint32_t)sp.tok) : 0;  // items whose tokens all stand before position 0: one unit each
    if (none > j) none = j;
    return none + pg_floor_sum(j - none, sp.kt, sp.tok, c + (none + 1) * sp.tok + sp.kt - 1);
}

EA_HD int64_t pg_head_units(const PgSeq &s, const PgSplit &sp) {
    const int j = pg_items(s, sp) - 1;
    return pg_units_before(s, sp, j) + pg_item_units(s, sp, j);
}

EA_HD int64_t pg_seq_units(const PgSeq &s, const PgSplit &sp) {
    return pg_served(s, sp) ? sp.heads * pg_head_units(s, sp) : 0;
}

// The item that holds unit u of one key-value head.
EA_HD int pg_item_of(const PgSeq &s, const PgSplit &sp, int64_t u) {
    int a = 0, b = pg_items(s, sp) - 1;
    while (a < b) {
        const int mid = a + (b - a + 1) / 2;
        if (pg_units_before(s, sp, mid) <= u) a = mid;
        else b = mid - 1;
    }
    return a;
}

// Units [pg_first(x), pg_first(x + 1)) of CTA x, of `parts` with work.
EA_HD int64_t pg_first(int64_t total, int parts, int x) {
    if (total <= INT32_MAX) {  // parts * parts < 2^32
        const uint32_t t = (uint32_t)total, q = t / (uint32_t)parts, r = t - q * (uint32_t)parts;
        return (int64_t)q * x + r * (uint32_t)x / (uint32_t)parts;
    }
    return total / parts * x + total % parts * x / parts;
}
// The CTAs whose first unit lies before unit u (0 < u <= total): total x / parts < u.
EA_HD int pg_before(int64_t total, int parts, int64_t u) {
    const int64_t a = u * parts;  // u <= 2^48, parts < 2^11
    if (a <= INT32_MAX && total <= INT32_MAX) return (int)(((uint32_t)a + (uint32_t)total - 1u) / (uint32_t)total);
    return (int)((a + total - 1) / total);
}
EA_HD int64_t pg_div(int64_t a, int b) { return a <= INT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b; }
EA_HD int pg_parts(int64_t total, int ctas) { return (int)(total < ctas ? total : ctas); }

// A CTA's share of the units.
struct PgShare {
    int64_t w0, off;   // first unit of the batch; the same within its sequence
    int64_t total;     // units of the batch
    int64_t count;     // units of this CTA
    int32_t seq, parts;
    PgSeq s;           // sequence `seq`
};

// The parts of items in a CTA's share, in order (Seqs: seqs(i) is sequence i,
// seqs.count() their number).
struct PgWalk {
    PgSeq s;
    int64_t left;            // units not taken yet
    int32_t seq, head, item;
    int32_t u0;              // first unit of the current item not taken yet
    int32_t units;           // units of the current item

    EA_HD void begin(const PgShare &sh, const PgSplit &sp) {
        left = sh.count;
        seq = sh.seq;
        head = item = u0 = units = 0;
        if (left <= 0) return;
        s = sh.s;
        if (pg_items(s, sp) == 1) {  // one item a head: no search
            units = pg_item_units(s, sp, 0);
            head = (int)pg_div(sh.off, units);
            u0 = (int)(sh.off - (int64_t)head * units);
            return;
        }
        const int64_t hu = pg_head_units(s, sp);
        head = (int)(sh.off / hu);
        const int64_t u = sh.off - head * hu;
        item = pg_item_of(s, sp, u);
        u0 = (int)(u - pg_units_before(s, sp, item));
        units = pg_item_units(s, sp, item);
    }

    // Units of the current part (0: none left).
    EA_HD int part() const { return (int)(left < units - u0 ? left : units - u0); }

    // Leave `n` units of the current part behind (n <= part()).
    template <class Seqs>
    EA_HD void step(int n, const PgSplit &sp, const Seqs &seqs) {
        left -= n;
        u0 += n;
        if (u0 < units || left <= 0) return;
        u0 = 0;
        if (++item == pg_items(s, sp)) {
            item = 0;
            if (++head == sp.heads) {
                head = 0;
                do s = seqs(++seq);
                while (!pg_served(s, sp) && seq + 1 < seqs.count());
            }
        }
        units = pg_item_units(s, sp, item);
    }
};

// Element offset of a vector (page, head, slot) / dim in the pool.
EA_HD int64_t pg_vec(const PgPool &c, int64_t page, int head, int slot) {
    return ((page * c.heads + head) << c.page_log2) + slot;
}

}  // namespace ea
