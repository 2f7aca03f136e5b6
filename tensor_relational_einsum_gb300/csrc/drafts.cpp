// drafts.cpp -- the entry points around drafted tokens: rotary positions,
// verification, keeping the accepted rows of the cache.
#include <algorithm>
#include <cmath>

#include "drafts.h"
#include "paged_host.h"

namespace ea {
namespace {

// The batch's rows, without its pages: what rotation and verification read.
ea_status rows_args(const char *what, const ea_page_batch *b, int64_t rows, bool lens) {
    if (!b || !b->starts || (lens && !b->lens)) return set_error(EA_ERR_ARG, "%s: NULL batch or batch array", what);
    if (off_4({b->starts, b->lens})) return set_error(EA_ERR_ARG, "%s: the batch's arrays must be aligned to 4 bytes", what);
    if (b->n_seqs < 1 || b->n_seqs > 65536) return set_error(EA_ERR_ARG, "%s: n_seqs %d out of [1, 65536]", what, b->n_seqs);
    if (b->max_new < 0) return set_error(EA_ERR_ARG, "%s: max_new %d", what, b->max_new);
    if (rows > INT32_MAX - 8191) return set_error(EA_ERR_UNSUPPORTED, "%s: more than %d rows", what, INT32_MAX - 8191);
    return EA_OK;
}

int32_t most_new(const ea_page_batch *b, int64_t rows) {
    return (int32_t)(b->max_new > 0 && b->max_new < rows ? b->max_new : rows);
}

// Bytes [p, p + n) share some with the batch's bounds or lengths.
bool in_rows(const ea_page_batch *b, const void *p, size_t n) {
    return b && (overlap(b->starts, ((size_t)b->n_seqs + 1) * 4, p, n) || overlap(b->lens, (size_t)b->n_seqs * 4, p, n));
}

bool overlap(const ea_relation_s *a, const ea_relation_s *b) { return ea::overlap(a->arena, a->bytes, b->arena, b->bytes); }

}  // namespace
}  // namespace ea

using namespace ea;

extern "C" ea_status ea_rotary(const ea_rotary_opts *opts, const ea_page_batch *batch, ea_relation q, ea_relation k,
                               ea_relation q_out, ea_relation k_out, void *stream) {
    return entry([&]() -> ea_status {
        const char *what = "ea_rotary";
        if (!opts || !opts->freqs || !q || !q_out || (k != nullptr) != (k_out != nullptr))
            return set_error(EA_ERR_ARG, "%s: NULL argument, or one of k and its result", what);
        const ea_rotary_opts &o = *opts;
        if ((batch != nullptr) == (o.positions != nullptr)) return set_error(EA_ERR_ARG, "%s: give a batch or positions", what);
        if (o.parents && !batch) return set_error(EA_ERR_ARG, "%s: parents belong to a batch", what);
        if (off_4({o.positions})) return set_error(EA_ERR_ARG, "%s: positions must be aligned to 4 bytes", what);
        if (o.layout != EA_ROTARY_INTERLEAVED && o.layout != EA_ROTARY_HALF) return set_error(EA_ERR_ARG, "%s: layout %d", what, o.layout);
        if (!std::isfinite(o.amplitude)) return set_error(EA_ERR_ARG, "%s: amplitude", what);
        RoParams p{};
        int64_t rows = 0, dim = 0;
        ea_relation in[2] = {q, k}, out[2] = {q_out, k_out};
        for (int w = 0; w < 2 && in[w]; w++) {
            int64_t r, h, d, ro, ho, dd;
            ea_status s = dense_rows(in[w], what, 2, &r, &h, &d);
            if (!s) s = dense_rows(out[w], what, 2, &ro, &ho, &dd);
            if (s) return s;
            if (w == 0) rows = r, dim = d;
            if (r != rows || d != dim || ro != r || ho != h || dd != d) return set_error(EA_ERR_SHAPE, "%s: q, k and their results have different rows, heads or columns", what);
            if (in[w]->dtype != q->dtype || out[w]->dtype != q->dtype) return set_error(EA_ERR_DTYPE, "%s: q, k and their results have different dtypes", what);
            if (h < 1 || h > 65535 || d > 65535) return set_error(EA_ERR_UNSUPPORTED, "%s: %lld heads of %lld columns", what, (long long)h, (long long)d);
            if (out[w]->arena != in[w]->arena && overlap(out[w], in[w])) return set_error(EA_ERR_ARG, "%s: a result overlaps its operand, but is not it", what);
            p.x[w] = in[w]->arena;
            p.y[w] = out[w]->arena;
            p.heads[w] = (int32_t)h;
        }
        if (k && (overlap(q_out, k) || overlap(k_out, q) || overlap(q_out, k_out))) return set_error(EA_ERR_ARG, "%s: q and k overlap", what);
        if (k && (p.x[0] == p.y[0]) != (p.x[1] == p.y[1])) return set_error(EA_ERR_ARG, "%s: both in place, or neither", what);
        if (o.dims < 2 || o.dims % 2 || o.dims > 2 * kRoPairs || o.offset < 0 || (int64_t)o.offset + o.dims > dim)
            return set_error(o.dims > 2 * kRoPairs ? EA_ERR_UNSUPPORTED : EA_ERR_SHAPE, "%s: columns %d to %lld of %lld (an even number, %d at most)", what,
                             o.offset, (long long)o.offset + o.dims, (long long)dim, 2 * kRoPairs);
        if (rows > INT32_MAX - 8191) return set_error(EA_ERR_UNSUPPORTED, "%s: more than %d rows", what, INT32_MAX - 8191);
        if (batch) {
            ea_status s = rows_args(what, batch, rows, true);
            if (!s && o.parents) s = tree_args(what, batch, o.parents, rows);
            if (s) return s;
        }
        for (int w = 0; w < 2 && out[w]; w++) {
            const void *a = out[w]->arena;
            const size_t n = out[w]->bytes;
            if (in_rows(batch, a, n) || ea::overlap(o.positions, rows * 4, a, n) || ea::overlap(o.parents, rows * 4, a, n))
                return set_error(EA_ERR_ARG, "%s: the batch, positions or parents lie in a result", what);
        }
        p.dim = (int32_t)dim;
        p.dims = o.dims;
        p.offset = o.offset;
        p.half = o.layout == EA_ROTARY_HALF;
        p.f32 = q->dtype == EA_F32;
        p.rows = rows;
        p.positions = o.positions;
        p.parents = o.parents;
        if (batch) {
            p.starts = batch->starts;
            p.lens = batch->lens;
            p.n_seqs = batch->n_seqs;
            p.max_new = most_new(batch, rows);
        }
        p.amplitude = o.amplitude == 0.0f ? 1.0f : o.amplitude;
        p.sign = o.backward ? -p.amplitude : p.amplitude;
        for (int i = 0; i < o.dims / 2; i++) {
            if (!std::isfinite(o.freqs[i])) return set_error(EA_ERR_ARG, "%s: frequency %d", what, i);
            double t = o.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
            t -= std::floor(t);
            t = t * 18446744073709551616.0;                  // 2^64: exact
            p.turn[i] = t >= 18446744073709551616.0 ? 0 : (uint64_t)t;
        }
        std::lock_guard<std::mutex> lk(g_mu);
        DevCtx *c;
        ea_status s = get_ctx(&c);
        if (s) return s;
        p.err = c->err;
        int64_t ctas = 0;
        if (rows > 0) {
            cudaError_t e = launch_rotary(p, c->num_sms, &ctas, (cudaStream_t)stream);
            if (e != cudaSuccess) return cuda_error(e, what);
        }
        note_launch(kRotary, ctas > 0, ctas);
        return EA_OK;
    });
}

extern "C" ea_status ea_verify_drafts(const ea_verify_opts *opts, const ea_page_batch *batch, ea_relation target, ea_relation draft,
                                      void *stream) {
    return entry([&]() -> ea_status {
        const char *what = "ea_verify_drafts";
        if (!opts || !target || !opts->sample || !opts->path || !opts->counts || !opts->picked)
            return set_error(EA_ERR_ARG, "%s: NULL argument", what);
        const ea_verify_opts &o = *opts;
        if (off_4({o.tokens, o.parents, o.accept, o.sample, o.path, o.counts, o.picked}))
            return set_error(EA_ERR_ARG, "%s: arrays must be aligned to 4 bytes", what);
        int64_t rows, vocab;
        ea_status s = dense_rows(target, what, 1, &rows, &vocab, nullptr);
        if (s) return s;
        if (rows > 0 && (!o.tokens || !o.accept)) return set_error(EA_ERR_ARG, "%s: NULL argument", what);
        if (vocab < 1 || vocab > INT32_MAX - 8191) return set_error(EA_ERR_UNSUPPORTED, "%s: a vocabulary of %lld", what, (long long)vocab);
        if (draft) {
            int64_t rows_d, vocab_d;
            s = dense_rows(draft, what, 1, &rows_d, &vocab_d, nullptr);
            if (s) return s;
            if (rows_d != rows || vocab_d != vocab) return set_error(EA_ERR_SHAPE, "%s: target and draft have different extents", what);
            if (draft->dtype != target->dtype) return set_error(EA_ERR_DTYPE, "%s: target and draft have different dtypes", what);
        }
        s = rows_args(what, batch, rows, false);
        if (s) return s;
        const int32_t most = most_new(batch, rows);
        if (most > kPgNodes) return set_error(EA_ERR_UNSUPPORTED, "%s: trees of up to %d nodes (%d at most; give max_new)", what, most, kPgNodes);
        if (o.width < 1 || o.width < most) return set_error(EA_ERR_ARG, "%s: paths of %d entries for trees of up to %d nodes", what, o.width, most);
        const size_t n = batch->n_seqs;
        const struct {
            const void *p;
            size_t bytes;
        } outs[3] = {{o.path, n * o.width * 4}, {o.counts, n * 4}, {o.picked, n * 4}},
          ins[6] = {{target->arena, target->bytes}, {draft ? draft->arena : nullptr, draft ? draft->bytes : 0}, {o.tokens, (size_t)rows * 4},
                    {o.parents, (size_t)rows * 4}, {o.accept, (size_t)rows * 4}, {o.sample, n * 4}};
        for (int i = 0; i < 3; i++) {
            bool bad = in_rows(batch, outs[i].p, outs[i].bytes);
            for (const auto &x : ins) bad |= ea::overlap(outs[i].p, outs[i].bytes, x.p, x.bytes);
            for (int j = 0; j < i; j++) bad |= ea::overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes);
            if (bad) return set_error(EA_ERR_ARG, "%s: a result overlaps an operand or another result", what);
        }
        std::lock_guard<std::mutex> lk(g_mu);
        DevCtx *c;
        s = get_ctx(&c);
        if (s) return s;
        VfParams p{};
        p.target = target->arena;
        p.draft = draft ? draft->arena : nullptr;
        p.tokens = o.tokens;
        p.parents = o.parents;
        p.starts = batch->starts;
        p.accept = o.accept;
        p.sample = o.sample;
        p.path = o.path;
        p.counts = o.counts;
        p.picked = o.picked;
        p.rows = rows;
        p.vocab = vocab;
        p.n_seqs = batch->n_seqs;
        p.max_new = most;
        p.width = o.width;
        p.bf16 = target->dtype == EA_BF16;
        p.err = c->err;
        int64_t ctas = 0;
        cudaError_t e = launch_verify(p, c->num_sms, &ctas, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_error(e, what);
        note_launch(kVerify, 1, ctas);
        return EA_OK;
    });
}

extern "C" ea_status ea_cache_keep(const ea_cache *caches, int32_t n_caches, const ea_page_batch *batch, const int32_t *path,
                                   int32_t width, const int32_t *counts, int32_t *lens_out, void *stream) {
    return entry([&]() -> ea_status {
        const char *what = "ea_cache_keep";
        if (!caches || !path || !counts || n_caches < 1) return set_error(EA_ERR_ARG, "%s: NULL argument or no cache", what);
        for (int i = 0; i < n_caches; i++)
            if (!caches[i]) return set_error(EA_ERR_ARG, "%s: NULL cache", what);
        ea_cache_s *f = caches[0];
        ea_status s = batch_args(batch, f->page, INT32_MAX - 8191);
        if (s) return s;
        if (batch->max_new < 1 || batch->max_new > kPgNodes)
            return set_error(EA_ERR_UNSUPPORTED, "%s: max_new %d (1 to %d nodes)", what, batch->max_new, kPgNodes);
        if (width < 1) return set_error(EA_ERR_ARG, "%s: paths of %d entries", what, width);
        if (off_4({path, counts, lens_out})) return set_error(EA_ERR_ARG, "%s: arrays must be aligned to 4 bytes", what);
        const size_t n = batch->n_seqs, path_bytes = n * width * 4;
        for (int i = 0; i < n_caches; i++) {
            const ea_cache_s *c = caches[i];
            if (c->format != f->format) return set_error(EA_ERR_DTYPE, "%s: caches of different formats", what);
            if (c->n_pages != f->n_pages || c->page != f->page || c->heads != f->heads || c->dim != f->dim)
                return set_error(EA_ERR_SHAPE, "%s: caches of different extents", what);
            if (c->device != f->device) return set_error(EA_ERR_ARG, "%s: caches on different devices", what);
        }
        // All arrays of the caches by address, so that neighbours tell of overlaps: layers are mostly made in order, and then
        // this insertion moves nothing.
        struct Span {
            const char *at;
            size_t bytes;
        };
        std::vector<Span> by;
        by.reserve(4 * (size_t)n_caches);
        const size_t cells = cache_bytes(f), scales = f->ks ? cells / (size_t)f->dim / (f->format == EA_CACHE_BF16 ? 2 : 1) : 0;
        auto put = [&](const void *p, size_t bytes) {
            size_t i = by.size();
            by.push_back({(const char *)p, bytes});
            for (; i > 0 && by[i - 1].at > (const char *)p; i--) std::swap(by[i - 1], by[i]);
        };
        for (int i = 0; i < n_caches; i++) put(caches[i]->k, cells);
        for (int i = 0; i < n_caches; i++) put(caches[i]->v, cells);
        for (int i = 0; scales && i < n_caches; i++) put(caches[i]->ks, scales);
        for (int i = 0; scales && i < n_caches; i++) put(caches[i]->vs, scales);
        for (size_t i = 1; i < by.size(); i++)
            if (by[i - 1].at + by[i - 1].bytes > by[i].at) return set_error(EA_ERR_ARG, "%s: caches overlap", what);
        const Span apart[] = {{(const char *)batch->pages, ((n - 1) * batch->page_stride + batch->max_pages) * 4},
                              {(const char *)batch->starts, (n + 1) * 4}, {(const char *)batch->lens, n * 4},
                              {(const char *)path, path_bytes}, {(const char *)counts, n * 4}, {(const char *)lens_out, n * 4}};
        for (const Span &x : apart) {
            if (!x.at) continue;
            // the first array that ends beyond x's beginning
            const auto i = std::partition_point(by.begin(), by.end(), [&](const Span &y) { return y.at + y.bytes <= x.at; });
            if (i != by.end() && i->at < x.at + x.bytes)
                return set_error(EA_ERR_ARG, "%s: the batch, the path or the lengths lie in a cache", what);
        }
        if (lens_out && (in_batch(batch, lens_out, n * 4) || overlap(lens_out, n * 4, path, path_bytes) || overlap(lens_out, n * 4, counts, n * 4)))
            return set_error(EA_ERR_ARG, "%s: lens_out overlaps the batch, the path or the counts", what);
        std::lock_guard<std::mutex> lk(g_mu);
        DevCtx *c;
        s = here(f, &c);
        if (s) return s;
        KpParams p{};
        p.t = table_of(batch, f->page, INT32_MAX - 8191);
        p.n_pages = f->n_pages;
        p.page_log2 = f->page_log2;
        p.heads = f->heads;
        p.row_bytes = f->dim * (f->format == EA_CACHE_BF16 ? 2 : 1);
        p.width = width;
        p.path = path;
        p.counts = counts;
        p.err = c->err;
        int64_t all = 0;
        int launches = 0;
        for (int i = 0; i < n_caches; i += kKeepCaches) {
            p.n_caches = std::min(kKeepCaches, n_caches - i);
            p.lens_out = i == 0 ? lens_out : nullptr;
            for (int j = 0; j < p.n_caches; j++) {
                p.k[j] = caches[i + j]->k;
                p.v[j] = caches[i + j]->v;
                p.ks[j] = caches[i + j]->ks;
                p.vs[j] = caches[i + j]->vs;
            }
            int64_t ctas = 0;
            cudaError_t e = launch_cache_keep(p, f->num_sms, &ctas, (cudaStream_t)stream);
            if (e != cudaSuccess) return cuda_error(e, what);
            all += ctas;
            launches++;
        }
        note_launch(kCacheRows, launches, all);
        return EA_OK;
    });
}
