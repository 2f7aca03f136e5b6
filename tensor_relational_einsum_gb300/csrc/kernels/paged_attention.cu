// paged_attention.cu -- attention over the paged cache, the plain way: one
// warp for a query row of one head.  Lanes take a key each for the scores (32
// keys at a time, fp32 sums), the running maximum and sum follow over the
// warp, and for the second product the lanes take D / 32 columns of V each.
#include "paged_common.cuh"

namespace ea {
namespace {

using namespace pg;

template <int D, bool E4M3>
__device__ __forceinline__ float cell(const PgPool &c, const char *pool, const uint8_t *scales, int64_t vec, int d) {
    if constexpr (E4M3) {
        const __half h = __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)pool[vec * D + d], __NV_E4M3));
        return __half2float(h) * scale_value(scales[vec]);
    } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(pool)[vec * D + d]);
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) plain_kernel(const __grid_constant__ PgAttn p, int min_rows) {
    __shared__ float s_q[4][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t at = (int64_t)blockIdx.x * 4 + warp;
    if (at >= p.t.rows * p.qheads) return;
    const int row = (int)(at / p.qheads), qh = (int)(at % p.qheads), head = qh / p.group;
    int a = 0, b = p.t.n_seqs - 1;
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (__ldg(p.t.starts + mid) <= row) a = mid;
        else b = mid - 1;
    }
    const PgSeq s = load_seq(p.t, a, p.c.page_log2, p.err);
    if (row < s.first || row >= s.first + s.n || (int64_t)s.n * p.group < min_rows) return;
    const int pos = s.len - s.n + (row - s.first);
    const int end = p.causal ? min(s.len, pos + 1) : s.len;
    const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(p.q) + at * D;
    for (int d = lane; d < D; d += 32) s_q[warp][d] = __bfloat162float(q[d]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int t0 = 0; t0 < end; t0 += 32) {
        const int t = t0 + lane;
        int64_t vec = 0;
        float x = -INFINITY;
        if (t < end) {
            const int g = load_page(p.t, p.c.n_pages, a, t >> p.c.page_log2, p.err);
            vec = pg_vec(p.c, g, head, t & ((1 << p.c.page_log2) - 1));
            x = 0.f;
            for (int d = 0; d < D; d++) x = fmaf(s_q[warp][d], cell<D, E4M3>(p.c, p.c.k, p.c.ks, vec, d), x);
            x *= p.scale;
        }
        float mx = x;
        for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const float m1 = fmaxf(m, mx), alpha = expf(m - m1), e = t < end ? expf(x - m1) : 0.f;
        float sum = e;
        for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        l = l * alpha + sum;
        m = m1;
        for (int i = 0; i < D / 32; i++) o[i] *= alpha;
        for (int j = 0; j < min(32, end - t0); j++) {
            const float w = __shfl_sync(0xffffffffu, e, j);
            const int64_t v = __shfl_sync(0xffffffffu, vec, j);
            for (int i = 0; i < D / 32; i++) o[i] = fmaf(w, cell<D, E4M3>(p.c, p.c.v, p.c.vs, v, 32 * i + lane), o[i]);
        }
    }
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.o) + at * D;
    for (int i = 0; i < D / 32; i++) out[32 * i + lane] = __float2bfloat16_rn(end > 0 ? o[i] / l : 0.f);
    if (p.m_out && lane == 0) {
        p.m_out[at] = m;
        p.l_out[at] = l;
    }
}

}  // namespace

cudaError_t launch_cache_attention(const PgAttn &p, int64_t *ctas, cudaStream_t st, int min_rows) {
    *ctas = (p.t.rows * p.qheads + 3) / 4;
    const unsigned n = (unsigned)*ctas;
    const bool e4m3 = p.c.fmt == EA_CACHE_E4M3;
    if (p.c.dim == 64) {
        if (e4m3) plain_kernel<64, true><<<n, 128, 0, st>>>(p, min_rows);
        else plain_kernel<64, false><<<n, 128, 0, st>>>(p, min_rows);
    } else {
        if (e4m3) plain_kernel<128, true><<<n, 128, 0, st>>>(p, min_rows);
        else plain_kernel<128, false><<<n, 128, 0, st>>>(p, min_rows);
    }
    return cudaGetLastError();
}

}  // namespace ea
