// paged_common.cuh -- device helpers shared by the paged cache's kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../paged.h"
#include "dev_common.cuh"

namespace ea {
namespace pg {

__device__ __forceinline__ void batch_fail(int *err) { atomicCAS(err, 0, (int)kDevBatch); }

// Sequence i of the table; out of range: raises the error word, no rows.
__device__ __forceinline__ PgSeq load_seq(const PgTable &t, int i, int *err) {
    PgSeq s;
    if (!pg_seq(__ldg(t.starts + i), __ldg(t.starts + i + 1), __ldg(t.lens + i), t.rows, t.max_new, t.cap, &s))
        batch_fail(err);
    return s;
}

// The kernels of an attention call overlap at their ends (programmatic
// dependent launch): each lets the next be placed as soon as it runs, and
// waits for the one before it to be complete, at the latest before it ends
// itself, so that the last one's end is the end of all.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch behind the stream's last kernel; `early`: it may be placed before
// that one has ended (the kernel calls wait_for_previous).
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool early, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A page number; out of range: raises the error word and names page 0, so
// that what follows stays inside the pool.
__device__ __forceinline__ int32_t check_page(int32_t g, int64_t n_pages, int *err) {
    if (g >= 0 && g < n_pages) return g;
    batch_fail(err);
    return 0;
}

// 32 bytes at once: as two stores of 16 each of them fills half a sector.
// Relations are aligned to 16 bytes only; off a 32-byte boundary it is two
// stores after all.
__device__ __forceinline__ void st_32(void *dst, const uint32_t *x) {
    if (((uintptr_t)dst & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// Four e4m3 bytes as f16: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// 2^e for -126 <= e <= 127; 0 below.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)max(e + 127, 0) << 23); }

// The value of a scale byte: 2^(b - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Scale byte of a vector whose largest magnitude has the fp32 bits `amax`:
// the least e with |x| <= 448 * 2^e (448 = 1.75 * 2^8), kept in [-126, 120].
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255u;  // an infinity or NaN
    if (amax == 0u) return 127u;
    const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(-126, min(120, e)) + 127);
}

}  // namespace pg
}  // namespace ea
