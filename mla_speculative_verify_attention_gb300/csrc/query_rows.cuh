// Query rows and key codes on their way to the tensor cores, for the kernels over the fp8 cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "internal.cuh"

namespace mla {

// Four e4m3 codes (byte i = code i) as four fp16 values; exact, NaN stays NaN.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    return make_uint2((uint32_t)lo.x | ((uint32_t)lo.y << 16), (uint32_t)hi.x | ((uint32_t)hi.y << 16));
}

// Two bf16 values (one word) times f, a power of two, as two fp16 values.
__device__ __forceinline__ uint32_t q_to_f16(uint32_t w, float f) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t q_to_bf16(uint32_t w, float f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// N query rows, a row a warp: rows first, first + step, ..; rows past nrows are zeros.
template <int N>
__device__ __forceinline__ void load_q_rows(uint4 (&v)[N][3], const __nv_bfloat16* q0, int first, int step, int nrows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int rr = first + u * step;
        const uint4* src = reinterpret_cast<const uint4*>(q0 + (int64_t)rr * D_QK);
#pragma unroll
        for (int c = 0; c < 3; ++c)
            v[u][c] = rr < nrows && c * 32 + lane < 72 ? __ldg(src + c * 32 + lane) : make_uint4(0, 0, 0, 0);
    }
}

// The exponent of each row's largest element (the warp holds the rows as load_q_rows left them), within
// what keeps 2^(14 - e) and 2^(e - 14) finite.
template <int N>
__device__ __forceinline__ void row_exponents(const uint4 (&v)[N][3], int (&e)[N]) {
    __nv_bfloat162 top[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        __nv_bfloat162 m[3];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const uint32_t w[4] = {v[u][c].x & 0x7fff7fffu, v[u][c].y & 0x7fff7fffu, v[u][c].z & 0x7fff7fffu,
                                   v[u][c].w & 0x7fff7fffu};
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
            m[c] = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        }
        top[u] = __hmax2(__hmax2(m[0], m[1]), m[2]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const uint32_t w = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&top[u]), o);
            top[u] = __hmax2(top[u], *reinterpret_cast<const __nv_bfloat162*>(&w));
        }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const float big = fmaxf(__low2float(top[u]), __high2float(top[u]));
        e[u] = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 127);
    }
}

}  // namespace mla
