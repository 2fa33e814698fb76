// The fp8 latent cache's own writer and reader.
//
// Append: a bf16 row x[0:576] is quantised as it is written,
//     scale = max_{d<512} |x[d]| / 448  (fp32),  code[d] = e4m3(x[d] / scale),
// 448 being the largest e4m3 value, e4m3() rounding to nearest even and saturating; the
// rope dims stay bf16.  One scale a token, so a row can be written without touching any
// other.  The maximum is over the finite values: an infinity saturates to +-448 and a NaN
// keeps the NaN code, so neither costs the other 511 values their precision.  A row without a
// finite value other than zero has scale 0, and reads back as zeros (and NaN).  Read: the reverse,
// scale * decode(code) in fp32 (28 bits rounded to 24) and that product in bf16.
//
// Both are bound by HBM (1152 B of bf16 row and 644 B of quantised row each way): one warp
// a row, 8 dims a lane and step, so that every load and store is a full line.
//
// Measured on GB300: append of 46080 rows 15.6 us (5.3 TB/s), read of 169817 scattered rows 48.2 us
// (6.3 TB/s); 72 and 4105 rows 1.7 and 2.3 us, a launch.  Append with the slot read and checked
// before the row is loaded takes 17.9 us, so the row's loads come first.
#include "../../include/mla_verify.h"
#include "fp8_decode.cuh"
#include "internal.cuh"

namespace mla {
namespace {

constexpr int KQ_THREADS = 128;
constexpr float E4M3_MAX = 448.f;

__device__ __forceinline__ void row8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// max |f|, NaN left out; with `finite`, infinities too.
__device__ __forceinline__ float max_abs8(const float (&f)[8], float m, bool finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(f[i]);
        m = fmaxf(m, finite && a == INFINITY ? 0.f : a);
    }
    return m;
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// x / scale, correctly rounded: with inv = 1 / scale correctly rounded, each step
// q + (x - q scale) inv brings a quotient that is a few units off to within one, and one that is
// within a unit to the correctly rounded one (Markstein 1990).  Taken as q - (q scale - x) inv: a zero
// of either sign then leaves q = +-0 as it is, where a correction that is added makes +0 of it.  Needs
// a scale well inside the normal range; five operations where the general division takes a dozen.
__device__ __forceinline__ float divide(float x, float scale, float inv) {
    float q = __fmul_rn(x, inv);
    q = fmaf(-fmaf(q, scale, -x), inv, q);
    return fmaf(-fmaf(q, scale, -x), inv, q);
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float scale, float inv, bool finite) {
    float r[8];
    if (finite && scale > 8.6736174e-19f && scale < 1.1529215e18f) {       // 2^-60, 2^60
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = divide(f[i], scale, inv);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = scale > 0.f ? __fdiv_rn(f[i], scale) : f[i];
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(r[4 * h], r[4 * h + 1]), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(r[4 * h + 2], r[4 * h + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    return make_uint2(w[0], w[1]);
}

__global__ void __launch_bounds__(KQ_THREADS)
    kv_append_quant_kernel(uint8_t* __restrict__ kv_lat, float* __restrict__ kv_scale,
                           __nv_bfloat16* __restrict__ kv_rope, int64_t n_pool, const int32_t* __restrict__ slots,
                           const __nv_bfloat16* __restrict__ rows, int n_rows, unsigned* status) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = ((int64_t)blockIdx.x * KQ_THREADS + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= n_rows) return;
    // the row is on its way before the slot is looked at
    const int s = __ldg(slots + i);
    const uint4* src = reinterpret_cast<const uint4*>(rows + i * D_QK);
    const uint4 ra = __ldg(src + lane), rb = __ldg(src + 32 + lane);
    const uint4 rope = lane < 8 ? __ldg(src + 64 + lane) : make_uint4(0, 0, 0, 0);
    if (s < 0 || (int64_t)s >= n_pool) {
        if (lane == 0) atomicOr(status, DEV_BAD_SLOT);
        return;
    }
    float a[8], b[8];
    row8(ra, a);
    row8(rb, b);
    float m = warp_max(max_abs8(b, max_abs8(a, 0.f, false), false));
    const bool finite = m < INFINITY;                  // (of what is not NaN)
    if (!finite) m = warp_max(max_abs8(b, max_abs8(a, 0.f, true), true));
    const float scale = __fdiv_rn(m, E4M3_MAX);
    uint2* lat = reinterpret_cast<uint2*>(kv_lat + (int64_t)s * D_V);
    const float inv = __frcp_rn(scale);
    lat[lane] = encode8(a, scale, inv, finite);
    lat[32 + lane] = encode8(b, scale, inv, finite);
    if (lane < 8) reinterpret_cast<uint4*>(kv_rope + (int64_t)s * 64)[lane] = rope;
    if (lane == 0) kv_scale[s] = scale;
}

__device__ __forceinline__ uint4 decode8(const uint2& c, float scale) {
    uint32_t o[4];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
        const float2 f = __half22float2(h);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(KQ_THREADS)
    kv_read_fp8_kernel(const uint8_t* __restrict__ kv_lat, const float* __restrict__ kv_scale,
                       const __nv_bfloat16* __restrict__ kv_rope, int64_t n_pool, const int32_t* __restrict__ slots,
                       __nv_bfloat16* __restrict__ out, int n_rows, unsigned* status) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = ((int64_t)blockIdx.x * KQ_THREADS + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= n_rows) return;
    const int s = slots[i];
    uint4* dst = reinterpret_cast<uint4*>(out + i * D_QK);
    if (s < 0 || (int64_t)s >= n_pool) {
        if (lane == 0) atomicOr(status, DEV_BAD_SLOT);
        const uint4 z = make_uint4(0, 0, 0, 0);
        dst[lane] = z;
        dst[32 + lane] = z;
        if (lane < 8) dst[64 + lane] = z;
        return;
    }
    const uint2* lat = reinterpret_cast<const uint2*>(kv_lat + (int64_t)s * D_V);
    const uint2 a = __ldg(lat + lane), b = __ldg(lat + 32 + lane);
    const float scale = __ldg(kv_scale + s);
    uint4 rope = make_uint4(0, 0, 0, 0);
    if (lane < 8) rope = __ldg(reinterpret_cast<const uint4*>(kv_rope + (int64_t)s * 64) + lane);
    dst[lane] = decode8(a, scale);
    dst[32 + lane] = decode8(b, scale);
    if (lane < 8) dst[64 + lane] = rope;
}

int check_cache(const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope, int64_t n_pool,
                const int32_t* slots, const void* rows, int n_rows) {
    if (n_rows < 0) return MLA_ERR_SHAPE;
    if (n_rows == 0) return MLA_OK;
    if (!kv_lat || !kv_scale || !kv_rope || !slots || !rows) return MLA_ERR_NULL;
    if (n_pool < 1 || n_pool > 0x7fffffffLL) return MLA_ERR_SHAPE;
    if (!aligned(kv_lat, 16) || !aligned(kv_rope, 16) || !aligned(rows, 16) || !aligned(kv_scale, 4) ||
        !aligned(slots, 4))
        return MLA_ERR_ALIGN;
    return MLA_OK;
}

unsigned warps_grid(int n_rows) { return (unsigned)(((int64_t)n_rows * 32 + KQ_THREADS - 1) / KQ_THREADS); }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_kv_append_quant(uint8_t* kv_lat, float* kv_scale, void* kv_rope, int64_t n_pool,
                                   const int32_t* slots, const void* rows, int n_rows, mla_stream_t stream) {
    int rc = check_cache(kv_lat, kv_scale, kv_rope, n_pool, slots, rows, n_rows);
    if (rc != MLA_OK || n_rows == 0) return rc;
    unsigned* status = nullptr;
    rc = device_state(nullptr, &status, nullptr);
    if (rc != MLA_OK) return rc;
    if (launch_dependent(kv_append_quant_kernel, dim3(warps_grid(n_rows)), dim3(KQ_THREADS), 0,
                         reinterpret_cast<cudaStream_t>(stream), kv_lat, kv_scale,
                         static_cast<__nv_bfloat16*>(kv_rope), n_pool, slots, static_cast<const __nv_bfloat16*>(rows),
                         n_rows, status) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    return MLA_OK;
}

extern "C" int mla_kv_read_fp8(const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope, int64_t n_pool,
                               const int32_t* slots, void* out, int n_rows, mla_stream_t stream) {
    int rc = check_cache(kv_lat, kv_scale, kv_rope, n_pool, slots, out, n_rows);
    if (rc != MLA_OK || n_rows == 0) return rc;
    unsigned* status = nullptr;
    rc = device_state(nullptr, &status, nullptr);
    if (rc != MLA_OK) return rc;
    if (launch_dependent(kv_read_fp8_kernel, dim3(warps_grid(n_rows)), dim3(KQ_THREADS), 0,
                         reinterpret_cast<cudaStream_t>(stream), kv_lat, kv_scale,
                         static_cast<const __nv_bfloat16*>(kv_rope), n_pool, slots,
                         static_cast<__nv_bfloat16*>(out), n_rows, status) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    return MLA_OK;
}
