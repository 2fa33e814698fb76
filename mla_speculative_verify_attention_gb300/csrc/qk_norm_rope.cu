// RMS norm of the latent dims and position rotation of the rope dims, for the queries'
// heads and the new key rows of a step in one launch:
//     y[d]         = x[d] * w[d] / sqrt(mean_{d<512} x[d]^2 + eps)            (d < 512; w NULL: x[d])
//     (y_a, y_b)   = (x_a cos - x_b sin, x_b cos + x_a sin), angle = position * inv_freq[i]
// with the pair (a, b) = 512 + (2i, 2i + 1) or 512 + (i, i + 32), i < 32.  Statistics and
// products are fp32; each output value is rounded to bf16 once.
//
// Angle: a position times a frequency in fp32 is off by position * 2^-25, a sixteenth of a
// radian at 2^20, and the GPU's few fp64 units would bound the kernel.  So the frequency is
// held in turns as a 64-bit binary fraction F = inv_freq / (2 pi) * 2^64, made once per
// block in fp64, and position * F modulo 2^64 is the angle's fraction of a turn: exact
// integer arithmetic but for F's own rounding (2^-53 relative).
//
// Bound by HBM: a row is read once and written once (2 x 1152 B).  A block serves up to eight rows
// of one token (heads, and the key row last): its four warps issue the loads of two rows each,
// one warp computes the 32 sines and cosines that the rows share while they are on their way,
// and each lane then handles one 16-byte piece of 8 dims a step.  Measured, 1152 tokens of 64
// heads (173 MB): 29.9 us, 5.8 TB/s; four rows a warp 31.9, eight warps of one row 33.6.
#include "../../include/mla_verify.h"
#include "internal.cuh"

#include <math.h>

namespace mla {
namespace {

constexpr int NR_WARPS = 4;
constexpr int NR_ROWS = 2;       // rows a warp has in flight

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(NR_WARPS * 32)
    qk_norm_rope_kernel(const __nv_bfloat16* q, const __nv_bfloat16* kv, const __nv_bfloat16* __restrict__ q_weight,
                        const __nv_bfloat16* __restrict__ kv_weight, const int32_t* __restrict__ positions,
                        const float* __restrict__ inv_freq, float eps, int interleaved, int H, int rows_per_block,
                        __nv_bfloat16* q_out, __nv_bfloat16* kv_out) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float s_cos[32], s_sin[32];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_q = q ? H : 0, rows = n_q + (kv ? 1 : 0);
    const int r0 = blockIdx.y * rows_per_block + warp, r_end = min(rows, (int)(blockIdx.y + 1) * rows_per_block);
    // all of the warp's rows are under way before the angles are made
    uint4 v[NR_ROWS][3];
#pragma unroll
    for (int u = 0; u < NR_ROWS; ++u) {
        const int r = r0 + u * NR_WARPS;
        if (r >= r_end) break;
        const uint4* src = reinterpret_cast<const uint4*>(r < n_q ? q + (t * H + r) * D_QK : kv + t * D_QK);
        v[u][0] = src[lane];
        v[u][1] = src[32 + lane];
        v[u][2] = lane < 8 ? src[64 + lane] : make_uint4(0, 0, 0, 0);
    }
    if (warp == 0) {
        const double turns = (double)inv_freq[lane] * 0.15915494309189533577;   // 1 / (2 pi)
        // the fraction of a turn, as a 64-bit binary fraction (whole turns drop out)
        const long long F = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
        const long long frac = (long long)((unsigned long long)F * (unsigned long long)(long long)positions[t]);
        float sn, cs;
        sincospif((float)(int)(frac >> 32) * 4.656612873077393e-10f, &sn, &cs);  // half turns: 2^-31
        s_cos[lane] = cs;
        s_sin[lane] = sn;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NR_ROWS; ++u) {
        const int r = r0 + u * NR_WARPS;
        if (r >= r_end) break;
        const bool is_q = r < n_q;
        uint4* dst = reinterpret_cast<uint4*>(is_q ? q_out + (t * H + r) * D_QK : kv_out + t * D_QK);
        const uint4* w = reinterpret_cast<const uint4*>(is_q ? q_weight : kv_weight);
        if (w) {
            float fa[8], fb[8], wt[8], ss = 0.f;
            unpack8(v[u][0], fa);
            unpack8(v[u][1], fb);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += fa[i] * fa[i] + fb[i] * fb[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.f / D_V) + eps);
            unpack8(__ldg(w + lane), wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) fa[i] = fa[i] * inv * wt[i];
            unpack8(__ldg(w + 32 + lane), wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) fb[i] = fb[i] * inv * wt[i];
            v[u][0] = pack8(fa);
            v[u][1] = pack8(fb);
        }
        dst[lane] = v[u][0];
        dst[32 + lane] = v[u][1];
        float x[8], y[8];
        unpack8(v[u][2], x);
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float cs = s_cos[(4 * lane + i) & 31], sn = s_sin[(4 * lane + i) & 31];
                y[2 * i] = x[2 * i] * cs - x[2 * i + 1] * sn;
                y[2 * i + 1] = x[2 * i + 1] * cs + x[2 * i] * sn;
            }
        } else {
            // lanes 0-3 hold the pairs' first halves, lanes 4-7 the second
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float other = __shfl_xor_sync(0xffffffffu, x[i], 4);
                const float cs = s_cos[(8 * lane + i) & 31], sn = s_sin[(8 * lane + i) & 31];
                y[i] = lane < 4 ? x[i] * cs - other * sn : x[i] * cs + other * sn;
            }
        }
        if (lane < 8) dst[64 + lane] = pack8(y);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const __nv_bfloat16* q, const __nv_bfloat16* kv, const __nv_bfloat16* q_weight,
                                const __nv_bfloat16* kv_weight, const int32_t* positions, const float* inv_freq,
                                float eps, int interleaved, int64_t T, int H, __nv_bfloat16* q_out,
                                __nv_bfloat16* kv_out, cudaStream_t stream) {
    const int rows = (q ? H : 0) + (kv ? 1 : 0);
    const int blocks = (rows + NR_WARPS * NR_ROWS - 1) / (NR_WARPS * NR_ROWS);
    const int rows_per_block = (rows + blocks - 1) / blocks;
    const dim3 grid((unsigned)T, (unsigned)blocks);
    return launch_dependent(qk_norm_rope_kernel, grid, dim3(NR_WARPS * 32), 0, stream, q, kv, q_weight, kv_weight,
                            positions, inv_freq, eps, interleaved, H, rows_per_block, q_out, kv_out);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_qk_norm_rope(const void* q, const void* kv, const void* q_weight, const void* kv_weight,
                                const int32_t* positions, const float* inv_freq, float eps, int interleaved,
                                int64_t n_tokens, int H, void* q_out, void* kv_out, mla_stream_t stream) {
    if (n_tokens < 0 || n_tokens > 0x7fffffffLL || H < 1 || H > MLA_MAX_HEADS) return MLA_ERR_SHAPE;
    if (n_tokens == 0) return MLA_OK;
    if ((!q && !kv) || (q && !q_out) || (kv && !kv_out) || !positions || !inv_freq) return MLA_ERR_NULL;
    if (!(eps >= 0.f) || !isfinite(eps)) return MLA_ERR_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(q_weight, 16) || !aligned(kv_weight, 16) ||
        !aligned(q_out, 16) || !aligned(kv_out, 16) || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return MLA_ERR_ALIGN;
    int rc = device_state(nullptr, nullptr, nullptr);
    if (rc != MLA_OK) return rc;
    using bf = __nv_bfloat16;
    if (launch_qk_norm_rope(static_cast<const bf*>(q), static_cast<const bf*>(kv), static_cast<const bf*>(q_weight),
                            static_cast<const bf*>(kv_weight), positions, inv_freq, eps, interleaved ? 1 : 0, n_tokens,
                            H, static_cast<bf*>(q_out), static_cast<bf*>(kv_out),
                            reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    return MLA_OK;
}
