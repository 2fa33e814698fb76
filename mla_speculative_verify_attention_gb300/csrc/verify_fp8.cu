// Verify attention over the fp8 latent cache: the drafts, lengths, slot table and masks of
// mla_verify_attn over keys k_j = [scale_j * decode(lat_j) | rope_j], output in bf16.
//
// One CTA handles eight query rows (a warp each) over one key split: the keys of a tile are
// dequantised once into shared memory, each warp forms their scores by warp sums, keeps the
// running maximum and sum of the softmax and accumulates 16 output dims a lane in fp32.
#include "../../include/mla_verify.h"
#include "fp8_decode.cuh"
#include "internal.cuh"

#include <math.h>
#include <string.h>

namespace mla {
namespace {

constexpr int VF_WARPS = 8;
constexpr int VF_KEYS = 16;

struct Fp8Args {
    const __nv_bfloat16* q;
    const uint8_t* lat;
    const float* kscale;
    const __nv_bfloat16* rope;
    int64_t n_pool;
    const int32_t* slot;
    int slot_stride;
    const int32_t* seq_lens;
    const uint8_t* mask;
    const uint64_t* mask_bits;
    int B, q_len, H;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    float* part_out;
    float* part_lse;
    int nsplit;
    unsigned* status;
};

__global__ void __launch_bounds__(VF_WARPS * 32) verify_fp8_kernel(const Fp8Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float keys[VF_KEYS][D_QK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x, b = blockIdx.z;
    const int rows = a.q_len * a.H;
    const int r = blockIdx.y * VF_WARPS + warp;
    const bool row_ok = r < rows;
    const int n = a.seq_lens[b];
    const bool bad_len = n < a.q_len || n > a.slot_stride;
    int k0 = 0, k1 = 0;
    if (!bad_len) split_range(n, a.nsplit, s, VF_KEYS, &k0, &k1);
    const int p = n - a.q_len;
    const int t = row_ok ? r / a.H : 0;
    float qv[18], acc[16];
#pragma unroll
    for (int i = 0; i < 18; ++i)
        qv[i] = row_ok ? __bfloat162float(a.q[((int64_t)b * rows + r) * D_QK + i * 32 + lane]) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int k = k0; k < k1; k += VF_KEYS) {
        __syncthreads();
        for (int j = warp; j < VF_KEYS; j += VF_WARPS) {
            if (k + j >= k1) break;
            int sl = a.slot[(int64_t)b * a.slot_stride + k + j];
            if (sl < 0 || sl >= a.n_pool) {
                sl = 0;
                if (lane == 0) atomicOr(a.status, DEV_BAD_SLOT);
            }
            const float sc = a.kscale[sl];
            for (int d = lane; d < D_V; d += 32) {
                const __half_raw h = __nv_cvt_fp8_to_halfraw(a.lat[(int64_t)sl * D_V + d], __NV_E4M3);
                keys[j][d] = sc * __half2float(__half(h));
            }
            for (int d = lane; d < 64; d += 32) keys[j][D_V + d] = __bfloat162float(a.rope[(int64_t)sl * 64 + d]);
        }
        __syncthreads();
        if (!row_ok) continue;
        for (int j = 0; j < VF_KEYS && k + j < k1; ++j) {
            const int dr = k + j - p;
            if (dr >= 0) {
                bool seen = dr <= t;
                if (a.mask_bits) seen = (a.mask_bits[(int64_t)b * a.q_len + t] >> dr) & 1ull;
                else if (a.mask) seen = a.mask[((int64_t)b * a.q_len + t) * a.q_len + dr] != 0;
                if (!seen) continue;
            }
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 18; ++i) x += qv[i] * keys[j][i * 32 + lane];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            x *= a.scale;
            const float mn = fmaxf(m, x), c = expf(m - mn), w = expf(x - mn);
            l = l * c + w;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = acc[i] * c + w * keys[j][i * 32 + lane];
            m = mn;
        }
    }
    if (!row_ok) return;
    if (bad_len && lane == 0) atomicOr(a.status, DEV_BAD_LEN);
    const float inv = l != 0.f ? 1.f / l : 0.f;             // a NaN sum (a NaN key that is seen) stays NaN
    const float lse = bad_len ? __int_as_float(0x7fc00000) : (l != 0.f ? m + logf(l) : -INFINITY);
    const int64_t row = (int64_t)b * rows + r;
    if (a.nsplit == 1) {
        for (int i = 0; i < 16; ++i) a.out[row * D_V + i * 32 + lane] = __float2bfloat16_rn(acc[i] * inv);
        if (lane == 0) a.lse[row] = lse;
    } else {
        for (int i = 0; i < 16; ++i) a.part_out[(row * a.nsplit + s) * D_V + i * 32 + lane] = acc[i] * inv;
        if (lane == 0) a.part_lse[row * a.nsplit + s] = lse;
    }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_verify_attn_fp8(const void* q, const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope,
                                   int64_t n_pool, const int32_t* slot_table, int slot_stride,
                                   const int32_t* seq_lens, const uint8_t* draft_mask, const uint64_t* draft_mask_bits,
                                   int B, int q_len, int H, float scale, void* out, float* lse, int nsplit,
                                   void* workspace, size_t ws_bytes, mla_stream_t stream) {
    if (B < 0 || B > 65535 || q_len < 1 || q_len > MLA_MAX_Q_LEN || H < 1 || H > MLA_MAX_HEADS) return MLA_ERR_SHAPE;
    if (nsplit < 0 || nsplit > MLA_MAX_NSPLIT) return MLA_ERR_NSPLIT;
    if (B == 0) return MLA_OK;
    if (!q || !kv_lat || !kv_scale || !kv_rope || !slot_table || !seq_lens || !out || !lse) return MLA_ERR_NULL;
    if (n_pool < 1 || n_pool > 0x7fffffffLL || slot_stride < q_len) return MLA_ERR_SHAPE;
    if ((long long)B * q_len * H > 0x7fffffffLL) return MLA_ERR_SHAPE;
    if (!isfinite(scale) || (draft_mask && draft_mask_bits)) return MLA_ERR_ARG;
    if (!aligned(q, 16) || !aligned(kv_lat, 16) || !aligned(kv_rope, 16) || !aligned(kv_scale, 4) ||
        !aligned(slot_table, 4) || !aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(draft_mask_bits, 8))
        return MLA_ERR_ALIGN;
    Fp8Args a;
    memset(&a, 0, sizeof a);
    int num_sms = 0;
    int rc = device_state(nullptr, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    const int ns = nsplit > 0 ? nsplit : mla_verify_auto_nsplit(B, q_len, H, slot_stride, num_sms, workspace ? ws_bytes : 0);
    const long long rows = (long long)B * q_len * H;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.lat = kv_lat; a.kscale = kv_scale; a.rope = static_cast<const __nv_bfloat16*>(kv_rope);
    a.n_pool = n_pool; a.slot = slot_table; a.slot_stride = slot_stride; a.seq_lens = seq_lens;
    a.mask = draft_mask; a.mask_bits = draft_mask_bits;
    a.B = B; a.q_len = q_len; a.H = H; a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out); a.lse = lse; a.nsplit = ns;
    if (ns > 1) {
        if (!workspace || ws_bytes < mla_verify_workspace_bytes(B, q_len, H, ns)) return MLA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return MLA_ERR_ALIGN;
        a.part_out = static_cast<float*>(workspace);
        a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)rows * ns * D_V * 4));
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_dependent(verify_fp8_kernel, dim3(ns, (q_len * H + VF_WARPS - 1) / VF_WARPS, B), dim3(VF_WARPS * 32), 0,
                         st, a) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    if (ns > 1 && launch_combine_bf16(a.part_out, a.part_lse, rows, ns, a.out, lse, st) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    return MLA_OK;
}
