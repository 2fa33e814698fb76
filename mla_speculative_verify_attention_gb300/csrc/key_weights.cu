// The weight that each cached key got from the rows of a step (mla_key_weights, mla_key_weights_fp8):
//     new_j = sum over rows r = (t, h) that count and see key j of exp(z_rj - lse_r)
//     out_j = decay * weights_j + new_j
// The attention's log-sum-exp is given, so there is no softmax to run: every (row, key) pair stands for itself.
//
// A warp a key; lane l holds dims 16 l .. 16 l + 15 of the latent and 2 l, 2 l + 1 of the rotated part.  The
// latent's sum and the rotated part's stay apart until the key's scale is known, as in the attention.
#include "../../include/mla_verify.h"
#include "internal.cuh"
#include "score_rules.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

namespace mla {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int WARPS = 8;

struct WeightArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kv;      // the bf16 cache, or
    const uint8_t* lat;           // the fp8 cache
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
    ScoreRules rules;
    const float* lse;
    const uint8_t* counted;
    const float* weights;
    float decay;
    float* out;
    unsigned* status;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool FP8>
__global__ void __launch_bounds__(32 * WARPS) key_weights_kernel(const WeightArgs a) {
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int n = a.seq_lens[b];
    if (n < a.q_len || n > a.slot_stride) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, DEV_BAD_LEN);
        return;
    }
    const int p = n - a.q_len;
    for (int64_t j = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); j < n; j += (int64_t)gridDim.x * WARPS) {
        const int64_t at = (int64_t)b * a.slot_stride + j;
        int sl = a.slot[at];
        if (sl < 0 || (int64_t)sl >= a.n_pool) {
            if (lane == 0) atomicOr(a.status, DEV_BAD_SLOT);
            sl = 0;
        }
        float k[16], r0, r1, ks = 1.f;
        if (FP8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.lat + (int64_t)sl * D_V) + lane);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3));
                k[2 * i] = __low2float(h);
                k[2 * i + 1] = __high2float(h);
            }
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(a.rope + (int64_t)sl * 64) + lane);
            r0 = bf_lo(x);
            r1 = bf_hi(x);
            ks = a.kscale[sl];
        } else {
            const uint4* row = reinterpret_cast<const uint4*>(a.kv + (int64_t)sl * D_QK);
            const uint4 v[2] = {__ldg(row + 2 * lane), __ldg(row + 2 * lane + 1)};
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) { k[2 * i] = bf_lo(w[i]); k[2 * i + 1] = bf_hi(w[i]); }
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(row + 64) + lane);
            r0 = bf_lo(x);
            r1 = bf_hi(x);
        }
        const int kp = a.rules.key_pos ? a.rules.key_pos[at] : (int)j, kd = a.rules.key_doc ? a.rules.key_doc[at] : -1;
        float sum = 0.f;
        for (int t = 0; t < a.q_len; ++t) {
            if (a.counted && !a.counted[b * a.q_len + t]) continue;
            bool draft_ok = j < p;
            if (!draft_ok) {
                const int i = (int)(j - p);
                draft_ok = a.mask_bits ? (a.mask_bits[(int64_t)b * a.q_len + t] >> i) & 1ull
                           : a.mask    ? a.mask[((int64_t)b * a.q_len + t) * a.q_len + i] != 0
                                       : i <= t;
            }
            for (int h = 0; h < a.H; ++h) {
                const RowRule rule = a.rules.row(b, t, h, p, a.slot_stride, false);
                if (!rule.sees(draft_ok, kp, kd)) break;
                const int64_t r = ((int64_t)b * a.q_len + t) * a.H + h;
                const uint4* row = reinterpret_cast<const uint4*>(a.q + r * D_QK);
                const uint4 v[2] = {__ldg(row + 2 * lane), __ldg(row + 2 * lane + 1)};
                const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
                const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(row + 64) + lane);
                float A = 0.f, C = bf_lo(x) * r0 + bf_hi(x) * r1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    A = fmaf(bf_lo(w[i]), k[2 * i], A);
                    A = fmaf(bf_hi(w[i]), k[2 * i + 1], A);
                }
                for (int o = 16; o; o >>= 1) {
                    A += __shfl_xor_sync(0xffffffffu, A, o);
                    C += __shfl_xor_sync(0xffffffffu, C, o);
                }
                float z = fmaf(A, ks, C) * (a.scale * LOG2E);
                if (a.rules.softcap > 0.f) z = capped(z * (2.f / a.rules.softcap)) * (a.rules.softcap * LOG2E);
                if (a.rules.slopes) z = fmaf((float)(kp - rule.pos), rule.slope, z);
                const float l = a.lse[r];
                if (l != -INFINITY) sum += ex2(fmaf(-l, LOG2E, z));
            }
        }
        if (lane == 0) a.out[at] = a.weights && j < p ? fmaf(a.decay, a.weights[at], sum) : sum;
    }
}

template <bool FP8>
int key_weights_call(WeightArgs a, const uint64_t* bits, cudaStream_t stream) {
    if (a.B < 0 || a.B > 65535 || a.q_len < 1 || a.q_len > MLA_MAX_Q_LEN || a.H < 1 || a.H > MLA_MAX_HEADS) return MLA_ERR_SHAPE;
    if (a.B == 0) return MLA_OK;
    if (!a.q || (FP8 ? !a.lat || !a.kscale || !a.rope : !a.kv) || !a.slot || !a.seq_lens || !a.lse || !a.out) return MLA_ERR_NULL;
    if (a.n_pool < 1 || a.n_pool > 0x7fffffffLL || a.slot_stride < a.q_len || a.slot_stride > MLA_MAX_FP8_KEYS) return MLA_ERR_SHAPE;
    if ((long long)a.B * a.q_len * a.H > 0x7fffffffLL) return MLA_ERR_SHAPE;
    if (!isfinite(a.scale) || !isfinite(a.decay) || (a.mask && bits)) return MLA_ERR_ARG;
    if (!aligned(a.q, 16) || !aligned(a.lat, 16) || !aligned(a.rope, 16) || !aligned(a.kscale, 4) || !aligned(a.kv, 16) ||
        !aligned(a.slot, 4) || !aligned(a.seq_lens, 4) || !aligned(a.lse, 4) || !aligned(a.weights, 4) ||
        !aligned(a.out, 4) || !aligned(bits, 8))
        return MLA_ERR_ALIGN;
    a.mask_bits = bits;
    int num_sms = 0;
    const int rc = device_state(nullptr, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    const int blocks = (int)min((a.slot_stride + WARPS - 1) / WARPS, max(1, 8 * num_sms / a.B));
    key_weights_kernel<FP8><<<dim3(blocks, a.B), 32 * WARPS, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH;
}

WeightArgs weight_args(const void* q, int64_t n_pool, const int32_t* slot_table, int slot_stride, const int32_t* seq_lens,
                       const uint8_t* draft_mask, int B, int q_len, int H, float scale, const ScoreRules& rules,
                       const float* lse, const uint8_t* counted, const float* weights, float decay, float* out) {
    WeightArgs a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_pool = n_pool; a.slot = slot_table; a.slot_stride = slot_stride; a.seq_lens = seq_lens; a.mask = draft_mask;
    a.B = B; a.q_len = q_len; a.H = H; a.scale = scale; a.rules = rules;
    a.lse = lse; a.counted = counted; a.weights = weights; a.decay = decay; a.out = out;
    return a;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_key_weights_fp8(const void* q, const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope,
                                   int64_t n_pool, const int32_t* slot_table, int slot_stride, const int32_t* seq_lens,
                                   const uint8_t* draft_mask, const uint64_t* draft_mask_bits, int B, int q_len, int H,
                                   float scale, float softcap, const float* slopes, const int32_t* key_pos, int window,
                                   const int32_t* prefix_lens, const int32_t* key_doc, const float* lse,
                                   const uint8_t* counted, const float* weights, float decay, float* out,
                                   mla_stream_t stream) {
    ScoreRules rules;
    const int rc = check_rules(softcap, slopes, key_pos, window, prefix_lens, key_doc, &rules);
    if (rc != MLA_OK) return rc;
    WeightArgs a = weight_args(q, n_pool, slot_table, slot_stride, seq_lens, draft_mask, B, q_len, H, scale, rules, lse,
                               counted, weights, decay, out);
    a.lat = kv_lat; a.kscale = kv_scale; a.rope = static_cast<const __nv_bfloat16*>(kv_rope);
    return key_weights_call<true>(a, draft_mask_bits, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_key_weights(const void* q, const void* kv_cache, int64_t n_pool, const int32_t* slot_table,
                               int slot_stride, const int32_t* seq_lens, const uint8_t* draft_mask,
                               const uint64_t* draft_mask_bits, int B, int q_len, int H, float scale, float softcap,
                               const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                               const int32_t* key_doc, const float* lse, const uint8_t* counted, const float* weights,
                               float decay, float* out, mla_stream_t stream) {
    ScoreRules rules;
    const int rc = check_rules(softcap, slopes, key_pos, window, prefix_lens, key_doc, &rules);
    if (rc != MLA_OK) return rc;
    WeightArgs a = weight_args(q, n_pool, slot_table, slot_stride, seq_lens, draft_mask, B, q_len, H, scale, rules, lse,
                               counted, weights, decay, out);
    a.kv = static_cast<const __nv_bfloat16*>(kv_cache);
    return key_weights_call<false>(a, draft_mask_bits, reinterpret_cast<cudaStream_t>(stream));
}
