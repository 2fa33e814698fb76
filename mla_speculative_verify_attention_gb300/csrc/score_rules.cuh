// Score rules of the long-context operators: what a score q.k goes through before the softmax, and
// which keys a draft sees.
//     z = scale q.k,   z = softcap tanh(z / softcap),   z += slopes[h] (pos(key) - pos(draft))
//     a key is seen iff its document is the draft's or negative, and it is either within the draft
//     mask and the window (pos(draft) - pos(key) < window) or in the prefix (pos(key) < prefix_lens[b])
// A draft's position and document are those of its own key.
#pragma once

#include <float.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "internal.cuh"

namespace mla {

// 2^x, relative error 2^-22 (denormal results are 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t bits_of(float2 x) {
    uint64_t v;
    memcpy(&v, &x, sizeof v);
    return v;
}
__device__ __forceinline__ float2 pair_of(uint64_t v) {
    float2 x;
    memcpy(&x, &v, sizeof x);
    return x;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
    return pair_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return pair_of(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// tanh(u) = u + u w P(w), w = u^2, for |u| <= 1: the polynomial of least relative error, 2^-24.1 (fitted by
// reweighted least squares on Chebyshev nodes); 2^-22.6 with the roundings of fp32.
__device__ __forceinline__ float2 tanh_near(float2 u) {
    const float2 w = mul2(u, u);
    float2 s = fma2(w, both(0.0010582641698420048f), both(-0.0062593379989266396f));
    s = fma2(s, w, both(0.020359758287668228f));
    s = fma2(s, w, both(-0.053498707711696625f));
    s = fma2(s, w, both(0.13326409459114075f));
    s = fma2(s, w, both(-0.33332985639572144f));
    return fma2(mul2(w, s), u, u);
}
// Farther out 1 - 2 / (e^2|u| + 1) with u's sign: the quotient, at most 0.24 there, is off by 1.5 2^-22 of itself.
__device__ __forceinline__ float tanh_far(float u) {
    const float e = ex2(fabsf(u) * 2.8853900817779268f) + 1.f;
    float q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(e));
    return copysignf(fmaf(-2.f, q, 1.f), u);
}
__device__ __forceinline__ float2 tanh2(float2 u) {
    const float2 near = tanh_near(u);
    return make_float2(fabsf(u.x) <= 1.f ? near.x : tanh_far(u.x), fabsf(u.y) <= 1.f ? near.y : tanh_far(u.y));
}

// A row's capped scores in log2 units are cap_out tanh(cap_in x), where c2 x are the uncapped ones.  Under the largest
// caps cap_in would lose its bits below 2^-126: there tanh is its argument for every x below 2^88, and so it is with
// PLAIN_IN.  Under the smallest ones cap_in stays finite: a score of 0 is 0.
constexpr float PLAIN_IN = 0x1p-100f;
__device__ __forceinline__ float cap_in(float c2, float softcap) {
    const float in = c2 / (softcap * 1.4426950408889634f);
    return fabsf(in) < 0x1p-126f ? PLAIN_IN : fminf(fmaxf(in, -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ float cap_out(float c2, float softcap, float in) {
    return in == PLAIN_IN ? c2 * 0x1p100f : softcap * 1.4426950408889634f;
}
// Caps are at most this: in log2 units they are below 2^128.
constexpr float MAX_CAP = 0x1.62e4p127f;

// One query row's part of the rules.
struct RowRule {
    int pos, lo, prefix, doc;      // keys below position `lo` are out of the window
    float slope;                   // in log2 units

    __device__ __forceinline__ bool sees(bool draft_ok, int key_pos, int key_doc) const {
        return ((draft_ok && key_pos >= lo) || key_pos < prefix) && (key_doc == doc || key_doc < 0);
    }
    // Of keys before the drafts with positions span.x .. span.y and documents span.z .. span.w: sees none, or all.
    __device__ __forceinline__ bool none(int4 span) const {
        return (span.y < lo && span.x >= prefix) || (span.z >= 0 && (doc < span.z || doc > span.w));
    }
    __device__ __forceinline__ bool all(int4 span) const {
        return (span.x >= lo || span.y < prefix) && (span.w < 0 || (span.z == span.w && span.z == doc));
    }
};

struct ScoreRules {
    float softcap = 0.f;                       // 0: none
    int window = 0;                            // 0: none
    const float* slopes = nullptr;             // [H]
    const int32_t* key_pos = nullptr;          // [B, slot_stride]; null: a key's index
    const int32_t* prefix_lens = nullptr;      // [B]
    const int32_t* key_doc = nullptr;          // [B, slot_stride]
    const int2* gaps = nullptr;                // [B], of launch_key_gaps
    int masked = 0;                            // a window, a prefix or documents,
    int spans = 0;                             // and positions or documents given key by key

    // The keys that have to be looked at: with given positions any of them may be visible.
    __host__ __device__ __forceinline__ KeySpan span() const {
        KeySpan s;
        s.gaps = gaps;
        if (!key_pos) {
            s.window = window;
            s.prefix_lens = prefix_lens;
        }
        return s;
    }
    // Rule of draft t, head h of stream b, whose draft 0 is key p; `skip`: nothing is read.
    __device__ __forceinline__ RowRule row(int b, int t, int h, int p, int slot_stride, bool skip) const {
        RowRule r;
        r.pos = p + t;
        r.doc = -1;
        r.lo = r.prefix = INT_MIN;
        r.slope = 0.f;
        if (skip) return r;
        const int64_t at = (int64_t)b * slot_stride + p + t;
        if (key_doc) r.doc = __ldg(key_doc + at);
        if (key_pos) r.pos = __ldg(key_pos + at);
        if (window > 0) r.lo = (int)max((long long)r.pos - window + 1, (long long)INT_MIN);
        if (prefix_lens) r.prefix = __ldg(prefix_lens + b);
        if (slopes) r.slope = __ldg(slopes + h) * 1.4426950408889634f;
        return r;
    }
};

// Whether keys that no draft sees can lie together without being known from the lengths alone.
inline bool has_gaps(const ScoreRules& r) { return r.key_doc || (r.key_pos && r.window > 0); }
// Finds (a cluster of eight CTAs for long streams) each stream's longest run of keys before the drafts that none of them sees (in whole groups of 32):
// gaps[b] = its first key, its keys.
cudaError_t launch_key_gaps(const ScoreRules& r, const int32_t* seq_lens, int B, int q_len, int slot_stride, int2* gaps,
                            cudaStream_t stream);

// MLA_OK, or what is wrong with the rules' arguments.
int check_rules(float softcap, const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                const int32_t* key_doc, ScoreRules* out);

}  // namespace mla
