// Score rules of the long-context operators: what a score q.k goes through before the softmax, and
// which keys a draft sees.
//     z = scale q.k,   z = softcap tanh(z / softcap),   z += slopes[h] (pos(key) - pos(draft))
//     a key is seen iff its document is the draft's or negative, and it is either within the draft
//     mask and the window (pos(draft) - pos(key) < window) or in the prefix (pos(key) < prefix_lens[b])
// A draft's position and document are those of its own key.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "internal.cuh"

namespace mla {

// 2^x, relative error 2^-22 (denormal results are 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(u) for a = 2 u log2(e).  Away from zero 1 - 2 / (2^a + 1): the quotient, at most 0.76, is off by
// 1.5 2^-22 of itself, so tanh by 2^-21.8 absolute, or 2^-19.8 of itself at the least u; below u = 1/4,
// where that would cancel, the odd series up to u^9 (the next term is 2^-26 of the sum).
__device__ __forceinline__ float capped(float a) {
    const float e = ex2(a) + 1.f;
    float q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(e));
    const float u = a * 0.34657359027997264f, w = u * u;         // ln(2) / 2
    float s = fmaf(w, 62.f / 2835.f, -17.f / 315.f);
    s = fmaf(w, s, 2.f / 15.f);
    s = fmaf(w, s, -1.f / 3.f);
    s = fmaf(w * s, u, u);
    return fabsf(a) < 0.72134752044448170f ? s : fmaf(-2.f, q, 1.f);   // u = 1/4
}

// One query row's part of the rules.
struct RowRule {
    int pos, lo, prefix, doc;      // keys below position `lo` are out of the window
    float slope;                   // in log2 units

    __device__ __forceinline__ bool sees(bool draft_ok, int key_pos, int key_doc) const {
        return ((draft_ok && key_pos >= lo) || key_pos < prefix) && (key_doc == doc || key_doc < 0);
    }
};

struct ScoreRules {
    float softcap = 0.f;                       // 0: none
    int window = 0;                            // 0: none
    const float* slopes = nullptr;             // [H]
    const int32_t* key_pos = nullptr;          // [B, slot_stride]; null: a key's index
    const int32_t* prefix_lens = nullptr;      // [B]
    const int32_t* key_doc = nullptr;          // [B, slot_stride]
    int masked = 0;                            // a window, a prefix or documents

    // The keys that have to be looked at: with given positions any of them may be visible.
    __host__ __device__ __forceinline__ KeySpan span() const {
        KeySpan s;
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

// MLA_OK, or what is wrong with the rules' arguments.
int check_rules(float softcap, const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                const int32_t* key_doc, ScoreRules* out);

}  // namespace mla
