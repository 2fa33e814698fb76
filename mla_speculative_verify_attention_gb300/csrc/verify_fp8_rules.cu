// mla_verify_attn_fp8_rules(): the attention of verify_fp8.cuh under score rules.
#include "verify_fp8.cuh"

namespace mla {

int check_rules(float softcap, const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                const int32_t* key_doc, ScoreRules* out) {
    if (!(softcap >= 0.f) || !isfinite(softcap) || window < 0) return MLA_ERR_ARG;
    if (!aligned(slopes, 4) || !aligned(key_pos, 4) || !aligned(prefix_lens, 4) || !aligned(key_doc, 4))
        return MLA_ERR_ALIGN;
    ScoreRules r;
    r.softcap = softcap; r.window = window; r.slopes = slopes; r.key_pos = key_pos; r.prefix_lens = prefix_lens;
    r.key_doc = key_doc;
    r.masked = window > 0 || prefix_lens || key_doc;
    r.spans = r.masked && (key_pos || key_doc);
    *out = r;
    return MLA_OK;
}

}  // namespace mla

using namespace mla;

extern "C" int mla_verify_attn_fp8_rules(const void* q, const uint8_t* kv_lat, const float* kv_scale,
                                         const void* kv_rope, int64_t n_pool, const int32_t* slot_table,
                                         int slot_stride, const int32_t* seq_lens, const uint8_t* draft_mask,
                                         const uint64_t* draft_mask_bits, int B, int q_len, int H, float scale,
                                         float softcap, const float* slopes, const int32_t* key_pos, int window,
                                         const int32_t* prefix_lens, const int32_t* key_doc, void* out, float* lse,
                                         int nsplit, void* workspace, size_t ws_bytes, mla_stream_t stream) {
    ScoreRules rules;
    const int rc = check_rules(softcap, slopes, key_pos, window, prefix_lens, key_doc, &rules);
    if (rc != MLA_OK) return rc;
    if (softcap == 0.f && !slopes && !rules.masked)      // no rule: positions alone change nothing
        return mla_verify_attn_fp8(q, kv_lat, kv_scale, kv_rope, n_pool, slot_table, slot_stride, seq_lens, draft_mask,
                                   draft_mask_bits, B, q_len, H, scale, out, lse, nsplit, workspace, ws_bytes, stream);
    return verify_fp8_call<true>(q, kv_lat, kv_scale, kv_rope, n_pool, slot_table, slot_stride, seq_lens, draft_mask,
                                 draft_mask_bits, B, q_len, H, scale, rules, out, lse, nsplit, workspace, ws_bytes,
                                 stream);
}
