// mla_verify_attn_fp8(): the kernel and its launches are in verify_fp8.cuh.
#include "verify_fp8.cuh"

using namespace mla;

extern "C" int mla_verify_attn_fp8(const void* q, const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope,
                                   int64_t n_pool, const int32_t* slot_table, int slot_stride,
                                   const int32_t* seq_lens, const uint8_t* draft_mask, const uint64_t* draft_mask_bits,
                                   int B, int q_len, int H, float scale, void* out, float* lse, int nsplit,
                                   void* workspace, size_t ws_bytes, mla_stream_t stream) {
    return verify_fp8_call<false>(q, kv_lat, kv_scale, kv_rope, n_pool, slot_table, slot_stride, seq_lens, draft_mask,
                                  draft_mask_bits, B, q_len, H, scale, ScoreRules{}, out, lse, nsplit, workspace,
                                  ws_bytes, stream);
}

extern "C" size_t mla_verify_fp8_workspace_bytes(int B, int q_len, int H, int max_seq, int num_sms) {
    if (B <= 0 || q_len < 1 || q_len > MLA_MAX_Q_LEN || H < 1 || H > MLA_MAX_HEADS || max_seq < 1 || num_sms < 1) return 0;
    int n_tiles, R_step, R;
    fp8_tiling(q_len * H, &n_tiles, &R_step, &R);
    const size_t uniform = mla_verify_workspace_bytes(B, q_len, H, fp8_auto_nsplit(B, n_tiles, R, max_seq, num_sms));
    const size_t slot_rows = (size_t)fp8_balanced_slots(B, n_tiles, num_sms) * q_len * H;
    const size_t balanced = align256(slot_rows * D_V * 4) + align256(slot_rows * 4);
    return balanced ? balanced : uniform;
}
