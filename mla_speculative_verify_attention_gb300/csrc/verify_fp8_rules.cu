// mla_verify_attn_fp8_rules(): the attention of verify_fp8.cuh under score rules.
#include "verify_fp8.cuh"

#include <cooperative_groups.h>

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int GAP_NT = 1024, GAP_CLUSTER = 8, GAP_UNROLL = 8;

// Of the groups start .. start + count - 1: hidden ones at the beginning, at the end, the longest run and where.
struct Run {
    int start, count, pre, suf, best, at;
};
__device__ __forceinline__ Run join(const Run& x, const Run& y) {
    Run z = {x.start, x.count + y.count, x.pre == x.count ? x.count + y.pre : x.pre,
             y.suf == y.count ? y.count + x.suf : y.suf, x.best, x.at};
    const int over = x.suf + y.pre;
    if (over > z.best) { z.best = over; z.at = x.start + x.count - x.suf; }
    if (y.best > z.best) { z.best = y.best; z.at = y.at; }
    return z;
}

// A cluster (of short streams, or of many, a CTA) a stream; a warp takes consecutive groups of 32 keys.
__global__ void __launch_bounds__(GAP_NT) key_gaps_kernel(const ScoreRules r, const int32_t* seq_lens, int q_len, int slot_stride,
                                                          int C, int2* gaps) {
    __shared__ Run warps[GAP_NT / 32], ctas[GAP_CLUSTER];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x / C, rank = blockIdx.x % C;
    const int n = seq_lens[b];
    if (n < q_len || n > slot_stride) {                  // (the cluster as a whole)
        if (rank == 0 && tid == 0) gaps[b] = make_int2(0, 0);
        return;
    }
    if (C > 1) cluster.barrier_arrive();                 // this CTA runs: the wait is where another's memory is written
    const int64_t row = (int64_t)b * slot_stride;
    const int p = n - q_len;
    // documents and window of all drafts together
    int lo = INT_MAX, first_doc = INT_MAX, last_doc = INT_MIN;
    for (int t = lane; t < q_len; t += 32) {
        const RowRule one = r.row(b, t, 0, p, slot_stride, false);
        lo = min(lo, one.lo);
        first_doc = min(first_doc, one.doc);
        last_doc = max(last_doc, one.doc);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    first_doc = __reduce_min_sync(0xffffffffu, first_doc);
    last_doc = __reduce_max_sync(0xffffffffu, last_doc);
    const int prefix = r.prefix_lens ? r.prefix_lens[b] : INT_MIN;
    const int groups = p / 32, per = (groups + C * (GAP_NT / 32) - 1) / (C * (GAP_NT / 32));
    Run mine = {min((rank * (GAP_NT / 32) + warp) * per, groups), 0, 0, 0, 0, 0};
    const int end = min(mine.start + per, groups);
    for (int g = mine.start; g < end; g += GAP_UNROLL) {
        int doc[GAP_UNROLL], pos[GAP_UNROLL];
#pragma unroll
        for (int i = 0; i < GAP_UNROLL; ++i) {
            const int j = min(g + i, end - 1) * 32 + lane;
            doc[i] = r.key_doc ? r.key_doc[row + j] : -1;
            pos[i] = r.key_pos ? r.key_pos[row + j] : j;
        }
#pragma unroll
        for (int i = 0; i < GAP_UNROLL; ++i) {
            const bool hidden = (doc[i] >= 0 && (doc[i] < first_doc || doc[i] > last_doc)) || (pos[i] < lo && pos[i] >= prefix);
            const bool all = __all_sync(0xffffffffu, hidden);
            if (g + i < end) mine = join(mine, Run{g + i, 1, all, all, all, g + i});
        }
    }
    auto reduce = [&](Run x, int lanes) {
        for (int o = 1; o < lanes; o <<= 1) {
            Run y;
            y.start = __shfl_down_sync(0xffffffffu, x.start, o);
            y.count = __shfl_down_sync(0xffffffffu, x.count, o);
            y.pre = __shfl_down_sync(0xffffffffu, x.pre, o);
            y.suf = __shfl_down_sync(0xffffffffu, x.suf, o);
            y.best = __shfl_down_sync(0xffffffffu, x.best, o);
            y.at = __shfl_down_sync(0xffffffffu, x.at, o);
            x = join(x, y);                              // (of lanes that are not a multiple of 2 o nobody reads it)
        }
        return x;
    };
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    Run all = {};
    if (warp == 0) all = reduce(warps[lane], 32);
    if (C > 1) {
        cluster.barrier_wait();                          // every CTA of the cluster runs
        if (tid == 0) *cluster.map_shared_rank(&ctas[rank], 0) = all;
        cluster.sync();
        if (rank > 0) return;
        if (warp == 0) all = reduce(ctas[lane % C], C);
    }
    if (tid == 0) gaps[b] = all.best > 0 ? make_int2(all.at * 32, all.best * 32) : make_int2(0, 0);
}

}  // namespace

cudaError_t launch_key_gaps(const ScoreRules& r, const int32_t* seq_lens, int B, int q_len, int slot_stride, int2* gaps,
                            cudaStream_t stream) {
    // (clusters of eight reach 120 of the SMs at once)
    int C = slot_stride > 8192 ? GAP_CLUSTER : 1;
    while (C > 1 && (long long)B * C > 120) C /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(GAP_NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, key_gaps_kernel, r, seq_lens, q_len, slot_stride, C, gaps);
}

int check_rules(float softcap, const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                const int32_t* key_doc, ScoreRules* out) {
    if (!(softcap >= 0.f) || !isfinite(softcap) || window < 0) return MLA_ERR_ARG;
    if (!aligned(slopes, 4) || !aligned(key_pos, 4) || !aligned(prefix_lens, 4) || !aligned(key_doc, 4))
        return MLA_ERR_ALIGN;
    ScoreRules r;
    r.softcap = fminf(softcap, MAX_CAP); r.window = window; r.slopes = slopes; r.key_pos = key_pos; r.prefix_lens = prefix_lens;
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
