// Eviction from a cache by accumulated weight (mla_kv_evict): K of a stream's n keys stay, their table
// entries move together.
//
// A block a stream.  Weights are compared as 32-bit integers in the order of the numbers; the K-th largest
// is found eight bits a pass with a histogram in shared memory (integer counts: no order of additions),
// then the keys are taken in order, a block's width at a time, each with its place from a scan.  A chunk
// is read before anything of it is written, and its places are not behind its own, so tables may be
// compacted in place.
#include "../../include/mla_verify.h"
#include "internal.cuh"

#include <limits.h>

namespace mla {
namespace {

constexpr int NT = 1024;

struct EvictArgs {
    const int32_t* slot;
    const int32_t* seq_lens;
    const float* weights;
    const int32_t* key_pos;
    const int32_t* key_doc;
    int slot_stride;
    const int32_t* budgets;
    int budget, sink, recent;
    int32_t* table_out;
    int32_t* lens_out;
    float* weights_out;
    int32_t* pos_out;
    int32_t* doc_out;
    int32_t* freed;
    int32_t* n_freed;
    unsigned* status;
};

// The number's place in the order: NaN above all, -0 beside 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Inclusive sum over the block of x, and the block's total.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                     // the sums of the scan before have been read
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return x + (w ? __shfl_sync(0xffffffffu, s, w - 1) : 0);
}

__global__ void __launch_bounds__(NT) kv_evict_kernel(const EvictArgs a) {
    __shared__ int hist[256], sums[32];
    __shared__ int found[2];
    const int b = blockIdx.x, tid = threadIdx.x, n = a.seq_lens[b];
    if (n < 0 || n > a.slot_stride) {
        __syncthreads();
        if (tid == 0) {
            atomicOr(a.status, DEV_BAD_LEN);
            a.lens_out[b] = n;
            if (a.n_freed) a.n_freed[b] = 0;
        }
        return;
    }
    const int64_t row = (int64_t)b * a.slot_stride;
    const int budget = max(0, a.budgets ? a.budgets[b] : a.budget);
    const int K = (int)min((long long)n, max((long long)budget, (long long)a.sink + a.recent));
    // of the keys lo .. hi - 1 the `want` largest stay
    const int lo = min(a.sink, n), hi = max(lo, (int)max((long long)n - a.recent, 0ll));
    int want = K - lo - (n - hi);
    uint32_t top = 0;                                    // the want-th largest's leading bits, then all
    if (want > 0 && want < hi - lo) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += NT) {
                const uint32_t u = order_of(a.weights[row + j]);
                if (shift == 24 || (u >> (shift + 8)) == (top >> (shift + 8))) atomicAdd(&hist[(u >> shift) & 255], 1);
            }
            __syncthreads();
            int total;
            const int mine = tid < 256 ? hist[255 - tid] : 0;
            const int upto = block_scan(mine, sums, &total);
            if (tid < 256 && upto >= want && upto - mine < want) {
                found[0] = 255 - tid;
                found[1] = want - (upto - mine);
            }
            __syncthreads();
            top |= (uint32_t)found[0] << shift;
            want = found[1];
            __syncthreads();
        }
    } else if (want <= 0) {
        top = 0xffffffffu;                               // none, not even of the largest
        want = 0;
    } else {
        want = INT_MAX;                                  // all: top = 0
    }
    int kept = 0, ties = 0;
    for (int j0 = 0; j0 < n; j0 += NT) {
        const int j = j0 + tid;
        uint32_t u = 0;
        float w = 0.f;
        int slot = 0, pos = j, doc = 0;
        if (j < n) {
            w = a.weights[row + j];
            slot = a.slot[row + j];
            if (a.key_pos) pos = a.key_pos[row + j];
            if (a.key_doc) doc = a.key_doc[row + j];
            u = order_of(w);
        }
        const bool mid = j >= lo && j < hi, tie = mid && u == top;
        int total;
        const int rank = block_scan(tie, sums, &total);
        const bool keep = j < n && (!mid || u > top || (tie && ties + rank <= want));
        ties += total;
        const int to = block_scan(keep, sums, &total) - 1 + kept;
        if (keep) {
            a.table_out[row + to] = slot;
            a.weights_out[row + to] = w;
            if (a.pos_out) a.pos_out[row + to] = pos;
            if (a.doc_out) a.doc_out[row + to] = doc;
        } else if (j < n && a.freed) {
            a.freed[row + j - (to + 1)] = slot;
        }
        kept += total;
    }
    if (tid == 0) {
        a.lens_out[b] = K;
        if (a.n_freed) a.n_freed[b] = n - K;
    }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_kv_evict(const int32_t* slot_table, const int32_t* seq_lens, const float* weights,
                            const int32_t* key_pos, const int32_t* key_doc, int B, int slot_stride,
                            const int32_t* budgets, int budget, int sink, int recent, int32_t* table_out,
                            int32_t* lens_out, float* weights_out, int32_t* pos_out, int32_t* doc_out, int32_t* freed,
                            int32_t* n_freed, mla_stream_t stream) {
    if (B < 0 || B > 65535 || slot_stride < 1 || slot_stride > MLA_MAX_FP8_KEYS) return MLA_ERR_SHAPE;
    if (sink < 0 || recent < 0) return MLA_ERR_ARG;
    if (B == 0) return MLA_OK;
    if (!slot_table || !seq_lens || !weights || !table_out || !lens_out || !weights_out) return MLA_ERR_NULL;
    if (!freed != !n_freed) return MLA_ERR_NULL;
    if (doc_out && !key_doc) return MLA_ERR_ARG;
    const void* all[] = {slot_table, seq_lens, weights, key_pos, key_doc, budgets, table_out,
                         lens_out, weights_out, pos_out, doc_out, freed, n_freed};
    for (const void* p : all)
        if (!aligned(p, 4)) return MLA_ERR_ALIGN;
    EvictArgs a = {slot_table, seq_lens, weights, key_pos, key_doc, slot_stride, budgets, budget, sink, recent, table_out,
                   lens_out, weights_out, pos_out, doc_out, freed, n_freed, nullptr};
    const int rc = device_state(nullptr, &a.status, nullptr);
    if (rc != MLA_OK) return rc;
    kv_evict_kernel<<<B, NT, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH;
}
