// Eviction from a cache by accumulated weight (mla_kv_evict): K of a stream's n keys stay, their table
// entries move together.
//
// A cluster of up to sixteen CTAs a stream.  Weights are compared as 32-bit integers in the order of the
// numbers; the K-th largest is found from histograms in shared memory (integer counts: no order of additions)
// over its first 13 bits, the next 11 and the last 8, as many of them as it takes.  The first pass keeps the
// integers in shared memory, up to 49152 a CTA, for the others.  Then the keys are taken in order, 8192 a CTA
// and round, the CTAs one behind the other, each key with its place from ballots and the counts of the warps
// and CTAs before it.  A round is read before anything of it is written, by all CTAs, and its places are not
// behind its own, so tables may be compacted in place.
#include "../../include/mla_verify.h"
#include "internal.cuh"

#include <cooperative_groups.h>
#include <limits.h>

#include <atomic>

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int NT = 1024;
constexpr int ITEMS = 8;                             // keys of a thread and round
constexpr int CHUNK = NT * ITEMS;
constexpr int MAX_CLUSTER = 16;
constexpr int BITS0 = 13, BITS1 = 11, BITS2 = 8;
constexpr int BINS = 1 << BITS0;
constexpr int MAX_KEPT = 49152;                      // integers that a CTA keeps in shared memory

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

struct Shared {
    int warp_sums[32];
    int slice[MAX_CLUSTER];                          // keys in every CTA's slice of the bins
    int found[3];                                    // bin, keys wanted of it, keys in it
    int totals[2][MAX_CLUSTER];                      // of every CTA's chunk: keys that stay | ties << 16
};

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
    const int before = __shfl_sync(0xffffffffu, s, (w + 31) & 31);
    return x + (w ? before : 0);
}

// Adds the lane's key to its bin, where it counts.  Weights that are all alike (zeros, say) meet in one bin: a
// warp of those adds once.
__device__ __forceinline__ void count(int* hist, bool counts, uint32_t bin) {
    const uint32_t first = __shfl_sync(0xffffffffu, bin, 0);
    if (__all_sync(0xffffffffu, counts && bin == first)) {
        if ((threadIdx.x & 31) == 0) atomicAdd(&hist[bin], 32);
    } else if (counts) {
        atomicAdd(&hist[bin], 1);
    }
}

// The bin, from the last one down, in which the cluster's `want`-th key lies; CTA r adds the r-th part of the
// bins up.  All histograms are zero afterwards.
__device__ __forceinline__ void find_bin(cg::cluster_group& cluster, int C, int rank, int* hist, int bins, Shared& s, int want) {
    const int tid = threadIdx.x;
    if (C > 1) cluster.sync();                           // every CTA has counted
    else __syncthreads();
    const int part = bins / C, per = (part + NT - 1) / NT, first = bins - 1 - rank * part;   // a thread's bins
    int mine[BINS / NT], sum = 0;
#pragma unroll
    for (int q = 0; q < BINS / NT; ++q) {
        mine[q] = 0;
        const int at = tid * per + q;
        if (q < per && at < part) {
            if (C == 1) mine[q] = hist[first - at];
            else
                for (int r = 0; r < C; ++r) mine[q] += *cluster.map_shared_rank(hist + first - at, r);
        }
        sum += mine[q];
    }
    int total, upto = block_scan(sum, s.warp_sums, &total);
    if (C > 1) {
        if (tid < C) *cluster.map_shared_rank(&s.slice[rank], tid) = total;
        cluster.sync();
        int before = 0;
        for (int r = 0; r < rank; ++r) before += s.slice[r];
        upto += before;
    }
    if (upto >= want && upto - sum < want) {             // one thread of the cluster
        int left = want - (upto - sum), q = 0;
#pragma unroll
        for (int k = 0; k < BINS / NT; ++k)
            if (k == q && left > mine[k]) { left -= mine[k]; ++q; }
        int in = 0;
#pragma unroll
        for (int k = 0; k < BINS / NT; ++k)
            if (k == q) in = mine[k];
        for (int r = 0; r < C; ++r) {
            int* f = C == 1 ? s.found : cluster.map_shared_rank(s.found, r);
            f[0] = first - (tid * per + q);
            f[1] = left;
            f[2] = in;
        }
    }
    for (int i = tid; i < bins; i += NT) hist[i] = 0;    // (read by now: behind the barriers of the scan or the cluster)
    if (C > 1) cluster.sync();
    else __syncthreads();
}

__global__ void __launch_bounds__(NT, 1) kv_evict_kernel(const EvictArgs a, int C, int cap) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared s;
    int* const hist = reinterpret_cast<int*>(smem);
    uint32_t* const held = reinterpret_cast<uint32_t*>(smem) + BINS;
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster.block_rank() : 0, b = blockIdx.x / C;
    const int n = a.seq_lens[b];
    for (int i = tid; i < BINS; i += NT) hist[i] = 0;
    if (C > 1) cluster.sync();                           // every CTA runs, and has read the length
    else __syncthreads();
    if (n < 0 || n > a.slot_stride) {
        if (rank == 0 && tid == 0) {
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
    // key i of the thread in round k, in the order of the stream: warps, then items, then lanes
    const int rounds = (int)(((long long)n + (long long)C * CHUNK - 1) / ((long long)C * CHUNK));
    const int mine0 = rank * CHUNK + warp * 32 * ITEMS + lane;
    // a key stays if its weight is above `top`, and of those equal to it the first `want`
    uint32_t top = 0;
    if (want > 0 && want < hi - lo) {
        for (int k = 0; k < rounds; ++k) {
            const long long j0 = (long long)k * C * CHUNK + mine0;
            float w[ITEMS];
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) w[i] = j0 + 32 * i < n ? a.weights[row + j0 + 32 * i] : 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const long long j = j0 + 32 * i;
                const uint32_t u = order_of(w[i]);
                const int at = k * CHUNK + i * NT + tid;
                if (at < cap) held[at] = u;
                count(hist, j >= lo && j < hi, u >> (32 - BITS0));
            }
        }
        int shift = 32 - BITS0;
        find_bin(cluster, C, rank, hist, BINS, s, want);
#pragma unroll 1
        for (;;) {
            top |= (uint32_t)s.found[0] << shift;
            want = s.found[1];
            const bool whole = want == s.found[2];
            if (whole) {                                 // the bin stays as a whole
                want = top ? 0 : INT_MAX;
                top = top ? top - 1 : 0;
            }
            if (whole || shift == 0) break;
            const int bits = shift == 32 - BITS0 ? BITS1 : BITS2, above = shift;
            shift -= bits;
            for (int k = 0; k < rounds; ++k) {
                const long long j0 = (long long)k * C * CHUNK + mine0;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    const long long j = j0 + 32 * i;
                    const int at = k * CHUNK + i * NT + tid;
                    const uint32_t u = at < cap ? held[at] : j < n ? order_of(a.weights[row + j]) : 0u;
                    if (j >= lo && j < hi && (u >> above) == (top >> above)) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1u)], 1);
                }
            }
            __syncthreads();                             // (found has been read)
            find_bin(cluster, C, rank, hist, 1 << bits, s, want);
        }
    } else if (want <= 0) {
        top = 0xffffffffu;                               // none, not even of the largest
        want = 0;
    } else {
        want = INT_MAX;                                  // all
    }
    int kept = 0, tied = 0;                              // before this round: keys above, ties
    for (int k = 0; k < rounds; ++k) {
        const long long j0 = (long long)k * C * CHUNK + mine0;
        float w[ITEMS];
        int slot[ITEMS], pos[ITEMS], doc[ITEMS];
        unsigned stay[ITEMS], tie[ITEMS];                // the warp's keys of item i
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const long long j = j0 + 32 * i;
            w[i] = 0.f;
            slot[i] = doc[i] = 0;
            pos[i] = (int)j;
            if (j < n) {
                w[i] = a.weights[row + j];
                slot[i] = a.slot[row + j];
                if (a.pos_out && a.key_pos) pos[i] = a.key_pos[row + j];
                if (a.doc_out) doc[i] = a.key_doc[row + j];
            }
        }
        int all = 0;                                     // the warp's: stay | ties << 16
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const long long j = j0 + 32 * i;
            const uint32_t u = order_of(w[i]);
            const bool mid = j >= lo && j < hi;
            stay[i] = __ballot_sync(0xffffffffu, j < n && (!mid || u > top));
            tie[i] = __ballot_sync(0xffffffffu, mid && u == top);
            all += __popc(stay[i]) | __popc(tie[i]) << 16;
        }
        __syncthreads();                                 // the sums of the round before have been read
        if (lane == 0) s.warp_sums[warp] = all;
        __syncthreads();
        int upto = s.warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int total = __shfl_sync(0xffffffffu, upto, 31);
        const int before_warp = __shfl_sync(0xffffffffu, upto, warp) - all;
        int before = 0, whole = total;
        if (C > 1) {
            if (tid < C) *cluster.map_shared_rank(&s.totals[k & 1][rank], tid) = total;
            cluster.sync();
            const int t = lane < C ? s.totals[k & 1][lane] : 0;
            // (sixteen chunks' counts pass 16 bits: added apart)
            int st = t & 0xffff, ti = t >> 16;
            int st_b = lane < rank ? st : 0, ti_b = lane < rank ? ti : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                st += __shfl_xor_sync(0xffffffffu, st, o);
                ti += __shfl_xor_sync(0xffffffffu, ti, o);
                st_b += __shfl_xor_sync(0xffffffffu, st_b, o);
                ti_b += __shfl_xor_sync(0xffffffffu, ti_b, o);
            }
            int up = kept + st_b + (before_warp & 0xffff), eq = tied + ti_b + (before_warp >> 16);
            kept += st;
            tied += ti;
            before = up;
            whole = eq;
        } else {
            before = kept + (before_warp & 0xffff);
            whole = tied + (before_warp >> 16);
            kept += total & 0xffff;
            tied += total >> 16;
        }
        const unsigned lower = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const long long j = j0 + 32 * i;
            const int eq = whole + __popc(tie[i] & lower);
            const int to = before + __popc(stay[i] & lower) + min(eq, want);
            const bool is_tie = (tie[i] >> lane) & 1u;
            if (((stay[i] >> lane) & 1u) || (is_tie && eq < want)) {
                a.table_out[row + to] = slot[i];
                a.weights_out[row + to] = w[i];
                if (a.pos_out) a.pos_out[row + to] = pos[i];
                if (a.doc_out) a.doc_out[row + to] = doc[i];
            } else if (j < n && a.freed) {
                a.freed[row + j - to] = slot[i];
            }
            before += __popc(stay[i]);
            whole += __popc(tie[i]);
        }
    }
    if (rank == 0 && tid == 0) {
        a.lens_out[b] = K;
        if (a.n_freed) a.n_freed[b] = n - K;
    }
}

// CTAs a stream: up to sixteen while they have a round each and the launch stays within one wave.
cudaError_t launch_kv_evict(const EvictArgs& a, int B, int num_sms, int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (BINS + MAX_KEPT) * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    int C = 1;
    while (C < MAX_CLUSTER && (long long)C * CHUNK < a.slot_stride && 2ll * C * B <= num_sms) C *= 2;
    const long long per_round = (long long)C * CHUNK, rounds = (a.slot_stride + per_round - 1) / per_round;
    const int cap = (int)min(rounds * CHUNK, (long long)MAX_KEPT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = (size_t)(BINS + cap) * 4;
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
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, a, C, cap);
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
    int num_sms = 0, dev = 0;
    const int rc = device_state(&dev, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    if (launch_kv_evict(a, B, num_sms, dev, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_LAUNCH;
    return MLA_OK;
}
