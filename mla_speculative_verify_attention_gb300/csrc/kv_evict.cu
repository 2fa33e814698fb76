// Eviction from a cache by accumulated weight (mla_kv_evict): K of a stream's n keys stay, their table
// entries move together.
//
// A cluster of up to sixteen CTAs a stream.  Weights are compared as 32-bit integers in the opposite order of the
// numbers; the K-th smallest is found from histograms in shared memory (integer counts: no order of additions)
// over its first 13 bits, the next 11 and the last 8, as many of them as it takes.  The first pass keeps the
// integers in shared memory, up to 40960 a CTA, for the others; the second lists the few that the third has to
// look at.  Then the keys are taken in order, each with its place from ballots and the counts of the keys
// before it, 8192 a CTA and round, the CTAs one behind the other.  A round is read before anything of it is
// written, by all CTAs, and its places are not behind its own, so tables may be compacted in place.
// Where several rounds are needed and no table is compacted in place, the cluster only leaves the border and
// each warp's counts in the workspace, and a second kernel over all SMs takes the keys.
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
constexpr int BINS = 1 << BITS0, ALL_BINS = BINS + (1 << BITS1) + (1 << BITS2);   // a pass its own
constexpr int GROUPS = 64;                           // of a pass's bins
constexpr int MAX_HELD = 40960;                      // integers that a CTA keeps in shared memory
constexpr int MAX_LIST = 4096;                       // and those of them that it lists

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
    struct Border* border;                           // workspace, or null: one kernel does it all
    int32_t* warp_counts;                            // [B][chunks * 32]: keys that stay | ties << 16, a warp's 256 keys
    int32_t* chunk_counts;                           // [B][chunks]: the same of a chunk of 8192
};

// What the first kernel leaves of a stream: a key j of lo .. hi - 1 stays if its integer is below `top`, and of
// those equal to it the first `want`; all others of the n keys stay.
struct Border {
    int n, lo, hi, want;
    uint32_t top;
};

// The number's place in the opposite order: NaN before all, -0 beside 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 0u : (u & 0x80000000u) ? u : ~(u | 0x80000000u);
}

constexpr uint32_t ZERO = 0x7fffffffu;               // order_of(0)
constexpr uint32_t NONE = 0xffffffffu;               // no number's: the last is that of -infinity, 0xff800000

// A thread's keys j0 + 32 i of the stream, and which of the warp's keys stay or tie.
struct Keys {
    float w[ITEMS];
    int slot[ITEMS], pos[ITEMS], doc[ITEMS];
    unsigned stay[ITEMS], tie[ITEMS];

    // Returns the warp's counts: stay | ties << 16.
    __device__ __forceinline__ int load(const EvictArgs& a, const Border& o, int64_t row, int j0, int items) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int j = j0 + 32 * i;
            w[i] = 0.f;
            slot[i] = doc[i] = 0;
            pos[i] = j;
            if (i < items && j < o.n) {
                w[i] = a.weights[row + j];
                slot[i] = a.slot[row + j];
                if (a.pos_out && a.key_pos) pos[i] = a.key_pos[row + j];
                if (a.doc_out) doc[i] = a.key_doc[row + j];
            }
        }
        int all = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (i >= items) break;
            const int j = j0 + 32 * i;
            const uint32_t u = order_of(w[i]);
            const bool mid = j >= o.lo && j < o.hi;
            stay[i] = __ballot_sync(0xffffffffu, j < o.n && (!mid || u < o.top));
            tie[i] = __ballot_sync(0xffffffffu, mid && u == o.top);
            all += __popc(stay[i]) | __popc(tie[i]) << 16;
        }
        return all;
    }
    // `before`, `equal`: keys before the warp's that stay for sure, and ties.
    __device__ __forceinline__ void write(const EvictArgs& a, const Border& o, int64_t row, int j0, int items, int before, int equal) const {
        const int lane = threadIdx.x & 31;
        const unsigned lower = (1u << lane) - 1u;
        before += min(equal, o.want);                    // with the ties that stay
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int j = j0 + 32 * i;
            if (i >= items || j - lane >= o.n) break;
            unsigned keep = stay[i];
            if (tie[i]) {                                // the first of them, as many as are wanted
                const int room = o.want - min(equal, o.want), m = __popc(tie[i]);
                equal += m;
                if (room >= m) keep |= tie[i];
                else if (room > 0) keep |= __ballot_sync(0xffffffffu, ((tie[i] >> lane) & 1u) && __popc(tie[i] & lower) < room);
            }
            const int to = before + __popc(keep & lower);
            before += __popc(keep);
            if ((keep >> lane) & 1u) {
                a.table_out[row + to] = slot[i];
                a.weights_out[row + to] = w[i];
                if (a.pos_out) a.pos_out[row + to] = pos[i];
                if (a.doc_out) a.doc_out[row + to] = doc[i];
            } else if (j < o.n && a.freed) {
                a.freed[row + j - to] = slot[i];
            }
        }
    }
};

struct Shared {
    int warp_sums[32];
    int groups[3][GROUPS];                           // a pass's keys in every sixty-fourth of the bins
    int found[3];                                    // bin, keys wanted of it, keys in it
    int listed;                                      // keys of the bin, as many as MAX_LIST in the list
    int totals[2][MAX_CLUSTER];                      // of every CTA's chunk: keys that stay | ties << 16
};

// A warp's search for the `want`-th of N <= 64 numbers in order, N / 32 (or 1) consecutive ones a lane: its
// index, what is wanted of it, and the number.  Any lane may have found it: the caller looks at `here`.
template <int PER>
__device__ __forceinline__ bool find_in_warp(const int (&v)[PER], int want, int* at, int* left, int* in) {
    const int lane = threadIdx.x & 31;
    int sum = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) sum += v[q];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    int rest = want - (upto - sum);
    const bool here = rest > 0 && upto >= want;
    bool done = false;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        if (!done) {
            *at = lane * PER + q;
            *in = v[q];
            done = rest <= v[q];
            if (!done) rest -= v[q];
        }
    }
    *left = rest;
    return here;
}

// The bin in which the cluster's `want`-th key lies.  Every CTA looks for itself: at all CTAs' sums of the 64
// groups of bins, then at the group's bins.  One cluster barrier: nobody writes these bins again.
template <int BINS_>
__device__ __forceinline__ void find_bin(cg::cluster_group& cluster, int C, int pass, int* hist, Shared& s, int want) {
    constexpr int G = BINS_ / GROUPS;                    // bins of a group: 128, 32 or 4
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __syncthreads();                                     // every warp has counted
    // two groups a warp
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int g = warp * 2 + h;
        int sum = 0;
#pragma unroll
        for (int q = 0; q < (G + 31) / 32; ++q)
            if (lane + 32 * q < G) sum += hist[g * G + 32 * q + lane];
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) s.groups[pass][g] = sum;
    }
    if (C > 1) cluster.sync();
    else __syncthreads();
    if (warp == 0) {
        int v[2] = {0, 0}, at = 0, left = 0, in = 0;
        if (C == 1) {
            v[0] = s.groups[pass][2 * lane];
            v[1] = s.groups[pass][2 * lane + 1];
        } else {
            int x[MAX_CLUSTER][2];
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {
                const int2 y = r < C ? *reinterpret_cast<const int2*>(cluster.map_shared_rank(&s.groups[pass][2 * lane], r)) : make_int2(0, 0);
                x[r][0] = y.x;
                x[r][1] = y.y;
            }
#pragma unroll
            for (int r = 0; r < MAX_CLUSTER; ++r) {
                v[0] += x[r][0];
                v[1] += x[r][1];
            }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, find_in_warp(v, want, &at, &left, &in));
        const int src = __ffs(hit) - 1;
        const int group = __shfl_sync(0xffffffffu, at, src), rest = __shfl_sync(0xffffffffu, left, src);
        constexpr int PER = (G + 31) / 32;
        int u[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) u[q] = 0;
        if (lane * PER < G) {
            const int* bins = hist + group * G + lane * PER;
            for (int r = 0; r < C; ++r) {
                const int* p = C == 1 ? bins : cluster.map_shared_rank(const_cast<int*>(bins), r);
#pragma unroll
                for (int q = 0; q < PER; ++q) u[q] += p[q];
            }
        }
        if (find_in_warp(u, rest, &at, &left, &in)) {
            s.found[0] = group * G + at;
            s.found[1] = left;
            s.found[2] = in;
        }
    }
    __syncthreads();
}

__global__ void __launch_bounds__(NT, 1) kv_evict_kernel(const EvictArgs a, int C, int cap) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared s;
    int* const hist = reinterpret_cast<int*>(smem);
    uint32_t* const list = reinterpret_cast<uint32_t*>(smem) + ALL_BINS;
    uint32_t* const held = list + MAX_LIST;
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster.block_rank() : 0, b = blockIdx.x / C;
    const int n = a.seq_lens[b];
    const int budget = max(0, a.budgets ? a.budgets[b] : a.budget);
    for (int i = tid; i < ALL_BINS / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    if (tid == 0) s.listed = 0;
    if (C > 1) cluster.sync();                           // every CTA runs, and has read the length
    else __syncthreads();
    if (n < 0 || n > a.slot_stride) {
        if (rank == 0 && tid == 0) {
            atomicOr(a.status, DEV_BAD_LEN);
            a.lens_out[b] = n;
            if (a.n_freed) a.n_freed[b] = 0;
            if (a.border) a.border[b] = Border{};
        }
        return;
    }
    const int64_t row = (int64_t)b * a.slot_stride;
    const float* const weights = a.weights + row;
    const int K = (int)min((long long)n, max((long long)budget, (long long)a.sink + a.recent));
    // of the keys lo .. hi - 1 the `want` heaviest stay
    const int lo = min(a.sink, n), hi = max(lo, (int)max((long long)n - a.recent, 0ll));
    int want = K - lo - (n - hi);
    // The thread's keys of round k are j0 + 32 i, in the order of the stream by warps, then items, then lanes.
    // (n + a round stays below 2^31: the table's width is at most 2^30.)
    // A stream of one round is shared out evenly: `items` keys a thread.
    const int items = a.border ? ITEMS : max(1, min(ITEMS, (n + C * NT - 1) / (C * NT)));
    const int step = C * NT * items, rounds = (n + step - 1) / step, mine0 = (rank * NT + warp * 32) * items + lane;
    // a key stays if its integer is below `top`, and of those equal to it the first `want`
    uint32_t top = 0;
    const bool formed = want > 0 && want < hi - lo;      // there is a choice: the integers are formed
    // Eight integers of the warp's 256 keys of round k (any eight: lane l those from 8 l on where they are held);
    // NONE for a key that is not among the lo .. hi - 1.
    auto eight = [&](int k, uint32_t (&u)[ITEMS]) {
        const int at = k * CHUNK + warp * 32 * ITEMS;
        if (at < cap) {
#pragma unroll
            for (int q = 0; q < ITEMS; q += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(held + at + lane * ITEMS + q);
                u[q] = v.x; u[q + 1] = v.y; u[q + 2] = v.z; u[q + 3] = v.w;
            }
        } else {
            const int j0 = k * step + mine0;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const bool mid = i < items && (unsigned)(j0 + 32 * i - lo) < (unsigned)(hi - lo);
                u[i] = mid ? order_of(weights[j0 + 32 * i]) : NONE;
            }
        }
    };
    if (formed) {
        float w[ITEMS], next[ITEMS];
        int zeros = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) next[i] = i < items && mine0 + 32 * i < n ? weights[mine0 + 32 * i] : 0.f;
        for (int k = 0; k < rounds; ++k) {
            const int j0 = k * step + mine0, at = k * CHUNK + warp * 32 * ITEMS + lane;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                w[i] = next[i];
                const int j = j0 + step + 32 * i;
                next[i] = j < n ? weights[j] : 0.f;
            }
            // (zeros, which may be many, are counted apart: they would wait for each other)
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const bool mid = i < items && (unsigned)(j0 + 32 * i - lo) < (unsigned)(hi - lo);
                const uint32_t u = mid ? order_of(w[i]) : NONE;
                if (at < cap) held[at + 32 * i] = u;
                if (i >= items) continue;
                if (u < NONE && u != ZERO) atomicAdd(&hist[u >> (32 - BITS0)], 1);
                zeros += u == ZERO;
            }
        }
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        if (lane == 0 && zeros) atomicAdd(&hist[ZERO >> (32 - BITS0)], zeros);
        find_bin<BINS>(cluster, C, 0, hist, s, want);
        int shift = 32 - BITS0;
        int* bins = hist + BINS;
        bool listed = false;
#pragma unroll 1
        for (;;) {
            top |= (uint32_t)s.found[0] << shift;
            want = s.found[1];
            if (want == s.found[2]) {                    // the bin stays as a whole
                top |= (1u << shift) - 1u;
                want = INT_MAX;
                break;
            }
            if (shift == 0) break;
            const int bits = shift == 32 - BITS0 ? BITS1 : BITS2, above = shift;
            shift -= bits;
            auto put = [&](uint32_t u) { atomicAdd(&bins[(u >> shift) & ((1u << bits) - 1u)], 1); };
            if (listed) {
                const int m = s.listed;
                for (int i = tid; i < m; i += NT)
                    if (list[i] - top < 1u << above) put(list[i]);
            } else {
                for (int k = 0; k < rounds; ++k) {
                    uint32_t u[ITEMS];
                    eight(k, u);
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) any |= u[i] - top < 1u << above;
                    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        const bool in = u[i] - top < 1u << above;
                        const unsigned m = __ballot_sync(0xffffffffu, in);
                        if (m == 0) continue;
                        int base = 0;
                        if (lane == 0) base = s.listed <= MAX_LIST ? atomicAdd(&s.listed, __popc(m)) : MAX_LIST;
                        base = __shfl_sync(0xffffffffu, base, 0) + __popc(m & ((1u << lane) - 1u));
                        if (in) {
                            if (base < MAX_LIST) list[base] = u[i];
                            put(u[i]);
                        }
                    }
                }
            }
            __syncthreads();                             // (found has been read, the list is there)
            listed = s.listed <= MAX_LIST;
            if (bits == BITS1) find_bin<1 << BITS1>(cluster, C, 1, bins, s, want);
            else find_bin<1 << BITS2>(cluster, C, 2, bins, s, want);
            bins += 1 << BITS1;
        }
    } else if (want <= 0) {
        want = 0;                                        // none, not even of the first
    } else {
        top = ~0u;                                       // all
        want = INT_MAX;
    }
    const Border o = {n, lo, hi, want, top};
    if (a.border) {
        // each warp's counts of its 256 keys, for the second kernel
        const int chunks = (a.slot_stride + CHUNK - 1) / CHUNK;
        for (int k = 0; k < rounds; ++k) {
            const int g = k * C + rank, w0 = k * step + (rank * NT + warp * 32) * items, w1 = w0 + 32 * items;
            int stay = 0, tie = 0;
            uint32_t u[ITEMS];
            if (formed) eight(k, u);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                stay += formed && u[i] < top;
                tie += formed && u[i] == top;
            }
            int all = __reduce_add_sync(0xffffffffu, stay | tie << 16);
            // and the warp's keys outside of lo .. hi - 1; without a choice all of those inside or none
            all += max(0, min(w1, lo) - min(w0, lo)) + max(0, min(w1, n) - max(min(w0, n), hi));
            if (!formed && want) all += max(0, min(w1, hi) - max(w0, lo));
            if (g >= chunks) break;
            if (lane == 0) {
                s.warp_sums[warp] = all;
                a.warp_counts[((int64_t)b * chunks + g) * 32 + warp] = all;
            }
            __syncthreads();
            if (warp == 0) {
                const int sum = __reduce_add_sync(0xffffffffu, s.warp_sums[lane]);
                if (lane == 0) a.chunk_counts[(int64_t)b * chunks + g] = sum;
            }
            __syncthreads();
        }
        if (rank == 0 && tid == 0) a.border[b] = o;
    } else {
        int kept = 0, tied = 0;                          // before this round: keys that stay, ties
        for (int k = 0; k < rounds; ++k) {
            const int j0 = k * step + mine0;
            Keys keys;
            const int all = keys.load(a, o, row, j0, items);
            __syncthreads();                             // the sums of the round before have been read
            if (lane == 0) s.warp_sums[warp] = all;
            __syncthreads();
            const int t = s.warp_sums[lane], total = __reduce_add_sync(0xffffffffu, t);
            const int before_warp = __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
            int before = kept + (before_warp & 0xffff), equal = tied + (before_warp >> 16);
            if (C > 1) {
                if (tid < C) *cluster.map_shared_rank(&s.totals[k & 1][rank], tid) = total;
                cluster.sync();
                // (sixteen chunks' counts pass 16 bits: added apart)
                const int c = lane < C ? s.totals[k & 1][lane] : 0, c_b = lane < rank ? c : 0;
                kept += __reduce_add_sync(0xffffffffu, c & 0xffff);
                tied += __reduce_add_sync(0xffffffffu, c >> 16);
                before += __reduce_add_sync(0xffffffffu, c_b & 0xffff);
                equal += __reduce_add_sync(0xffffffffu, c_b >> 16);
            } else {
                kept += total & 0xffff;
                tied += total >> 16;
            }
            keys.write(a, o, row, j0, items, before, equal);
        }
    }
    if (rank == 0 && tid == 0) {
        a.lens_out[b] = K;
        if (a.n_freed) a.n_freed[b] = n - K;
    }
    if (C > 1) cluster.sync();                           // nobody looks at this CTA's shared memory any more
}

// The second kernel: a CTA 2048 keys, a warp 256.
constexpr int TAKE_NT = 256, TAKE_KEYS = TAKE_NT * ITEMS;
__global__ void __launch_bounds__(TAKE_NT) kv_evict_take(const EvictArgs a) {
    __shared__ int sums[2][TAKE_NT / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y;
    const Border o = a.border[b];
    const int first = blockIdx.x * TAKE_KEYS;
    if (first >= o.n) return;                            // (a bad length: 0 keys)
    const int64_t row = (int64_t)b * a.slot_stride;
    const int chunks = (a.slot_stride + CHUNK - 1) / CHUNK, chunk = first / CHUNK;
    Keys keys;
    const int j0 = first + warp * 32 * ITEMS + lane;
    keys.load(a, o, row, j0, ITEMS);
    int before = 0, equal = 0;
    for (int g = tid; g < chunk; g += TAKE_NT) {
        const int c = a.chunk_counts[(int64_t)b * chunks + g];
        before += c & 0xffff;
        equal += c >> 16;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = equal;
    }
    __syncthreads();
    before = equal = 0;
#pragma unroll
    for (int w = 0; w < TAKE_NT / 32; ++w) {
        before += sums[0][w];
        equal += sums[1][w];
    }
    const int me = (first - chunk * CHUNK) / (32 * ITEMS) + warp;   // the warp's place in its chunk
    const int c = lane < me ? a.warp_counts[((int64_t)b * chunks + chunk) * 32 + lane] : 0;
    before += __reduce_add_sync(0xffffffffu, c & 0xffff);
    equal += __reduce_add_sync(0xffffffffu, c >> 16);
    if (j0 - lane < o.n) keys.write(a, o, row, j0, ITEMS, before, equal);
}

// CTAs a stream: up to sixteen while they have a round each and the launch stays within one wave.
int evict_cluster(int B, int slot_stride, int num_sms) {
    int C = 1;
    while (C < MAX_CLUSTER && (long long)C * CHUNK < slot_stride && 2ll * C * B <= num_sms) C *= 2;
    return C;
}

cudaError_t launch_kv_evict(const EvictArgs& a, int B, int C, int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (ALL_BINS + MAX_LIST + MAX_HELD) * 4);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const long long per_round = (long long)C * CHUNK, rounds = (a.slot_stride + per_round - 1) / per_round;
    const int cap = (int)min(rounds * CHUNK, (long long)MAX_HELD);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = (size_t)(ALL_BINS + MAX_LIST + cap) * 4;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_kernel, a, C, cap);
    if (e != cudaSuccess || !a.border) return e;
    return launch_dependent(kv_evict_take, dim3((a.slot_stride + TAKE_KEYS - 1) / TAKE_KEYS, B), dim3(TAKE_NT), 0, stream, a);
}

size_t evict_workspace(int B, int slot_stride) {
    const size_t chunks = ((size_t)slot_stride + CHUNK - 1) / CHUNK;
    return align256((size_t)B * sizeof(Border)) + (size_t)B * chunks * 33 * 4;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_kv_evict(const int32_t* slot_table, const int32_t* seq_lens, const float* weights,
                            const int32_t* key_pos, const int32_t* key_doc, int B, int slot_stride,
                            const int32_t* budgets, int budget, int sink, int recent, int32_t* table_out,
                            int32_t* lens_out, float* weights_out, int32_t* pos_out, int32_t* doc_out, int32_t* freed,
                            int32_t* n_freed, void* workspace, size_t ws_bytes, mla_stream_t stream) {
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
    if (!aligned(workspace, 4)) return MLA_ERR_ALIGN;
    EvictArgs a = {slot_table, seq_lens, weights, key_pos, key_doc, slot_stride, budgets, budget, sink, recent, table_out,
                   lens_out, weights_out, pos_out, doc_out, freed, n_freed, nullptr, nullptr, nullptr, nullptr};
    int num_sms = 0, dev = 0;
    const int rc = device_state(&dev, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    const int C = evict_cluster(B, slot_stride, num_sms);
    const bool in_place = table_out == slot_table || weights_out == weights || (pos_out && pos_out == key_pos) || (doc_out && doc_out == key_doc);
    if ((long long)C * CHUNK < slot_stride && !in_place && workspace && ws_bytes >= evict_workspace(B, slot_stride)) {
        const size_t chunks = ((size_t)slot_stride + CHUNK - 1) / CHUNK;
        a.border = static_cast<Border*>(workspace);
        a.chunk_counts = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256((size_t)B * sizeof(Border)));
        a.warp_counts = a.chunk_counts + (size_t)B * chunks;
    }
    if (launch_kv_evict(a, B, C, dev, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_LAUNCH;
    return MLA_OK;
}

extern "C" size_t mla_kv_evict_workspace_bytes(int B, int slot_stride, int num_sms) {
    if (B <= 0 || B > 65535 || slot_stride < 1 || slot_stride > MLA_MAX_FP8_KEYS || num_sms < 1) return 0;
    return (long long)evict_cluster(B, slot_stride, num_sms) * CHUNK < slot_stride ? evict_workspace(B, slot_stride) : 0;
}
