// Eviction from a cache by accumulated weight (mla_kv_evict): K of a stream's n keys stay, their table
// entries move together.
//
// Weights are compared as 32-bit integers in the opposite order of the numbers; the K-th smallest is found from
// histograms in shared memory (integer counts: no order of additions) over its first 13 bits, the next 11 and
// the last 8, as many of them as it takes.  Then the keys are taken, each with its place from ballots and the
// counts of the keys before it.
//
// Streams of up to 8192 keys a CTA: a cluster of up to sixteen CTAs a stream, in one kernel; a thread keeps its
// eight integers in registers.  Everything is read before anything is written, so tables may be compacted
// in place.
// One stream of 4105 keys takes 7.3 to 8.9 us captured: dependent reads, counts and barriers.
// Longer ones: all SMs share the streams out in chunks of 8192 keys.  One kernel adds the histograms up in the
// workspace; the next counts what stays for sure and lists the keys of the border's bin, of which each
// stream's last CTA to finish finds the border and adds those that stay to the counts; the third takes the
// keys.  64 streams of up to 46 thousand keys take 25.6 us, two of a million 27.5, dependent kernels of which each
// starts during the one before it; the bytes alone would take 3.2 and 4.1.  A table that is compacted in place passes
// through the workspace and comes back by one kernel more: 36.9 and 35.7 us (behind the copies that restore the tables).
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
    // workspace of the wide form
    int32_t* hist;                                   // [B][GROUPS + BINS], zeroed: sums of the groups of bins, the bins
    int32_t* done;                                   // [B][2], zeroed: CTAs that have listed, keys listed
    int32_t* lens;                                   // [B]: keys (0: a bad length)
    struct Border* border;                           // [B]
    int32_t* chunk_counts;                           // [B][chunks]: keys that stay | ties << 16
    int32_t* warp_counts;                            // [B][chunks * 32]: the same of a warp's 256 keys
    uint2* list;                                     // [B][slot_stride]: integer and index of a key
};

// How a stream's keys are chosen: a key j of lo .. hi - 1 stays if its integer is below `top`, and of
// those equal to it the first `want`; all others of the n keys stay.
struct Border {
    int n, K, lo, hi, want;
    uint32_t top;
};

// The number's place in the opposite order: NaN before all, -0 beside 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 0u : (u & 0x80000000u) ? u : ~(u | 0x80000000u);
}

constexpr uint32_t ZERO = 0x7fffffffu;               // order_of(0)
constexpr uint32_t NONE = 0xffffffffu;               // no number's: the last is that of -infinity, 0xff800000

// What a stream's lengths say.
struct Plan {
    int n, K, lo, hi, want;                              // of the keys lo .. hi - 1 the `want` heaviest stay
    bool bad, formed;                                    // a bad length; there is a choice
};
__device__ __forceinline__ Plan plan_of(const EvictArgs& a, int b) {
    Plan p;
    p.n = a.seq_lens[b];
    p.bad = p.n < 0 || p.n > a.slot_stride;
    const int n = p.bad ? 0 : p.n, budget = max(0, a.budgets ? a.budgets[b] : a.budget);
    p.K = (int)min((long long)n, max((long long)budget, (long long)a.sink + a.recent));
    p.lo = min(a.sink, n);
    p.hi = max(p.lo, (int)max((long long)n - a.recent, 0ll));
    p.want = p.K - p.lo - (n - p.hi);
    p.formed = p.want > 0 && p.want < p.hi - p.lo;
    return p;
}
// Without a choice: all of them or none.
__device__ __forceinline__ Border without_choice(const Plan& p) {
    return p.want <= 0 ? Border{p.bad ? 0 : p.n, p.K, p.lo, p.hi, 0, 0u} : Border{p.n, p.K, p.lo, p.hi, INT_MAX, ~0u};
}
__device__ __forceinline__ void write_lens(const EvictArgs& a, int b, const Plan& p) {
    if (p.bad) atomicOr(a.status, DEV_BAD_LEN);
    a.lens_out[b] = p.bad ? p.n : p.K;
    if (a.n_freed) a.n_freed[b] = p.bad ? 0 : p.n - p.K;
}

// A thread's keys j0 + 32 i of the stream, and which of them stay (bit i) or tie
// (bit 16 + i).  N: keys of a thread, up to 16; DOCS: with documents.
template <int N, bool DOCS>
struct Keys {
    float w[N];
    int slot[N], pos[N], doc[N];
    unsigned mine;

    __device__ __forceinline__ void fetch_weights(const EvictArgs& a, int n, int64_t row, int j0, int items) {
        const float* const at = a.weights + row + j0;    // (items lie at fixed offsets from here)
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = i < items && j0 + 32 * i < n ? at[32 * i] : 0.f;
    }
    __device__ __forceinline__ void fetch_slots(const EvictArgs& a, int n, int64_t row, int j0, int items) {
        const int32_t* const slots = a.slot + row + j0;
#pragma unroll
        for (int i = 0; i < N; ++i) slot[i] = i < items && j0 + 32 * i < n ? slots[32 * i] : 0;
    }
    __device__ __forceinline__ void fetch(const EvictArgs& a, int n, int64_t row, int j0, int items) {
        if (a.pos_out) {
            const int32_t* const at = a.key_pos + row + j0;
#pragma unroll
            for (int i = 0; i < N; ++i) pos[i] = a.key_pos && i < items && j0 + 32 * i < n ? at[32 * i] : j0 + 32 * i;
        }
        if (DOCS && a.doc_out) {
            const int32_t* const at = a.key_doc + row + j0;
#pragma unroll
            for (int i = 0; i < N; ++i) doc[i] = i < items && j0 + 32 * i < n ? at[32 * i] : 0;
        }
    }
    // Returns the warp's counts: stay | ties << 16.
    __device__ __forceinline__ int choose(const Border& o, int j0, int items) {
        mine = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = j0 + 32 * i;
            const uint32_t u = order_of(w[i]);
            const bool in = i < items && j < o.n, mid = j >= o.lo && j < o.hi;
            mine |= (unsigned)(in && (!mid || u < o.top)) << i | (unsigned)(in && mid && u == o.top) << (16 + i);
        }
        return __reduce_add_sync(0xffffffffu, __popc(mine & 0xffffu) | __popc(mine >> 16) << 16);
    }
    // `before`, `equal`: keys before the warp's that stay for sure, and ties.
    __device__ __forceinline__ void write(const EvictArgs& a, const Border& o, int64_t row, int j0, int items, int before, int equal) const {
        const int lane = threadIdx.x & 31;
        const unsigned lower = (1u << lane) - 1u;
        before += min(equal, o.want);                    // with the ties that stay
        const bool ties = __any_sync(0xffffffffu, mine >> 16);
        int32_t* const table = a.table_out + row;
        float* const weights = a.weights_out + row;
        int32_t *const positions = a.pos_out + row, *const docs = a.doc_out + row;   // (where there are any)
        int32_t* const freed = a.freed + row + j0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = j0 + 32 * i;
            if (i >= items || j - lane >= o.n) break;
            unsigned keep = __ballot_sync(0xffffffffu, (mine >> i) & 1u);
            if (ties) {                                  // the first of them, as many as are wanted
                const unsigned tie = __ballot_sync(0xffffffffu, (mine >> (16 + i)) & 1u);
                const int room = o.want - min(equal, o.want), m = __popc(tie);
                equal += m;
                if (room >= m) keep |= tie;
                else if (room > 0) keep |= __ballot_sync(0xffffffffu, ((tie >> lane) & 1u) && __popc(tie & lower) < room);
            }
            const int to = before + __popc(keep & lower);
            before += __popc(keep);
            const bool stays = (keep >> lane) & 1u;
            if (stays || (j < o.n && a.freed)) *(stays ? table + to : freed + (32 * i - to)) = slot[i];
            if (stays) {
                weights[to] = w[i];
                if (a.pos_out) positions[to] = pos[i];
                if (DOCS && a.doc_out) docs[to] = doc[i];
            }
        }
    }
};

struct Shared {
    int warp_sums[32];
    int groups[3][GROUPS];                           // a pass's keys in every sixty-fourth of the bins
    int found[3];                                    // bin, keys wanted of it, keys in it
    int listed;                                      // the wide form: keys of the bin
    int totals[MAX_CLUSTER];                         // of every CTA: keys that stay | ties << 16
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
#pragma unroll 4
            for (int r = 0; r < C; ++r) {
                const int2 y = *reinterpret_cast<const int2*>(cluster.map_shared_rank(&s.groups[pass][2 * lane], r));
                v[0] += y.x;
                v[1] += y.y;
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

// Takes the bin that was found over the `shift` last bits into the border; true where it is known then.
__device__ __forceinline__ bool narrow(const Shared& s, int shift, uint32_t* top, int* want) {
    *top |= (uint32_t)s.found[0] << shift;
    *want = s.found[1];
    if (*want < s.found[2]) return shift == 0;
    *top |= (1u << shift) - 1u;                          // the bin stays as a whole
    *want = INT_MAX;
    return true;
}

__global__ void __launch_bounds__(NT, 1) kv_evict_kernel(const EvictArgs a, int C) {
    __shared__ __align__(16) int hist[ALL_BINS];
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster.block_rank() : 0, b = blockIdx.x / C;
    const Plan p = plan_of(a, b);
    // The thread's keys are j0 + 32 i, `items` of them, in the order of the stream by warps, then items, then lanes.
    const int64_t row = (int64_t)b * a.slot_stride;
    const int items = p.bad ? 1 : max(1, min(ITEMS, (p.n + C * NT - 1) / (C * NT)));
    const int j0 = (rank * NT + warp * 32) * items + lane, n = p.bad ? 0 : p.n;
    Keys<ITEMS, true> keys;
    keys.fetch_weights(a, n, row, j0, items);
    keys.fetch_slots(a, n, row, j0, items);
    for (int i = tid; i < ALL_BINS / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    if (C > 1) cluster.sync();                           // every CTA runs, and has read the length
    else __syncthreads();
    if (p.bad) {
        if (rank == 0 && tid == 0) write_lens(a, b, p);
        return;
    }
    Border o = without_choice(p);
    if (p.formed) {
        auto integer = [&](int i) -> uint32_t {          // NONE for a key that is not among the lo .. hi - 1
            return i < items && (unsigned)(j0 + 32 * i - p.lo) < (unsigned)(p.hi - p.lo) ? order_of(keys.w[i]) : NONE;
        };
        int zeros = 0;                                   // (counted apart: they would wait for each other)
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t u = integer(i);
            if (u < NONE && u != ZERO) atomicAdd(&hist[u >> (32 - BITS0)], 1);
            zeros += u == ZERO;
        }
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        if (lane == 0 && zeros) atomicAdd(&hist[ZERO >> (32 - BITS0)], zeros);
        find_bin<BINS>(cluster, C, 0, hist, s, p.want);
        o.top = 0;
        int shift = 32 - BITS0;
        int* bins = hist + BINS;
#pragma unroll 1
        while (!narrow(s, shift, &o.top, &o.want)) {
            const int bits = shift == 32 - BITS0 ? BITS1 : BITS2, above = shift;
            shift -= bits;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const uint32_t u = integer(i);
                if (u - o.top < 1u << above) atomicAdd(&bins[(u >> shift) & ((1u << bits) - 1u)], 1);
            }
            if (bits == BITS1) find_bin<1 << BITS1>(cluster, C, 1, bins, s, o.want);
            else find_bin<1 << BITS2>(cluster, C, 2, bins, s, o.want);
            bins += 1 << BITS1;
        }
    }
    keys.fetch(a, n, row, j0, items);
    const int all = keys.choose(o, j0, items);
    if (lane == 0) s.warp_sums[warp] = all;
    __syncthreads();
    const int t = s.warp_sums[lane], total = __reduce_add_sync(0xffffffffu, t);
    const int before_warp = __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
    int before = before_warp & 0xffff, equal = before_warp >> 16;
    if (C > 1) {
        if (tid < C) *cluster.map_shared_rank(&s.totals[rank], tid) = total;
        cluster.sync();                                  // (and everything has been read)
        const int c = lane < rank ? s.totals[lane] : 0;  // (sixteen CTAs' counts pass 16 bits: added apart)
        before += __reduce_add_sync(0xffffffffu, c & 0xffff);
        equal += __reduce_add_sync(0xffffffffu, c >> 16);
    }
    keys.write(a, o, row, j0, items, before, equal);
    if (rank == 0 && tid == 0) write_lens(a, b, p);
}

// ---- the wide form.  Keys mine + 32 i of chunk blockIdx.x, as in the one above; integers of keys that are not
// among the lo .. hi - 1 are NONE.
__device__ __forceinline__ void chunk_keys(const EvictArgs& a, int b, const Plan& p, uint32_t (&u)[ITEMS]) {
    const int j0 = blockIdx.x * CHUNK + (threadIdx.x >> 5) * 32 * ITEMS + (threadIdx.x & 31);
    const float* const at = a.weights + (int64_t)b * a.slot_stride + j0;
    float w[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) w[i] = j0 + 32 * i < p.n ? at[32 * i] : 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) u[i] = (unsigned)(j0 + 32 * i - p.lo) < (unsigned)(p.hi - p.lo) ? order_of(w[i]) : NONE;
}

// Each of these kernels starts while the one before it ends, and reads the call's inputs before it waits for it:
// what came before the call has ended by then, since each lets the next one start after a wait of its own, and only
// the last ones write outside of the workspace.
__global__ void __launch_bounds__(256) kv_evict_zero(int4* ws, int n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) ws[i] = make_int4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(NT, 2) kv_evict_count(const EvictArgs a) {
    __shared__ __align__(16) int hist[BINS];
    const int tid = threadIdx.x, b = blockIdx.y;
    const Plan p = plan_of(a, b);
    if (!p.formed || blockIdx.x * CHUNK >= p.n) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (blockIdx.x == 0 && tid == 0) a.lens[b] = p.bad ? 0 : p.n;
        return;
    }
    for (int i = tid; i < BINS / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    uint32_t u[ITEMS];
    chunk_keys(a, b, p, u);
    __syncthreads();
    int zeros = 0;                                       // (counted apart: they would wait for each other)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (u[i] < NONE && u[i] != ZERO) atomicAdd(&hist[u[i] >> (32 - BITS0)], 1);
        zeros += u[i] == ZERO;
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if ((tid & 31) == 0 && zeros) atomicAdd(&hist[ZERO >> (32 - BITS0)], zeros);
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && tid == 0) a.lens[b] = p.n;
    // a warp two groups of bins
    int* const out = a.hist + (int64_t)b * (GROUPS + BINS);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        constexpr int G = BINS / GROUPS;
        const int g = (tid >> 5) * 2 + h;
        int sum = 0;
#pragma unroll
        for (int q = 0; q < G / 32; ++q) {
            const int i = g * G + 32 * q + (tid & 31), c = hist[i];
            if (c) atomicAdd(&out[GROUPS + i], c);
            sum += c;
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if ((tid & 31) == 0 && sum) atomicAdd(&out[g], sum);
    }
}

constexpr int HELD = 4096;
__global__ void __launch_bounds__(NT, 2) kv_evict_border(const EvictArgs a) {
    __shared__ __align__(16) int hist[ALL_BINS - BINS];
    __shared__ uint2 held[HELD];                         // the list's first keys
    __shared__ Shared s;
    __shared__ int base, last;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
    const Plan p = plan_of(a, b);
    uint32_t u[ITEMS];
    if (!p.bad) chunk_keys(a, b, p, u);
    for (int i = tid; i < (ALL_BINS - BINS) / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!p.formed && blockIdx.x == 0 && tid == 0) a.border[b] = without_choice(p);
    if (p.bad || blockIdx.x * CHUNK >= p.n) return;
    Border o = without_choice(p);
    int shift = 32 - BITS0;
    bool known = true;
    if (p.formed && tid < 32) {
        // the border's bin: its group, then the bin
        constexpr int PER = BINS / GROUPS / 32;
        const int* const in = a.hist + (int64_t)b * (GROUPS + BINS);
        int v[2] = {__ldcg(in + 2 * lane), __ldcg(in + 2 * lane + 1)}, at = 0, left = 0, keys = 0;
        const unsigned hit = __ballot_sync(0xffffffffu, find_in_warp(v, p.want, &at, &left, &keys));
        const int src = __ffs(hit) - 1, group = __shfl_sync(0xffffffffu, at, src), rest = __shfl_sync(0xffffffffu, left, src);
        int w[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) w[q] = __ldcg(in + GROUPS + group * 32 * PER + lane * PER + q);
        if (find_in_warp(w, rest, &at, &left, &keys)) {
            s.found[0] = group * 32 * PER + at;
            s.found[1] = left;
            s.found[2] = keys;
        }
        if (lane == 0) s.listed = 0;
    }
    __syncthreads();
    if (p.formed) {
        o.top = 0;
        known = narrow(s, shift, &o.top, &o.want);
    }
    // what stays for sure, and the ties: of the warp's keys, of the chunk's
    const int warp = tid >> 5, w0 = blockIdx.x * CHUNK + warp * 32 * ITEMS, w1 = w0 + 32 * ITEMS;
    int stay = 0, tie = 0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        stay += u[i] < o.top;
        tie += known && u[i] == o.top && u[i] != NONE;
    }
    int all = __reduce_add_sync(0xffffffffu, stay | tie << 16);
    all += max(0, min(w1, p.lo) - min(w0, p.lo)) + max(0, min(w1, p.n) - max(min(w0, p.n), p.hi));
    if (lane == 0) {
        s.warp_sums[warp] = all;
        a.warp_counts[((int64_t)b * gridDim.x + blockIdx.x) * 32 + warp] = all;
    }
    __syncthreads();
    if (warp == 0) {
        all = __reduce_add_sync(0xffffffffu, s.warp_sums[lane]);
        if (lane == 0) a.chunk_counts[(int64_t)b * gridDim.x + blockIdx.x] = all;
    }
    if (!p.formed) return;
    uint2* const list = a.list + (int64_t)b * a.slot_stride;
    if (!known) {
        // the bin's keys go to the list, in any order
        int mine = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) mine += u[i] - o.top < 1u << shift;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        int at = 0;
        if (lane == 31 && upto) at = atomicAdd(&s.listed, upto);
        at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
        __syncthreads();
        if (tid == 0) base = s.listed ? atomicAdd(&a.done[2 * b + 1], s.listed) : 0;
        __syncthreads();
        at += base;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (u[i] - o.top < 1u << shift) list[at++] = make_uint2(u[i], w0 + 32 * i + lane);
    }
    // the stream's last CTA goes on (one thread's fences stand for all: the barriers order the others' accesses)
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last = atomicAdd(&a.done[2 * b], 1) == (p.n - 1) / CHUNK;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    if (!known) {
        const int m = __ldcg(&a.done[2 * b + 1]);
        int* bins = hist;
#pragma unroll 1
        do {
            const int bits = shift == 32 - BITS0 ? BITS1 : BITS2, above = shift;
            shift -= bits;
            for (int first = tid; first < m; first += 4 * NT) {
                uint2 key[4];                            // (read before any is counted)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = first + q * NT;
                    key[q] = i >= m ? make_uint2(NONE, 0) : shift == 0 && i < HELD ? held[i] : __ldcg(list + i);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = first + q * NT;
                    if (shift > 0 && i < min(m, HELD)) held[i] = key[q];
                    if (key[q].x - o.top < 1u << above) atomicAdd(&bins[(key[q].x >> shift) & ((1u << bits) - 1u)], 1);
                }
            }
            if (bits == BITS1) find_bin<1 << BITS1>(cluster, 1, 1, bins, s, o.want);
            else find_bin<1 << BITS2>(cluster, 1, 2, bins, s, o.want);
            bins += 1 << BITS1;
        } while (!narrow(s, shift, &o.top, &o.want));
        // those that stay or tie go to the counts; a chunk's keys lie together in the list, and a warp adds them up
        for (int i = tid; i - lane < m; i += NT) {
            const uint2 key = i >= m ? make_uint2(NONE, 0) : i < HELD ? held[i] : __ldcg(list + i);
            const bool mine = key.x <= o.top;
            const int chunk = mine ? (int)(key.y / CHUNK) : -1;
            const unsigned group = __match_any_sync(0xffffffffu, chunk), below = __ballot_sync(0xffffffffu, key.x < o.top) & group;
            if (mine) {
                atomicAdd(&a.warp_counts[(int64_t)b * gridDim.x * 32 + key.y / (32 * ITEMS)], key.x < o.top ? 1 : 1 << 16);
                if (lane == __ffs(group) - 1)
                    atomicAdd(&a.chunk_counts[(int64_t)b * gridDim.x + chunk], __popc(below) | __popc(group & ~below) << 16);
            }
        }
    }
    if (tid == 0) a.border[b] = o;
}

// A CTA 2048 keys, a warp 256.
constexpr int TAKE_NT = 256, TAKE_ITEMS = 8, TAKE_KEYS = TAKE_NT * TAKE_ITEMS;
template <bool DOCS>
__global__ void __launch_bounds__(TAKE_NT, DOCS ? 4 : 5) kv_evict_take(const EvictArgs a) {
    __shared__ int sums[2][TAKE_NT / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y;
    const int first = blockIdx.x * TAKE_KEYS;
    const int64_t row = (int64_t)b * a.slot_stride;
    const int chunks = (a.slot_stride + CHUNK - 1) / CHUNK, chunk = first / CHUNK;
    const int me = (first - chunk * CHUNK) / (32 * ITEMS) + warp * (TAKE_ITEMS / ITEMS);   // of the warp's first keys' counts
    const int j0 = first + warp * 32 * TAKE_ITEMS + lane, n = a.lens[b];
    if (first >= n && blockIdx.x > 0) return;            // (the stream's first CTA writes its lengths)
    Keys<TAKE_ITEMS, DOCS> keys;
    keys.fetch_weights(a, n, row, j0, TAKE_ITEMS);
    keys.fetch_slots(a, n, row, j0, TAKE_ITEMS);
    keys.fetch(a, n, row, j0, TAKE_ITEMS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Border o = a.border[b];
    // (only here, by the one thread that still reads the length: lens_out may be seq_lens)
    if (blockIdx.x == 0 && tid == 0) write_lens(a, b, plan_of(a, b));
    const int c = lane < me ? a.warp_counts[((int64_t)b * chunks + chunk) * 32 + lane] : 0;
    int before = 0, equal = 0;
    for (int g = tid; g < chunk; g += TAKE_NT) {
        const int k = a.chunk_counts[(int64_t)b * chunks + g];
        before += k & 0xffff;
        equal += k >> 16;
    }
    if (first >= o.n) return;                            // (a bad length: 0 keys)
    keys.choose(o, j0, TAKE_ITEMS);
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
    before += __reduce_add_sync(0xffffffffu, c & 0xffff);
    equal += __reduce_add_sync(0xffffffffu, c >> 16);
    if (j0 - lane < o.n) keys.write(a, o, row, j0, TAKE_ITEMS, before, equal);
}

// What was to be compacted in place comes back from the workspace (`from`: null where it was not).
struct Back {
    const int32_t *table, *pos, *doc;
    const float* weights;
};
__global__ void __launch_bounds__(TAKE_NT) kv_evict_back(const EvictArgs a, const Back from) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y, n = a.border[b].n, K = n ? a.border[b].K : 0;
    const int64_t row = (int64_t)b * a.slot_stride;
    for (int j = blockIdx.x * TAKE_KEYS + threadIdx.x, e = min(K, (int)(blockIdx.x + 1) * TAKE_KEYS); j < e; j += TAKE_NT) {
        if (from.table) a.table_out[row + j] = from.table[row + j];
        if (from.weights) a.weights_out[row + j] = from.weights[row + j];
        if (from.pos) a.pos_out[row + j] = from.pos[row + j];
        if (from.doc) a.doc_out[row + j] = from.doc[row + j];
    }
}

// CTAs a stream: up to sixteen while that leaves them 8192 keys or more and the launch stays within one wave: clusters
// do not reach every SM (measured: 7 of sixteen CTAs run at once, 15 of eight, 36 of four, 76 of two).  A second wave
// costs as much as the first (8 streams of 130000 keys, sixteen CTAs each, 29.4 us, in the wide form 18.2; 16 of
// 65000, eight each, 25.1 and 18.3), one wave less than the wide form (7 streams of 130000 keys 16.5 and 18.6).
int evict_cluster(int B, int slot_stride, int num_sms) {
    int C = 1;
    while (C < MAX_CLUSTER && (long long)C * CHUNK < slot_stride) {
        const int beyond = C == 8 ? 40 : C == 4 ? 32 : C == 2 ? 8 : 0;   // SMs without a whole cluster of 2 C CTAs
        if (2ll * C * B > num_sms - beyond) break;
        C *= 2;
    }
    return C;
}

cudaError_t launch_kv_evict(const EvictArgs& a, int B, int C, int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(NT);
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
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, a, C);
}

// The wide form's workspace: what has to be zero first, and (in place) four tables at its end.
struct Wide {
    size_t zeroed, lens, border, chunk_counts, warp_counts, list, tables, total;
};
Wide evict_workspace(int B, int slot_stride, bool in_place) {
    const size_t chunks = ((size_t)slot_stride + CHUNK - 1) / CHUNK, table = align256((size_t)B * slot_stride * 4);
    Wide w;
    w.zeroed = align256((size_t)B * (GROUPS + BINS + 2) * 4);
    w.lens = w.zeroed;
    w.border = w.lens + align256((size_t)B * 4);
    w.chunk_counts = w.border + align256((size_t)B * sizeof(Border));
    w.warp_counts = w.chunk_counts + align256((size_t)B * chunks * 4);
    w.list = w.warp_counts + align256((size_t)B * chunks * 32 * 4);
    w.tables = w.list + 2 * table;
    w.total = w.tables + (in_place ? 4 * table : 0);
    return w;
}

cudaError_t launch_kv_evict_wide(EvictArgs a, int B, bool in_place, void* workspace, cudaStream_t stream) {
    const Wide w = evict_workspace(B, a.slot_stride, in_place);
    char* const ws = static_cast<char*>(workspace);
    a.hist = reinterpret_cast<int32_t*>(ws);
    a.done = a.hist + (size_t)B * (GROUPS + BINS);
    a.lens = reinterpret_cast<int32_t*>(ws + w.lens);
    a.border = reinterpret_cast<Border*>(ws + w.border);
    a.chunk_counts = reinterpret_cast<int32_t*>(ws + w.chunk_counts);
    a.warp_counts = reinterpret_cast<int32_t*>(ws + w.warp_counts);
    a.list = reinterpret_cast<uint2*>(ws + w.list);
    const int vectors = (int)(w.zeroed / 16);            // (at most 65535 streams' 33 KB)
    cudaError_t e = launch_dependent(kv_evict_zero, dim3((unsigned)min((vectors + 255) / 256, 1024)), dim3(256), 0, stream,
                                     reinterpret_cast<int4*>(ws), vectors);
    const dim3 grid((a.slot_stride + CHUNK - 1) / CHUNK, B), take((a.slot_stride + TAKE_KEYS - 1) / TAKE_KEYS, B);
    if (e == cudaSuccess) e = launch_dependent(kv_evict_count, grid, dim3(NT), 0, stream, a);
    if (e == cudaSuccess) e = launch_dependent(kv_evict_border, grid, dim3(NT), 0, stream, a);
    EvictArgs t = a;
    Back from = {};
    if (in_place) {
        const size_t table = align256((size_t)B * a.slot_stride * 4);
        char* const to = ws + w.tables;
        if (a.table_out == a.slot) from.table = t.table_out = reinterpret_cast<int32_t*>(to);
        if (a.weights_out == a.weights) from.weights = t.weights_out = reinterpret_cast<float*>(to + table);
        if (a.pos_out && a.pos_out == a.key_pos) from.pos = t.pos_out = reinterpret_cast<int32_t*>(to + 2 * table);
        if (a.doc_out && a.doc_out == a.key_doc) from.doc = t.doc_out = reinterpret_cast<int32_t*>(to + 3 * table);
    }
    if (e == cudaSuccess) e = launch_dependent(a.doc_out ? kv_evict_take<true> : kv_evict_take<false>, take, dim3(TAKE_NT), 0, stream, t);
    if (e == cudaSuccess && in_place) e = launch_dependent(kv_evict_back, take, dim3(TAKE_NT), 0, stream, a, from);
    return e;
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
    if (!aligned(workspace, 16)) return MLA_ERR_ALIGN;
    EvictArgs a = {slot_table, seq_lens, weights, key_pos, key_doc, slot_stride, budgets, budget, sink, recent, table_out,
                   lens_out, weights_out, pos_out, doc_out, freed, n_freed};
    int num_sms = 0, dev = 0;
    const int rc = device_state(&dev, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    const int C = evict_cluster(B, slot_stride, num_sms);
    const bool in_place = table_out == slot_table || weights_out == weights || (pos_out && pos_out == key_pos) || (doc_out && doc_out == key_doc);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((long long)C * CHUNK >= slot_stride) {
        if (launch_kv_evict(a, B, C, dev, st) != cudaSuccess) return MLA_ERR_LAUNCH;
        return MLA_OK;
    }
    if (!workspace || ws_bytes < evict_workspace(B, slot_stride, in_place).total) return MLA_ERR_WORKSPACE;
    if (launch_kv_evict_wide(a, B, in_place, workspace, st) != cudaSuccess) return MLA_ERR_LAUNCH;
    return MLA_OK;
}

extern "C" size_t mla_kv_evict_workspace_bytes(int B, int slot_stride, int in_place, int num_sms) {
    if (B <= 0 || B > 65535 || slot_stride < 1 || slot_stride > MLA_MAX_FP8_KEYS || num_sms < 1) return 0;
    return (long long)evict_cluster(B, slot_stride, num_sms) * CHUNK < slot_stride ? evict_workspace(B, slot_stride, in_place != 0).total : 0;
}
