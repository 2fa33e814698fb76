// Acceptance of drafted tokens by rejection sampling down a draft chain or tree, from given
// random numbers, so that the tokens that come out are distributed as the target's own.
//
// Node 0 is the stream's last committed token; node i's token was drawn from the drafter's
// distribution q_c after its parent c, and p_c is the target's.  At the current node c
// (c = 0 at first), with R = p_c and S = 1, the children are tried in index order:
//     child k is accepted, and becomes the current node, iff u_k q_c(x_k) S < R(x_k);
//     otherwise R <- max(R - S q_c, 0) and S <- sum R.
// When no child is left the next token is drawn from R: the lowest i with
// R(0) + .. + R(i) > u_next sum R.  R and S are the unnormalised residual distribution and
// its normaliser, and the maxima telescope: after rejections with normalisers S_0 = 1,
// S_1, .. the residual is R(x) = max(p(x) - A q(x), 0) with A = S_0 + S_1 + .., so one
// multiply-add an element from the two rows replaces a running copy of R.  Without a drafter
// (drafts that were not drawn but chosen) q is one at the token: a rejection takes the token
// out of p.
//
// Exactness: the tokens are whole numbers, so a sum that is off near a border gives another
// token.  p - A q is formed with its fp32 rounding error kept beside it (Dekker 1971, Knuth:
// two-sum and the product's error by a fused multiply-add), rounded to a multiple of 2^-44
// (residual.cuh) and summed as a 64-bit integer: sums do not depend on their order or on how the
// vocabulary is split, and the GPU's few fp64 units see a handful of operations a node.
//
// Bound by HBM, one pass over the row pair of the node the walk stops at (8 V bytes a
// stream; a pass more for each sibling tried after a rejection, mostly from L2), and by
// latency for few streams.  A cluster of CTAs shares a stream: each CTA owns a contiguous
// part of the vocabulary, each of its warps a contiguous part of that, and the partial sums
// meet in distributed shared memory.  Every CTA repeats the walk (a few dozen operations),
// so only sums cross CTAs.
//
// Measured on GB300 (GPU time a call): one chain of 8 drafts over 32000 tokens 6.5 us, a chain of
// dependent reads and one cluster barrier; 64 chains of 15 over 131072 tokens 20.0 us, of which
// the pass over 67 MB takes 12 us (5.6 TB/s); 64 trees of 16 nodes 41.9 us: the mean stream
// makes 1.9 passes, the slowest six, and each pass after the first takes 4.5 us for its 128 KB a CTA,
// plus 2 us for barrier and walk.  For the 64 trees (at 47.4 us, before loads ran a batch ahead): clusters
// of 4 61 us, of 16 (two waves) 54 us, blocks of 512 threads 59 us.  Copies to shared memory five
// vectors ahead: the same for trees, 0.4 us more for chains.
#include "../../include/mla_verify.h"
#include "internal.cuh"
#include "residual.cuh"

#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr int DV_THREADS = 256;
constexpr int DV_WARPS = DV_THREADS / 32;
constexpr int DV_MAX_CLUSTER = 16;                   // (more than eight CTAs: opted into per device)
constexpr int DV_BATCH = 2;                          // vectors of each row that a thread has in flight
constexpr long long MOST = 1ll << 49;                // a thread's sum at most (32): 4096 of them do not overflow

struct DraftArgs {
    const float* p;               // [B, q_len, V]
    const float* q;               // [B, q_len, V] or nullptr
    const int32_t* tokens;        // [B, q_len]
    const int32_t* parents;       // [B, q_len] or nullptr = chain
    const float* u;               // [B, q_len]
    const float* u_next;          // [B]
    int q_len;
    int V;
    int32_t* n_accepted;          // [B]
    int32_t* out_tokens;          // [B, q_len]
    int32_t* path;                // [B, q_len]
    unsigned* status;
};

// A probability as it counts: NaN and negative as 0, above 1 as 1.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// floor(u T) for u in [0, 1), T >= 0; at most T (u of 1 and more), and 0 for a negative u or a NaN.
__device__ __forceinline__ long long floor_product(float u, long long T) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return T;
    const unsigned bits = __float_as_uint(u), e = bits >> 23;
    const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);     // u = m 2^-shift, shift >= 24
    const int shift = 150 - (int)max(e, 1u);
    const unsigned long long lo = m * (unsigned long long)T, hi = __umul64hi(m, (unsigned long long)T);
    return (long long)(shift < 64 ? hi << (64 - shift) | lo >> shift : (shift < 128 ? hi >> (shift - 64) : 0ull));
}

// A residual row: p and q of the current node.  Positions k run over whole vectors of four that
// start on 16-byte boundaries, `shift` elements before the row; element x = k - shift.
struct Row {
    const float* p;
    const float* q;
    int V, shift;
};

__device__ __forceinline__ void load4(const float* row, int x, int V, float (&f)[4]) {
    if (x >= 0 && x + 4 <= V) {
        const float4 t = __ldg(reinterpret_cast<const float4*>(row + x));
        f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = x + j >= 0 && x + j < V ? __ldg(row + x + j) : 0.f;
    }
}

// Sum of the residual over positions lo, lo + step, .. < hi (vectors of four).
template <int FORM>
__device__ __forceinline__ long long sum_row(const Row& r, const Coef& c, int lo, int hi, int step) {
    long long sum = 0;
    const int end = min(hi, r.V + r.shift);
    float p[DV_BATCH][4], q[DV_BATCH][4], pn[DV_BATCH][4], qn[DV_BATCH][4];
    auto load = [&](int k, float (&p)[DV_BATCH][4], float (&q)[DV_BATCH][4]) {
#pragma unroll
        for (int u = 0; u < DV_BATCH; ++u) {
            const int x = k + u * step < end ? k + u * step - r.shift : r.V;   // past the end: all zero
            load4(r.p, x, r.V, p[u]);
            if (FORM != FROM_P) load4(r.q, x, r.V, q[u]);
        }
    };
    load(lo, p, q);
    for (int k = lo; k < end; k += DV_BATCH * step) {
        load(k + DV_BATCH * step, pn, qn);
        Few few = {0, 0};
#pragma unroll
        for (int u = 0; u < DV_BATCH; ++u)
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                add_residuals<FORM>(prob(p[u][j]), prob(p[u][j + 1]), FORM != FROM_P ? prob(q[u][j]) : 0.f,
                                    FORM != FROM_P ? prob(q[u][j + 1]) : 0.f, c, few);
        sum += few.sum(4 * DV_BATCH);
#pragma unroll
        for (int u = 0; u < DV_BATCH; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) { p[u][j] = pn[u][j]; if (FORM != FROM_P) q[u][j] = qn[u][j]; }
    }
    return sum;
}

__device__ __forceinline__ long long one(const Row& r, const Coef& c, int form, int x) {
    return residual<MINUS_AQ>(prob(r.p[x]), form == FROM_P ? 0.f : prob(r.q[x]), c);
}

// The same sum over lo .. < hi by one thread, for short pieces (one form for all: equal to MINUS_Q at
// A = 1, and to FROM_P at q = 0).
__device__ __forceinline__ long long sum_piece(const Row& r, const Coef& c, int form, int lo, int hi) {
    long long sum = 0;
    const int end = min(hi, r.V + r.shift);
#pragma unroll 1
    for (int k = lo; k < end; k += 4) {
        float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
        load4(r.p, k - r.shift, r.V, p);
        if (form != FROM_P) load4(r.q, k - r.shift, r.V, q);
        Few few = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; j += 2)
            add_residuals<MINUS_AQ>(prob(p[j]), prob(p[j + 1]), prob(q[j]), prob(q[j + 1]), c, few);
        sum += few.sum(4);
    }
    return sum;
}

__device__ __forceinline__ long long sum_range(const Row& r, const Coef& c, int form, int lo, int hi, int step) {
    if (form == FROM_P) return sum_row<FROM_P>(r, c, lo, hi, step);
    if (form == MINUS_Q) return sum_row<MINUS_Q>(r, c, lo, hi, step);
    return sum_row<MINUS_AQ>(r, c, lo, hi, step);
}

struct Shared {
    int tok[MLA_MAX_Q_LEN];
    float u[MLA_MAX_Q_LEN], pt[MLA_MAX_Q_LEN], qt[MLA_MAX_Q_LEN];   // p and q of the node's token at its parent
    unsigned long long kids[MLA_MAX_Q_LEN];            // bit i: node i is a child
    unsigned long long first;                          // bit i: node i passes as the first child tried
    unsigned long long todo;                           // children of the current node that are still to try
    int removed[MLA_MAX_Q_LEN];                        // tokens taken out of p (no drafter), and their p
    long long removed_p[MLA_MAX_Q_LEN];
    int acc[MLA_MAX_Q_LEN];                            // accepted nodes
    int n_acc, n_removed, cur, done, sum_wanted;
    double A, S;
    int have_S, have_sum;                              // S is known; the sums are those of p at `cur` (no drafter)
    long long sum;
    long long warp_sum[2][DV_WARPS];
    long long cta_sum[2][DV_MAX_CLUSTER];              // of every CTA of the cluster
    long long scan[DV_WARPS];
};

__device__ __forceinline__ bool is_removed(const Shared& s, int x) {
    for (int i = 0; i < s.n_removed; ++i)
        if (s.removed[i] == x) return true;
    return false;
}

__global__ void __launch_bounds__(DV_THREADS, 4) draft_verify_kernel(const DraftArgs a, int C, int per_cta, int per_warp) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    const int b = blockIdx.x / C, rank = blockIdx.x % C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t V = a.V;
    const int64_t base = (int64_t)b * a.q_len;
    const bool drafter = a.q != nullptr;
    // ---- the nodes: parent, token, random number and both probabilities of the token
    if (tid < MLA_MAX_Q_LEN) s.kids[tid] = 0;
    if (tid == 0) {
        s.first = 0;
        s.n_acc = 0; s.n_removed = 0; s.cur = 0; s.done = 0;
        s.A = 0.0; s.S = 1.0; s.have_S = 1; s.have_sum = 0;
    }
    __syncthreads();
    if (tid > 0 && tid < a.q_len) {
        const int i = tid;
        const int par = a.parents ? a.parents[base + i] : i - 1;
        const int tok = a.tokens[base + i];
        const float u = a.u[base + i];
        if (par < -1 || par >= i || (par >= 0 && (tok < 0 || tok >= a.V))) {
            if (rank == 0) atomicOr(a.status, DEV_BAD_DRAFT);
        } else if (par >= 0) {
            const float pt = prob(a.p[(base + par) * V + tok]);
            const float qt = drafter ? prob(a.q[(base + par) * V + tok]) : 1.f;
            s.tok[i] = tok;
            s.u[i] = u;
            s.pt[i] = pt;
            s.qt[i] = qt;
            atomicOr(&s.kids[par], 1ull << i);
            if ((double)u * (double)qt < (double)pt) atomicOr(&s.first, 1ull << i);   // exact: 48 bits
        }
    }
    __syncthreads();
    if (tid == 0) s.todo = s.kids[0];
    const int cta_lo = rank * per_cta, my_lo = cta_lo + warp * per_warp, my_hi = my_lo + per_warp;
    int phase = 0, form = FROM_P;
    bool fallback = false, started = false;
    long long total = 0, before = 0;                   // sums over the vocabulary, and before this CTA's part
    Row row;
    Coef c;
    for (;;) {
        // ---- walk until a test needs a sum that is not there, or no child is left
        if (tid == 0 && !fallback) {
            unsigned long long todo = s.todo;
            while (todo && s.have_S) {
                const int i = __ffsll((long long)todo) - 1;
                todo &= todo - 1;
                bool yes;
                if (s.A == 0.0) {
                    yes = (s.first >> i) & 1;
                } else {
                    const double qx = s.qt[i];
                    const double r = drafter ? (double)s.pt[i] - s.A * qx : (is_removed(s, s.tok[i]) ? 0.0 : (double)s.pt[i]);
                    yes = (double)s.u[i] * qx * s.S < r;
                }
                if (yes) {
                    s.acc[s.n_acc++] = i;
                    s.cur = i;
                    s.A = 0.0; s.S = 1.0;
                    s.n_removed = 0;
                    s.have_sum = 0;
                    todo = s.kids[i];
                } else if (drafter) {
                    s.A += s.S;
                    s.have_S = 0;
                } else {
                    s.A = 1.0;                         // some rejection
                    if (!is_removed(s, s.tok[i])) {
                        s.removed[s.n_removed] = s.tok[i];
                        s.removed_p[s.n_removed++] = residual<FROM_P>(s.pt[i], 0.f, c);
                    }
                    s.have_S = s.have_sum;             // p's sum less the tokens taken out
                    if (s.have_sum) {
                        long long left = s.sum;
                        for (int j = 0; j < s.n_removed; ++j) left -= s.removed_p[j];
                        s.S = (double)left * UNIT;
                    }
                }
            }
            s.todo = todo;
            s.done = todo == 0;
            s.sum_wanted = drafter || !s.have_sum;
        }
        __syncthreads();
        const bool done = s.done;
        // ---- sum of the residual (without a drafter: of p) over this CTA's part of the vocabulary
        if (s.sum_wanted) {
            const int64_t at = (base + s.cur) * V;
            row.p = a.p + at;
            row.q = drafter ? a.q + at : nullptr;
            row.V = a.V;
            row.shift = (int)(at & 3);
            form = !drafter || s.A == 0.0 ? FROM_P : (s.A == 1.0 ? MINUS_Q : MINUS_AQ);
            c.ah = (float)s.A;
            c.al = (float)(s.A - (double)c.ah);
            phase ^= 1;
            long long sum = min(sum_range(row, c, form, my_lo + lane * 4, my_hi, 128), MOST);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) s.warp_sum[phase][warp] = sum;
            __syncthreads();
            if (!started) cluster.barrier_wait();      // every CTA of the cluster runs
            started = true;
            if (tid < C) {
                long long t = 0;
                for (int w = 0; w < DV_WARPS; ++w) t += s.warp_sum[phase][w];
                *cluster.map_shared_rank(&s.cta_sum[phase][rank], tid) = t;
            }
            cluster.sync();
            const long long v = lane < C ? s.cta_sum[phase][lane] : 0;
            total = v;
            before = lane < rank ? v : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                total += __shfl_xor_sync(0xffffffffu, total, o);
                before += __shfl_xor_sync(0xffffffffu, before, o);
            }
        }
        long long left = total;
        for (int j = 0; j < s.n_removed; ++j) left -= s.removed_p[j];
        if (done && (left > 0 || fallback)) break;     // a fallback without a sum: no probability anywhere
        __syncthreads();                               // everyone has read the walk's state
        if (tid == 0) {
            if (done) {                                // nothing left of the residual: p itself
                s.A = 0.0;
                s.n_removed = 0;
                s.sum_wanted = drafter;
            } else {
                s.sum = total;
                s.have_sum = !drafter;
                s.S = (double)left * UNIT;
                s.have_S = 1;
            }
        }
        if (done) fallback = true;
    }
    // ---- the next token: the element at which the running sum passes u_next times the whole
    long long mine_all = s.cta_sum[phase][rank];
    for (int j = 0; j < s.n_removed; ++j) {
        const int k = s.removed[j] + row.shift;
        total -= s.removed_p[j];
        if (k < cta_lo) before -= s.removed_p[j];
        else if (k < cta_lo + per_cta) mine_all -= s.removed_p[j];
    }
    if (total > 0) {
        // cum > u T  <=>  cum > floor(u T), in whole numbers
        long long thr = floor_product(a.u_next[b], total);
        if (thr > total - 1) thr = total - 1;
        thr -= before;
        if (thr >= 0 && thr < mine_all) {                          // in this CTA's part (uniform over the CTA)
            int w = 0;
            for (; w < DV_WARPS - 1; ++w) {
                long long ws = s.warp_sum[phase][w];
                for (int j = 0; j < s.n_removed; ++j) {
                    const int k = s.removed[j] + row.shift - cta_lo;
                    if (k >= w * per_warp && k < (w + 1) * per_warp) ws -= s.removed_p[j];
                }
                if (thr < ws) break;
                thr -= ws;
            }
            // the block takes that warp's part, a contiguous piece a thread; then the warp whose
            // piece it is, an element a lane
            const int piece = ((per_warp + DV_THREADS - 1) / DV_THREADS + 3) / 4 * 4;
            const int lo = cta_lo + w * per_warp, hi = lo + per_warp;
            const int k0 = lo + tid * piece, k1 = min(k0 + piece, hi);
            long long mine = 0;
            if (k0 < k1) {
                mine = min(sum_piece(row, c, form, k0, k1), MOST);
                for (int j = 0; j < s.n_removed; ++j) {
                    const int k = s.removed[j] + row.shift;
                    if (k >= k0 && k < k1) mine -= s.removed_p[j];
                }
            }
            auto scan = [&](long long v) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += t;
                }
                return v;
            };
            long long cum = scan(mine);
            if (lane == 31) s.scan[warp] = cum;
            __syncthreads();
            for (int i = 0; i < warp; ++i) cum += s.scan[i];
            const bool here = cum > thr && cum - mine <= thr;
            const unsigned hit = __ballot_sync(0xffffffffu, here);               // one lane of the block
            // (none where a sum was cut off at MOST: the row is no distribution)
            if (!__syncthreads_or(here) && tid == 0) a.out_tokens[base + s.n_acc] = -1;
            if (hit) {
                const int L = __ffs(hit) - 1;
                thr -= __shfl_sync(0xffffffffu, cum - mine, L);
                const int x0 = __shfl_sync(0xffffffffu, k0, L) - row.shift, x1 = __shfl_sync(0xffffffffu, k1, L) - row.shift;
                for (int x = x0 + lane;; x += 32) {
                    long long v = 0;
                    if (x >= 0 && x < min(x1, a.V) && !is_removed(s, x)) v = one(row, c, form, x);
                    const long long upto = scan(v);
                    const unsigned at = __ballot_sync(0xffffffffu, upto > thr);
                    if (at || x - lane + 32 >= x1) {
                        if (lane == (at ? __ffs(at) - 1 : 0)) a.out_tokens[base + s.n_acc] = x >= 0 && x < a.V ? x : -1;
                        break;
                    }
                    thr -= __shfl_sync(0xffffffffu, upto, 31);
                }
            }
        }
    } else if (rank == 0 && tid == 0) {
        a.out_tokens[base + s.n_acc] = -1;
        atomicOr(a.status, DEV_BAD_DRAFT);
    }
    if (rank == 0 && tid < a.q_len) {
        if (tid == 0) a.n_accepted[b] = s.n_acc;
        const bool in = tid < s.n_acc;
        a.path[base + tid] = in ? s.acc[tid] : -1;
        if (tid != s.n_acc) a.out_tokens[base + tid] = in ? s.tok[s.acc[tid]] : -1;
    }
}

}  // namespace

// CTAs a stream: up to sixteen while the launch stays within one wave of four CTAs an SM and a
// thread has a vector of each row at least.
cudaError_t launch_draft_verify(const DraftArgs& a, int B, int num_sms, int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(draft_verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    int C = 1;
    while (C < DV_MAX_CLUSTER && (int64_t)C * DV_THREADS * 4 < a.V && 2ll * C * B <= 4ll * num_sms) C *= 2;
    // whole vectors of 128 elements a warp step; three elements more for the largest shift
    const int64_t span = (int64_t)a.V + 3;
    const int64_t per_warp = ((span + (int64_t)C * DV_WARPS - 1) / ((int64_t)C * DV_WARPS) + 127) / 128 * 128;
    const int64_t per_cta = per_warp * DV_WARPS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(DV_THREADS);
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
    return cudaLaunchKernelEx(&cfg, draft_verify_kernel, a, C, (int)per_cta, (int)per_warp);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_draft_verify(const float* target_probs, const float* draft_probs, const int32_t* draft_tokens,
                                const int32_t* parents, const float* u_accept, const float* u_next, int B, int q_len,
                                int vocab, int32_t* n_accepted, int32_t* tokens, int32_t* path, mla_stream_t stream) {
    if (B < 0 || B > 65535 || q_len < 1 || q_len > MLA_MAX_Q_LEN || vocab < 1 || vocab > MLA_MAX_VOCAB)
        return MLA_ERR_SHAPE;
    if (B == 0) return MLA_OK;
    if (!target_probs || !draft_tokens || !u_accept || !u_next || !n_accepted || !tokens || !path) return MLA_ERR_NULL;
    if (!aligned(target_probs, 16) || !aligned(draft_probs, 16) || !aligned(draft_tokens, 4) || !aligned(parents, 4) ||
        !aligned(u_accept, 4) || !aligned(u_next, 4) || !aligned(n_accepted, 4) || !aligned(tokens, 4) ||
        !aligned(path, 4))
        return MLA_ERR_ALIGN;
    DraftArgs a;
    a.p = target_probs; a.q = draft_probs; a.tokens = draft_tokens; a.parents = parents;
    a.u = u_accept; a.u_next = u_next; a.q_len = q_len; a.V = vocab;
    a.n_accepted = n_accepted; a.out_tokens = tokens; a.path = path;
    int num_sms = 0, dev = 0;
    int rc = device_state(&dev, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    if (launch_draft_verify(a, B, num_sms, dev, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_LAUNCH;
    return MLA_OK;
}
