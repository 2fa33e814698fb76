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
// two-sum and the product's error by a fused multiply-add), rounded to a multiple of 2^-45
// and summed as a 64-bit integer: sums do not depend on their order or on how the
// vocabulary is split, and the GPU's few fp64 units see a handful of operations a node.
//
// Bound by HBM, one pass over the row pair of the node the walk stops at (8 V bytes a
// stream; a pass more for each sibling tried after a rejection, mostly from L2), and by
// latency for few streams.  A cluster of CTAs shares a stream: each CTA owns a contiguous
// part of the vocabulary, each of its warps a contiguous part of that, and the partial sums
// meet in distributed shared memory.  Every CTA repeats the walk (a few dozen operations),
// so only sums cross CTAs.
#include "../../include/mla_verify.h"
#include "internal.cuh"

#include <cooperative_groups.h>
#include <math.h>

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr int DV_THREADS = 512;
constexpr int DV_WARPS = DV_THREADS / 32;
constexpr int DV_MAX_CLUSTER = 8;
constexpr double UNIT = 1.0 / 35184372088832.0;      // 2^-45, the unit of the integer sums

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
__device__ __forceinline__ float prob(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

// max(p - A q, 0) in units of 2^-45, A = ah + al.
__device__ __forceinline__ long long residual(float p, float q, float ah, float al) {
    // (explicit roundings: a contracted multiply-add would lose the errors' meaning)
    const float ph = __fmul_rn(ah, q);
    const float pe = fmaf(al, q, fmaf(ah, q, -ph));   // A q = ph + pe
    const float d = __fsub_rn(p, ph);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), ph), pe);   // p - A q = d + e where d > 0
    if (!(d + e > 0.f)) return 0;
    // adding 1.5 * 2^23 rounds to an integer and leaves it in the low mantissa bits
    constexpr float MAGIC = 12582912.f;
    const float th = fmaf(d, 4194304.f, MAGIC);                               // d * 2^22
    const float hi = th - MAGIC;
    const float rem = fmaf(hi, -2.384185791015625e-07f, d) + e;               // |rem| <= 2^-23
    const float tl = fmaf(rem, 35184372088832.f, MAGIC);                      // rem * 2^45
    return (long long)(__float_as_int(th) - 0x4B400000) * 8388608ll + (__float_as_int(tl) - 0x4B400000);
}

struct Shared {
    int par[MLA_MAX_Q_LEN], tok[MLA_MAX_Q_LEN];
    float u[MLA_MAX_Q_LEN], pt[MLA_MAX_Q_LEN], qt[MLA_MAX_Q_LEN];   // p and q of the node's token at its parent
    int removed[MLA_MAX_Q_LEN];                        // tokens taken out of p (no drafter)
    int acc[MLA_MAX_Q_LEN];                            // accepted nodes
    int n_acc, n_removed, cur, node, done;
    double A, S;
    int have_S;
    long long warp_sum[2][DV_WARPS];
    long long cta_sum[2];
    long long scan[DV_WARPS];
    int found;
};

__device__ __forceinline__ bool is_removed(const Shared& s, int x) {
    for (int i = 0; i < s.n_removed; ++i)
        if (s.removed[i] == x) return true;
    return false;
}

__global__ void __launch_bounds__(DV_THREADS) draft_verify_kernel(const DraftArgs a, int C, int per_cta, int per_warp) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.x / C, rank = blockIdx.x % C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t V = a.V;
    const int64_t base = (int64_t)b * a.q_len;
    const bool drafter = a.q != nullptr;
    // ---- the nodes: parent, token, random number and both probabilities of the token
    if (tid < a.q_len) {
        const int i = tid;
        int par = a.parents ? a.parents[base + i] : i - 1;
        const int tok = a.tokens[base + i];
        bool bad = false;
        if (i == 0) {
            par = -2;                                  // the root is nobody's child
        } else if (par < -1 || par >= i || (par >= 0 && (tok < 0 || tok >= a.V))) {
            bad = true;
        }
        if (bad) {
            par = -2;
            if (rank == 0) atomicOr(a.status, DEV_BAD_DRAFT);
        }
        float pt = 0.f, qt = 1.f;
        if (par >= 0) {
            pt = prob(a.p[(base + par) * V + tok]);
            if (drafter) qt = prob(a.q[(base + par) * V + tok]);
        }
        s.par[i] = par;
        s.tok[i] = tok;
        s.u[i] = a.u[base + i];
        s.pt[i] = pt;
        s.qt[i] = qt;
    }
    if (tid == 0) {
        s.n_acc = 0; s.n_removed = 0; s.cur = 0; s.node = 1; s.done = 0;
        s.A = 0.0; s.S = 1.0; s.have_S = 1;
    }
    __syncthreads();
    const int64_t my_lo = (int64_t)rank * per_cta + (int64_t)warp * per_warp;
    int64_t my_hi = my_lo + per_warp;
    if (my_hi > (int64_t)(rank + 1) * per_cta) my_hi = (int64_t)(rank + 1) * per_cta;
    int phase = 0;
    bool fallback = false;
    long long total = 0, before = 0;
    for (;;) {
        // ---- walk until a test needs the residual's sum, or the tree ends
        if (tid == 0 && !fallback) {
            int i = s.node;
            for (; i < a.q_len; ++i) {
                if (s.par[i] != s.cur) continue;
                if (!s.have_S) break;
                const double qx = s.qt[i];
                double r;
                if (drafter) {
                    r = (double)s.pt[i] - s.A * qx;
                } else {
                    r = is_removed(s, s.tok[i]) ? 0.0 : (double)s.pt[i];
                }
                if ((double)s.u[i] * qx * s.S < r) {
                    s.acc[s.n_acc++] = i;
                    s.cur = i;
                    s.A = 0.0; s.S = 1.0; s.have_S = 1;
                    s.n_removed = 0;
                } else {
                    s.A += s.S;
                    s.have_S = 0;
                    if (!drafter && !is_removed(s, s.tok[i])) s.removed[s.n_removed++] = s.tok[i];
                }
            }
            s.node = i;
            s.done = i >= a.q_len;
        }
        __syncthreads();
        // ---- sum of the residual over this CTA's part of the vocabulary
        const int64_t row = (base + s.cur) * V;
        const bool use_q = drafter && s.A > 0.0;
        const float ah = (float)s.A, al = (float)(s.A - (double)ah);
        const float* p = a.p + row;
        const float* q = use_q ? a.q + row : nullptr;
        // vectors of four start on 16-byte boundaries, `shift` elements before the row
        const int shift = (int)(row & 3);
        long long sum = 0;
        for (int64_t k = my_lo + lane * 4; k < my_hi; k += 128) {
            const int64_t x = k - shift;
            if (x >= V) break;
            float pv[4], qv[4] = {0.f, 0.f, 0.f, 0.f};
            if (x >= 0 && x + 4 <= V) {
                const float4 t = __ldg(reinterpret_cast<const float4*>(p + x));
                pv[0] = t.x; pv[1] = t.y; pv[2] = t.z; pv[3] = t.w;
                if (use_q) {
                    const float4 w = __ldg(reinterpret_cast<const float4*>(q + x));
                    qv[0] = w.x; qv[1] = w.y; qv[2] = w.z; qv[3] = w.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = x + j >= 0 && x + j < V;
                    pv[j] = in ? p[x + j] : 0.f;
                    if (use_q) qv[j] = in ? q[x + j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += residual(prob(pv[j]), prob(qv[j]), ah, al);
        }
        if (!drafter && !fallback)
            for (int j = lane; j < s.n_removed; j += 32) {
                const int64_t x = s.removed[j] + shift;
                if (x >= my_lo && x < my_hi) sum -= residual(prob(p[s.removed[j]]), 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s.warp_sum[phase][warp] = sum;
        __syncthreads();
        if (tid == 0) {
            long long t = 0;
            for (int w = 0; w < DV_WARPS; ++w) t += s.warp_sum[phase][w];
            s.cta_sum[phase] = t;
        }
        cluster.sync();
        total = before = 0;
        for (int r = 0; r < C; ++r) {
            const long long v = *cluster.map_shared_rank(&s.cta_sum[phase], r);
            if (r < rank) before += v;
            total += v;
        }
        const bool done = s.done;
        if (done && (total > 0 || fallback)) break;    // a fallback without a sum: no probability anywhere
        __syncthreads();                               // everyone has read the walk's state
        if (tid == 0) {
            if (done) {                                // nothing left of the residual: p itself
                s.A = 0.0;
                s.n_removed = 0;
            } else {
                s.S = (double)total * UNIT;
                s.have_S = 1;
            }
        }
        if (done) fallback = true;
        phase ^= 1;
    }
    // ---- the next token: the element at which the running sum passes u_next * total
    int next = -1;
    if (total > 0) {
        const double want = (double)a.u_next[b] * (double)total;
        long long thr = want > 0.0 ? (long long)want : 0;          // floor; cum > u T  <=>  cum > floor(u T)
        if (thr > total - 1) thr = total - 1;
        thr -= before;
        if (thr >= 0 && thr < s.cta_sum[phase]) {                  // in this CTA's part (uniform over the CTA)
            int w = 0;
            while (thr >= s.warp_sum[phase][w]) thr -= s.warp_sum[phase][w++];
            const int64_t row = (base + s.cur) * V;
            const bool use_q = drafter && s.A > 0.0;
            const float ah = (float)s.A, al = (float)(s.A - (double)ah);
            const int shift = (int)(row & 3);
            const int64_t lo = (int64_t)rank * per_cta + (int64_t)w * per_warp - shift;
            if (tid == 0) s.found = 0;
            for (int64_t k = lo; k < lo + per_warp; k += DV_THREADS) {
                const int64_t x = k + tid;
                long long v = 0;
                if (x >= 0 && x < V && x < lo + per_warp && (drafter || !is_removed(s, (int)x)))
                    v = residual(prob(a.p[row + x]), use_q ? prob(a.q[row + x]) : 0.f, ah, al);
                long long c = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, c, o);
                    if (lane >= o) c += t;
                }
                __syncthreads();                       // s.scan of the previous chunk has been read
                if (lane == 31) s.scan[warp] = c;
                __syncthreads();
                long long all = 0, mine = 0;
                for (int i = 0; i < DV_WARPS; ++i) {
                    if (i < warp) mine += s.scan[i];
                    all += s.scan[i];
                }
                if (mine + c > thr && mine + c - v <= thr) s.found = (int)x;   // exactly one thread, v > 0
                if (all > thr) break;
                thr -= all;
            }
            __syncthreads();
            next = s.found;
            if (tid == 0) a.out_tokens[base + s.n_acc] = next;
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
    cluster.sync();                                    // no CTA leaves while another may read its sums
}

}  // namespace

cudaError_t launch_draft_verify(const DraftArgs& a, int B, cudaStream_t stream) {
    int C = 1;
    while (C < DV_MAX_CLUSTER && (int64_t)C * DV_THREADS * 4 < a.V) C *= 2;
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
    int rc = device_state(nullptr, &a.status, nullptr);
    if (rc != MLA_OK) return rc;
    if (launch_draft_verify(a, B, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MLA_ERR_LAUNCH;
    return MLA_OK;
}
