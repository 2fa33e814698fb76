// The weight that each cached key got from the rows of a step (mla_key_weights, mla_key_weights_fp8):
//     new_j = sum over rows r = (t, h) that count and see key j of exp(z_rj - lse_r)
//     out_j = decay * weights_j + new_j
// The attention's log-sum-exp is given, so there is no softmax to run: every (row, key) pair stands for
// itself, and a key's sum needs nothing of another key.
//
// One CTA handles up to 128 query rows of one stream over one range of its keys, in tiles of 48 keys, on
// the 5th-generation tensor cores: all of Q sits in TMEM (288 columns), the scores of two tiles beside it.
//   gather   16 warps, three keys of a tile each.  fp8 cache: rows into registers, two tiles ahead, and as
//            exact fp16 values into a 128-byte-swizzled stage; bf16 cache: 16-byte cp.async into the stage
//   A, C     tcgen05.mma M=128 (query rows) x N=48 (keys) x K=576; over the fp8 cache the latent's sum A and the
//            rotated part's C apart, as in verify_fp8.cuh: z = s_j A + C needs no rounding of a key
//   weights  one thread a query row: exp2(c z - lse), then the sum over a warp's 32 rows by halving exchanges
//            (16 keys in 16 shuffles), the four warps' sums in shared memory
// More than 128 rows: a row tile a CTA, whose sums meet in the workspace (4 bytes a key and row tile; a
// second small kernel adds them in order).  Sums have a fixed order: equal calls give equal bits.
#include "../../include/mla_verify.h"
#include "internal.cuh"
#include "query_rows.cuh"
#include "score_rules.cuh"
#include "tc_ptx.cuh"

#include <math.h>

#include <atomic>

namespace mla {
namespace {

using namespace tc;

constexpr float LOG2E = 1.4426950408889634f;
constexpr int NK = 48;                               // keys per tile
constexpr int MAX_R = 128;                           // query rows per CTA
constexpr int NT = 768;
constexpr int GATHER0 = 8, GATHER_WARPS = 16;        // warps 0-3 weights, 4 products, 0-7 Q to TMEM, 8-23 gather
constexpr int WK = NK / GATHER_WARPS;                // keys of a tile per gather warp
constexpr int STAGES = 4;
constexpr int RING = STAGES + 2;                     // key scales outlive their stage by the two tiles of scores
constexpr int NCHUNK = D_QK / 64;
constexpr int REGION = NK * 128;                     // one 64-dim chunk of a stage
constexpr int STAGE_BYTES = NCHUNK * REGION;         // 55296 B
constexpr int Q_CHUNK = MAX_R * 128;                 // Q on its way to TMEM lies in stages 1 to 3
constexpr uint32_t TMEM_COLS = 512;
constexpr int D_COL = NCHUNK * 32, D_STEP = 2 * NK;  // scores of tile i at D_COL + (i & 1) D_STEP: A, then C
static_assert(D_COL + 2 * D_STEP <= (int)TMEM_COLS, "TMEM");
static_assert(NCHUNK * Q_CHUNK <= (STAGES - 1) * STAGE_BYTES, "Q's way station");

enum { B_KV_FULL = 0, B_KV_EMPTY = B_KV_FULL + STAGES, B_S_FULL = B_KV_EMPTY + STAGES, B_S_FREE = B_S_FULL + 2,
       B_Q_FULL = B_S_FREE + 2, B_COUNT };

struct Misc {
    uint64_t bars[B_COUNT];
    uint32_t tmem;
    volatile int abort;
    float row_exp[MAX_R];                            // the power of two that a query row was divided by
    float key_scale[RING][NK];
    int key_pos[RING][NK], key_doc[RING][NK];
    float sums[2][4][NK];                            // a tile's sums over the rows of each weights warp
};
constexpr int SMEM = STAGES * STAGE_BYTES + (int)sizeof(Misc);
static_assert(SMEM <= 232448, "opt-in shared memory per block on sm_103");

struct WeightArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kv;      // the bf16 cache, or
    const uint8_t* lat;           // the fp8 cache
    const float* kscale;
    const __nv_bfloat16* rope;
    int64_t n_pool;
    const int32_t* slot;
    int slot_stride;
    const int32_t* seq_lens;
    const uint8_t* mask;
    const uint64_t* mask_bits;
    int B, q_len, H;
    float scale;
    ScoreRules rules;
    const float* lse;
    const uint8_t* counted;
    const float* weights;
    float decay;
    float* out;
    float* part;                  // [row tile][B, slot_stride], used with several row tiles
    int R_step;                   // rows per tile
    int nsplit;                   // key ranges of a stream, or (balanced) of all streams
    int balanced;
    int debug_stall;
    unsigned* status;
};

// Key ranges of B <= 64 streams of unequal length: chunks of whole tiles, the smallest with which all
// streams together need no more than S ranges.  Every warp finds the same; range x's stream and keys.
__device__ __forceinline__ void balanced_range(const WeightArgs& a, int S, int x, int* b, int* begin, int* end, int* index,
                                               int* count) {
    const int lane = threadIdx.x & 31;
    const KeySpan span = a.rules.span();
    int n[2];
    long long total = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        n[h] = i < a.B ? a.seq_lens[i] : -1;
        n[h] = n[h] >= a.q_len && n[h] <= a.slot_stride ? span.seen(i, n[h], a.q_len) : i < a.B ? 0 : -1;
        total += max(n[h], 0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // a stream without keys takes a range too (its length is reported there)
    unsigned c = total < (1ll << 30) ? ((unsigned)total + S - 1u) / S : (unsigned)((total + S - 1) / S);
    c = max(c + NK - 1u, (unsigned)NK) / NK * NK;
    int ns[2], all;
    for (;; c += max(1u, c / (64u * NK)) * NK) {         // (steps of a sixty-fourth: a few dozen at most)
        ns[0] = n[0] < 0 ? 0 : max(1, (int)((n[0] + c - 1u) / c));
        ns[1] = n[1] < 0 ? 0 : max(1, (int)((n[1] + c - 1u) / c));
        all = ns[0] + ns[1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if (all <= S) break;                             // (S >= B: one range a stream always fits)
    }
    int run = 0;
    *b = -1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = ns[h];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        v += run;
        run = __shfl_sync(0xffffffffu, v, 31);
        const unsigned m = __ballot_sync(0xffffffffu, x < v);
        if (m && *b < 0) {
            const int L = __ffs(m) - 1;
            *b = L + 32 * h;
            *count = __shfl_sync(0xffffffffu, ns[h], L);
            *index = x - (__shfl_sync(0xffffffffu, v, L) - *count);
            const int len = __shfl_sync(0xffffffffu, n[h], L);
            *begin = (int)min((long long)len, (long long)*index * c);
            *end = (int)min((long long)len, (*index + 1ll) * c);
        }
    }
}

// Sums of e[k] over the warp's lanes: lane 2 k (and 2 k + 1) ends up with key k's.
__device__ __forceinline__ float sum_rows(float (&e)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 8; half > 0; half >>= 1) {
        const bool up = lane & (2 * half);
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? e[i] : e[i + half], keep = up ? e[i + half] : e[i];
            e[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * half);
        }
    }
    return e[0] + __shfl_xor_sync(0xffffffffu, e[0], 1);
}

__device__ __forceinline__ void give_up(Misc* M, unsigned* status) {
    if (atomicExch(const_cast<int*>(&M->abort), 1) == 0) atomicOr(status, DEV_TIMEOUT);
}

template <bool FP8, bool RULES>
__global__ void __launch_bounds__(NT, 1) key_weights_kernel(const WeightArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Misc* const M = reinterpret_cast<Misc*>(smem + STAGES * STAGE_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = a.q_len * a.H, row0 = blockIdx.y * a.R_step, nrows = min(a.R_step, rows - row0);
    const bool direct = gridDim.y == 1;

    // ---- the keys of this CTA: visible ones k_begin .. k_end - 1 of stream b, range `index` of `count`
    int b = blockIdx.z, k_begin = 0, k_end = 0, index = blockIdx.x, count = a.nsplit;
    if (a.balanced) {
        balanced_range(a, a.nsplit, blockIdx.x, &b, &k_begin, &k_end, &index, &count);
        if (b < 0) return;
    }
    const int n = a.seq_lens[b];
    if (n < a.q_len || n > a.slot_stride) {
        if (tid == 0) atomicOr(a.status, DEV_BAD_LEN);
        return;
    }
    int gap_at = 0, gap = 0;
    if (RULES) a.rules.span().gap(b, n, a.q_len, &gap_at, &gap);
    if (!a.balanced) split_range(n - gap, a.nsplit, index, NK, &k_begin, &k_end);
    const int T = (k_end - k_begin + NK - 1) / NK;
    const int p = n - gap - a.q_len;                     // first draft among the visible keys
    const int64_t stream0 = (int64_t)b * a.slot_stride;
    float* const part = direct ? a.out : a.part + (int64_t)blockIdx.y * a.B * a.slot_stride;

    // keys that no draft sees: their former weights decay
    if (RULES && direct) {
        const int share = (gap + count - 1) / count, g0 = index * share, g1 = min(gap, g0 + share);
        for (int g = g0 + tid; g < g1; g += NT)
            a.out[stream0 + gap_at + g] = a.weights ? a.decay * a.weights[stream0 + gap_at + g] : 0.f;
    }
    if (T <= 0) return;
    if (smem_u32(smem) & 1023u) {                        // the swizzled layouts need a 1024-byte aligned base
        if (tid == 0) atomicOr(a.status, DEV_TIMEOUT);
        return;
    }

    if (warp == 4) {
        tmem_alloc(&M->tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (tid == 5 * 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&M->bars[B_KV_FULL + i], FP8 ? GATHER_WARPS : 32 * GATHER_WARPS);
            mbar_init(&M->bars[B_KV_EMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M->bars[B_S_FULL + i], 1);
            mbar_init(&M->bars[B_S_FREE + i], 4);
        }
        mbar_init(&M->bars[B_Q_FULL], 8);
        M->abort = 0;
        mbar_init_fence();
    }

    // ---- Q rows warp, warp + 24, warp + 48 and so on into stages 1 to 3 (chunks of 128 rows of 128 B, swizzled)
    uint8_t* const q_tmp = smem + STAGE_BYTES;
    const __nv_bfloat16* q0 = a.q + ((int64_t)b * rows + row0) * D_QK;
    for (int first = warp; first < nrows; first += 3 * (NT / 32)) {
        uint4 v[3][3];
        load_q_rows(v, q0, first, NT / 32, nrows);
        int exps[3];
        if (FP8) row_exponents<3>(v, exps);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            const int rr = first + u * (NT / 32);
            if (rr >= nrows) break;
            const float mul = FP8 ? __int_as_float((14 - exps[u] + 127) << 23) : 1.f;
            if (FP8 && lane == 0) M->row_exp[rr] = __int_as_float((exps[u] - 14 + 127) << 23);
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const int pc = c * 32 + lane;
                if (pc >= 72) break;
                uint4 o = v[u][c];
                if (FP8 && pc < 64) o = make_uint4(q_to_f16(o.x, mul), q_to_f16(o.y, mul), q_to_f16(o.z, mul), q_to_f16(o.w, mul));
                else if (FP8) o = make_uint4(q_to_bf16(o.x, mul), q_to_bf16(o.y, mul), q_to_bf16(o.z, mul), q_to_bf16(o.w, mul));
                *reinterpret_cast<uint4*>(q_tmp + (pc >> 3) * Q_CHUNK + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4)) = o;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;

    if (warp < 8) {
        // ---- Q to TMEM: warps w and w + 4 the rows of quadrant w, chunks in turn
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int r = (warp & 3) * 32 + lane;
        if ((warp & 3) * 32 < nrows) {
#pragma unroll 1
            for (int c = warp >> 2; c < NCHUNK; c += 2) {
                uint32_t h[32];
                const uint8_t* src = q_tmp + c * Q_CHUNK + r * 128;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + ((j ^ (r & 7)) << 4));
                    h[4 * j] = v.x; h[4 * j + 1] = v.y; h[4 * j + 2] = v.z; h[4 * j + 3] = v.w;
                }
                tmem_st32(tmem + lane_base + c * 32, h);
            }
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M->bars[B_Q_FULL]);
    }

    if (warp == 4) {
        // ================= A and C =================
        const uint32_t id_a = FP8 ? idesc_f16(128, NK, false, false) : idesc_bf16(128, NK, false, false);
        const uint32_t id_c = idesc_bf16(128, NK, false, false);
        const uint64_t dk = smem_desc_sw128(smem_u32(smem), 16, 1024);
        bool ok = mbar_wait_warp(&M->bars[B_Q_FULL], 0, &M->abort);
        int i = 0;                                       // tiles issued
        for (; i < T && ok; ++i) {
            const int st = i % STAGES;
            ok = mbar_wait_warp(&M->bars[B_KV_FULL + st], (i / STAGES) & 1, &M->abort);
            if (ok && i >= 2) ok = mbar_wait_warp(&M->bars[B_S_FREE + (i & 1)], ((i - 2) / 2) & 1, &M->abort);
            if (!ok) break;
            fence_proxy_async_smem();                    // keys (generic proxy) -> tensor-core reads
            tc_fence_after();
            const uint64_t st16 = (uint64_t)(st * STAGE_BYTES) >> 4;
            const uint32_t d = tmem + D_COL + (i & 1) * D_STEP;
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D_QK / 16; ++ks) {
                    const int c = ks >> 2;
                    const uint64_t kd = dk + st16 + (uint32_t)((c * REGION + (ks & 3) * 32) >> 4);
                    if (FP8 && c == NCHUNK - 1) mma_bf16_ta(d + NK, tmem + ks * 8, kd, id_c, (ks & 3) > 0);
                    else mma_bf16_ta(d, tmem + ks * 8, kd, id_a, ks > 0);
                }
                mma_commit(&M->bars[B_KV_EMPTY + st]);
                mma_commit(&M->bars[B_S_FULL + (i & 1)]);
            }
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0) give_up(M, a.status);
            if (i > 0) mbar_drain(&M->bars[B_S_FULL + ((i - 1) & 1)], ((i - 1) / 2) & 1);
        }
        __syncwarp();
    } else if (warp >= GATHER0) {
        // ================= gather: keys WK w .. WK w + 2 of every tile =================
        const int w = warp - GATHER0;
        bool bad_slot = false;
        const int32_t* slot_row = a.slot + stream0;
        // key l & 3 of tile t (past the range: its last key), and its index in the stream
        auto key_at = [&](int t) -> int {
            const int v = min(k_begin + t * NK + WK * w + min(lane & 3, WK - 1), k_end - 1);
            return RULES && v >= gap_at ? v + gap : v;
        };
        // lane l holds the slot of key l & 3 of tile t0 + (l >> 2), for the current group of eight tiles and
        // the next; indices are checked when their group becomes current
        auto load_slots = [&](int t0) -> int {
            const int t = t0 + (lane >> 2);
            return t < T ? __ldg(slot_row + key_at(t)) : 0;
        };
        int cur = load_slots(0), nxt = load_slots(8);
        auto slots_of = [&](int j) -> int {
            if ((j & 7) == 0) {
                if (j > 0) {
                    cur = nxt;
                    nxt = load_slots(j + 8);
                }
                if (cur < 0 || (int64_t)cur >= a.n_pool) { bad_slot = true; cur = 0; }
            }
            return __shfl_sync(0xffffffffu, cur, ((j & 7) << 2) + (lane & 3));
        };
        // the stage is free: its products are done, and Q has left it
        auto stage_free = [&](int i) -> bool {
            if ((i >= STAGES && !mbar_wait_warp(&M->bars[B_KV_EMPTY + i % STAGES], ((i - STAGES) / STAGES) & 1, &M->abort)) ||
                (i == 1 && !mbar_wait_warp(&M->bars[B_Q_FULL], 0, &M->abort))) {
                if (lane == 0) give_up(M, a.status);
                return false;
            }
            return true;
        };
        if constexpr (FP8) {
            struct Raw {
                uint4 lat[WK], rope;
                float scale;
                int pos, doc;                            // RULES
            };
            auto load_tile = [&](Raw& r, int j) {
                if (j >= T) return;
                const int sl = slots_of(j);
#pragma unroll
                for (int it = 0; it < WK; ++it)
                    r.lat[it] = ld_stream(reinterpret_cast<const uint4*>(a.lat + (int64_t)__shfl_sync(0xffffffffu, sl, it) * D_V) + lane);
                const int rs = __shfl_sync(0xffffffffu, sl, lane >> 3);
                if (lane < 8 * WK) r.rope = ld_stream(reinterpret_cast<const uint4*>(a.rope + (int64_t)rs * 64) + (lane & 7));
                r.scale = __ldg(a.kscale + sl);
                if (RULES) {
                    if (a.rules.key_pos) r.pos = __ldg(a.rules.key_pos + stream0 + key_at(j));
                    if (a.rules.key_doc) r.doc = __ldg(a.rules.key_doc + stream0 + key_at(j));
                }
            };
            // lane l widens dims 16 l .. 16 l + 15: 16-byte pieces j0, j0 + 1 of region l / 4.  Lanes of odd
            // regions store their second piece first, so each store covers all eight 16-byte bank groups.
            const int region = lane >> 2, j0 = (lane & 3) * 2, odd = region & 1;
            auto widen_tile = [&](const Raw& r, int i) -> bool {
                if (!stage_free(i)) return false;
                const int st = i % STAGES;
                uint8_t* base = smem + st * STAGE_BYTES;
#pragma unroll
                for (int it = 0; it < WK; ++it) {
                    const int key = WK * w + it;
                    const uint2 h0 = widen4(r.lat[it].x), h1 = widen4(r.lat[it].y), h2 = widen4(r.lat[it].z), h3 = widen4(r.lat[it].w);
                    const uint4 lo = make_uint4(h0.x, h0.y, h1.x, h1.y), hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
                    uint8_t* row = base + region * REGION + key * 128;
                    *reinterpret_cast<uint4*>(row + (((j0 + odd) ^ (key & 7)) << 4)) = odd ? hi : lo;
                    *reinterpret_cast<uint4*>(row + (((j0 + 1 - odd) ^ (key & 7)) << 4)) = odd ? lo : hi;
                }
                if (lane < 8 * WK) {
                    const int key = WK * w + (lane >> 3);
                    *reinterpret_cast<uint4*>(base + (NCHUNK - 1) * REGION + key * 128 + (((lane & 7) ^ (key & 7)) << 4)) = r.rope;
                }
                if (lane < WK) {
                    M->key_scale[i % RING][WK * w + lane] = r.scale >= 0.f ? r.scale : __int_as_float(0x7fc00000);
                    if (RULES) {
                        M->key_pos[i % RING][WK * w + lane] = a.rules.key_pos ? r.pos : key_at(i);
                        M->key_doc[i % RING][WK * w + lane] = a.rules.key_doc ? r.doc : -1;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !(a.debug_stall && i == 0)) mbar_arrive(&M->bars[B_KV_FULL + st]);
                return true;
            };
            Raw r0, r1;
            load_tile(r0, 0);
            load_tile(r1, 1);
            for (int i = 0; i < T; i += 2) {
                if (!__all_sync(0xffffffffu, widen_tile(r0, i))) break;
                load_tile(r0, i + 2);
                if (i + 1 >= T) break;
                if (!__all_sync(0xffffffffu, widen_tile(r1, i + 1))) break;
                load_tile(r1, i + 3);
            }
        } else {
            for (int i = 0; i < T; ++i) {
                const int sl = slots_of(i), st = i % STAGES;
                if (!__all_sync(0xffffffffu, stage_free(i))) break;
                const uint32_t base = smem_u32(smem) + st * STAGE_BYTES;
#pragma unroll
                for (int it = 0; it < (WK * 72 + 31) / 32; ++it) {
                    const int f = it * 32 + lane, kk = min(f / 72, WK - 1), pc = f % 72, key = WK * w + kk;
                    const int row_slot = __shfl_sync(0xffffffffu, sl, kk);
                    if (f < WK * 72)
                        cp_async16(base + (pc >> 3) * REGION + key * 128 + (((pc & 7) ^ (key & 7)) << 4),
                                   a.kv + (int64_t)row_slot * D_QK + pc * 8);
                }
                if (RULES && lane < WK) {
                    if (a.rules.key_pos) cp_async4(smem_u32(&M->key_pos[i % RING][WK * w + lane]), a.rules.key_pos + stream0 + key_at(i));
                    if (a.rules.key_doc) cp_async4(smem_u32(&M->key_doc[i % RING][WK * w + lane]), a.rules.key_doc + stream0 + key_at(i));
                }
                if (!(a.debug_stall && i == 0)) cp_async_arrive_noinc(&M->bars[B_KV_FULL + st]);
            }
            cp_async_wait_all();
        }
        if (bad_slot) atomicOr(a.status, DEV_BAD_SLOT);
    } else if (warp < 4) {
        // ================= weights =================
        const int r = warp * 32 + lane;                  // query row of this thread (lane of A and C)
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const bool row_ok = r < nrows, rows_used = warp * 32 < nrows;
        const int t = row_ok ? (row0 + r) / a.H : 0;
        const float lse = row_ok ? a.lse[(int64_t)b * rows + row0 + r] : 0.f;
        const bool live = row_ok && lse != -INFINITY && (!a.counted || a.counted[(int64_t)b * a.q_len + t]);
        const bool any_live = __any_sync(0xffffffffu, live);
        // drafts this row sees, bit i = draft i (q_len <= 64)
        uint64_t vis = 0;
        if (live) {
            if (a.mask_bits) {
                vis = a.mask_bits[(int64_t)b * a.q_len + t];
            } else if (a.mask) {
                for (int d = 0; d < a.q_len; ++d)
                    vis |= (uint64_t)(a.mask[((int64_t)b * a.q_len + t) * a.q_len + d] != 0 ? 1u : 0u) << d;
            } else {
                vis = t >= 63 ? ~0ull : (2ull << t) - 1;
            }
        }
        const float c2 = live ? a.scale * LOG2E * (FP8 ? M->row_exp[r] : 1.f) : 0.f;
        const float off = -lse * LOG2E;
        RowRule rule;
        if (RULES) rule = a.rules.row(b, t, row_ok ? (row0 + r) % a.H : 0, p + gap, a.slot_stride, false);
        const float cap_in = RULES && a.rules.softcap > 0.f ? 2.f * c2 / a.rules.softcap : 0.f;
        const float cap_out = RULES ? a.rules.softcap * LOG2E : 0.f;
        for (int i = 0; i < T; ++i) {
            const int buf = i & 1, k0 = k_begin + i * NK;
            // the key that this thread writes, and its former weight
            const int v = k0 + tid;
            const int64_t at = stream0 + (RULES && v >= gap_at ? v + gap : v);
            const bool mine = tid < NK && v < k_end;
            float old = 0.f;
            if (direct && mine && a.weights && v < p) old = a.weights[at];
            const bool ok = mbar_wait_warp(&M->bars[B_S_FULL + buf], (i / 2) & 1, &M->abort);
            tc_fence_after();
            if (ok && rows_used) {
#pragma unroll
                for (int g = 0; g < NK / 16; ++g) {
                    uint32_t va[16], vc[16];
                    const uint32_t d = tmem + lane_base + D_COL + buf * D_STEP + 16 * g;
                    tmem_ld16(d, va);
                    if (FP8) tmem_ld16(d + NK, vc);
                    tmem_ld_wait();
                    float e[16];
                    const int kg = k0 + 16 * g;
                    const float* ks = M->key_scale[i % RING] + 16 * g;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float dot = FP8 ? fmaf(__uint_as_float(va[k]), ks[k], __uint_as_float(vc[k])) : __uint_as_float(va[k]);
                        float x;
                        if (RULES) {
                            x = a.rules.softcap > 0.f ? fmaf(capped(dot * cap_in), cap_out, off) : fmaf(dot, c2, off);
                            if (a.rules.slopes) {
                                const int kp = FP8 || a.rules.key_pos ? M->key_pos[i % RING][16 * g + k]
                                                                      : (kg + k >= gap_at ? kg + k + gap : kg + k);
                                x = fmaf((float)(kp - rule.pos), rule.slope, x);
                            }
                        } else {
                            x = fmaf(dot, c2, off);
                        }
                        e[k] = live ? ex2(x) : 0.f;
                    }
                    if (RULES && a.rules.masked) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int j = kg + k - p;    // draft index, < 0: before the drafts
                            const int kp = FP8 || a.rules.key_pos ? M->key_pos[i % RING][16 * g + k]
                                                                  : (kg + k >= gap_at ? kg + k + gap : kg + k);
                            const int kd = FP8 || a.rules.key_doc ? M->key_doc[i % RING][16 * g + k] : -1;
                            if (!rule.sees(j < 0 || ((vis >> (j & 63)) & 1ull), kp, kd)) e[k] = 0.f;
                        }
                    } else if (kg + 16 > p) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int j = kg + k - p;
                            if (j >= 0 && !((vis >> (j & 63)) & 1ull)) e[k] = 0.f;
                        }
                    }
                    const float s = any_live ? sum_rows(e) : 0.f;
                    if ((lane & 1) == 0) M->sums[buf][warp][16 * g + (lane >> 1)] = s;
                }
                tc_fence_before();
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&M->bars[B_S_FREE + buf]);
            if (bar_red_or(1, 128, !ok)) {               // the sums are there, or a warp gives up
                if (!ok && lane == 0) give_up(M, a.status);
                break;
            }
            if (mine) {
                float s = M->sums[buf][0][tid];
#pragma unroll
                for (int q = 1; q < 4; ++q)
                    if (q * 32 < nrows) s += M->sums[buf][q][tid];
                part[at] = direct && a.weights && v < p ? fmaf(a.decay, old, s) : s;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// The row tiles' sums of each key, added in order.
__global__ void __launch_bounds__(256) key_weights_join(const WeightArgs a, int n_tiles) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y, n = a.seq_lens[b];
    if (n < a.q_len || n > a.slot_stride) return;
    int gap_at, gap;
    a.rules.span().gap(b, n, a.q_len, &gap_at, &gap);
    const int64_t step = (int64_t)a.B * a.slot_stride;
    for (int j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) {
        const int64_t at = (int64_t)b * a.slot_stride + j;
        float s = 0.f;
        if (j < gap_at || j >= gap_at + gap) {
            s = a.part[at];
            for (int i = 1; i < n_tiles; ++i) s += a.part[at + i * step];
        }
        a.out[at] = a.weights && j < n - a.q_len ? fmaf(a.decay, a.weights[at], s) : s;
    }
}

void weight_tiling(int rows, int* n_tiles, int* R_step) {
    *n_tiles = (rows + MAX_R - 1) / MAX_R;
    *R_step = (rows + *n_tiles - 1) / *n_tiles;
}

// Key ranges of a stream: the least of waves of CTAs x (a CTA's start + its tiles).
int weight_nsplit(int B, int n_tiles, int max_seq, int num_sms) {
    const long long fixed = 6, tiles = ((long long)max_seq + NK - 1) / NK;
    const long long most = min(tiles, 8ll * num_sms / ((long long)B * n_tiles) + 1);
    long long best = 1, best_cost = 0;
    for (long long want = 1; want <= most; ++want) {
        const long long per_cta = (tiles + want - 1) / want, ns = (tiles + per_cta - 1) / per_cta;   // none empty
        const long long cost = ((long long)B * n_tiles * ns + num_sms - 1) / num_sms * (fixed + per_cta);
        if (want == 1 || cost < best_cost) { best = ns; best_cost = cost; }
    }
    return (int)best;
}

template <bool FP8, bool RULES>
cudaError_t launch_weights(const WeightArgs& a, dim3 grid, int dev, cudaStream_t stream) {
    auto* k = key_weights_kernel<FP8, RULES>;
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(k, grid, dim3(NT), (size_t)SMEM, stream, a);
}

template <bool FP8>
int key_weights_call(WeightArgs a, const uint64_t* bits, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    if (a.B < 0 || a.B > 65535 || a.q_len < 1 || a.q_len > MLA_MAX_Q_LEN || a.H < 1 || a.H > MLA_MAX_HEADS) return MLA_ERR_SHAPE;
    if (a.B == 0) return MLA_OK;
    if (!a.q || (FP8 ? !a.lat || !a.kscale || !a.rope : !a.kv) || !a.slot || !a.seq_lens || !a.lse || !a.out) return MLA_ERR_NULL;
    if (a.n_pool < 1 || a.n_pool > 0x7fffffffLL || a.slot_stride < a.q_len || a.slot_stride > MLA_MAX_FP8_KEYS) return MLA_ERR_SHAPE;
    if ((long long)a.B * a.q_len * a.H > 0x7fffffffLL) return MLA_ERR_SHAPE;
    if (!isfinite(a.scale) || !isfinite(a.decay) || (a.mask && bits)) return MLA_ERR_ARG;
    if (!aligned(a.q, 16) || !aligned(a.lat, 16) || !aligned(a.rope, 16) || !aligned(a.kscale, 4) || !aligned(a.kv, 16) ||
        !aligned(a.slot, 4) || !aligned(a.seq_lens, 4) || !aligned(a.lse, 4) || !aligned(a.weights, 4) ||
        !aligned(a.out, 4) || !aligned(bits, 8))
        return MLA_ERR_ALIGN;
    a.mask_bits = bits;
    const size_t need = mla_key_weights_workspace_bytes(a.B, a.q_len, a.H, a.slot_stride);
    if (need) {
        if (!workspace || ws_bytes < need) return MLA_ERR_WORKSPACE;
        if (!aligned(workspace, 4)) return MLA_ERR_ALIGN;
        a.part = static_cast<float*>(workspace);
    }
    int num_sms = 0, dev = 0, n_tiles;
    const int rc = device_state(&dev, &a.status, &num_sms);
    if (rc != MLA_OK) return rc;
    weight_tiling(a.q_len * a.H, &n_tiles, &a.R_step);
    a.debug_stall = take_debug_stall() ? 1 : 0;
    const int slots = num_sms / n_tiles;
    if (a.B >= 2 && a.B <= BALANCED_MAX_STREAMS && slots >= 2 * a.B) {
        a.balanced = 1;
        a.nsplit = slots;
    } else {
        a.nsplit = weight_nsplit(a.B, n_tiles, a.rules.span().most(a.slot_stride, a.q_len), num_sms);
    }
    const dim3 grid(a.nsplit, n_tiles, a.balanced ? 1 : a.B);
    const ScoreRules& r = a.rules;
    const bool ruled = r.softcap > 0.f || r.slopes || r.masked;
    if ((ruled ? launch_weights<FP8, true>(a, grid, dev, stream) : launch_weights<FP8, false>(a, grid, dev, stream)) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    if (n_tiles > 1) {
        const int blocks = (int)min(((long long)a.slot_stride + 255) / 256, max(1ll, 16ll * num_sms / a.B));
        if (launch_dependent(key_weights_join, dim3(blocks, a.B), dim3(256), 0, stream, a, n_tiles) != cudaSuccess)
            return MLA_ERR_LAUNCH;
    }
    return MLA_OK;
}

WeightArgs weight_args(const void* q, int64_t n_pool, const int32_t* slot_table, int slot_stride, const int32_t* seq_lens,
                       const uint8_t* draft_mask, int B, int q_len, int H, float scale, const ScoreRules& rules,
                       const float* lse, const uint8_t* counted, const float* weights, float decay, float* out) {
    WeightArgs a{};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_pool = n_pool; a.slot = slot_table; a.slot_stride = slot_stride; a.seq_lens = seq_lens; a.mask = draft_mask;
    a.B = B; a.q_len = q_len; a.H = H; a.scale = scale; a.rules = rules;
    a.lse = lse; a.counted = counted; a.weights = weights; a.decay = decay; a.out = out;
    return a;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_key_weights_fp8(const void* q, const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope,
                                   int64_t n_pool, const int32_t* slot_table, int slot_stride, const int32_t* seq_lens,
                                   const uint8_t* draft_mask, const uint64_t* draft_mask_bits, int B, int q_len, int H,
                                   float scale, float softcap, const float* slopes, const int32_t* key_pos, int window,
                                   const int32_t* prefix_lens, const int32_t* key_doc, const float* lse,
                                   const uint8_t* counted, const float* weights, float decay, float* out,
                                   void* workspace, size_t ws_bytes, mla_stream_t stream) {
    ScoreRules rules;
    const int rc = check_rules(softcap, slopes, key_pos, window, prefix_lens, key_doc, &rules);
    if (rc != MLA_OK) return rc;
    WeightArgs a = weight_args(q, n_pool, slot_table, slot_stride, seq_lens, draft_mask, B, q_len, H, scale, rules, lse,
                               counted, weights, decay, out);
    a.lat = kv_lat; a.kscale = kv_scale; a.rope = static_cast<const __nv_bfloat16*>(kv_rope);
    return key_weights_call<true>(a, draft_mask_bits, workspace, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int mla_key_weights(const void* q, const void* kv_cache, int64_t n_pool, const int32_t* slot_table,
                               int slot_stride, const int32_t* seq_lens, const uint8_t* draft_mask,
                               const uint64_t* draft_mask_bits, int B, int q_len, int H, float scale, float softcap,
                               const float* slopes, const int32_t* key_pos, int window, const int32_t* prefix_lens,
                               const int32_t* key_doc, const float* lse, const uint8_t* counted, const float* weights,
                               float decay, float* out, void* workspace, size_t ws_bytes, mla_stream_t stream) {
    ScoreRules rules;
    const int rc = check_rules(softcap, slopes, key_pos, window, prefix_lens, key_doc, &rules);
    if (rc != MLA_OK) return rc;
    WeightArgs a = weight_args(q, n_pool, slot_table, slot_stride, seq_lens, draft_mask, B, q_len, H, scale, rules, lse,
                               counted, weights, decay, out);
    a.kv = static_cast<const __nv_bfloat16*>(kv_cache);
    return key_weights_call<false>(a, draft_mask_bits, workspace, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t mla_key_weights_workspace_bytes(int B, int q_len, int H, int slot_stride) {
    if (B <= 0 || q_len < 1 || q_len > MLA_MAX_Q_LEN || H < 1 || H > MLA_MAX_HEADS || slot_stride < 1) return 0;
    int n_tiles, R_step;
    weight_tiling(q_len * H, &n_tiles, &R_step);
    return n_tiles > 1 ? (size_t)n_tiles * B * slot_stride * 4 : 0;
}
