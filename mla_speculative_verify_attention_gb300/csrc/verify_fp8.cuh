// Verify attention over the fp8 latent cache: the drafts, lengths, slot table and masks of
// mla_verify_attn over keys k_j = [s_j * code_j | rope_j] (e4m3 codes, one fp32 scale s_j a
// key), output in bf16, on the 5th-generation tensor cores (tcgen05, TMEM).
//
// Mathematics.  The codes go to the tensor cores as they are: every e4m3 value is an fp16
// value, and so is a bf16 query after its row is brought to [2^14, 2^15) by a power of two, as
// long as it is within 2^-31 of the row's largest (smaller ones lose bits below 2^-24, 2^-38 of the
// largest).  So the products code * q are exact, and a score has no error but its fp32 sum's.  With
// A = sum_d q_d code_jd and C = sum_d q_d rope_jd in two fp32 accumulators,
//     x_j  = c (s_j A + C)                              score in log2 units, c = scale log2(e) 2^e_row
//     y_j  = x_j + log2 s_j,   P_j = 2^(y_j - m)        fp16, m the running maximum of y
//     out  = sum_j P_j code_j / l,   l = sum_j P_j / s_j,   lse = (m + log2 l) ln 2
// so a key's scale enters its probability's weight, in fp32, and the value product again
// runs on the bare codes.  m is shifted by 7 so that P fills the fp16 range up to 2^15 (the
// maximum may lag by 2^8 before O is rescaled).  P's rounding is relative 2^-11, and absolute 2^-25
// below 2^-14: a key whose weight is less than 2^-32 of the row's largest may add nothing to out, while l,
// which takes P before the rounding, still counts it.  Scales below 2^-90 (rows of zeros) count as
// 2^-90 in the weight.
//
// One CTA handles up to 72 (in one form 96) query rows (r = t * H + h of one stream) over one key
// split, in tiles of 48 keys:
//   gather   eight warps read the tile's raw rows (512 code bytes, 128 rope bytes, scale) from
//            the slot table straight into registers, two tiles ahead, and widen them
//            (e4m3x2 -> f16x2, one instruction a pair) into a 128-byte-swizzled stage
//   A, C     tcgen05.mma M=128 (query rows) x N=48 (keys): K=512 in fp16, K=64 (rope) in bf16;
//            as many 64-dim chunks of Q as TMEM has columns for sit there
//   P        one thread a query row: mask, running maximum and sum, P to shared memory
//   O^T     += code^T P^T: M=128 (value dims) x N=rows x K=48 keys, four 128-dim chunks in TMEM
//
// What bounds it, with long streams: the gather's warps, 1.9 us a tile at 72 rows (time stamps a role,
// mixed batch of eight streams): 0.95 us until the loads of a tile are issued, behind those in flight,
// 0.7 for the widening and its stores, 0.25 waiting for a free stage, one after the other in each warp.
// The scores wait 0.6 us a tile for keys, the softmax works 1.05 and waits 0.8.  Neither the matrix
// operands' 1900 cycles of shared memory (128 B a cycle; 0.95 us) nor the HBM bytes, 0.7 us, are the
// period.  The mixed batch with 200 thousand keys takes 76 us a call.  A tile is 48 keys because three such
// stages fit beside Q (two of 64 keys wait for each other: 83 us; two of 48: 81 us).  Two forms that
// were measured and not kept: codes as the matrix units' fp8 operands for scores and values, without
// any widening (keys as rows of the scores, Q in two e4m3 pieces, P in three; half of the
// shared-memory traffic, but only one tile of 128 keys fits, and scores, P and values follow each
// other: 79 us, and 26 instead of 17 us at one tile a CTA, whose code is three times as long); rows
// called into L2 four tiles ahead (80 us).  Partial rows in fp16: within 2 us either way.
// With few keys: the chain of first reads (length, slots, rows), the queries' conversion, the first pass
// through the code and the epilogue's partial rows: 15.1 us a call at one tile a CTA and 72 rows.
//
// The RULES form (mla_verify_attn_fp8_rules): x goes through the cap and the bias in log2 units before log2 s_j is added
// (score_rules.cuh).  The bias's part that belongs to the row, slope x (row's position - the stream's last), is added
// to the log-sum-exp instead of to every key (up to 64 in size: half a step of such a sum is 2^-18; where it is larger the
// differences of positions are taken).  The gather leaves the positions' distances and, a warp, the
// least and greatest position and document of its six keys; from those a row knows most tiles to be seen whole or
// not at all; of others a lane looks at a key for one draft after the other.  Rules cost the softmax up to 0.6 us a tile
// (32 streams of 64 rows, nine tiles a CTA: none 39 us a call, a bias 41, a cap 47, documents of which half are
// hidden 41) and a first pass through their code.
//
// Warps (512 threads): 0 issues A and C, 1 issues O^T (whole warp, one elected lane), 4-7 Q,
// softmax and epilogue (TMEM lane quadrant = warp % 4), 8-15 gather and widening (six keys of
// a tile each).  The launch's 512 x 128 registers are shared out again per warpgroup: 72 a
// thread for warps 0-3, 168 for the softmax (a row's 48 scores in two parts), 136 for the gather
// (two tiles in flight): 128 x (72 + 168 + 2 x 136) = 65536, the launch's total.  Every mbarrier
// wait is bounded: the first to give up sets the abort flag and the status bit, and every role
// leaves.
#pragma once

#include "../../include/mla_verify.h"
#include "internal.cuh"
#include "query_rows.cuh"
#include "score_rules.cuh"
#include "tc_ptx.cuh"

#include <math.h>
#include <string.h>

#include <atomic>

namespace mla {
namespace {

using namespace tc;

constexpr int NK = 48;                               // keys per tile
constexpr int MAX_R = 96;                            // query rows per CTA: 72 beside three key stages,
constexpr int MAX_R3 = 72;                           // 96 beside two
constexpr int NT = 512;
constexpr int WIDE_WARPS = 8;
constexpr int WK = NK / WIDE_WARPS;                  // keys of a tile per gather warp
constexpr int MAX_STAGES = 3;
constexpr int NCHUNK = D_QK / 64;                    // 8 latent chunks and the rope chunk
constexpr int REGION = NK * 128;                     // one 64-dim chunk of a stage
constexpr int STAGE_BYTES = NCHUNK * REGION;         // 55296 B
constexpr uint32_t TMEM_COLS = 512;
constexpr int A_COL = 0, C_COL = NK, O_COL = 2 * NK; // TMEM columns: A, C, O^T (4 R), Q chunks
constexpr float TAU = 8.0f;                          // lazy rescale threshold (log2 units)
constexpr float P_SHIFT = 7.0f;
constexpr float MIN_SCALE = 8.0779356694631609e-28f; // 2^-90
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int MAX_SMEM = 232448;                     // opt-in shared memory per block on sm_103

enum { B_KV_FULL = 0, B_KV_EMPTY = B_KV_FULL + MAX_STAGES, B_S_FULL = B_KV_EMPTY + MAX_STAGES, B_S_FREE, B_P_FULL, B_Q_FULL,
       B_COUNT };
constexpr int BAR_BYTES = 128;
static_assert(B_COUNT * 8 + 8 <= BAR_BYTES, "barrier area");

struct Layout {
    int kv, p, misc, total;                          // the Q chunks start at 0
};
// RQ: rows of a Q chunk (whole groups of eight).  The MMA reads 128 rows a chunk: what lies
// behind the last, in the next chunk or the key stages, gives scores that nobody uses.
__host__ __device__ inline Layout layout_for(int R, int RQ, int nq_s, int stages, bool rules) {
    Layout L;
    L.kv = (nq_s * RQ * 128 + 1023) / 1024 * 1024;
    L.p = L.kv + stages * STAGE_BYTES;
    L.misc = (L.p + R * NK * 2 + 127) / 128 * 128;
    // barriers, TMEM base and abort flag; a key's scale, log2, inverse (and distance); a row's factor (and spans)
    L.total = L.misc + BAR_BYTES + MAX_STAGES * NK * (rules ? 16 : 12) + 512 + (rules ? MAX_STAGES * WIDE_WARPS * 16 : 0);
    return L;
}

struct Fp8Args {
    const __nv_bfloat16* q;
    const uint8_t* lat;
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
    __nv_bfloat16* out;           // used when nsplit == 1
    float* lse;
    float* part_out;              // layouts of VerifyArgs
    float* part_lse;
    int nsplit;
    int balanced, bal_G;
    int R, RQ, R_step;            // MMA rows (of 16), Q rows in shared memory (of 8), rows per tile
    int debug_stall;
    unsigned* status;
    unsigned long long* rescales;
    ScoreRules rules;             // (the RULES form)
};

struct Misc {
    uint64_t* bars;
    uint32_t* tmem_slot;
    volatile int* abort;
    float2* key_sl;               // [stage][NK]: scale (NaN: the key holds a NaN), log2 of the clamped scale;
                                  // the RULES form: [stage][2][NK], scales, then logarithms
    float* key_inv;               // [stage][NK]: 1 / clamped scale (finite: a masked key's P of 0 stays 0)
    float* row_f;                 // [128]: the power of two that a query row was divided by, alpha while the
                                  // loop runs, 1 / l in the epilogue (the row's own thread reads the first)
    float* key_far;               // [stage][NK], the RULES form: position less the stream's last
    int4* key_span;               // [stage][gather warp]: least and largest position, least and largest document
};
__device__ __forceinline__ Misc misc_at(uint8_t* smem, int off) {
    Misc m;
    m.bars = reinterpret_cast<uint64_t*>(smem + off);
    m.tmem_slot = reinterpret_cast<uint32_t*>(smem + off + BAR_BYTES - 8);
    m.abort = reinterpret_cast<volatile int*>(smem + off + BAR_BYTES - 4);
    m.key_sl = reinterpret_cast<float2*>(smem + off + BAR_BYTES);
    m.key_inv = reinterpret_cast<float*>(smem + off + BAR_BYTES + MAX_STAGES * NK * 8);
    m.row_f = reinterpret_cast<float*>(smem + off + BAR_BYTES + MAX_STAGES * NK * 12);
    m.key_far = m.row_f + 128;
    m.key_span = reinterpret_cast<int4*>(m.key_far + MAX_STAGES * NK);
    return m;
}

__device__ __forceinline__ void give_up(const Misc& m, unsigned* status) {
    if (atomicExch(const_cast<int*>(m.abort), 1) == 0) atomicOr(status, DEV_TIMEOUT);
}

// Those rows in fp16 (the rope chunk in bf16), each divided by row_exp, the power of two that brings
// its largest element into [2^14, 2^15): chunks below NQT to q_tmp (bound for TMEM), the others to q_s;
// rows of 128 B, 128-byte swizzle, RQ rows a chunk.
template <int N, int NQT>
__device__ __forceinline__ void store_q_rows(const uint4 (&v)[N][3], uint8_t* q_s, uint8_t* q_tmp, float* row_exp,
                                             int first, int step, int end, int RQ) {
    const int lane = threadIdx.x & 31;
    int exps[N];
    row_exponents<N>(v, exps);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int rr = first + u * step;
        const int e = exps[u];
        const float mul = __int_as_float((14 - e + 127) << 23);
        if (rr >= end) continue;
        if (lane == 0) row_exp[rr] = __int_as_float((e - 14 + 127) << 23);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const int pc = c * 32 + lane, ch = pc >> 3;
            const uint4 x = v[u][c];
            if (pc < 64) {
                const uint4 o = make_uint4(q_to_f16(x.x, mul), q_to_f16(x.y, mul), q_to_f16(x.z, mul), q_to_f16(x.w, mul));
                uint8_t* chunk = ch < NQT ? q_tmp + ch * RQ * 128 : q_s + (ch - NQT) * RQ * 128;
                *reinterpret_cast<uint4*>(chunk + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4)) = o;
            } else if (pc < 72) {
                const uint4 o = make_uint4(q_to_bf16(x.x, mul), q_to_bf16(x.y, mul), q_to_bf16(x.z, mul), q_to_bf16(x.w, mul));
                *reinterpret_cast<uint4*>(q_s + (NCHUNK - 1 - NQT) * RQ * 128 + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4)) = o;
            }
        }
    }
    fence_proxy_async_smem();                            // generic stores -> tensor-core reads
}

// NQT: latent chunks of Q in TMEM (the others, and the rope chunk, in shared memory); STAGES: key stages;
// RULES: scores under a.rules.
template <int NQT, int STAGES, bool RULES>
__global__ void __launch_bounds__(NT, 1) verify_fp8_kernel(const Fp8Args a) {
    constexpr int NQS = NCHUNK - NQT;
    extern __shared__ __align__(1024) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int R = a.R, RQ = a.RQ;
    const Layout L = layout_for(R, RQ, NQS, STAGES, RULES);
    const Misc M = misc_at(smem, L.misc);
    const uint32_t q_addr = smem_u32(smem), kv_addr = smem_u32(smem + L.kv), p_addr = smem_u32(smem + L.p);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int s = blockIdx.x, b = blockIdx.z;
    const int rows = a.q_len * a.H;
    const int row0 = blockIdx.y * a.R_step;
    const int nrows = min(a.R_step, rows - row0);
    const bool misaligned = (q_addr & 1023u) != 0;       // the swizzled layouts need a 1024-byte aligned base
    int n, k_begin = 0, k_end = 0;
    bool bad_len;
    if (a.balanced) {
        const BalancedPlan P = balanced_plan(a.seq_lens, a.B, a.q_len, a.slot_stride, a.bal_G, NK, NK,
                                             RULES ? a.rules.span() : KeySpan{});
        balanced_slot(P, blockIdx.x, &b, &s);
        if (b < 0) return;                               // slot beyond the streams' need
        n = __shfl_sync(0xffffffffu, b < 32 ? P.n[0] : P.n[1], b & 31);
        bad_len = n < a.q_len || n > a.slot_stride;
        if (!bad_len) {
            k_begin = (int)min((long long)n, (long long)s * P.chunk);
            k_end = (int)min((long long)n, (long long)(s + 1) * P.chunk);
        }
    } else {
        n = a.seq_lens[b];
        bad_len = n < a.q_len || n > a.slot_stride;
        if (RULES && !bad_len) n = a.rules.span().seen(b, n, a.q_len);
        if (!bad_len) split_range(n, a.nsplit, s, NK, &k_begin, &k_end);
    }
    // RULES: n counts the keys that some draft can see (ScoreRules::span); key v of these is key
    // v + (v >= gap_at ? gap : 0) of the stream
    int gap_at = 0, gap = 0;
    if (RULES && !bad_len) a.rules.span().gap(b, a.seq_lens[b], a.q_len, &gap_at, &gap);
    const int64_t part_row0 = a.balanced ? (int64_t)blockIdx.x * rows + row0
                                         : ((int64_t)b * rows + row0) * a.nsplit + s;
    const int64_t part_row_step = a.balanced ? 1 : a.nsplit;
    const int T = misaligned ? 0 : (k_end - k_begin + NK - 1) / NK;
    const int p = n - a.q_len;                           // first draft key
    // First key of the i-th tile.  Under a bias by distance the tiles come from the last one back: near keys
    // usually weigh most, and from the first tile on the maximum would rise with every tile, and O^T be rescaled.
    auto tile_at = [&](int i) -> int { return k_begin + (RULES && a.rules.slopes ? T - 1 - i : i) * NK; };

    // ---- set-up: barriers and TMEM
    if (warp == 0) {
        tmem_alloc(M.tmem_slot, TMEM_COLS);
        tmem_relinquish();
    } else if (tid == 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&M.bars[B_KV_FULL + i], WIDE_WARPS);
            mbar_init(&M.bars[B_KV_EMPTY + i], 1);
        }
        mbar_init(&M.bars[B_S_FULL], 1);
        mbar_init(&M.bars[B_S_FREE], 4);
        mbar_init(&M.bars[B_P_FULL], 4);
        mbar_init(&M.bars[B_Q_FULL], 4);
        *M.abort = misaligned ? 1 : 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *M.tmem_slot;
    const int q_col = O_COL + 4 * R;                     // Q chunk c < NQT: columns q_col + 32 c ..
    // The query rows' conversion: by the softmax warps, the last sixth of the rows by warps 2 and 3;
    // chunks bound for TMEM pass through the last key stage.
    const __nv_bfloat16* q0 = a.q + ((int64_t)b * rows + row0) * D_QK;
    uint8_t* const q_tmp = smem + L.kv + (STAGES - 1) * STAGE_BYTES;
    constexpr int Q_ROWS = STAGES == 3 ? MAX_R3 : MAX_R, Q_SOFT = Q_ROWS / 6 * 5, Q_THREADS = 128 + 64;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
        // ================= A and C =================
        if (T > 0) {
            const uint32_t id_a = idesc_f16(128, NK, false, false), id_c = idesc_bf16(128, NK, false, false);
            const uint64_t dq = smem_desc_sw128(q_addr, 16, 1024), dk = smem_desc_sw128(kv_addr, 16, 1024);
            const uint32_t q_region16 = (uint32_t)(RQ * 128) >> 4;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&M.bars[B_Q_FULL], 0, M.abort));
            fence_proxy_async_smem();
            int i = 0;                                   // tiles issued
            for (; i < T && ok; ++i) {
                const int st = i % STAGES;
                ok = mbar_wait(&M.bars[B_KV_FULL + st], (i / STAGES) & 1, M.abort);
                if (ok && i >= 1) ok = mbar_wait(&M.bars[B_S_FREE], (i - 1) & 1, M.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t st16 = (uint64_t)(st * STAGE_BYTES) >> 4;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D_QK / 16; ++ks) {
                        const int c = ks >> 2;
                        const uint64_t kd = dk + st16 + (uint32_t)((c * REGION + (ks & 3) * 32) >> 4);
                        if (c < NQT) {
                            mma_bf16_ta(tmem + A_COL, tmem + q_col + ks * 8, kd, id_a, ks > 0);
                        } else {
                            const uint64_t qd = dq + (uint32_t)(c - NQT) * q_region16 + (uint32_t)(ks & 3) * 2;
                            if (c < NCHUNK - 1) mma_bf16(tmem + A_COL, qd, kd, id_a, ks > 0);
                            else mma_bf16(tmem + C_COL, qd, kd, id_c, (ks & 3) > 0);
                        }
                    }
                    mma_commit(&M.bars[B_S_FULL]);
                }
                __syncwarp();
            }
            if (!ok) {
                if (lane == 0) give_up(M, a.status);
                if (i > 0) mbar_drain(&M.bars[B_S_FULL], (i - 1) & 1);
            }
        }
        __syncwarp();
        } else if (warp == 1) {
        // ================= O^T =================
        const uint32_t id_o = idesc_f16(128, R, true, false);
        // codes^T: M-major, 64-dim chunks REGION apart, 8-key groups 1024 B apart
        const uint64_t dv = smem_desc_sw128(kv_addr, REGION, 1024);
        // P: K-major, no swizzle, 8-key blocks R * 16 B apart, 8-row blocks 128 B apart
        const uint64_t dp = smem_desc(p_addr, R * 16, 128);
        bool ok = true;
        int j = 0;                                       // tiles issued
        for (; j < T && ok; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait(&M.bars[B_P_FULL], j & 1, M.abort));
            if (!ok) break;
            tc_fence_after();
            const uint64_t st16 = (uint64_t)((j % STAGES) * STAGE_BYTES) >> 4;
            if (elect_one()) {
#pragma unroll
                for (int ci = 0; ci < 4; ++ci)
#pragma unroll
                    for (int kk = 0; kk < NK / 16; ++kk)
                        mma_bf16(tmem + O_COL + ci * R, dv + st16 + (uint64_t)((2 * ci * REGION + kk * 2048) >> 4),
                                 dp + (uint64_t)((kk * 2 * R * 16) >> 4), id_o, j > 0 || kk > 0);
                mma_commit(&M.bars[B_KV_EMPTY + j % STAGES]);
            }
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0) give_up(M, a.status);
            if (j > 0) mbar_drain(&M.bars[B_KV_EMPTY + (j - 1) % STAGES], ((j - 1) / STAGES) & 1);
        }
        __syncwarp();
        } else if (T > 0) {
            for (int first = Q_SOFT + warp - 2; first < min(RQ, Q_ROWS); first += 6) {
                uint4 v[3][3];
                load_q_rows(v, q0, first, 2, nrows);
                store_q_rows<3, NQT>(v, smem, q_tmp, M.row_f, first, 2, RQ, RQ);
            }
            bar_arrive(4, Q_THREADS);
        }
    } else if (warp >= 8) {
        // ================= gather and widening: keys WK w .. WK w + 5 of every tile =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int w = warp - 8;
        bool bad_slot = false;
        const int32_t* slot_row = a.slot + (int64_t)b * a.slot_stride;
        // lane l holds the slot of key WK w + (l & 7) of tile t0 + (l >> 3), for the current group of
        // four tiles and the next; indices are checked when their group becomes current
        auto load_slots = [&](int t0) -> int {
            const int t = t0 + (lane >> 3);
            if (t >= T) return 0;
            const int v = min(tile_at(t) + WK * w + min(lane & 7, WK - 1), k_end - 1);   // past the split: a valid key
            return __ldg(slot_row + (RULES && v >= gap_at ? v + gap : v));
        };
        int cur = load_slots(0), nxt = load_slots(4);
        struct Raw {
            uint4 lat[WK], rope[2];
            float scale;
            int pos, doc;                                // RULES
        };
        const int last_pos = RULES && a.rules.key_pos && !bad_len ? __ldg(a.rules.key_pos + (int64_t)b * a.slot_stride + p + gap + a.q_len - 1)
                                                                  : p + gap + a.q_len - 1;
        auto load_tile = [&](Raw& r, int j) {
            if (j >= T) return;
            if ((j & 3) == 0) {
                if (j > 0) {
                    cur = nxt;
                    nxt = load_slots(j + 4);
                }
                if (cur < 0 || (int64_t)cur >= a.n_pool) { bad_slot = true; cur = 0; }
            }
            const int sl = __shfl_sync(0xffffffffu, cur, ((j & 3) << 3) + (lane & 7));   // key WK w + (lane & 7)
#pragma unroll
            for (int it = 0; it < WK; ++it)
                r.lat[it] = ld_stream(reinterpret_cast<const uint4*>(a.lat + (int64_t)__shfl_sync(0xffffffffu, sl, it) * D_V) + lane);
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const int f = it * 32 + lane, rs = __shfl_sync(0xffffffffu, sl, f >> 3);
                if (f < 8 * WK) r.rope[it] = ld_stream(reinterpret_cast<const uint4*>(a.rope + (int64_t)rs * 64) + (f & 7));
            }
            r.scale = __ldg(a.kscale + sl);
            if (RULES) {
                const int v = min(tile_at(j) + WK * w + min(lane & 7, WK - 1), k_end - 1);
                r.pos = v >= gap_at ? v + gap : v;
                r.doc = a.rules.key_doc ? __ldg(a.rules.key_doc + (int64_t)b * a.slot_stride + r.pos) : -1;
                if (a.rules.key_pos) r.pos = __ldg(a.rules.key_pos + (int64_t)b * a.slot_stride + r.pos);
            }
        };
        // lane l widens dims 16 l .. 16 l + 15: 16-byte pieces j0, j0 + 1 of region l / 4.  Lanes of odd
        // regions store their second piece first, so each store covers all eight 16-byte bank groups.
        const int region = lane >> 2, j0 = (lane & 3) * 2, odd = region & 1;
        auto widen_tile = [&](const Raw& r, int i) -> bool {
            const int st = i % STAGES;
            // the last stage first holds the Q chunks on their way to TMEM; the warp goes on or leaves as a whole
            if ((i >= STAGES && !mbar_wait_warp(&M.bars[B_KV_EMPTY + st], ((i - STAGES) / STAGES) & 1, M.abort)) ||
                (i == STAGES - 1 && !mbar_wait_warp(&M.bars[B_Q_FULL], 0, M.abort))) {
                if (lane == 0) give_up(M, a.status);
                return false;
            }
            uint8_t* base = smem + L.kv + st * STAGE_BYTES;
            __half2 top = __half2half2(__ushort_as_half(0));
#pragma unroll
            for (int it = 0; it < WK; ++it) {
                const int key = WK * w + it;
                const uint2 h0 = widen4(r.lat[it].x), h1 = widen4(r.lat[it].y), h2 = widen4(r.lat[it].z), h3 = widen4(r.lat[it].w);
                const uint32_t hw[8] = {h0.x, h0.y, h1.x, h1.y, h2.x, h2.y, h3.x, h3.y};
#pragma unroll
                for (int e = 0; e < 8; ++e) top = __hmax2_nan(top, *reinterpret_cast<const __half2*>(&hw[e]));
                const uint4 lo = make_uint4(hw[0], hw[1], hw[2], hw[3]), hi = make_uint4(hw[4], hw[5], hw[6], hw[7]);
                uint8_t* row = base + region * REGION + key * 128;
                *reinterpret_cast<uint4*>(row + (((j0 + odd) ^ (key & 7)) << 4)) = odd ? hi : lo;
                *reinterpret_cast<uint4*>(row + (((j0 + 1 - odd) ^ (key & 7)) << 4)) = odd ? lo : hi;
            }
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const int f = it * 32 + lane;
                const int key = WK * w + (f >> 3);
                if (f < 8 * WK) *reinterpret_cast<uint4*>(base + (NCHUNK - 1) * REGION + key * 128 + (((f & 7) ^ (key & 7)) << 4)) = r.rope[it];
            }
            // A NaN code must reach the rows that see its key and no other, but as a value it would
            // meet the zero probabilities of the others: it is stored as 0 and the key's scale
            // becomes NaN.  (Rare: the second look is taken only where a lane met one.)
            float sc = r.scale >= 0.f ? r.scale : __int_as_float(0x7fc00000);
            if (__any_sync(0xffffffffu, __hisnan(__low2half(top)) || __hisnan(__high2half(top)))) {
#pragma unroll 1
                for (int it = 0; it < WK; ++it) {
                    const int key = WK * w + it;
                    uint32_t* row = reinterpret_cast<uint32_t*>(base + region * REGION + key * 128);
                    bool found = false;
                    for (int e = 0; e < 8; ++e) {
                        uint32_t* at = row + ((((j0 + (e >> 2)) ^ (key & 7)) << 2) + (e & 3));
                        const uint32_t v = *at;
                        const bool n0 = (v & 0x7c00u) == 0x7c00u, n1 = (v & 0x7c000000u) == 0x7c000000u;
                        if (n0 || n1) {
                            found = true;
                            *at = (n0 ? 0u : v & 0xffffu) | (n1 ? 0u : v & 0xffff0000u);
                        }
                    }
                    if (__any_sync(0xffffffffu, found) && (lane & 7) == it) sc = __int_as_float(0x7fc00000);
                }
            }
            if (lane < WK) {
                const float cl = fmaxf(sc, MIN_SCALE);
                if (RULES) {
                    float* sl = reinterpret_cast<float*>(M.key_sl + st * NK);
                    sl[WK * w + lane] = sc;
                    sl[NK + WK * w + lane] = log2f(cl);
                    M.key_far[st * NK + WK * w + lane] = (float)((long long)r.pos - last_pos);
                } else {
                    M.key_sl[st * NK + WK * w + lane] = make_float2(sc, log2f(cl));
                }
                M.key_inv[st * NK + WK * w + lane] = 1.f / cl;
            }
            if (RULES && a.rules.spans) {                // (every lane holds one of the warp's keys)
                const int4 span = make_int4(__reduce_min_sync(0xffffffffu, r.pos), __reduce_max_sync(0xffffffffu, r.pos),
                                            __reduce_min_sync(0xffffffffu, r.doc), __reduce_max_sync(0xffffffffu, r.doc));
                if (lane == 0) M.key_span[st * WIDE_WARPS + w] = span;
            }
            fence_proxy_async_smem();                    // generic stores -> tensor-core reads
            __syncwarp();
            if (lane == 0 && !(a.debug_stall && i == 0)) mbar_arrive(&M.bars[B_KV_FULL + st]);
            return true;
        };
        Raw r0, r1;
        // (The votes on what every lane knows keep the warp together behind lane 0's arrival: without them
        // 70.2 instead of 68.8 us on the mixed batch.)
        load_tile(r0, 0);
        load_tile(r1, 1);
        for (int i = 0; i < T; i += 2) {
            if (!__all_sync(0xffffffffu, widen_tile(r0, i))) break;
            load_tile(r0, i + 2);
            if (i + 1 >= T) break;
            if (!__all_sync(0xffffffffu, widen_tile(r1, i + 1))) break;
            load_tile(r1, i + 3);
        }
        if (bad_slot) atomicOr(a.status, DEV_BAD_SLOT);
    } else {
        // ================= Q, softmax, epilogue =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int quad = warp & 3;                       // TMEM lane quadrant of this warp
        const int r = quad * 32 + lane;                  // query row of this thread (lane of A and C)
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const bool row_ok = r < nrows;
        if (T > 0) {
            constexpr int QB = 8;
            for (int first = quad; first < min(RQ, Q_SOFT); first += 4 * QB) {
                uint4 v[QB][3];
                load_q_rows(v, q0, first, 4, min(nrows, Q_SOFT));
                store_q_rows<QB, NQT>(v, smem, q_tmp, M.row_f, first, 4, min(RQ, Q_SOFT), RQ);
            }
            bar_sync(4, Q_THREADS);
            // a thread a row: the TMEM chunks
            if (quad * 32 < RQ) {
#pragma unroll 1
                for (int c = 0; c < NQT; ++c) {
                    uint32_t h[32];
                    const uint8_t* src = q_tmp + c * RQ * 128 + min(r, RQ - 1) * 128;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + ((j ^ (r & 7)) << 4));
                        h[4 * j] = v.x; h[4 * j + 1] = v.y; h[4 * j + 2] = v.z; h[4 * j + 3] = v.w;
                    }
                    tmem_st32(tmem + lane_base + q_col + c * 32, h);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.bars[B_Q_FULL]);
        }
        const int t = row_ok ? (row0 + r) / a.H : 0;
        // drafts this row sees, bit i = draft i (q_len <= 64)
        uint64_t vis = 0;
        if (row_ok) {
            if (a.mask_bits) {
                vis = a.mask_bits[(int64_t)b * a.q_len + t];
            } else if (a.mask) {
                for (int d = 0; d < a.q_len; ++d)
                    vis |= (uint64_t)(a.mask[((int64_t)b * a.q_len + t) * a.q_len + d] != 0 ? 1u : 0u) << d;
            } else {
                vis = t >= 63 ? ~0ull : (2ull << t) - 1;
            }
        }
        const float c2 = T > 0 && row_ok ? a.scale * LOG2E * M.row_f[r] : 0.f;
        const int plain_end = min(p, k_end);             // keys below this need no mask (of drafts)
        RowRule rule;
        if (RULES) rule = a.rules.row(b, t, row_ok ? (row0 + r) % a.H : 0, p + gap, a.slot_stride, bad_len);
        const float in = RULES && a.rules.softcap > 0.f ? cap_in(c2, a.rules.softcap) : 0.f;
        const float capped = RULES && a.rules.softcap > 0.f ? cap_out(c2, a.rules.softcap, in) : 0.f;
        // The bias is slope (key's distance from the stream's last position - the row's): the second part, the same
        // for all of the row's keys, waits for the log-sum-exp.  Where it is large (bits would be lost beside it), or
        // the distances are no fp32 numbers, the warp takes the differences of positions instead.
        float bias0 = 0.f;
        bool far = false;
        if (RULES && a.rules.slopes && !bad_len) {
            const int64_t last_at = (int64_t)b * a.slot_stride + p + gap + a.q_len - 1;
            const long long off = (long long)rule.pos - (a.rules.key_pos ? __ldg(a.rules.key_pos + last_at) : p + gap + a.q_len - 1);
            far = __any_sync(0xffffffffu, off > (1 << 24) || off < -(1 << 24) || !(fabsf((float)off * rule.slope) <= 64.f));
            if (!far) bias0 = -(float)off * rule.slope;
        }
        const bool rows_used = quad * 32 < R;
        // position and document of visible key v (behind the split: of its last)
        auto key_index = [&](int v) -> int64_t {
            v = min(v, k_end - 1);
            return (int64_t)b * a.slot_stride + (v >= gap_at ? v + gap : v);
        };
        auto key_pos = [&](int v) -> int {
            return a.rules.key_pos ? __ldg(a.rules.key_pos + key_index(v)) : (v >= gap_at ? v + gap : v);
        };
        auto key_doc = [&](int v) -> int { return a.rules.key_doc ? __ldg(a.rules.key_doc + key_index(v)) : -1; };
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < T; ++i) {
            const int st = i % STAGES;
            ok = mbar_wait(&M.bars[B_KV_FULL + st], (i / STAGES) & 1, M.abort);     // the keys' scales
            ok = ok && mbar_wait(&M.bars[B_S_FULL], i & 1, M.abort);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            float x[NK];
            float mt = -INFINITY;
            const int k0 = tile_at(i);
            const float2* sl = M.key_sl + st * NK;
            const float* inv = M.key_inv + st * NK;
            if (ok && !rows_used) {                      // no row of this warp is in the tile
                __syncwarp();
                if (lane == 0) mbar_arrive(&M.bars[B_S_FREE]);
            } else if (ok) {
                uint32_t va[NK / 16][16], vc[NK / 16][16];
#pragma unroll
                for (int h = 0; h < NK / 16; ++h) {
                    tmem_ld16(tmem + lane_base + A_COL + 16 * h, va[h]);
                    tmem_ld16(tmem + lane_base + C_COL + 16 * h, vc[h]);
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&M.bars[B_S_FREE]);
                if constexpr (!RULES) {
#pragma unroll
                for (int k = 0; k < NK; k += 2) {
                    const float4 c = *reinterpret_cast<const float4*>(sl + k);
                    x[k] = fmaf(fmaf(__uint_as_float(va[k / 16][k % 16]), c.x, __uint_as_float(vc[k / 16][k % 16])), c2, c.y);
                    x[k + 1] = fmaf(fmaf(__uint_as_float(va[k / 16][k % 16 + 1]), c.z, __uint_as_float(vc[k / 16][k % 16 + 1])), c2, c.w);
                }
                } else {
                    // (four keys a read of shared memory: its queue is the gather's too)
                    const float4* ks = reinterpret_cast<const float4*>(sl);
                    const float4* kl = ks + NK / 4;
                    const bool cap = a.rules.softcap > 0.f;
                    auto pair = [&](int k) { return make_float2(x[k], x[k + 1]); };
                    auto put = [&](int k, float2 y) { x[k] = y.x; x[k + 1] = y.y; };
                    auto accs = [](const uint32_t (&v)[NK / 16][16], int k) {
                        return make_float2(__uint_as_float(v[k / 16][k % 16]), __uint_as_float(v[k / 16][k % 16 + 1]));
                    };
#pragma unroll
                    for (int k = 0; k < NK; k += 4) {
                        const float4 c = ks[k / 4];
                        put(k, fma2(accs(va, k), make_float2(c.x, c.y), accs(vc, k)));
                        put(k + 2, fma2(accs(va, k + 2), make_float2(c.z, c.w), accs(vc, k + 2)));
                    }
                    float gain = c2;
                    if (cap) {
                        float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < NK; k += 2) {
                            put(k, mul2(pair(k), both(in)));
                            top[k & 2] = fmaxf(top[k & 2], fabsf(x[k]));
                            top[(k & 2) + 1] = fmaxf(top[(k & 2) + 1], fabsf(x[k + 1]));
                        }
                        // scores within the cap, as nearly all are, take the polynomial alone
                        if (__all_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= 1.f)) {
#pragma unroll
                            for (int k = 0; k < NK; k += 2) put(k, tanh_near(pair(k)));
                        } else {
#pragma unroll
                            for (int k = 0; k < NK; k += 2) put(k, tanh2(pair(k)));
                        }
                        gain = capped;
                    }
#pragma unroll
                    for (int k = 0; k < NK; k += 4) {
                        const float4 c = kl[k / 4];
                        put(k, fma2(pair(k), both(gain), make_float2(c.x, c.y)));
                        put(k + 2, fma2(pair(k + 2), both(gain), make_float2(c.z, c.w)));
                    }
                    if (a.rules.slopes) {
                        if (!far) {
                            const float4* kf = reinterpret_cast<const float4*>(M.key_far + st * NK);
#pragma unroll
                            for (int k = 0; k < NK; k += 4) {
                                const float4 c = kf[k / 4];
                                put(k, fma2(make_float2(c.x, c.y), both(rule.slope), pair(k)));
                                put(k + 2, fma2(make_float2(c.z, c.w), both(rule.slope), pair(k + 2)));
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < NK; ++k)
                                x[k] = fmaf((float)(key_pos(k0 + k) - rule.pos), rule.slope, x[k]);
                        }
                    }
                    // bit k: the row sees key k0 + k
                    uint64_t see = ~0ull;
                    if (k0 + NK > plain_end) {
                        const int before = p - k0;       // keys of the tile before the drafts
                        if (before < 64) see = before > 0 ? vis << before | ((1ull << before) - 1) : before > -64 ? vis >> -before : 0;
                    }
                    if (a.rules.masked) {
                        // the tile's keys as a whole, and each of them only where that does not decide
                        int4 span;
                        if (a.rules.spans) {
                            const int4 part = M.key_span[st * WIDE_WARPS + (lane & (WIDE_WARPS - 1))];
                            span = make_int4(__reduce_min_sync(0xffffffffu, part.x), __reduce_max_sync(0xffffffffu, part.y),
                                             __reduce_min_sync(0xffffffffu, part.z), __reduce_max_sync(0xffffffffu, part.w));
                        } else {
                            const int z = min(k0 + NK, k_end) - 1;
                            span = make_int4(k0 >= gap_at ? k0 + gap : k0, z >= gap_at ? z + gap : z, -1, -1);
                        }
                        const bool none = rule.none(span);
                        // (drafts in the prefix are seen whatever their mask says)
                        if (__all_sync(0xffffffffu, none || (rule.all(span) && (k0 + NK <= p || span.x >= rule.prefix)))) {
                            if (none) see = 0;
                        } else {
                            see = 0;
                            // lane l looks at keys l and 32 + (l & 15), for one draft of the warp's rows after the other
                            const int v0 = k0 + lane, v1 = k0 + 32 + (lane & 15);
                            const int pos0 = key_pos(v0), pos1 = key_pos(v1), doc0 = key_doc(v0), doc1 = key_doc(v1);
                            unsigned todo = __ballot_sync(0xffffffffu, row_ok);
#pragma unroll 1
                            while (todo) {
                                const int lead = __ffs(todo) - 1;
                                RowRule one;
                                one.lo = __shfl_sync(0xffffffffu, rule.lo, lead);
                                one.prefix = __shfl_sync(0xffffffffu, rule.prefix, lead);
                                one.doc = __shfl_sync(0xffffffffu, rule.doc, lead);
                                const uint64_t drafts = __shfl_sync(0xffffffffu, vis, lead);
                                const int j0 = v0 - p, j1 = v1 - p;   // draft indices, < 0: before the drafts
                                const uint64_t lower = __ballot_sync(0xffffffffu, one.sees(j0 < 0 || ((drafts >> (j0 & 63)) & 1ull), pos0, doc0));
                                const uint64_t upper = __ballot_sync(0xffffffffu, one.sees(j1 < 0 || ((drafts >> (j1 & 63)) & 1ull), pos1, doc1));
                                const int its = __shfl_sync(0xffffffffu, t, lead);   // (by every lane: not behind row_ok)
                                const bool mine = row_ok && t == its;
                                if (mine) see = lower | (upper & 0xffffull) << 32;
                                todo &= ~__ballot_sync(0xffffffffu, mine);
                            }
                        }
                    }
                    if (k0 + NK > k_end) see &= (1ull << (k_end - k0)) - 1;
                    if (__any_sync(0xffffffffu, (see & ((1ull << NK) - 1)) != (1ull << NK) - 1)) {
#pragma unroll
                        for (int k = 0; k < NK; ++k)
                            if (!((see >> k) & 1ull)) x[k] = -INFINITY;
                    }
                }
                // rows past the tile need no mask of their own: nothing reads their P
                if (!RULES && k0 + NK > plain_end) {
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        const int j = k0 + k;
                        if (!(j < k_end && (j < p || ((vis >> (j - p)) & 1ull)))) x[k] = -INFINITY;
                    }
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int k = 4; k < NK; ++k) mx[k & 3] = fmaxf(mx[k & 3], x[k]);
                mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            }
            const bool need = ok && row_ok && mt > m + TAU;
            float alpha = 1.f;
            if (need) {
                alpha = ex2(m - mt);
                l *= alpha;
                m = mt;
            }
            uint32_t pk[NK / 2];
            if (ok && rows_used) {
                const float mu = m == -INFINITY ? 0.f : m - P_SHIFT;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int k = 0; k < NK; k += 4) {
                    const float4 iv = *reinterpret_cast<const float4*>(inv + k);
                    const float p0 = ex2(x[k] - mu), p1 = ex2(x[k + 1] - mu), p2 = ex2(x[k + 2] - mu), p3 = ex2(x[k + 3] - mu);
                    l0 = fmaf(p0, iv.x, l0);             // the sum keeps fp32 probabilities
                    l1 = fmaf(p1, iv.y, l1);
                    l0 = fmaf(p2, iv.z, l0);
                    l1 = fmaf(p3, iv.w, l1);
                    const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
                    pk[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                    pk[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                }
                l += l0 + l1;
            }
            // P's buffer and O^T are free once O^T of the tile before is done
            if (ok && i >= 1) ok = mbar_wait(&M.bars[B_KV_EMPTY + (i - 1) % STAGES], ((i - 1) / STAGES) & 1, M.abort);
            if (bar_red_or(1, 128, need || !ok)) {
                if (bar_red_or(1, 128, !ok)) { ok = false; break; }
                if (i >= 1) {
                    // O^T column r (query row r) *= alpha_r; thread = TMEM lane = value dim
                    if (r == 0) atomicAdd(a.rescales, 1ull);
                    M.row_f[r] = alpha;
                    bar_sync(2, 128);
                    tc_fence_after();
                    for (int ci = 0; ci < 4; ++ci)
                        for (int c0 = 0; c0 < R; c0 += 16) {
                            uint32_t v[16];
                            const uint32_t ta = tmem + lane_base + O_COL + ci * R + c0;
                            tmem_ld16(ta, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj) v[jj] = __float_as_uint(__uint_as_float(v[jj]) * M.row_f[c0 + jj]);
                            tmem_st16(ta, v);
                        }
                    tmem_st_wait();
                }
            }
            if (r < R) {
                // P (B operand, K-major, no swizzle): keys 8 kb .. 8 kb + 7 of row r at kb * (R * 16) + r * 16
#pragma unroll
                for (int kb = 0; kb < NK / 8; ++kb)
                    *reinterpret_cast<uint4*>(smem + L.p + kb * (R * 16) + r * 16) =
                        make_uint4(pk[4 * kb], pk[4 * kb + 1], pk[4 * kb + 2], pk[4 * kb + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.bars[B_P_FULL]);
        }
        if (ok && T > 0) ok = mbar_wait(&M.bars[B_KV_EMPTY + (T - 1) % STAGES], ((T - 1) / STAGES) & 1, M.abort);
        const bool failed = bar_red_or(1, 128, !ok);
        if (failed) give_up(M, a.status);
        tc_fence_after();

        float rinv, lse_v;
        if (bad_len) { rinv = 0.f; lse_v = __int_as_float(0x7fc00000); }
        else if (l != 0.f) { rinv = 1.f / l; lse_v = (m - P_SHIFT + log2f(l) + (RULES ? bias0 : 0.f)) * LN2; }   // NaN stays NaN
        else { rinv = 0.f; lse_v = -INFINITY; }
        M.row_f[r] = rinv;
        const int64_t grow0 = (int64_t)b * rows + row0;
        const bool direct = !a.balanced && a.nsplit == 1;
        if (row_ok) {
            if (direct) a.lse[grow0 + r] = lse_v;
            else a.part_lse[part_row0 + r * part_row_step] = lse_v;
        }
        bar_sync(2, 128);
        // O^T -> rows: thread = TMEM lane = value dim; the four 128-dim chunks of a group of 16 rows
        // are loaded from TMEM together
        const bool have_o = T > 0 && !failed;
        for (int c0 = 0; c0 < nrows; c0 += 16) {
            uint32_t v[4][16];
            if (have_o) {
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_ld16(tmem + lane_base + O_COL + e * R + c0, v[e]);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int jj = 0; jj < 16; ++jj) v[e][jj] = 0u;
            }
#pragma unroll
            for (int jj = 0; jj < 16; ++jj) {
                const int rr = c0 + jj;
                if (rr >= nrows) break;
                const float ri = M.row_f[rr];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float o = have_o ? __uint_as_float(v[e][jj]) * ri : 0.f;
                    const int d = e * 128 + quad * 32 + lane;
                    if (direct) a.out[(grow0 + rr) * D_V + d] = __float2bfloat16_rn(o);
                    else a.part_out[(part_row0 + rr * part_row_step) * D_V + d] = o;
                }
            }
        }
    }

    // ---- teardown; the combine launched after this kernel may now be scheduled
    tc_fence_before();
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 32) {
        if (bad_len) atomicOr(a.status, DEV_BAD_LEN);
        if (misaligned) atomicOr(a.status, DEV_TIMEOUT);
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int NQT, int STAGES, bool RULES>
cudaError_t launch_one(const Fp8Args& a, dim3 grid, int dev, cudaStream_t stream) {
    auto* k = verify_fp8_kernel<NQT, STAGES, RULES>;
    const int smem = layout_for(a.R, a.RQ, NCHUNK - NQT, STAGES, RULES).total;
    if (a.RQ > (STAGES == 3 ? MAX_R3 : MAX_R) || smem > MAX_SMEM || O_COL + 4 * a.R + 32 * NQT > (int)TMEM_COLS ||
        NQT * a.RQ * 128 > STAGE_BYTES)                  // (the TMEM chunks' way station)
        return cudaErrorInvalidConfiguration;
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
        // the warpgroups' shares have to be in the launch's registers, or their request would wait for ever
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, k);
        if (e != cudaSuccess) return e;
        if (at.numRegs * NT < 128 * (72 + 168 + 2 * 136)) return cudaErrorInvalidConfiguration;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(k, grid, dim3(NT), (size_t)smem, stream, a);
}

// Row tiles of a stream: of up to 72 rows beside three key stages; 73 to 96 rows are one tile beside
// two (measured, sixteen streams of 80 rows and 3000 keys: 41.1 us, as two tiles of 40 rows 49.4).  With
// more rows the fewer and larger tiles cost as much as they save (one stream of 576 rows and 4105 keys: six
// tiles of 96 rows 26.8 us, eight of 72 25.6).
void fp8_tiling(int rows, int* n_tiles, int* R_step, int* R) {
    tc_tiling(rows, MAX_R, n_tiles, R_step, R);
    int n3, step3, r3;
    tc_tiling(rows, MAX_R3, &n3, &step3, &r3);
    if (n3 < 2 * *n_tiles) { *n_tiles = n3; *R_step = step3; *R = r3; }
}

// The automatic split count of a uniform call: the least of
//     waves of CTAs x (start and epilogue of a CTA + its tiles) + the merge
// over the counts from one to a tile a split, the longest stream's keys in whole tiles.  The times (ns)
// are measured: a CTA of 16 rows starts and ends in 6 us and takes 1.6 us a tile, one of 72 rows 10 and
// 1.8; the merge 3 us.  (One stream of 72 rows: 265 keys, six splits of a tile 15.0 us, three of two
// 16.6, one of six 20.2; 64 streams of 128 rows and 2000 keys: one split 95 us, two 120.)
int fp8_auto_nsplit(int B, int n_tiles, int R, int max_seq, int num_sms) {
    const long long fixed = 5000 + 70 * R, tile = 1500 + 5 * R, merge = 3000;
    const long long tiles = ((long long)max_seq + NK - 1) / NK;
    const long long most = min(min(tiles, (long long)MLA_MAX_NSPLIT), 8ll * num_sms / ((long long)B * n_tiles) + 1);
    long long best = 1, best_cost = 0;
    for (long long want = 1; want <= most; ++want) {
        const long long per_cta = (tiles + want - 1) / want, ns = (tiles + per_cta - 1) / per_cta;   // none empty
        const long long waves = ((long long)B * n_tiles * ns + num_sms - 1) / num_sms;
        const long long cost = waves * (fixed + per_cta * tile) + (ns > 1 ? merge : 0);
        if (want == 1 || cost < best_cost) { best = ns; best_cost = cost; }
    }
    return (int)best;
}

// Split slots of the balanced split of B streams (0: not taken).
int fp8_balanced_slots(int B, int n_tiles, int num_sms) {
    const int slots = num_sms / n_tiles;
    return B >= 2 && B <= BALANCED_MAX_STREAMS && slots - B >= B ? slots : 0;
}

// As many Q chunks in TMEM as fit beside the scores and O^T: 1 at 96 MMA rows, 3 at 80, 5 up to 64, 7 up to 48.
template <bool RULES>
cudaError_t launch_verify_fp8(const Fp8Args& a, int n_tiles, int dev, cudaStream_t stream) {
    const dim3 grid(a.nsplit, n_tiles, a.balanced ? 1 : a.B);
    if (a.R <= 48) return launch_one<7, 3, RULES>(a, grid, dev, stream);
    if (a.R <= 64) return launch_one<5, 3, RULES>(a, grid, dev, stream);
    if (a.RQ <= MAX_R3) return launch_one<3, 3, RULES>(a, grid, dev, stream);
    if (a.R <= 80) return launch_one<3, 2, RULES>(a, grid, dev, stream);
    return launch_one<1, 2, RULES>(a, grid, dev, stream);
}

// Looking for keys that no draft sees costs 5 us, a tile 1.7: worth it where half of six tiles a CTA go.  (Measured,
// documents, without and with: 32 streams of 2047 keys x 64 rows, nine tiles a CTA, all keys seen 45.4 and 50.7 us, half
// 47.8 and 37.6, a tenth 45.2 and 31.6; 8 streams of 46000 keys x 72 rows 148 and 153, 149 and 92, 149 and 38.)
constexpr int GAP_TILES = 6;

// The checks and launches of a call.
template <bool RULES>
int verify_fp8_call(const void* q, const uint8_t* kv_lat, const float* kv_scale, const void* kv_rope, int64_t n_pool,
                    const int32_t* slot_table, int slot_stride, const int32_t* seq_lens, const uint8_t* draft_mask,
                    const uint64_t* draft_mask_bits, int B, int q_len, int H, float scale, const ScoreRules& rules,
                    void* out, float* lse, int nsplit, void* workspace, size_t ws_bytes, mla_stream_t stream) {
    if (B < 0 || B > 65535 || q_len < 1 || q_len > MLA_MAX_Q_LEN || H < 1 || H > MLA_MAX_HEADS) return MLA_ERR_SHAPE;
    if (nsplit < 0 || nsplit > MLA_MAX_NSPLIT) return MLA_ERR_NSPLIT;
    if (B == 0) return MLA_OK;
    if (!q || !kv_lat || !kv_scale || !kv_rope || !slot_table || !seq_lens || !out || !lse) return MLA_ERR_NULL;
    // (key positions are 32-bit, up to a tile and a split count past the last)
    if (n_pool < 1 || n_pool > 0x7fffffffLL || slot_stride < q_len || slot_stride > MLA_MAX_FP8_KEYS) return MLA_ERR_SHAPE;
    if ((long long)B * q_len * H > 0x7fffffffLL) return MLA_ERR_SHAPE;
    if (!isfinite(scale) || (draft_mask && draft_mask_bits)) return MLA_ERR_ARG;
    if (!aligned(q, 16) || !aligned(kv_lat, 16) || !aligned(kv_rope, 16) || !aligned(kv_scale, 4) ||
        !aligned(slot_table, 4) || !aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(draft_mask_bits, 8))
        return MLA_ERR_ALIGN;
    Fp8Args a{};
    int num_sms = 0, dev = 0;
    int rc = device_state(&dev, &a.status, &num_sms, &a.rescales);
    if (rc != MLA_OK) return rc;
    int n_tiles;
    fp8_tiling(q_len * H, &n_tiles, &a.R_step, &a.R);
    a.RQ = (a.R_step + 7) / 8 * 8;
    const long long per_stream = (long long)q_len * H, rows = B * per_stream;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.lat = kv_lat; a.kscale = kv_scale; a.rope = static_cast<const __nv_bfloat16*>(kv_rope);
    a.n_pool = n_pool; a.slot = slot_table; a.slot_stride = slot_stride; a.seq_lens = seq_lens;
    a.mask = draft_mask; a.mask_bits = draft_mask_bits;
    a.B = B; a.q_len = q_len; a.H = H; a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out); a.lse = lse;
    a.rules = rules;
    a.debug_stall = take_debug_stall() ? 1 : 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // Looks for the keys that no draft sees, where the workspace has room for the answer behind `used` bytes and
    // the CTAs have GAP_TILES tiles or more to gain from.
    auto look_for_gaps = [&](size_t used, int splits) -> bool {
        if (!RULES || !has_gaps(rules)) return true;
        used = align256(used);
        if (!workspace || !aligned(workspace, 8) || used + (size_t)B * sizeof(int2) > ws_bytes) return true;
        const long long tiles = ((long long)slot_stride + NK - 1) / NK * (a.balanced ? B : 1);
        if (tiles < (long long)GAP_TILES * splits) return true;
        int2* const gaps = reinterpret_cast<int2*>(static_cast<char*>(workspace) + used);
        a.rules.gaps = gaps;
        return launch_key_gaps(rules, seq_lens, B, q_len, slot_stride, gaps, st) == cudaSuccess;
    };
    const int slots = nsplit == 0 && workspace && aligned(workspace, 256) ? fp8_balanced_slots(B, n_tiles, num_sms) : 0;
    if (slots) {
        // streams of unequal length: all their keys in equal chunks over one wave of CTAs
        const size_t out_b = align256((size_t)slots * per_stream * D_V * 4);
        if (out_b + align256((size_t)slots * per_stream * 4) <= ws_bytes) {
            a.balanced = 1;
            a.bal_G = slots - B;
            a.nsplit = slots;
            a.part_out = static_cast<float*>(workspace);
            a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + out_b);
            if (!look_for_gaps(out_b + (size_t)slots * per_stream * 4, slots)) return MLA_ERR_LAUNCH;
            if (launch_verify_fp8<RULES>(a, n_tiles, dev, st) != cudaSuccess) return MLA_ERR_LAUNCH;
            VerifyArgs c;                              // what the combine reads of a split call
            memset(&c, 0, sizeof c);
            c.seq_lens = seq_lens; c.B = B; c.q_len = q_len; c.H = H; c.slot_stride = slot_stride;
            c.nsplit = a.nsplit; c.bal_G = a.bal_G; c.part_out = a.part_out; c.part_lse = a.part_lse; c.lse = lse;
            if (launch_combine_balanced_bf16(c, a.out, NK, RULES ? a.rules.span() : KeySpan{}, st) != cudaSuccess) return MLA_ERR_LAUNCH;
            return MLA_OK;
        }
    }
    int ns = nsplit;
    if (ns == 0) {
        ns = fp8_auto_nsplit(B, n_tiles, a.R, RULES ? rules.span().most(slot_stride, q_len) : slot_stride, num_sms);
        while (ns > 1 && mla_verify_workspace_bytes(B, q_len, H, ns) > (workspace ? ws_bytes : 0)) --ns;
    }
    a.nsplit = ns;
    if (ns > 1) {
        if (!workspace || ws_bytes < mla_verify_workspace_bytes(B, q_len, H, ns)) return MLA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return MLA_ERR_ALIGN;
        a.part_out = static_cast<float*>(workspace);
        a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)rows * ns * D_V * 4));
    }
    if (!look_for_gaps(ns > 1 ? mla_verify_workspace_bytes(B, q_len, H, ns) : 0, ns)) return MLA_ERR_LAUNCH;
    if (launch_verify_fp8<RULES>(a, n_tiles, dev, st) != cudaSuccess) return MLA_ERR_LAUNCH;
    if (ns > 1 && launch_combine_bf16(a.part_out, a.part_lse, rows, ns, a.out, lse, st) != cudaSuccess)
        return MLA_ERR_LAUNCH;
    return MLA_OK;
}

}  // namespace
}  // namespace mla
