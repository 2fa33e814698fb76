// The weight that each cached key got from the rows of a step (mla_key_weights, mla_key_weights_fp8):
//     new_j = sum over rows r = (t, h) that count and see key j of exp(z_rj - lse_r)
//     out_j = decay * weights_j + new_j
// The attention's log-sum-exp is given, so there is no softmax to run: every (row, key) pair stands for
// itself, and a key's sum needs nothing of another key.
//
// Scores over the fp8 cache.  The codes are operands of the 8-bit matrix products as they lie in the cache,
// nothing is widened.  A bf16 query, its row brought to [2^7, 2^8) by a power of two, goes in two e4m3 pieces:
// h, its first four bits, and l = 2^4 (q - h), the other four.  That is exact down to 2^-13 of the row's
// largest element, and within 2^-20 of the largest below.  With the pieces' sums over the latent dims H and
// L and the rotated part's C in three fp32 accumulators,
//     z_j = scale 2^e (s_j (H + 2^-4 L) + C)
// so neither keys nor scales are rounded.  (Measured on the products: 512 terms are summed to 2^-25 of the
// sum of their magnitudes, as with fp16 operands.)  The bf16 cache takes three sums over 192 dims: a long chain of
// products into one accumulator loses more, 1.3e-6 of the weights instead of 4e-7 (16 streams of 86 keys, 24 rows).
//
// One CTA handles up to 128 query rows of one stream over one range of its keys, in tiles of 32 keys, on
// the 5th-generation tensor cores: all of Q sits in TMEM (288 columns), the scores of two tiles beside it.
//   gather   four warps, eight keys of a tile each: 16-byte cp.async from the slot table's rows into
//            128-byte-swizzled stages, ten of them (fp8; 200 KB under way) or six (bf16)
//   scores   tcgen05.mma M=128 (query rows) x N=32 (keys), Q from TMEM
//   weights  sixteen warps, a thread a query row and 16 keys, in two sets that take tiles in turn:
//            exp2(c z - lse), then the sum over a warp's 32 rows by halving exchanges (16 keys in 16
//            shuffles), the four warps' sums in shared memory.  Up to 64 rows stand in TMEM twice, and
//            a thread takes 8 keys: a warp reaches one quadrant of the lanes only, the one of its own
//            scheduler, and two of the four schedulers would have nothing to do
//
// What bounds it.  Eight streams of 9 x 8 rows, 190 thousand keys: 31.5 us captured, the gather: scattered rows of 512
// bytes come from HBM at 4.3 TB/s at most, with cp.async from 1 to 16 warps as with bulk copies of a row (through
// registers 3.4; from L2 8.7, 8.1 and 6.5).  The bf16 cache, 32 streams of 64 rows, 108 MB: 24.3 us, 4.5 TB/s.  64 x 64 rows
// over 4160 keys: 31.6 us, 6 of them the queries' conversion of a CTA, the rest 33 tiles between products (0.4 us a
// tile) and score warps.  One tile: 8.3 us.  Forms that were measured and not kept: keys as rows of the products (M = 128
// keys, Q as the other operand, from shared memory) 33.6, 37.8 (bf16) and 48 us; rows by gathering tensor copies, 69
// cycles for 128 bytes of four rows; eight score warps 42 us on the first; codes widened to bf16, tiles of 48 keys, the first
// form here, 50.6.
//
// Masks are decided for a warp's keys as a whole from their least and greatest position and document, key by
// key only where that does not do (8 streams of 46000 keys, documents: 70 us, key by key throughout 95).
//
// More than 128 rows: a row tile a CTA, whose sums meet in the workspace (4 bytes a key and row tile; a
// second small kernel adds them in order).  Sums have a fixed order: equal calls give equal bits.
#include "../../include/mla_verify.h"
#include "internal.cuh"
#include "query_rows.cuh"
#include "score_rules.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

#include <math.h>

#include <atomic>

namespace mla {
namespace {

using namespace tc;

constexpr float LOG2E = 1.4426950408889634f;
constexpr int NK = 32;                               // keys per tile
constexpr int MAX_R = 128;                           // query rows per CTA
constexpr int NT = 768;
constexpr int SCORE_WARPS = 16, MMA_WARP = 16, GATHER0 = 20, GATHER_WARPS = 4;   // (18 and 19 only bring Q)
constexpr int WK = NK / GATHER_WARPS;                // keys of a tile per gather warp
constexpr int MAX_STAGES = 10;
// What belongs to a key outlives its stage: a set reads it after it has freed the scores for the tile after
// next, whose products let the gather go on to the tile a ring further.
constexpr int RING = MAX_STAGES + 4;
constexpr int REGION = NK * 128;                     // one 128-byte chunk of a stage's rows
constexpr int Q_CHUNKS = 9;
constexpr uint32_t TMEM_COLS = 512;
constexpr int D_COL = Q_CHUNKS * 32, D_STEP = 3 * NK;  // scores of tile i at D_COL + (i & 1) D_STEP: H, L, C
static_assert(D_COL + 2 * D_STEP <= (int)TMEM_COLS, "TMEM");

// A stage: fp8 four chunks of 128 codes and one of the rotated part, bf16 nine of 64 dims.
template <bool FP8>
struct Shape {
    static constexpr int CHUNKS = FP8 ? 5 : 9, STAGES = FP8 ? MAX_STAGES : 6, STAGE_BYTES = CHUNKS * REGION;
    // Q on its way to TMEM lies in the stages from this one on, in chunks of whole groups of eight rows
    static __device__ __forceinline__ int q_stage(int nrows) {
        return STAGES - (Q_CHUNKS * ((nrows + 7) / 8) * 1024 + STAGE_BYTES - 1) / STAGE_BYTES;
    }
    static_assert(STAGES % 2 == 0, "two warps take them in turn");
    static_assert(Q_CHUNKS * MAX_R * 128 <= (STAGES - 2) * STAGE_BYTES, "Q's way station");
};

enum { B_KV_FULL = 0, B_KV_EMPTY = B_KV_FULL + MAX_STAGES, B_S_FULL = B_KV_EMPTY + MAX_STAGES, B_S_FREE = B_S_FULL + 2,
       B_Q_FULL = B_S_FREE + 2, B_COUNT };

struct Misc {
    uint64_t bars[B_COUNT];
    uint32_t tmem;
    volatile int abort;
    float row_exp[MAX_R];                            // the power of two that a query row was divided by
    float key_scale[RING][NK];
    int key_pos[RING][NK], key_doc[RING][NK];
    float sums[2][2][4][NK];                         // of a set's two last tiles: sums over each quadrant's rows
};
template <bool FP8>
constexpr int smem_bytes() { return Shape<FP8>::STAGES * Shape<FP8>::STAGE_BYTES + (int)sizeof(Misc); }
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "opt-in shared memory per block on sm_103");

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

// Key ranges of B <= 64 streams of unequal length: chunks of whole tiles with which all streams together need no
// more than S ranges, from what it takes if the last chunks are half full on.  Every warp finds the same;
// range x's stream and keys.
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
    const unsigned parts = S - a.B / 2;
    unsigned c = total < (1ll << 30) ? ((unsigned)total + parts - 1u) / parts : (unsigned)((total + parts - 1) / parts);
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

// Sums of e[k], k < N, over the warp's lanes: lane l ends up with key (l N) / 32's.
template <int N>
__device__ __forceinline__ float sum_rows(float (&e)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = N / 2, with = 16; half > 0; half >>= 1, with >>= 1) {
        const bool up = lane & with;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = up ? e[i] : e[i + half], keep = up ? e[i + half] : e[i];
            e[i] = keep + __shfl_xor_sync(0xffffffffu, send, with);
        }
    }
    float s = e[0];
#pragma unroll
    for (int with = 16 / N; with > 0; with >>= 1) s += __shfl_xor_sync(0xffffffffu, s, with);
    return s;
}

// N (8 or 16) consecutive TMEM columns.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld8(taddr, r); }

__device__ __forceinline__ void give_up(Misc* M, unsigned* status) {
    if (atomicExch(const_cast<int*>(&M->abort), 1) == 0) atomicOr(status, DEV_TIMEOUT);
}

// Two bf16 values (one word) of a row times f, a power of two that brings the row below 1, as the e4m3 pieces of
// 2^8 times that: h in the two high bytes of the halves of .x, l in those of .y.  A half of fp16 below 1 has
// e4m3's exponent of 2^8 times the number in its lower four exponent bits, denormals alike, so the piece is the
// half's first bits.
__device__ __forceinline__ uint2 q_pieces(uint32_t w, __nv_bfloat162 f) {
    const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), f);
    const uint32_t qw = *reinterpret_cast<const uint32_t*>(&q);
    const __half2 x = __floats2half2_rn(__uint_as_float(qw << 16), __uint_as_float(qw & 0xffff0000u));
    const uint32_t hw = *reinterpret_cast<const uint32_t*>(&x) & 0xff80ff80u;
    const __half2 l = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&hw)), __float2half2_rn(16.f));
    const uint32_t lw = *reinterpret_cast<const uint32_t*>(&l);
    auto bits = [](uint32_t v) { return ((v << 1) & 0x7fff7fffu) | (v & 0x80008000u); };
    return make_uint2(bits(hw), bits(lw));
}

// One query row in its place in shared memory, chunk c's 128 bytes at row + c * q_chunk (16-byte pieces swizzled
// by `swz`), from nine chunks of 64 bf16 dims to four chunks of h, four of l and the rotated part; the power
// of two that it was divided by.  Whole warp.  A row with an infinity or a NaN becomes NaN.
__device__ __forceinline__ float convert_row(uint8_t* row, int q_chunk, int swz) {
    const int lane = threadIdx.x & 31;
    uint4 v[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const int pc = c * 32 + lane;
        v[c] = pc < 72 ? *reinterpret_cast<const uint4*>(row + (pc >> 3) * q_chunk + (((pc & 7) ^ swz) << 4)) : make_uint4(0, 0, 0, 0);
    }
    // the largest magnitude, as 16 bits of bf16: what is not finite lies above all numbers
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const uint32_t x = __vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu);
        most = __vmaxu2(most, __vmaxu2(x, __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
    }
    most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
    const int e = min(max((int)(most >> 7) - 127, -100), 127);
    const uint32_t spoil = most >= 0x7f80u ? 0x7f7f7f7fu : 0u;
    const uint32_t fb = e < 126 ? (uint32_t)(126 - e) << 7 : 0x40u >> (e - 126), fw = fb | fb << 16;   // 2^(-1 - e), twice
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&fw);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int pc = c * 32 + lane;
        const uint4 o = v[c];
        const uint2 x = q_pieces(o.x, f), y = q_pieces(o.y, f), z = q_pieces(o.z, f), w = q_pieces(o.w, f);
        uint8_t* at = row + (pc >> 4) * q_chunk + ((((pc & 15) >> 1) ^ swz) << 4) + (pc & 1) * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(__byte_perm(x.x, y.x, 0x7531) | spoil, __byte_perm(z.x, w.x, 0x7531) | spoil);
        *reinterpret_cast<uint2*>(at + 4 * q_chunk) = make_uint2(__byte_perm(x.y, y.y, 0x7531) | spoil, __byte_perm(z.y, w.y, 0x7531) | spoil);
    }
    if (lane < 8) {
        const float m = __uint_as_float((uint32_t)(7 - e + 127) << 23);
        const uint4 o = v[2];
        *reinterpret_cast<uint4*>(row + 8 * q_chunk + ((lane ^ swz) << 4)) =
            make_uint4(q_to_bf16(o.x, m), q_to_bf16(o.y, m), q_to_bf16(o.z, m), q_to_bf16(o.w, m));
    }
    return __uint_as_float((uint32_t)(e - 7 + 127) << 23);
}

// KW: keys of a tile per score warp, 16, or 8 with up to 64 rows.
template <bool FP8, bool RULES, int KW>
__global__ void __launch_bounds__(NT, 1) key_weights_kernel(const WeightArgs a) {
    using S = Shape<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Misc* const M = reinterpret_cast<Misc*>(smem + S::STAGES * S::STAGE_BYTES);
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
        const int share = (gap + count - 1) / count;
        const long long g0 = (long long)index * share, g1 = min((long long)gap, g0 + share);
        for (long long g = g0 + tid; g < g1; g += NT)
            a.out[stream0 + gap_at + g] = a.weights ? a.decay * a.weights[stream0 + gap_at + g] : 0.f;
    }
    if (T <= 0) return;
    if (smem_u32(smem) & 1023u) {                        // the swizzled layouts need a 1024-byte aligned base
        if (tid == 0) atomicOr(a.status, DEV_TIMEOUT);
        return;
    }

    if (warp == MMA_WARP) {
        tmem_alloc(&M->tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (tid == (MMA_WARP + 1) * 32) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&M->bars[B_KV_FULL + i], 32 * GATHER_WARPS);
            mbar_init(&M->bars[B_KV_EMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M->bars[B_S_FULL + i], 2);
            mbar_init(&M->bars[B_S_FREE + i], SCORE_WARPS / 2);
        }
        mbar_init(&M->bars[B_Q_FULL], SCORE_WARPS);
        M->abort = 0;
        mbar_init_fence();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = M->tmem;
    const int quad = warp & 3;                           // TMEM lane quadrant of this warp
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const int r = (quad * 32 + lane) & (KW == 16 ? 127 : 63);   // query row of this lane of A and the scores
    const int q_stage = S::q_stage(nrows);

    if (warp < GATHER0) {
        // ---- Q's rows, in nine chunks of 64 dims, rows of 128 B, swizzled; fp8: a warp a row, in pieces
        uint8_t* const q_tmp = smem + q_stage * S::STAGE_BYTES;
        const int q_chunk = (nrows + 7) / 8 * 1024;
        const __nv_bfloat16* q0 = a.q + ((int64_t)b * rows + row0) * D_QK;
        for (int rr = warp; rr < nrows; rr += GATHER0) {
            const uint32_t dst = smem_u32(q_tmp) + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4) + (lane >> 3) * q_chunk;
            const __nv_bfloat16* src = q0 + (int64_t)rr * D_QK + lane * 8;
            cp_async16(dst, src);
            cp_async16(dst + 4 * q_chunk, src + 256);
            if (lane < 8) cp_async16(dst + 8 * q_chunk, src + 512);
        }
        cp_async_wait_all();
        if (FP8) {
            __syncwarp();                                // (a warp converts the rows that it brought)
#pragma unroll 1
            for (int rr = warp; rr < nrows; rr += GATHER0) {
                const float e = convert_row(q_tmp + rr * 128, q_chunk, rr & 7);
                if (lane == 0) M->row_exp[rr] = e;
            }
        }
        bar_sync(3, 32 * GATHER0);
        if (warp < SCORE_WARPS) {
            // ---- Q to TMEM: a quadrant's four warps take its chunks in turn
            const int rr = min(r, nrows - 1);            // (lanes behind the last row: nobody reads their scores)
            if ((r & ~31) < nrows) {
#pragma unroll 1
                for (int c = warp >> 2; c < Q_CHUNKS; c += SCORE_WARPS / 4) {
                    uint32_t h[32];
                    const uint8_t* src = q_tmp + c * q_chunk + rr * 128;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + ((j ^ (rr & 7)) << 4));
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
    }

    if (warp == MMA_WARP || warp == MMA_WARP + 1) {
        // ================= scores: two warps take the tiles in turn, so that one's waits pass in the other's products
        const uint32_t id_f8 = idesc_e4m3(128, NK), id_bf = idesc_bf16(128, NK, false, false);
        const uint64_t dk = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const int buf = warp - MMA_WARP;
        const uint32_t d = tmem + D_COL + buf * D_STEP;
        bool ok = mbar_wait_warp(&M->bars[B_Q_FULL], 0, &M->abort);
        int i = buf, st = buf;                           // tile, stage
        uint32_t round = 0;
        for (; i < T && ok; i += 2) {
            ok = mbar_wait_warp(&M->bars[B_KV_FULL + st], round, &M->abort);
            if (ok && i >= 2) ok = mbar_wait_warp(&M->bars[B_S_FREE + buf], ((i - 2) >> 1) & 1, &M->abort);
            if (!ok) break;
            fence_proxy_async_smem();                    // cp.async (generic proxy) data -> tensor-core reads
            tc_fence_after();
            // (the address is the descriptor's low word; shared memory's 227 KB never carry into the high one)
            const uint32_t lo = (uint32_t)dk + (uint32_t)((st * S::STAGE_BYTES) >> 4);
            const uint64_t hi = dk & 0xffffffff00000000ull;
            if (elect_one()) {
                if (FP8) {
#pragma unroll
                    for (int ks = 0; ks < D_V / 32; ++ks) {
                        const uint64_t kd = hi | (lo + (uint32_t)(((ks >> 2) * REGION + (ks & 3) * 32) >> 4));
                        mma_f8_ta(d, tmem + ks * 8, kd, id_f8, ks > 0);
                        mma_f8_ta(d + NK, tmem + 128 + ks * 8, kd, id_f8, ks > 0);
                    }
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ta(d + 2 * NK, tmem + 256 + ks * 8, hi | (lo + (uint32_t)((4 * REGION + ks * 32) >> 4)), id_bf, ks > 0);
                } else {
#pragma unroll
                    for (int ks = 0; ks < D_QK / 16; ++ks)
                        mma_bf16_ta(d + ks / 12 * NK, tmem + ks * 8, hi | (lo + (uint32_t)(((ks >> 2) * REGION + (ks & 3) * 32) >> 4)), id_bf, ks % 12 > 0);
                }
                mma_commit(&M->bars[B_KV_EMPTY + st]);
                mma_commit(&M->bars[B_S_FULL + buf]);
                mbar_arrive(&M->bars[B_S_FULL + buf]);   // hands on what came with the keys: scales, positions
            }
            __syncwarp();
            st += 2;
            if (st >= S::STAGES) { st -= S::STAGES; round ^= 1; }
        }
        if (!ok) {
            if (lane == 0) give_up(M, a.status);
            if (i >= 2) mbar_drain(&M->bars[B_S_FULL + buf], ((i - 2) >> 1) & 1);
        }
        __syncwarp();
    } else if (warp >= GATHER0) {
        // ================= gather: keys WK w .. WK w + 7 of every tile =================
        const int w = warp - GATHER0;
        bool bad_slot = false;
        const int32_t* slot_row = a.slot + stream0;
        // key l & 7 of tile t (past the range: its last key), as an index in the stream
        auto key_at = [&](int t) -> int {
            const int v = min(k_begin + t * NK + WK * w + (lane & 7), k_end - 1);
            return RULES && v >= gap_at ? v + gap : v;
        };
        // lane l holds the slot of key l & 7 of tile t0 + (l >> 3), for the current group of four tiles and
        // the four after it (a load waits behind the stages' 200 KB that are under way); indices are
        // checked when their group becomes current
        auto load_slots = [&](int t0) -> int {
            const int t = t0 + (lane >> 3);
            return t < T ? __ldg(slot_row + key_at(t)) : 0;
        };
        int cur = load_slots(0), next[4], st = 0, ring = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) next[g] = load_slots(4 * g + 4);
        uint32_t round = 1;                              // (the wait for a fresh stage passes at once)
        for (int i = 0; i < T; ++i) {
            if ((i & 3) == 0) {
                if (i > 0) {
                    cur = next[0];
#pragma unroll
                    for (int g = 0; g < 3; ++g) next[g] = next[g + 1];
                    next[3] = load_slots(i + 16);
                }
                if (cur < 0 || (int64_t)cur >= a.n_pool) { bad_slot = true; cur = 0; }
            }
            const int sl = __shfl_sync(0xffffffffu, cur, ((i & 3) << 3) + (lane & 7));
            // the stage is free: its products are done, and Q has left it
            if (!mbar_wait_warp(&M->bars[B_KV_EMPTY + st], round, &M->abort) ||
                (i == q_stage && !mbar_wait_warp(&M->bars[B_Q_FULL], 0, &M->abort))) {
                if (lane == 0) give_up(M, a.status);
                break;
            }
            const uint32_t base = smem_u32(smem) + st * S::STAGE_BYTES;
            if (FP8) {
#pragma unroll
                for (int it = 0; it < WK; ++it) {        // lane l takes 16-byte piece l of a row's codes
                    const int key = WK * w + it;
                    cp_async16(base + (lane >> 3) * REGION + key * 128 + (((lane & 7) ^ (key & 7)) << 4),
                               a.lat + (int64_t)__shfl_sync(0xffffffffu, sl, it) * D_V + lane * 16);
                }
#pragma unroll
                for (int it = 0; it < WK / 4; ++it) {    // and of four rows' rotated parts
                    const int kk = it * 4 + (lane >> 3), key = WK * w + kk;
                    cp_async16(base + 4 * REGION + key * 128 + (((lane & 7) ^ (key & 7)) << 4),
                               a.rope + (int64_t)__shfl_sync(0xffffffffu, sl, kk) * 64 + (lane & 7) * 8);
                }
                if (lane < WK) cp_async4(smem_u32(&M->key_scale[ring][WK * w + lane]), a.kscale + sl);
            } else {
#pragma unroll
                for (int it = 0; it < WK * 72 / 32; ++it) {
                    const int f = it * 32 + lane, kk = f / 72, pc = f % 72, key = WK * w + kk;
                    cp_async16(base + (pc >> 3) * REGION + key * 128 + (((pc & 7) ^ (key & 7)) << 4),
                               a.kv + (int64_t)__shfl_sync(0xffffffffu, sl, kk) * D_QK + pc * 8);
                }
            }
            if (RULES && lane < WK) {
                const int64_t at = stream0 + key_at(i);
                if (a.rules.key_pos) cp_async4(smem_u32(&M->key_pos[ring][WK * w + lane]), a.rules.key_pos + at);
                if (a.rules.key_doc) cp_async4(smem_u32(&M->key_doc[ring][WK * w + lane]), a.rules.key_doc + at);
            }
            if (!(a.debug_stall && i == 0)) cp_async_arrive_noinc(&M->bars[B_KV_FULL + st]);
            if (++st == S::STAGES) { st = 0; round ^= 1; }
            if (++ring == RING) ring = 0;
        }
        cp_async_wait_all();
        if (bad_slot) atomicOr(a.status, DEV_BAD_SLOT);
    } else if (warp < SCORE_WARPS) {
        // ================= weights: keys g .. g + KW - 1 of every second tile =================
        const int set = warp >> 3, g = KW * (((warp >> 2) & 1) + (KW == 16 ? 0 : quad & 2)), rq = r >> 5;
        const bool row_ok = r < nrows, rows_used = rq * 32 < nrows, writer = (warp & 7) == 0;
        const int t = row_ok ? (row0 + r) / a.H : 0;
        const float lse = row_ok ? a.lse[(int64_t)b * rows + row0 + r] : 0.f;
        const bool live = row_ok && lse != -INFINITY && (!a.counted || a.counted[(int64_t)b * a.q_len + t]);
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
        const float in = RULES && a.rules.softcap > 0.f ? cap_in(c2, a.rules.softcap) : 0.f;
        const bool any_live = __any_sync(0xffffffffu, live);
        constexpr uint32_t ALL_KEYS = (1u << KW) - 1u;
        int ring = set;
        for (int i = set; i < T; i += 2) {
            const int k0 = k_begin + i * NK;
            // the key that this lane of the set's first warp writes, and its former weight
            const int v = k0 + lane;
            const int64_t at = stream0 + (RULES && v >= gap_at ? v + gap : v);
            const bool mine = writer && v < k_end, has_old = mine && direct && a.weights && v < p;
            const float old = has_old ? a.weights[at] : 0.f;
            float(*const sums)[NK] = M->sums[set][(i >> 1) & 1];
            const bool ok = mbar_wait_warp(&M->bars[B_S_FULL + set], (i >> 1) & 1, &M->abort);
            tc_fence_after();
            const int kg = k0 + g;
            // masked: bit k: the row sees key kg + k
            uint32_t see = ALL_KEYS;
            bool some = any_live;
            if (RULES && a.rules.masked && ok) {
                if (kg + KW > p) {
                    const int before = p - kg;           // keys before the drafts
                    see &= before > 0 ? (uint32_t)(vis << before) | ((1u << before) - 1u) : before > -64 ? (uint32_t)(vis >> -before) : 0u;
                }
                // the warp's keys as a whole, and one by one only where that does not decide
                const int at_k = g + lane % KW, v_k = min(kg + lane % KW, k_end - 1);
                const int kp = a.rules.key_pos ? M->key_pos[ring][at_k] : v_k + (v_k >= gap_at ? gap : 0);
                const int kd = a.rules.key_doc ? M->key_doc[ring][at_k] : -1;
                const int4 span = make_int4(__reduce_min_sync(0xffffffffu, kp), __reduce_max_sync(0xffffffffu, kp),
                                            __reduce_min_sync(0xffffffffu, kd), __reduce_max_sync(0xffffffffu, kd));
                const bool none = !live || rule.none(span);
                // (drafts in the prefix are seen whatever their mask says)
                if (__all_sync(0xffffffffu, none || (rule.all(span) && (kg + KW <= p || span.x >= rule.prefix)))) {
                    if (none) see = 0;
                } else {
                    see = 0;
#pragma unroll 1
                    for (int k = 0; k < KW; ++k) {
                        const int pos = __shfl_sync(0xffffffffu, kp, k), doc = __shfl_sync(0xffffffffu, kd, k);
                        const int j = kg + k - p;        // draft index, < 0: before the drafts
                        see |= (uint32_t)(rule.sees(j < 0 || ((vis >> (j & 63)) & 1ull), pos, doc)) << k;
                    }
                }
                if (!live) see = 0;
                some = __any_sync(0xffffffffu, see);
            }
            if (ok && some) {
                uint32_t va[KW], vl[KW], vc[KW];
                const uint32_t d = tmem + lane_base + D_COL + set * D_STEP + g;
                tmem_ld(d, va);
                tmem_ld(d + NK, vl);
                tmem_ld(d + 2 * NK, vc);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&M->bars[B_S_FREE + set]);
                float e[KW];
                const float* ks = M->key_scale[ring] + g;
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    const float x = __uint_as_float(va[k]), y = __uint_as_float(vl[k]), z = __uint_as_float(vc[k]);
                    const float dot = FP8 ? fmaf(fmaf(y, 0.0625f, x), ks[k], z) : x + y + z;
                    e[k] = RULES && a.rules.softcap > 0.f ? dot * in : fmaf(dot, c2, off);
                }
                if (RULES && a.rules.softcap > 0.f) {
                    const float out = cap_out(c2, a.rules.softcap, in);   // (held over the tiles: 35.7 instead of 35.2 us)
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < KW; ++k) top = fmaxf(top, fabsf(e[k]));
                    // scores within the cap, as nearly all are, take the polynomial alone
                    if (__all_sync(0xffffffffu, top <= 1.f)) {
#pragma unroll
                        for (int k = 0; k < KW; k += 2) {
                            const float2 y = fma2(tanh_near(make_float2(e[k], e[k + 1])), both(out), both(off));
                            e[k] = y.x;
                            e[k + 1] = y.y;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < KW; k += 2) {
                            const float2 y = fma2(tanh2(make_float2(e[k], e[k + 1])), both(out), both(off));
                            e[k] = y.x;
                            e[k + 1] = y.y;
                        }
                    }
                }
                if (RULES && a.rules.slopes) {
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        const int kp = a.rules.key_pos ? M->key_pos[ring][g + k] : kg + k + (kg + k >= gap_at ? gap : 0);
                        e[k] = fmaf((float)(kp - rule.pos), rule.slope, e[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < KW; ++k) e[k] = live ? ex2(e[k]) : 0.f;
                if (RULES && a.rules.masked) {
                    if (__any_sync(0xffffffffu, see != ALL_KEYS)) {
#pragma unroll
                        for (int k = 0; k < KW; ++k)
                            if (!((see >> k) & 1u)) e[k] = 0.f;
                    }
                } else if (kg + KW > p) {
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        const int j = kg + k - p;
                        if (j >= 0 && !((vis >> (j & 63)) & 1ull)) e[k] = 0.f;
                    }
                }
                const float s = sum_rows<KW>(e);
                if (lane % (32 / KW) == 0) sums[rq][g + lane / (32 / KW)] = s;
            } else {
                if (rows_used && lane < KW) sums[rq][g + lane] = 0.f;
                if (ok && lane == 0) mbar_arrive(&M->bars[B_S_FREE + set]);
            }
            if (bar_red_or(1 + set, 32 * SCORE_WARPS / 2, !ok)) {   // the sums are there, or a warp gives up
                if (!ok && lane == 0) give_up(M, a.status);
                // the set's keys from here on have no sum
                for (; writer && i < T; i += 2) {
                    const int u = k_begin + i * NK + lane;
                    if (u < k_end) part[stream0 + (RULES && u >= gap_at ? u + gap : u)] = __int_as_float(0x7fc00000);
                }
                break;
            }
            if (mine) {
                float s = sums[0][lane];
#pragma unroll
                for (int q = 1; q < 4; ++q)
                    if (q * 32 < nrows) s += sums[q][lane];
                part[at] = has_old ? fmaf(a.decay, old, s) : s;
            }
            ring = ring + 2 >= RING ? ring + 2 - RING : ring + 2;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
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

// Tiles of a CTA from which on keys that no draft sees are looked for (launch_key_gaps), at a price of 5 us.  (Measured,
// documents, without and with: 64 streams of 2000 keys x 64 rows, 27 tiles a CTA, all keys seen 30.2 and 34.6 us, half
// 29.5 and 24.7, a tenth 28.8 and 17.1; 8 streams of 46000 keys x 72 rows 70 and 75, 70 and 47, 70 and 21.)
constexpr int GAP_TILES = 16;

template <bool FP8, bool RULES, int KW>
cudaError_t launch_weights(const WeightArgs& a, dim3 grid, int dev, cudaStream_t stream) {
    auto* k = key_weights_kernel<FP8, RULES, KW>;
    static std::atomic<bool> attr_set[64];
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<FP8>());
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(k, grid, dim3(NT), (size_t)smem_bytes<FP8>(), stream, a);
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
    const size_t gaps_at = align256(need), gaps_end = gaps_at + (size_t)a.B * sizeof(int2);
    const long long tiles = ((long long)a.slot_stride + NK - 1) / NK * (a.balanced ? a.B : 1);
    if (has_gaps(a.rules) && workspace && aligned(workspace, 8) && gaps_end <= ws_bytes && tiles >= (long long)GAP_TILES * a.nsplit) {
        int2* const gaps = reinterpret_cast<int2*>(static_cast<char*>(workspace) + gaps_at);
        if (launch_key_gaps(a.rules, a.seq_lens, a.B, a.q_len, a.slot_stride, gaps, stream) != cudaSuccess) return MLA_ERR_LAUNCH;
        a.rules.gaps = gaps;
    }
    const ScoreRules& r = a.rules;
    const bool ruled = r.softcap > 0.f || r.slopes || r.masked;
    const bool twice = a.R_step <= 64;
    const cudaError_t e = ruled ? twice ? launch_weights<FP8, true, 8>(a, grid, dev, stream) : launch_weights<FP8, true, 16>(a, grid, dev, stream)
                                : twice ? launch_weights<FP8, false, 8>(a, grid, dev, stream) : launch_weights<FP8, false, 16>(a, grid, dev, stream);
    if (e != cudaSuccess) return MLA_ERR_LAUNCH;
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
    if (B <= 0 || B > 65535 || q_len < 1 || q_len > MLA_MAX_Q_LEN || H < 1 || H > MLA_MAX_HEADS || slot_stride < q_len ||
        slot_stride > MLA_MAX_FP8_KEYS)
        return 0;
    int n_tiles, R_step;
    weight_tiling(q_len * H, &n_tiles, &R_step);
    return n_tiles > 1 ? (size_t)n_tiles * B * slot_stride * 4 : 0;
}
