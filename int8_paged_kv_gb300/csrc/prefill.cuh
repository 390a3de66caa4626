// Prompt attention over the paged int8 caches on 5th-generation tensor cores:
// pa_q8_prefill (prefill.cu) and, under a sliding window with sinks (WIN),
// pa_q8_window_prefill (prefill_window.cu).
//
// out[i, h] = sum_t w_t V_t / sum_t w_t with w_t = 2^(z_t - R),
// z_t = log2(e) scale (q_i . K_t), over the tokens t < sees_i; one pass over
// the context with a running reference R per row.
//
// Rows.  The G query heads of a kv head share its K and V, so the rows of a
// tile are (token, head) pairs: 128 / G tokens x G heads fill the 128 lanes of
// an accumulator, and a tile of a causal prompt spans few tokens.  A CTA works
// on one tile or a pair of tiles of one kv head (an item), against tiles of TN
// context tokens.
//
// Precision.  Codes are exact in f16.  q is scaled by 2^-e per row (e its
// largest exponent), so f16 and bf16 rows are exact in one f16 part, up to
// 2^-25 of the row's largest value, and f32 rows keep 22 bits in two.  The
// weight that meets the code of token t is p_t vs_t (vs: the token's V scale),
// rounded to one f16 (16-bit rows: 2^-11 of itself, below their own rounding)
// or two (f32 rows: 2^-22), neither finer than 2^-25.  R moves with the scales too:
// a job's largest p times its largest vs stays below 2^15, and R is raised only when
// it must be, then to leave 2^7; so 2^-25 is at most 2^-32 of the largest such
// product, whatever the weight.  Sums of p and all accumulators are f32.
//
// Masks.  A token that a row does not see has p = 0 by selection, whatever its
// words hold, and does not enter the row's reference.  A token on a page that does
// not exist gets zero scales, so it counts as zero vectors.  (Masked out by a bit
// per token, every call would take longer: bf16 pairs of tiles 0.3%, f32 rows and
// head size 256 1.3 to 1.6%.)
//
// Windows (WIN).  The tokens that a CTA's rows see are the first few of the sequence
// and a run up to the last row's.  They stand side by side in the K/V tiles, without the
// tokens between them (Seen), in groups of four as in the cache; a row's window is then
// two bounds on the places, and its mask in the jobs at their edges a bit per place.
//
// Rates, causal operations (4 per row, head, dimension and token seen) over the
// call's time, whole prompts of up to 4096 tokens, 32 heads on 8, head size 128:
// bf16 812 TFLOP/s, f32 481 (two products for each: 962); 16 heads on 1, head
// size 256, up to 2048 tokens: f16 629, f32 457 (914).  cuBLAS reaches 1972 in
// bf16.  Of an item's 83,000 cycles (bf16, 28 K/V tiles) 70,000 are the loop: 2500 per 64
// tokens of a pair of row tiles, for which the MMAs need 1090.  What the loop waits
// for is instruction latency: 16 warps run five programs, 6.5 KB the largest, and
// issue 0.5 instructions a cycle and SM quarter; 7% of the instruction cache's
// requests miss, and what adds code to a loop loses 5-10%.  The
// rest: 4400 for Q (its latency from HBM, half hidden by the prefetch), 3700 to
// the first logits, 3000 to write, 3000 between CTAs.
#pragma once

#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "device_util.cuh"
#include "kernels.h"
#include "launch.h"
#include "pa_q8.h"

namespace pa_q8 {
namespace {

// How a CTA's two S buffers are used.  Pair: two row tiles take turns on each
// K/V tile, each with its own accumulator.  Split: one row tile, the even K/V
// tiles to one accumulator and the odd ones to the other, joined at the end.
// Single: one row tile and one accumulator (head size 256 fills TMEM).
enum Mode { kPair, kSplit, kSingle };

// Jobs after which an accumulator of f32 rows is added to sums of its own.  A job is
// 8 steps (MMAs of 16 tokens), and each cuts off about 1e-7 of what the accumulator
// holds where all terms have one sign: 1.2e-5 at a flush when nearly all weight came
// with the first job, a third of that when it came evenly.
constexpr int kFlush = 16;
// Under a window, which nearly every row has in full, every 6.  A sum of j jobs comes out j 1.3e-7 of the
// result off beside the 3e-7 to 5e-7 of the other roundings (2-norm, normal values), and 6 is the most that keeps
// all windows and head sizes below 1e-6: 0.90e-6, with 7 1.00e-6, with 8 1.13e-6, with 12 1.54e-6 (f32 products
// and sums in order 0.3e-6 to 1.1e-6).  A first flush takes a call 15% to 25% longer, as the warpgroup that flushes
// moves all columns while no weights are written; later ones less (8 prompts of up to 4096 rows, 6 for 8: 32 heads on 8,
// head size 128, windows of 700, 800, 1024 and 1500: 528, 566, 676, 796 us -> 527, 665, 710, 806; 16 heads on 1,
// head size 256, windows of 300, 500, 700 and 1500: 174, 204, 274, 375 us -> 174, 240, 277, 396; without a flush
// 240 under 700).
constexpr int kWindowFlush = 6;

// 64 tokens a job leave room in TMEM for the weights beside the logits.
constexpr int kTN = 64;

template <int D_, int NP_, Mode MODE_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int NP = NP_;                        // f16 parts of q and of the weights
    static constexpr Mode MODE = MODE_;
    static constexpr int W = D / 4 + 1;                   // words per token vector
    static constexpr int TN = kTN;                        // context tokens per job
    static constexpr int SUB = D == 256 ? 1 : 2;          // jobs' worth of tokens in a K/V tile: the conversion
    static constexpr int CT = SUB * TN;                   // warps need that much at a time to hide their latencies
    static constexpr int NT = MODE == kPair ? 2 : 1;      // row tiles
    static constexpr int NS = MODE == kSingle ? 1 : 2;    // accumulators, softmax warpgroups
    static constexpr int KST = D == 64 ? 4 : 2;           // K tiles in shared memory
    static constexpr int VST = D == 256 ? 3 - NP : KST;
    static constexpr int DEPTH = 4;                       // scale tables
    // Conversion warps.  Single: a job has twice the codes, and with 4 warps they were what it
    // waited for (f16 552 -> 633 TFLOP/s, f32 468 -> 495 with 8).
    static constexpr int CONV = NS == 1 ? 8 : 4;
    static constexpr int THREADS = 128 * (NS + 1) + 32 * CONV;    // softmax, conversion, issue warpgroups
    static constexpr int ROWS = 128 * NT;
    // Registers a thread by role, 4 x 128 in all, the threads' share at launch.  Each kernel has the
    // split in which the compiler spills none (the other one: head size 64, f32 461 us for 423,
    // bf16 579 for 562; head size 128, Pair 1% more, f32 13%).
    static constexpr bool WIDE = D == 128 && (MODE == kPair || NP == 2);
    static constexpr int REGS_SOFTMAX = MODE == kSingle ? 208 : 160;
    static constexpr int REGS_CONV = WIDE ? 112 : 104;
    static constexpr int REGS_ISSUE = MODE == kSingle ? 96 : WIDE ? 80 : 88;
    static_assert(NS * REGS_SOFTMAX + CONV / 4 * REGS_CONV + REGS_ISSUE <= 512, "registers at launch");
    static constexpr uint32_t Q_PART = 128u * D * 2;      // bytes of one f16 part of one row tile
    static constexpr uint32_t KV_TILE = (uint32_t)CT * D * 2;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = Q_OFF + NT * NP * Q_PART;
    static constexpr uint32_t V_OFF = K_OFF + KST * KV_TILE;
    static constexpr uint32_t TAB_OFF = V_OFF + VST * KV_TILE;
    static constexpr uint32_t TAB = (2 * CT + 4) * 4;     // K scales, V scales, largest |V scale| of each job, whether
                                                          // one of them is not finite
    static constexpr uint32_t QF_OFF = TAB_OFF + DEPTH * TAB;
    static constexpr uint32_t X_OFF = QF_OFF + ROWS * 4;  // Split: R, sum and Rs of both accumulators
    static constexpr uint32_t BAR_OFF = X_OFF + (MODE == kSplit ? 2 * 3 * 128 * 4 : 0);
    static constexpr int BARS = 2 * KST + 2 * VST + 2 * DEPTH + 8 + 2;
    static constexpr uint32_t SMEM = BAR_OFF + BARS * 8 + 16;
    // TMEM columns: S twice, the weights' parts twice (two f16 a column), the accumulators
    static constexpr int TM_P = 2 * TN, TM_O = TM_P + TN * NP, TM_Q = TM_O + NS * D;
    // ... and, in what is left, the first QT columns of 32 f16 pairs (64 head
    // dimensions) of each Q tile and part: QK reads them from there and leaves
    // shared memory, 40% busy, to the conversion (1% faster)
    static constexpr int QT_ROOM = (512 - TM_Q) / (32 * NT * NP);
    static constexpr int QT = QT_ROOM < D / 64 ? QT_ROOM : D / 64;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
    static_assert(SMEM > 232448 / 2, "one CTA per SM: each takes all of TMEM");
    static_assert(TM_Q + NT * NP * QT * 32 <= 512, "TMEM");
};

struct Plan {                          // in the workspace
    uint32_t *head;                    // entries, K/V tiles that pay for a piece, split items
    uint32_t *first;                   // [num_seqs + 1] items before a sequence's first
    uint4 *entries;                    // [cap_entries], most K/V tiles first: a CTA's work per kv head slice: seq,
                                       // row tile, first K/V tile, slot of its record (none: the whole item)
    uint4 *items;                      // [cap_items]: seq, tile, K/V tiles, first slot
    uint4 *splits;                     // [cap_slots]: of the items in pieces: seq, tile, first slot, pieces
    float *part;                       // [slots][groups][ROWS][D + 4]
    float *sums;                       // [SMs][accumulators][D / 4][128][4], or none
    uint32_t *places;                  // a bit per place in sums: taken
    int64_t cap_items, cap_entries, cap_slots;
};

struct Geometry {
    int group;                         // query heads of a kv head
    int heads;                         // of them in one tile: min(group, 128)
    uint32_t over_heads;               // ceil(2^16 / heads): row / heads == row * over_heads >> 16 for rows < 128
    int tokens;                        // tokens in a row tile: 128 / heads
    int span;                          // tokens of an item: NT * tokens
    int groups;                        // CTAs per (row tile, K/V piece): kv heads x head slices
    int slices;
};

struct Params {
    PrefillArgs a;
    Plan plan;
    Geometry g;
    int log2B;
    float scale_log2;
    int rows;                          // rows of an item (128 NT)
    int tn;                            // context tokens per K/V tile
    int may_split;
    int fine;                          // there is room for fine pieces
};

// Items are cut into pieces, each with a CTA and a record of its own, when there
// are too few of them to keep the SMs equally busy.  With p = (K/V tiles of all)
// / SMs: coarsely, an item longer than 2 p into pieces of about p, so that few
// items fill one wave; or finely, into pieces of about p / kFine, which even out
// between the SMs however the items divide.  A piece costs the time of kCost
// tiles; the way that should end first is taken.  (Two prompts of 512 rows behind
// 130,000 and 60,000 tokens, 256 CTAs: 2634 us uncut, 1695 finely; 128 equal CTAs
// of 8192 tokens: 196 us uncut, 270 finely.)
constexpr int kMinPiece = 512;         // context tokens that pay for a piece of their own
constexpr int kFine = 8;
constexpr float kCost = 2.0f;          // 10,000 cycles
constexpr int kMaySplit = 4;           // CTAs per SM, uncut, above which nothing is cut

// Whether fine pieces can pay: ctas items of `longest` tiles at most, `share` tiles per SM,
// the shorter half of them `low` long on average.
__device__ inline bool fine_pays(float sms, float ctas, float longest, float share, float low, float min_piece) {
    const float fine = fmaxf(share / kFine, min_piece);
    const float coarse = ctas <= sms ? fminf(longest, share * (1.0f + ctas / sms))
                                     : fmaxf(fminf(longest, 1.5f * share), share + 0.5f * low);
    return share * (1.0f + kCost / fine) + 0.5f * fine < coarse;
}

// Pieces of an item of this many K/V tiles, and their length but the last's.
__device__ __forceinline__ uint32_t pieces_of(uint32_t tiles, uint32_t piece, uint32_t &len) {
    const uint32_t n = max(1u, tiles / piece);
    len = max(1u, (tiles + n - 1) / n);
    return tiles ? (tiles + len - 1) / len : 1u;
}

__device__ __forceinline__ uint32_t context_of(const PrefillArgs &a, uint32_t s) {
    return (uint32_t)min((int64_t)a.context_lens[s], (int64_t)a.max_blocks_per_seq * a.block_size);
}

// Rows of a sequence; none when its bounds are out of order.
__device__ __forceinline__ uint32_t rows_of(const PrefillArgs &a, uint32_t s, uint32_t &lo) {
    lo = a.query_starts[s];
    const uint32_t hi = a.query_starts[s + 1];
    return hi < lo || hi > a.num_rows ? 0u : hi - lo;
}

// Tokens that the last row of tokens [i0, i0 + span) of a sequence sees.
__device__ __forceinline__ int most_seen(uint32_t c, uint32_t n, uint32_t i0, int span) {
    const int64_t last = min((int64_t)i0 + span, (int64_t)n) - 1;
    return (int)max((int64_t)0, (int64_t)c - ((int64_t)n - 1 - last));
}

// The tokens that the rows of tokens [i0, i0 + span) of a sequence see, side by side: places
// 0 .. total - 1.  Without a window they are the tokens.  Under one, place u is token u below
// `lead` (the sinks) and u + shift from there on; both are multiples of 4, so four places from
// a multiple of 4 on are four tokens of one page, one of which at least is seen.
template <bool WIN>
struct Seen {
    int lead, shift, total;
    __device__ Seen(const PrefillArgs &a, uint32_t c, uint32_t n, uint32_t i0, int span) : lead(0), shift(0) {
        total = most_seen(c, n, i0, span);
        if constexpr (WIN) {
            // the first row's window; from 0 on where the sinks reach it
            const int first = (int)max((int64_t)0, (int64_t)c - n + i0 + 1 - a.window) & ~3, sinks = (a.sinks + 3) & ~3;
            if (sinks < first) {
                lead = sinks;
                shift = first - sinks;
                total -= shift;
            }
        }
    }
    __device__ __forceinline__ int token(int u) const { return WIN && u >= lead ? u + shift : u; }
};

// ---------------------------------------------------------------- planning
//
// One CTA: the items of all sequences, cut into pieces when they are too few
// to fill the SMs, in descending order of their K/V tiles (the last wave then
// ends with the short ones).  Dependent loads and barriers, 7.5 us from cold
// caches; the main kernel's first CTAs set up meanwhile.
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;

// Exclusive sum of x over the CTA's threads (or largest x before this thread's).
template <bool MAX = false>
__device__ uint32_t scan_plan(uint32_t x, uint32_t &total) {
    auto join = [](uint32_t a, uint32_t b) { return MAX ? max(a, b) : a + b; };
    __shared__ uint32_t part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum = join(sum, y);
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    uint32_t w = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, d);
        if (lane >= d) w = join(w, y);
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const uint32_t before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0u;
    const uint32_t left = __shfl_up_sync(0xFFFFFFFFu, sum, 1);
    __syncthreads();
    return lane ? join(before, left) : before;
}

template <bool WIN>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Params P) {
    __shared__ uint32_t bucket[kBuckets];
    __shared__ unsigned long long sum_tiles, low_tiles;
    __shared__ uint32_t longest, low_items;
    grid_dependents_launch();
    const PrefillArgs &a = P.a;
    const int tid = threadIdx.x;
    bucket[tid] = 0;
    if (tid < (a.num_sms + 31) / 32) P.plan.places[tid] = 0;
    if (tid == 0) {
        sum_tiles = low_tiles = 0;
        longest = low_items = 0;
    }
    uint32_t items = 0, bound = 0;                       // bound: the largest start so far
    for (int s0 = 0; s0 < a.num_seqs; s0 += kPlanThreads) {
        const int s = s0 + tid;
        uint32_t t = 0, lo = 0, n = 0, top;
        if (s < a.num_seqs) n = rows_of(a, s, lo);
        // a sequence that begins below an earlier bound would share its rows
        const uint32_t before = max(bound, scan_plan<true>(s < a.num_seqs ? lo : 0u, top));
        bound = max(bound, top);
        if (s < a.num_seqs) {
            if (lo < before) n = 0;
            if (!n && a.query_starts[s + 1] != lo) flag_error(a.status, kDevBadRows);
            t = (n + P.g.span - 1) / P.g.span;
        }
        uint32_t total;
        const uint32_t at = items + scan_plan(t, total);
        if (s < a.num_seqs) P.plan.first[s] = at;
        items += total;
    }
    if (tid == 0) P.plan.first[a.num_seqs] = items;
    __syncthreads();
    // item i: its sequence (the last one whose first item is not behind i)
    auto item_of = [&](uint32_t i, uint32_t &s, uint32_t &tile) {
        int lo = 0, hi = a.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (P.plan.first[mid] <= i) lo = mid;
            else hi = mid;
        }
        s = lo;
        tile = i - P.plan.first[lo];
        uint32_t row0;
        const uint32_t n = rows_of(a, s, row0);
        return (uint32_t)((Seen<WIN>(a, context_of(a, s), n, tile * P.g.span, P.g.span).total + P.tn - 1) / P.tn);
    };
    uint32_t piece = 0x7FFFFFFFu;
    const uint32_t ctas = items * P.g.groups;
    const uint32_t sms = a.num_sms;
    if (P.may_split && ctas < kMaySplit * sms) {
        // each thread keeps to its items, so it may read what it wrote
        unsigned long long sum = 0;
        uint32_t top = 0;
        for (uint32_t i = tid; i < items; i += kPlanThreads) {
            uint32_t s, tile;
            const uint32_t tiles = item_of(i, s, tile);
            P.plan.items[i] = make_uint4(s, tile, tiles, 0u);
            sum += tiles;
            top = max(top, tiles);
        }
        if (sum) {
            atomicAdd(&sum_tiles, sum);
            atomicMax(&longest, top);
        }
        __syncthreads();
        uint32_t low = 0, lows = 0;                          // items up to the mean
        for (uint32_t i = tid; i < items; i += kPlanThreads) {
            const uint32_t tiles = P.plan.items[i].z;
            if ((unsigned long long)tiles * items <= sum_tiles) {
                low += tiles;
                ++lows;
            }
        }
        if (lows) {
            atomicAdd(&low_tiles, (unsigned long long)low);
            atomicAdd(&low_items, lows);
        }
        __syncthreads();
        const unsigned long long all = sum_tiles * P.g.groups;
        const uint32_t ends = sms * (P.fine && fine_pays((float)sms, (float)ctas, (float)longest, (float)all / sms,
                                                         (float)low_tiles / (float)max(low_items, 1u),
                                                         (float)(kMinPiece / P.tn)) ? kFine : 1);
        piece = max((uint32_t)(kMinPiece / P.tn), (uint32_t)((all + ends - 1) / ends));
    }
    uint32_t slots = 0, splits = 0;
    for (uint32_t i0 = 0; i0 < items; i0 += kPlanThreads) {
        const uint32_t i = i0 + tid;
        uint32_t s = 0, tile = 0, tiles = 0, np = 0;
        if (i < items) {
            uint32_t len;
            tiles = item_of(i, s, tile);
            np = pieces_of(tiles, piece, len);
            for (uint32_t p = 0; p < np; ++p)
                atomicAdd(&bucket[kBuckets - 1 - min(min(tiles - p * len, len), (uint32_t)kBuckets - 1)], 1u);
        }
        if (P.may_split) {
            uint32_t total, count;
            const uint32_t at = slots + scan_plan(np > 1 ? np : 0u, total);
            const uint32_t k = splits + scan_plan(np > 1 ? 1u : 0u, count);
            if (i < items) P.plan.items[i].w = at;
            if (np > 1 && k < P.plan.cap_slots) P.plan.splits[k] = make_uint4(s, tile, at, np);
            slots += total;
            splits += count;
        }
    }
    __syncthreads();
    uint32_t entries;
    const uint32_t at0 = scan_plan(bucket[tid], entries);
    bucket[tid] = at0;
    __syncthreads();
    for (uint32_t i = tid; i < items; i += kPlanThreads) {
        uint32_t s, tile;
        const uint32_t tiles = item_of(i, s, tile);
        uint32_t len;
        const uint32_t np = pieces_of(tiles, piece, len);
        const uint32_t slot = P.may_split ? P.plan.items[i].w : 0u;
        for (uint32_t p = 0; p < np; ++p) {
            const uint32_t at =
                atomicAdd(&bucket[kBuckets - 1 - min(min(tiles - p * len, len), (uint32_t)kBuckets - 1)], 1u);
            if (at < P.plan.cap_entries)
                P.plan.entries[at] = make_uint4(s, tile, p * len, np > 1 ? slot + p : 0xFFFFFFFFu);
        }
    }
    if (tid == 0) {
        P.plan.head[0] = (uint32_t)min((int64_t)entries, P.plan.cap_entries);
        P.plan.head[1] = piece;
        P.plan.head[2] = splits;
    }
}

// ---------------------------------------------------------------- main kernel

// 32 columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

// Wait for this warp's TMEM loads; the 32 values may be used only behind it.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void behind32(float *v) {
#pragma unroll
    for (int k = 0; k < 32; k += 8)
        asm volatile("" : "+f"(v[k]), "+f"(v[k + 1]), "+f"(v[k + 2]), "+f"(v[k + 3]), "+f"(v[k + 4]), "+f"(v[k + 5]),
                          "+f"(v[k + 6]), "+f"(v[k + 7]));
}

// 16 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&o)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7]),
                   "=f"(o[8]), "=f"(o[9]), "=f"(o[10]), "=f"(o[11]), "=f"(o[12]), "=f"(o[13]), "=f"(o[14]), "=f"(o[15])
                 : "r"(addr) : "memory");
}

// 16 packed words into 16 columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_st16_nowait(uint32_t addr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                    "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Descriptor of a tile of 128-byte rows under the 128-byte swizzle (8-row
// groups 1024 bytes apart); lbo: bytes between 64-element column blocks of an
// MN-major operand.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo) {
    return umma_smem_desc(saddr, lbo, 1024) | ((uint64_t)2 << 61);
}

// Byte offset of f16 element (row, k) in such a tile of `rows` rows.
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t k, uint32_t rows) {
    return (k >> 6) * rows * 128 + row * 128 + ((((k >> 3) & 7) ^ (row & 7)) << 4) + (k & 7) * 2;
}

// One lane of a converged warp.  (The compiler knows that one thread runs what
// this guards and keeps MMA descriptors in uniform registers; behind lane == 0
// an MMA took 180-390 cycles to issue.)
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// The word `off` bytes into a cache, loaded where this stands, not where the
// value is used.
__device__ __forceinline__ uint32_t load_here(const uint32_t *cache, uint64_t off) {
    uint32_t x;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x) : "l"(reinterpret_cast<const uint8_t *>(cache) + off));
    return x;
}

// Wait for the phase with this parity, until *abort is set or, for this
// thread, about a second passed (then *abort is set).  Time is read from the
// SM's clock, and first after 64 tries: a wait that succeeds costs 17 cycles.
// (Sleeping or suspended between the tries: no gain in the warps that issue,
// 5% lost in the others.)
constexpr long long kWaitCycles = 2000000000ll;
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile uint32_t *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            const long long t = clock64();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitCycles) {
                *abort = 1u;
                return false;
            }
        }
    }
}

// Where one kv head's vectors of a sequence are.
struct Pages {
    const uint32_t *row;                                  // the sequence's block table
    uint32_t page16, head16;                              // a page's and a head's place in it, in 16-byte units
    uint32_t in_page, row_bytes;
    int log2B;
    __device__ Pages(const PrefillArgs &a, uint32_t seq, int kvh, int words, int log2B_)
        : row(a.block_tables + (int64_t)seq * a.max_blocks_per_seq), in_page(a.block_size - 1), row_bytes(words * 4),
          log2B(log2B_) {
        head16 = (uint32_t)a.block_size * words / 4;      // block_size is a multiple of 4
        page16 = head16 * a.num_kv_heads;
        head16 *= kvh;
    }
    __device__ uint32_t find(int token) const { return __ldg(row + (token >> log2B)); }
    __device__ uint64_t offset(uint32_t page, int token) const {
        return (((uint64_t)page * page16 + head16) << 4) + (token & in_page) * row_bytes;
    }
};

template <int N> __device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, float (&x)[N]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (N == 2) {
            const float2 v = *reinterpret_cast<const float2 *>(p);
            x[0] = v.x; x[1] = v.y;
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p + k);
                x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
            }
        }
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t *>(p);
        else if constexpr (N == 4) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
        else *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
                const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&w[k]));
                x[2 * k] = v.x; x[2 * k + 1] = v.y;
            } else {
                x[2 * k] = __uint_as_float(w[k] << 16);
                x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        }
    }
}

// 16 bytes of a row of T.
template <typename T>
__device__ __forceinline__ uint4 chunk_of(const float *x) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (std::is_same<T, __half>::value) {
                w[k] = pack_f16x2(x[2 * k], x[2 * k + 1]);
            } else {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Warp roles (warpgroups, in this order; every link is an mbarrier, every wait
// bounded and abortable):
//  - softmax, one warpgroup per accumulator: a thread owns one row.  S row from
//    TMEM -> z, mask, reference -> p -> p vs as f16 parts in TMEM.
//  - conversion (4 warps; Single, whose jobs have twice the codes: 8): codes
//    of the tile's tokens from global memory (a
//    token's vector is one coalesced read; the next tile's words are in flight
//    in registers) -> f16 tiles of 128-byte rows, K's for QK's B operand
//    (K-major), V's for PV's (MN-major).
//  - tables (1 warp): the tile's K scales (times scale log2 e), V scales and
//    largest |V scale|.
//  - issue (two threads): job n of one (row tile, K/V tile) is S[n & 1] = Q K^T,
//    by one thread as soon as S[n & 1] was read, and O += P V, by the other.
//    S and P are apart, so a row's next logits are there when its weights are
//    written, and the tensor core works on one job while two softmaxes run.
// Barriers: k_full / v_full (the conversion warps), t_full (the table
// warp), k_free / v_free (commit of the last MMA on a tile whose place is
// needed again), t_free (the softmax warps that read the table), s_full[2]
// (commit of QK), s_free[2] and p_full[2] (4 softmax warps), pv_done[2]
// (commit of PV).
//
// The tensor cores cut what they add at an accumulator's last bits, always toward
// zero, about 1e-7 of it at every step, which adds up over a long context that one CTA
// walks (131,072 tokens: 4e-4 to 7e-4 of the result for V with a mean, 8e-4 when the
// first tokens have nearly all weight, 7e-5 for V around zero).  16-bit rows are left
// with that.  With f32 rows, every FLUSH jobs the softmax warps add the accumulator to
// f32 sums in the workspace and PV starts it anew: 3.6e-6, 1.2e-5 and 2.1e-6, at any
// length.  (Every 32 jobs: twice that, and 7% faster; every 8: half, 13% slower.)
// There are as many places for sums as
// SMs, each of which has one CTA at a time; a CTA takes a free one and gives it
// back.
template <typename T, typename C, bool WIN>
__global__ void __launch_bounds__(C::THREADS, 1) prefill_kernel(Params P) {
    constexpr int D = C::D, TN = C::TN, CT = C::CT, SUB = C::SUB, NP = C::NP, NS = C::NS, W = C::W;
    constexpr int FLUSH = NP == 1 ? 1 << 29 : WIN ? kWindowFlush : kFlush;    // 16-bit rows: never
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t s0 = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = s0 + C::BAR_OFF;
    auto k_full = [&](int st) { return bars + 8 * st; };
    auto k_free = [&](int st) { return bars + 8 * (C::KST + st); };
    auto v_full = [&](int st) { return bars + 8 * (2 * C::KST + st); };
    auto v_free = [&](int st) { return bars + 8 * (2 * C::KST + C::VST + st); };
    constexpr int BT = 2 * C::KST + 2 * C::VST, B2 = BT + 2 * C::DEPTH;
    auto t_full = [&](int tab) { return bars + 8 * (BT + tab); };
    auto t_free = [&](int tab) { return bars + 8 * (BT + C::DEPTH + tab); };
    auto s_full = [&](int b) { return bars + 8 * (B2 + b); };
    auto s_free = [&](int b) { return bars + 8 * (B2 + 2 + b); };
    auto p_full = [&](int b) { return bars + 8 * (B2 + 4 + b); };
    auto pv_done = [&](int b) { return bars + 8 * (B2 + 6 + b); };
    auto drained = [&](int i) { return bars + 8 * (B2 + 8 + i); };
    volatile uint32_t *tmem_at = reinterpret_cast<volatile uint32_t *>(smem + C::BAR_OFF + C::BARS * 8);
    volatile uint32_t *abort = tmem_at + 1, *place = tmem_at + 2;

    // the grid is the plan's upper bound
    const uint32_t entry = blockIdx.x / P.g.groups, cta = blockIdx.x % P.g.groups;
    if (P.may_split && blockIdx.x >= P.a.num_sms) {
        grid_dependency_wait();
        if (entry >= P.plan.head[0]) return;
    }
    // the first wave: set up while the planning kernel ends
    if (warp == 0) tmem_alloc(s0 + C::BAR_OFF + C::BARS * 8, 512);
    if (tid == 32) {
        for (int i = 0; i < C::BARS; ++i) {
            const bool by_conv = i < C::KST || (i >= 2 * C::KST && i < 2 * C::KST + C::VST);
            const bool by_softmax = i >= B2 + 2 && i < B2 + 6;
            const bool table = i >= BT + C::DEPTH && i < B2;
            mbar_init(bars + 8 * i, table ? 4 * NS : by_conv ? C::CONV : by_softmax ? 4 : 1);
        }
        *abort = 0u;
        fence_mbar_init();
    }
    grid_dependency_wait();

    const PrefillArgs &a = P.a;
    if (entry >= P.plan.head[0]) {
        __syncthreads();
        if (warp == 0) tmem_dealloc(*tmem_at, 512);
        return;
    }
    const int kvh = cta / P.g.slices, slice = cta % P.g.slices;
    const uint4 e = P.plan.entries[entry];
    uint32_t row0;
    const uint32_t n = rows_of(a, e.x, row0), c = context_of(a, e.x);
    const Seen<WIN> seen(a, c, n, e.y * P.g.span, P.g.span);
    const int seen_all = seen.total;                         // places of tokens, as all of them below
    const int j0 = (int)e.z;
    uint32_t piece_len;
    pieces_of((uint32_t)(seen_all + CT - 1) / CT, P.plan.head[1], piece_len);
    const int tiles = min((seen_all + CT - 1) / CT - j0, (int)piece_len);
    const int steps = min(tiles * SUB, (seen_all + TN - 1) / TN - j0 * SUB);     // of TN tokens
    const int jobs = C::MODE == kPair ? 2 * steps : steps;
    // whether accumulator x is flushed before the end
    auto flushes = [&](int x) { return NP == 2 && (C::MODE == kSingle ? jobs : (jobs - x + 1) / 2) > FLUSH; };
    // whether job x begins a new sum of its accumulator
    auto restarts = [](int x) { return (C::MODE == kSingle ? x : x >> 1) % FLUSH == 0; };
    if (flushes(0) && tid == 0) {
        // the SM's own place is free, unless its number is not below the count of SMs (CTAs that
        // all looked from place 0 on queued for it: a kernel that flushes took half again as long)
        uint32_t p;
        asm("mov.u32 %0, %%smid;" : "=r"(p));
        p %= (uint32_t)a.num_sms;
        for (int tries = 0;; p = (p + 1) % (uint32_t)a.num_sms) {
            if (!(atomicOr(P.plan.places + p / 32, 1u << (p & 31)) >> (p & 31) & 1u)) break;
            if (++tries > 1 << 20) {                         // never with one CTA per SM
                *abort = 1u;
                break;
            }
        }
        __threadfence();
        *place = p;
    }
    const int head0 = slice * P.g.heads;                                 // first head of the kv head's group
    const int heads = min(P.g.heads, P.g.group - head0);

    // ---- Q: f16 parts of q 2^-e into the swizzled tiles.  Each lane has two
    // runs of 8 elements of a row, so D / 16 lanes share one and a warp has
    // several in hand; all its loads are under way before the first is used.
    // (A warp per row, loads behind a branch per row: 8600 cycles an item, not 4600.)
    if (tiles > 0) {
        constexpr int LPR = D / 16, RPW = 32 / LPR;          // lanes of a row, rows of a warp at once
        constexpr int WARPS = C::THREADS / 32;
        constexpr int ROUNDS = (C::ROWS + WARPS * RPW - 1) / (WARPS * RPW);
        constexpr int BATCH = ROUNDS > 4 ? (ROUNDS + 1) / 2 : ROUNDS;
        const int l = lane % LPR;
#pragma unroll 1
        for (int u0 = 0; u0 < ROUNDS; u0 += BATCH) {
            alignas(16) T q[BATCH][16];
            bool have[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int r = ((u0 + u) * WARPS + warp) * RPW + lane / LPR;
                const int rt = r & 127, tok = (int)(rt * P.g.over_heads >> 16), h = rt - tok * P.g.heads;
                const uint32_t i = e.y * P.g.span + (r >> 7) * P.g.tokens + tok;
                have[u] = r < C::ROWS && tok < P.g.tokens && h < heads && i < n;
                // rows that do not exist: loaded from the first one that does, and made zeros
                const T *p = static_cast<const T *>(a.q) + (int64_t)(row0 + (have[u] ? i : 0u)) * a.q_stride +
                             (int64_t)(kvh * P.g.group + head0 + (have[u] ? h : 0)) * D + 8 * l;
                constexpr int V = 8 * sizeof(T) / 16;
#pragma unroll
                for (int c = 0; c < 2 * V; ++c)
                    reinterpret_cast<uint4 *>(q[u])[c] =
                        __ldg(reinterpret_cast<const uint4 *>(p + c / V * (D / 2)) + c % V);
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int r = ((u0 + u) * WARPS + warp) * RPW + lane / LPR, rt = r & 127;
                float x[2][8], mx = 0.0f;
                load_row(q[u], x[0]);
                load_row(q[u] + 8, x[1]);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k / 8][k % 8] = have[u] ? x[k / 8][k % 8] : 0.0f;
#pragma unroll
                for (int k = 0; k < 16; k += 2) mx = max3f(mx, fabsf(x[k / 8][k % 8]), fabsf(x[k / 8][k % 8 + 1]));
#pragma unroll
                for (int d = 1; d < LPR; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
                if (r >= C::ROWS) continue;
                const int eq = mx > 0.0f ? max(-126, min(126, (int)(__float_as_uint(mx) >> 23) - 127)) : 0;
                const float down = __uint_as_float((uint32_t)(127 - eq) << 23);
                if (l == 0)
                    reinterpret_cast<float *>(smem + C::QF_OFF)[r] = __uint_as_float((uint32_t)(127 + eq) << 23);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t hi[4];
                    [[maybe_unused]] uint32_t lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float y0 = x[c][2 * k] * down, y1 = x[c][2 * k + 1] * down;
                        if constexpr (NP == 2) split_f16x2(y0, y1, hi[k], lo[k]);
                        else hi[k] = pack_f16x2(y0, y1);
                    }
                    uint8_t *dst = smem + C::Q_OFF + (r >> 7) * NP * C::Q_PART + swz(rt, 8 * l + c * (D / 2), 128);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (NP == 2)
                        *reinterpret_cast<uint4 *>(dst + C::Q_PART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    const uint32_t tO = tmem + C::TM_O;
    if constexpr (C::QT > 0) {
        // the softmax warpgroups' threads carry a Q row each
        if (warp < 4 * C::NT && tiles > 0) {
            const int rt = tid & 127, nt = warp >> 2;
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int q = 0; q < C::QT; ++q) {
                    uint32_t v[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<uint4 *>(v + 4 * x) = *reinterpret_cast<const uint4 *>(
                            smem + C::Q_OFF + (nt * NP + p) * C::Q_PART + swz(rt, 64 * q + 8 * x, 128));
                    const uint32_t at = tmem + C::TM_Q + (nt * NP + p) * (32 * C::QT) + 32 * q +
                                        ((uint32_t)(32 * (warp & 3)) << 16);
                    tmem_st16_nowait(at, v);
                    tmem_st16_nowait(at + 16, v + 16);
                }
            tmem_wait_st();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    bool issued = false;

    constexpr int ISSUE = 4 * NS + C::CONV;                  // first warp of the issue warpgroup
    if (warp >= ISSUE) {
        // -------------------------------------------------- issue and tables
        set_regs_down<C::REGS_ISSUE>();
        // descriptors of the first tiles; offsets within and between tiles add to them in 16-byte units
        auto step_of = [](int job) { return C::MODE == kPair ? job >> 1 : job; };
        if (warp == ISSUE && elect_one()) {
            constexpr uint32_t ID_QK = umma_idesc_f16(128, TN);
            const uint64_t dQ = swizzled_desc(s0 + C::Q_OFF, 16), dK = swizzled_desc(s0 + C::K_OFF, 16);
            for (int job = 0; job < jobs; ++job) {
                const int step = step_of(job), j = step / SUB, st = j % C::KST, b = job & 1;
                const bool first = step % SUB == 0 && (C::MODE != kPair || b == 0);
                const bool last = step % SUB == SUB - 1 && (C::MODE != kPair || b == 1);
                if (first && !wait_for(k_full(st), (j / C::KST) & 1, abort)) break;
                if (job >= 2 && !wait_for(s_free(b), ((job >> 1) - 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t aK = dK + st * (C::KV_TILE / 16) + (step % SUB) * (TN * 128 / 16);
                const uint64_t aQ = dQ + (C::MODE == kPair ? b : 0) * (NP * C::Q_PART / 16);
                // the small parts first: what they add is not cut at the full sum's last bit
#pragma unroll (NP == 2 ? 1 : D / 64)
                for (int x = 0; x < NP * (D / 64); ++x) {
                    const int p = NP - 1 - x / (D / 64), y = x % (D / 64);
                    const uint64_t bK = aK + y * (CT * 128 / 16);
                    if (y < C::QT) {
                        const uint32_t tQ = tmem + C::TM_Q + ((C::MODE == kPair ? b : 0) * NP + p) * (32 * C::QT) + 32 * y;
#pragma unroll
                        for (int d = 0; d < 4; ++d) umma_f16_ta(tmem + b * TN, tQ + 8 * d, bK + 2 * d, ID_QK, x + d > 0);
                    } else {
                        const uint64_t bQ = aQ + (p * C::Q_PART + y * 128 * 128) / 16;
#pragma unroll
                        for (int d = 0; d < 4; ++d) umma_f16(tmem + b * TN, bQ + 2 * d, bK + 2 * d, ID_QK, x + d > 0);
                    }
                }
                umma_commit(s_full(b));
                if (last && j + C::KST < tiles) umma_commit(k_free(st));
                issued = true;
            }
        } else if (warp == ISSUE + 1 && elect_one()) {
            constexpr uint32_t ID_PV = umma_idesc_f16(128, D) | 1u << 16;       // B is MN-major
            const uint64_t dV = swizzled_desc(s0 + C::V_OFF, CT * 128);
            for (int job = 0; job < jobs; ++job) {
                const int step = step_of(job), j = step / SUB, st = j % C::VST, b = job & 1;
                const bool first = step % SUB == 0 && (C::MODE != kPair || b == 0);
                const bool last = step % SUB == SUB - 1 && (C::MODE != kPair || b == 1);
                if (first && !wait_for(v_full(st), (j / C::VST) & 1, abort)) break;
                if (!wait_for(p_full(b), (job >> 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t aV = dV + st * (C::KV_TILE / 16) + (step % SUB) * (TN * 128 / 16);
                const uint32_t tP = tmem + C::TM_P + b * (NP * TN / 2);
                const bool more = NP == 2 ? !restarts(job) : job > (C::MODE == kSingle ? 0 : 1);
#pragma unroll (NP == 2 ? 1 : NP)
                for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < TN / 16; ++k)
                        umma_f16_ta(tO + (C::MODE == kSingle ? 0 : b * D), tP + p * (TN / 2) + 8 * k,
                                    aV + k * (2048 / 16), ID_PV, more || p < NP - 1 || k > 0);
                umma_commit(pv_done(b));
                if (last && j + C::VST < tiles) umma_commit(v_free(st));
                issued = true;
            }
        }
        __syncwarp();
        if (warp == ISSUE + 3) {
            // the rows of the CTA that comes to this place about next, on their way to L2 (bf16
            // pairs of tiles 797 -> 815 TFLOP/s, f32 rows 502 -> 522)
            const uint32_t next = (blockIdx.x + (uint32_t)a.num_sms) / P.g.groups;
            if (next < P.plan.head[0]) {
                const uint4 e2 = P.plan.entries[next];
                const uint32_t cta2 = (blockIdx.x + (uint32_t)a.num_sms) % P.g.groups;
                const int first2 = (int)(cta2 % P.g.slices) * P.g.heads;
                const uint32_t bytes = (uint32_t)min(P.g.heads, P.g.group - first2) * D * (uint32_t)sizeof(T);
                uint32_t row2;
                const uint32_t n2 = rows_of(a, e2.x, row2);
                for (uint32_t t = e2.y * P.g.span + lane; t < min(n2, (e2.y + 1) * P.g.span); t += 32)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                     static_cast<const T *>(a.q) + (int64_t)(row2 + t) * a.q_stride +
                                     (int64_t)((int)(cta2 / P.g.slices) * P.g.group + first2) * D),
                                 "r"(bytes)
                                 : "memory");
            }
        }
        if (warp == ISSUE + 2) {
            // tokens lane + 32 u of a tile; the next tile's scales and the pages of
            // the one after it are in flight
            constexpr int PER = CT / 32;
            const Pages pages(a, e.x, kvh, W, P.log2B);
            float ks[PER], vs[PER];
            uint32_t page[PER];
            auto token = [&](int j, int u) { return (j0 + j) * CT + 32 * u + lane; };
            auto find = [&](int j) {
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    page[u] = token(j, u) < seen_all ? pages.find(seen.token(token(j, u))) : 0u;
            };
            auto load = [&](int j) {
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    ks[u] = vs[u] = 0.0f;                    // tokens no row sees, or on no page
                    if (token(j, u) >= seen_all) continue;
                    if (page[u] < a.num_blocks) {
                        const uint64_t off = pages.offset(page[u], seen.token(token(j, u))) + (W - 1) * 4;
                        ks[u] = __uint_as_float(load_here(a.key_cache, off));
                        vs[u] = __uint_as_float(load_here(a.value_cache, off));
                    } else {
                        flag_error(a.status, kDevBadBlock);
                    }
                }
            };
            find(0);
            load(0);
            find(1);
            for (int j = 0; j < tiles; ++j) {
                const int tab = j % C::DEPTH;
                if (j >= C::DEPTH &&
                    !__all_sync(0xFFFFFFFFu, wait_for(t_free(tab), (j / C::DEPTH - 1) & 1, abort)))
                    break;
                float *table = reinterpret_cast<float *>(smem + C::TAB_OFF + tab * C::TAB);
#pragma unroll
                for (int u = 0; u < PER; u += 2) {
                    uint32_t top = 0;                        // the largest finite |V scale| of a job
                    [[maybe_unused]] bool odd = false;       // whether one is not finite
#pragma unroll
                    for (int x = u; x < u + 2; ++x) {
                        table[32 * x + lane] = ks[x] * P.scale_log2;
                        table[CT + 32 * x + lane] = vs[x];
                        const uint32_t bits = __float_as_uint(vs[x]) & 0x7FFFFFFFu;
                        odd = odd || bits >= 0x7F800000u;
                        top = max(top, bits < 0x7F800000u ? bits : 0u);
                    }
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
                    if (lane == 0) table[2 * CT + u / 2] = __uint_as_float(top);
                    if constexpr (WIN) {
                        odd = __any_sync(0xFFFFFFFFu, odd);
                        if (lane == 0) table[2 * CT + SUB + u / 2] = odd ? 1.0f : 0.0f;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(t_full(tab));
                load(j + 1);
                find(j + 2);
            }
        }
    } else if (warp >= 4 * NS) {
        // ------------------------------------------------------- conversion
        set_regs_down<C::REGS_CONV>();
        const int cw = warp - 4 * NS;
        constexpr int TPW = CT / C::CONV;                    // tokens of a tile per warp
        constexpr int NW = TPW * (W - 1) / 32;               // words of a tile per lane
        const Pages pages(a, e.x, kvh, W, P.log2B);
        const F16Consts fc;
        uint32_t kw[NW], vw[NW];
        uint32_t page = 0;
        uint64_t off = 0;                                    // of this lane's token of the tile loaded last
        // this lane's token of tile j (lanes above TPW repeat the ones below)
        auto token = [&](int j) { return (j0 + j) * CT + cw * TPW + (lane % TPW); };
        auto find = [&](int j) { page = token(j) < seen_all ? pages.find(seen.token(token(j))) : 0u; };
        // The words of the warp's tokens, four tokens at a time: they are on one
        // page, W words apart.  Behind the last token that is seen, the other
        // tokens of its four are on the same page and read with it; fours that
        // hold none, or lie on a page that does not exist, read page 0's first
        // vectors.
        // word i of this lane: of token token_at(i) of the warp's tokens
        auto token_at = [&](int i) { return D == 64 ? 2 * i + (lane >> 4) : D == 128 ? i : i >> 1; };
        auto word_at = [&](int i) { return D == 64 ? lane & 15 : D == 128 ? lane : lane + 32 * (i & 1); };
        auto locate = [&](int j) {
            off = token(j) < seen_all && page < a.num_blocks ? pages.offset(page, seen.token(token(j))) : 0;
        };
        auto load = [&](const uint32_t *cache, uint64_t at, uint32_t (&w)[NW]) {
            constexpr int PER4 = 4 * NW / TPW;               // words of four tokens per lane
#pragma unroll
            for (int f = 0; f < TPW / 4; ++f) {
                const uint64_t from = __shfl_sync(0xFFFFFFFFu, at, 4 * f) + 4 * word_at(0) +
                                      4 * W * (D == 64 ? lane >> 4 : 0);
#pragma unroll
                for (int i = 0; i < PER4; ++i)
                    w[f * PER4 + i] = load_here(cache, from + (D == 64 ? 8 * W * i : D == 128 ? 4 * W * i
                                                                       : 4 * W * (i >> 1) + 128 * (i & 1)));
            }
        };
        auto convert = [&](uint8_t *tile, const uint32_t (&w)[NW]) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                uint2 v;
                codes4_to_f16x2(w[i], v.x, v.y, fc);
                *reinterpret_cast<uint2 *>(tile + swz(cw * TPW + token_at(i), 4 * word_at(i), CT)) = v;
            }
        };
        auto ready = [&](uint32_t bar) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // K(0), then K(j + 1) ahead of V(j): logits do not wait for a V tile's
        // place.  A tile's words are asked for when the registers are free, one
        // conversion (of the other cache) before they are used.
        find(0);
        locate(0);
        load(a.key_cache, off, kw);
        find(1);
        for (int j = 0; j <= tiles; ++j) {
            const uint64_t off_v = off;                      // tile j's
            if (j < tiles) {
                const int st = j % C::KST;
                if (j >= C::KST &&
                    !__all_sync(0xFFFFFFFFu, wait_for(k_free(st), (j / C::KST - 1) & 1, abort)))
                    break;
                convert(smem + C::K_OFF + st * C::KV_TILE, kw);
                locate(j + 1);
                load(a.key_cache, off, kw);                  // K(j + 1)
                find(j + 2);
                ready(k_full(st));
            }
            if (j > 0) {
                const int v = j - 1, st = v % C::VST;
                if (v >= C::VST &&
                    !__all_sync(0xFFFFFFFFu, wait_for(v_free(st), (v / C::VST - 1) & 1, abort)))
                    break;
                convert(smem + C::V_OFF + st * C::KV_TILE, vw);
                ready(v_full(st));
            }
            if (j < tiles) load(a.value_cache, off_v, vw);   // V(j)
        }
    } else {
        // ---------------------------------------------------------- softmax
        set_regs_up<C::REGS_SOFTMAX>();
        const int wg = warp >> 2;                            // accumulator
        const int rt = tid & 127;                            // row of the tile
        const int nt = C::MODE == kPair ? wg : 0;
        const int tok = (int)(rt * P.g.over_heads >> 16), h = rt - tok * P.g.heads;
        const uint32_t i = e.y * P.g.span + nt * P.g.tokens + tok;
        const bool row_ok = tok < P.g.tokens && h < heads && i < n;
        // rows that do not exist are computed as if they saw everything, and not stored
        const int sees = row_ok ? (int)max((int64_t)0, (int64_t)c - ((int64_t)n - 1 - i)) - seen.shift : seen_all;
        const int sees_min = (int)__reduce_min_sync(0xFFFFFFFFu, (unsigned)sees);
        // under a window it sees the places from `from` on, and the sinks
        const int from = WIN && row_ok ? max(0, sees - a.window) : 0;
        const int from_max = WIN ? (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)from) : 0;
        const float qf = tiles > 0 ? reinterpret_cast<const float *>(smem + C::QF_OFF)[nt * 128 + rt] : 1.0f;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tOw = tO + (C::MODE == kSingle ? 0 : wg * D) + lanes;
        float R = -INFINITY, Rs = -INFINITY;                 // references of the accumulator and of the sums
        float2 l2 = make_float2(0.0f, 0.0f);
        bool ok = true, flushed = false;
        // the row's sums of accumulator x: four columns of the 128 rows together, so that a warp's
        // accesses are whole lines
        auto sums_of = [&](int x) {
            return reinterpret_cast<float4 *>(P.plan.sums + ((int64_t)*place * NS + x) * 128 * D) + rt;
        };
        float4 *sums = flushes(0) ? sums_of(C::MODE == kSingle ? 0 : wg) : nullptr;
        // MASK: 1 the rows do not see all tokens of the job; 2 under a window, one of the tokens has a V
        // scale that is not finite besides, which a weight of zero alone does not hide
        auto tile_job = [&](auto mask_c, int job, int step, int b) {
            constexpr int MASK = decltype(mask_c)::value;
            const int tab = step / SUB % C::DEPTH, sub = step % SUB;
            // this job's K scales; its V scales are CT further, the largest of them at `vtop`
            const float *table = reinterpret_cast<const float *>(smem + C::TAB_OFF + tab * C::TAB) + sub * TN;
            const float vtop = reinterpret_cast<const float *>(smem + C::TAB_OFF + tab * C::TAB)[2 * CT + sub];
            const uint32_t tS = tmem + b * TN + lanes;
            float z[TN];
#pragma unroll
            for (int k = 0; k < TN; k += 32) tmem_ld32_nowait(tS + k, z + k);
            float vmax = vtop;
            const int rel = sees - (j0 * SUB + step) * TN;   // columns below it are seen
            [[maybe_unused]] uint32_t cols[TN / 32] = {};    // ... those whose bits are set, under a window
            if constexpr (MASK > 0 && WIN) {
                const int at = (j0 * SUB + step) * TN;
#pragma unroll
                for (int k = 0; k < TN / 32; ++k) {
                    // bits below x
                    auto below = [&](int x) {
                        const int y = x - 32 * k;
                        return y >= 32 ? 0xFFFFFFFFu : y <= 0 ? 0u : (1u << y) - 1u;
                    };
                    cols[k] = below(rel) & (~below(from - at) | below(a.sinks - at));
                }
            }
            auto hides = [&](int k) { return WIN ? !(cols[k / 32] >> (k % 32) & 1u) : k >= rel; };
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < TN; k += 32) behind32(z + k);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(b));
            if constexpr (MASK > 0 && !WIN) {
                vmax = 0.0f;
#pragma unroll
                for (int k = 0; k < TN; ++k) {
                    const float v = fabsf(table[CT + k]);
                    if (!hides(k) && v < INFINITY) vmax = fmaxf(vmax, v);
                }
            }
            [[maybe_unused]] float top_v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < TN; k += 4) {
                const float4 s4 = *reinterpret_cast<const float4 *>(table + k);
                float2 x = mul_f2(make_float2(z[k], z[k + 1]), make_float2(s4.x, s4.y));
                float2 y = mul_f2(make_float2(z[k + 2], z[k + 3]), make_float2(s4.z, s4.w));
                if constexpr (MASK > 0 && WIN) {
                    // one test a column for its logit and its V scale
                    const float4 v4 = *reinterpret_cast<const float4 *>(table + CT + k);
                    auto column = [&](int i, float &c, float v) {
                        if (hides(k + i)) c = -INFINITY;
                        else if (MASK == 1 || fabsf(v) < INFINITY) top_v[i] = fmaxf(top_v[i], fabsf(v));
                    };
                    column(0, x.x, v4.x);
                    column(1, x.y, v4.y);
                    column(2, y.x, v4.z);
                    column(3, y.y, v4.w);
                } else if constexpr (MASK > 0) {
                    if (hides(k)) x.x = -INFINITY;
                    if (hides(k + 1)) x.y = -INFINITY;
                    if (hides(k + 2)) y.x = -INFINITY;
                    if (hides(k + 3)) y.y = -INFINITY;
                }
                z[k] = x.x; z[k + 1] = x.y; z[k + 2] = y.x; z[k + 3] = y.y;
                mx[(k >> 1) & 2] = max3f(mx[(k >> 1) & 2], x.x, x.y);
                mx[((k >> 1) & 2) + 1] = max3f(mx[((k >> 1) & 2) + 1], y.x, y.y);
            }
            if constexpr (MASK > 0 && WIN) vmax = fmaxf(fmaxf(top_v[0], top_v[1]), fmaxf(top_v[2], top_v[3]));
            // 2^et > the tile's V scales; the reference must keep p vs below 2^15
            const float et = (float)max(-80, (int)(__float_as_uint(vmax) >> 23) - 126);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qf + et;
            const bool raise = top > R + 15.0f;              // also when R is still -inf
            if (__any_sync(0xFFFFFFFFu, raise)) {
                const float Rn = raise ? top - 7.0f : R;
                const float f = R == -INFINITY ? 0.0f : fast_exp2(R - Rn);
                R = Rn;
                l2.x *= f;
                l2.y *= f;
                const int before = C::MODE == kSingle ? job - 1 : job - 2;   // the accumulator's last PV
                if (before >= 0 && (NP == 1 || !restarts(job))) {     // (else PV starts it anew)
                    ok = wait_for(pv_done(before & 1), (before >> 1) & 1, abort);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; return; }
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D; k += 16) {
                        float o[16];
                        tmem_ld16(tOw + k, o);
                        uint32_t u[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(o[x] * f);
                        tmem_st16_nowait(tOw + k, u);
                    }
                }
            }
            if (job >= 2) {                                  // P[b] was read
                ok = wait_for(pv_done(b), ((job >> 1) - 1) & 1, abort);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; return; }
                tc_fence_after();
            }
            const uint32_t tP = tmem + C::TM_P + b * (NP * TN / 2) + lanes;
            const float ref = R == -INFINITY ? 0.0f : R;
            const float2 q2 = make_float2(qf, qf), r2 = make_float2(-ref, -ref);
            float2 la = make_float2(0.0f, 0.0f), lb = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k0 = 0; k0 < TN; k0 += 32) {
                uint32_t hi[16];
                [[maybe_unused]] uint32_t lo[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(table + CT + k0 + k);
                    float2 x = fma_f2(make_float2(z[k0 + k], z[k0 + k + 1]), q2, r2);
                    float2 y = fma_f2(make_float2(z[k0 + k + 2], z[k0 + k + 3]), q2, r2);
                    x = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    la = add_f2(la, x);
                    lb = add_f2(lb, y);
                    x = mul_f2(x, make_float2(v4.x, v4.y));
                    y = mul_f2(y, make_float2(v4.z, v4.w));
                    if constexpr (MASK == 2 || (MASK == 1 && !WIN)) {
                        if (hides(k0 + k)) x.x = 0.0f;
                        if (hides(k0 + k + 1)) x.y = 0.0f;
                        if (hides(k0 + k + 2)) y.x = 0.0f;
                        if (hides(k0 + k + 3)) y.y = 0.0f;
                    }
                    if constexpr (NP == 2) {
                        split_f16x2_fma(x.x, x.y, hi[k / 2], lo[k / 2]);
                        split_f16x2_fma(y.x, y.y, hi[k / 2 + 1], lo[k / 2 + 1]);
                    } else {
                        hi[k / 2] = pack_f16x2(x.x, x.y);
                        hi[k / 2 + 1] = pack_f16x2(y.x, y.y);
                    }
                }
                tmem_st16_nowait(tP + k0 / 2, hi);
                if constexpr (NP == 2) tmem_st16_nowait(tP + TN / 2 + k0 / 2, lo);
            }
            l2 = add_f2(l2, add_f2(la, lb));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(p_full(b));
                // Split: each softmax warpgroup has one of a tile's two jobs
                if (C::MODE == kSplit || sub == SUB - 1) mbar_arrive(t_free(tab));
            }
        };
        // A job of which this warp's rows see nothing: weights of zero, and nothing else moves.  (The
        // two row tiles of a pair see different ones: bf16, 17,762 rows, 32 heads on 8, under 256 tokens 245 -> 241 us,
        // under 1024 381 -> 372.  Where there is one tile, few jobs are like that: head size 256, f32, 1.5% slower.)
        constexpr bool ZEROS = WIN && C::MODE == kPair;
        [[maybe_unused]] const int sees_max = ZEROS ? (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)max(0, sees)) : 0;
        [[maybe_unused]] const int from_min = ZEROS ? (int)__reduce_min_sync(0xFFFFFFFFu, (unsigned)from) : 0;
        [[maybe_unused]] auto zero_job = [&](int job, int step, int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(b));
            if (job >= 2) {                                  // P[b] was read
                ok = wait_for(pv_done(b), ((job >> 1) - 1) & 1, abort);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; return; }
                tc_fence_after();
            }
            const uint32_t zero[16] = {};
#pragma unroll
            for (int k = 0; k < NP * TN / 2; k += 16) tmem_st16_nowait(tmem + C::TM_P + b * (NP * TN / 2) + lanes + k, zero);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(p_full(b));
                if (C::MODE == kSplit || step % SUB == SUB - 1) mbar_arrive(t_free(step / SUB % C::DEPTH));
            }
        };
        for (int job = C::MODE == kSingle ? 0 : wg; job < jobs; job += NS) {
            const int step = C::MODE == kPair ? job >> 1 : job, j = step / SUB, b = job & 1;
            ok = wait_for(t_full(j % C::DEPTH), (j / C::DEPTH) & 1, abort) &&
                 wait_for(s_full(b), (job >> 1) & 1, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            tc_fence_after();
            if (NP == 2 && job >= (C::MODE == kSingle ? FLUSH : 2 * FLUSH) && restarts(job)) {
                // the accumulator, added to the row's sums
                const int before = C::MODE == kSingle ? job - 1 : job - 2;
                ok = wait_for(pv_done(before & 1), (before >> 1) & 1, abort);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                // without waiting for the sums where no row of the warp has a new reference: this
                // thread alone adds to its places, so in a fixed order
                const float f = Rs == R ? 1.0f : fast_exp2(Rs - R);
                const bool same = __all_sync(0xFFFFFFFFu, f == 1.0f);
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    float4 *at = sums + k / 4 * 128;
                    tmem_ld32(tOw + k, o);
                    if (flushed && same) {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(at + x * 128), "f"(o[4 * x]),
                                         "f"(o[4 * x + 1]), "f"(o[4 * x + 2]), "f"(o[4 * x + 3])
                                         : "memory");
                        continue;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        float4 v = flushed ? __ldcg(at + x * 128) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        v = make_float4(fmaf(v.x, f, o[4 * x]), fmaf(v.y, f, o[4 * x + 1]), fmaf(v.z, f, o[4 * x + 2]),
                                        fmaf(v.w, f, o[4 * x + 3]));
                        __stcg(at + x * 128, v);
                    }
                }
                Rs = R;
                flushed = true;
            }
            const int at = (j0 * SUB + step) * TN;
            if (at + TN > sees_min || (WIN && at < from_max && at + TN > a.sinks)) {
                const float *table = reinterpret_cast<const float *>(smem + C::TAB_OFF + j % C::DEPTH * C::TAB);
                if (ZEROS && (at >= sees_max || (at >= a.sinks && at + TN <= from_min))) zero_job(job, step, b);
                else if (!WIN || table[2 * CT + SUB + step % SUB] == 0.0f) tile_job(std::integral_constant<int, 1>(), job, step, b);
                else tile_job(std::integral_constant<int, WIN ? 2 : 1>(), job, step, b);
            } else {
                tile_job(std::integral_constant<int, 0>(), job, step, b);
            }
            if (!ok) break;
        }
        // ---- the row's result: normalised, or as the piece's record
        const int mine = C::MODE == kSingle ? jobs - 1
                       : jobs - 1 - ((jobs - 1 - wg) & 1);    // the accumulator's last job (< 0: none)
        const bool any = C::MODE == kSingle ? jobs > 0 : jobs > wg;
        if (ok && any) {
            ok = wait_for(pv_done(mine & 1), (mine >> 1) & 1, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        if (!ok) *abort = 1u;
        float l = l2.x + l2.y;
        // of the accumulators (f) and of their sums relative to them (g)
        float f0 = 1.0f, f1 = 0.0f, g0 = Rs == R ? 1.0f : fast_exp2(Rs - R), g1 = 0.0f;
        bool both = false;
        if (C::MODE == kSplit) {
            // the two accumulators' references and sums, exchanged by the two threads of a row
            float *x = reinterpret_cast<float *>(smem + C::X_OFF);
            x[wg * 384 + rt] = R;
            x[wg * 384 + 128 + rt] = l;
            x[wg * 384 + 256 + rt] = Rs;
            tc_fence_before();
            named_barrier(1, 256);
            const float R0 = x[rt], l0 = x[128 + rt], R1 = x[384 + rt], l1 = x[512 + rt];
            const float Rs0 = x[256 + rt], Rs1 = x[640 + rt];
            g0 = Rs0 == R0 ? 1.0f : fast_exp2(Rs0 - R0);
            g1 = Rs1 == R1 ? 1.0f : fast_exp2(Rs1 - R1);
            const float Rm = fmaxf(R0, R1);
            f0 = R0 == -INFINITY ? 0.0f : fast_exp2(R0 - Rm);
            f1 = R1 == -INFINITY ? 0.0f : fast_exp2(R1 - Rm);
            // a sum that is NaN stays so, though its reference never moved
            l = (l0 == 0.0f ? 0.0f : l0 * (l0 == l0 ? f0 : 1.0f)) + (l1 == 0.0f ? 0.0f : l1 * (l1 == l1 ? f1 : 1.0f));
            R = Rm;
            both = jobs > 1;
        }
        if (*abort == 0u) {
            tc_fence_after();
            const bool piece = e.w != 0xFFFFFFFFu;
            T *dst = static_cast<T *>(a.out) + (int64_t)(row0 + i) * a.out_stride +
                     (int64_t)(kvh * P.g.group + head0 + h) * D;
            float *rec = P.plan.part + (((int64_t)e.w * P.g.groups + cta) * C::ROWS + nt * 128 + rt) * (D + 4);
            const float inv = piece ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
            f0 *= inv;
            f1 *= inv;
            if (piece && row_ok && (C::MODE != kSplit || wg == 0)) {
                rec[D] = R;
                rec[D + 1] = l;
            }
            // 32 columns of accumulator x
            auto gather = [&](int x, float g, int k, float (&o)[32]) {
                tmem_ld32((C::MODE == kSplit ? tO + x * D + lanes : tOw) + k, o);
                if constexpr (NP == 2) {
                    if (!flushes(x)) return;
                    const float4 *at = sums_of(x) + k / 4 * 128;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float4 v = __ldcg(at + y * 128);
                        o[4 * y] = fmaf(v.x, g, o[4 * y]);
                        o[4 * y + 1] = fmaf(v.y, g, o[4 * y + 1]);
                        o[4 * y + 2] = fmaf(v.z, g, o[4 * y + 2]);
                        o[4 * y + 3] = fmaf(v.w, g, o[4 * y + 3]);
                    }
                }
            };
            // 32 columns of the row (a row without weights has zeros, whatever its accumulator
            // holds; selected where that costs the kernel at hand no spilled registers)
            auto columns = [&](int k, float (&o)[32]) {
                const bool none = tiles <= 0 || l == 0.0f;
                if (tiles > 0) {
                    gather(C::MODE == kPair ? wg : 0, g0, k, o);
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = NP == 1 && none ? 0.0f : o[x] * f0;
                    if (both) {
                        float o1[32];
                        gather(1, g1, k, o1);
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = fmaf(o1[x], f1, o[x]);
                    }
                }
                if (NP == 1 ? tiles <= 0 || (both && none) : none) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0.0f;
                }
            };
            // Through shared memory, so that each store writes whole lines: up to
            // 128 bytes a row at a time.  The place is the row tile's Q (its last
            // QK is done; Split: and what follows it, since all MMAs are).
            // (Rows written by their threads: 5700 cycles an item, not 3000; f32 10,100, not 3900.)
            auto write = [&](auto *row) {
                using O = std::remove_pointer_t<decltype(row)>;
                constexpr int COLS = C::MODE == kSplit ? D / 2 : D;
                constexpr int CH = COLS * sizeof(O) < 128 ? COLS * sizeof(O) / 16 : 8;   // 16-byte chunks of a row
                constexpr int STEP = CH * 16 / sizeof(O);                                // columns
                const int k_lo = C::MODE == kSplit ? wg * COLS : 0;
                uint8_t *buf = smem + C::Q_OFF + (C::MODE == kPair ? nt * C::Q_PART : 0) +
                               (C::MODE == kSplit ? warp : warp & 3) * (32 * 16 * CH);
                auto chunk_at = [&](int r, int c) { return buf + r * (16 * CH) + ((c ^ (r / (8 / CH))) & (CH - 1)) * 16; };
                const uint32_t exist = __ballot_sync(0xFFFFFFFFu, row_ok);
                O *rows[CH];                                  // the rows that this lane writes a chunk of
#pragma unroll
                for (int x = 0; x < CH; ++x)
                    rows[x] = reinterpret_cast<O *>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(row),
                                                                x * (32 / CH) + lane / CH)) +
                              lane % CH * (16 / (int)sizeof(O));
#pragma unroll 1
                for (int k = k_lo; k < k_lo + COLS; k += STEP) {
#pragma unroll
                    for (int k0 = 0; k0 < STEP; k0 += 32) {
                        float o[32];
                        columns(k + k0, o);
#pragma unroll
                        for (int x = 0; x < 32; x += 16 / sizeof(O)) {
                            const uint4 v = chunk_of<O>(o + x);
                            *reinterpret_cast<uint4 *>(chunk_at(lane, (k0 + x) * (int)sizeof(O) / 16)) = v;
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < CH; ++x) {
                        const int r = x * (32 / CH) + lane / CH;
                        const uint4 v = *reinterpret_cast<const uint4 *>(chunk_at(r, lane % CH));
                        if (exist >> r & 1u) *reinterpret_cast<uint4 *>(rows[x] + k) = v;
                    }
                    __syncwarp();
                }
            };
            if (piece) write(rec);
            else write(dst);
        }
    }
    tc_fence_before();
    __syncthreads();
    const bool failed = *abort != 0u;
    if (failed && issued) {
        // the MMAs in flight end before their memory goes
        umma_commit(drained(warp & 1));
        mbar_wait(drained(warp & 1), 0);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && flushes(0)) {
        __threadfence();                                     // the sums' last readers are behind the barrier
        atomicAnd(P.plan.places + *place / 32, ~(1u << (*place & 31)));
    }
    if (failed && tid == 0) flag_error(a.status, kDevWaitTimeout);
}

// ------------------------------------------------------------------- join
//
// A warp per row of a split item: the pieces' records, weighted by their
// references.  Pieces in order, so the sum does not depend on the schedule.
// Bound by the records, D + 4 floats a row and piece, read once.
constexpr int kJoinPerSm = 8;

template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(Params P) {
    grid_dependency_wait();
    const PrefillArgs &a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t per = P.rows / 8;                         // CTAs of one piece's rows
    const uint64_t units = (uint64_t)P.plan.head[2] * P.g.groups * per;
    for (uint64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int r = (int)(u % per) * 8 + warp;
        const uint32_t cta = (uint32_t)(u / per) % P.g.groups;
        const uint4 it = P.plan.splits[u / per / P.g.groups];
        const int rt = r & 127, tok = (int)(rt * P.g.over_heads >> 16), h = rt - tok * P.g.heads;
        const int kvh = cta / P.g.slices, head0 = (cta % P.g.slices) * P.g.heads;
        uint32_t row0;
        const uint32_t n = rows_of(a, it.x, row0);
        const uint32_t i = it.y * P.g.span + (r >> 7) * P.g.tokens + tok;
        if (tok >= P.g.tokens || h >= min(P.g.heads, P.g.group - head0) || i >= n) continue;
        constexpr int PER = D / 32;
        const int64_t step = (int64_t)P.g.groups * P.rows * (D + 4);
        const float *rec = P.plan.part + (((int64_t)it.z * P.g.groups + cta) * P.rows + r) * (D + 4);
        float Rm = -INFINITY;
        for (uint32_t p = lane; p < it.w; p += 32) Rm = fmaxf(Rm, rec[p * step + D]);
#pragma unroll
        for (int d = 16; d; d >>= 1) Rm = fmaxf(Rm, __shfl_xor_sync(0xFFFFFFFFu, Rm, d));
        float l = 0.0f, o[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) o[k] = 0.0f;
#pragma unroll 4
        for (uint32_t p = 0; p < it.w; ++p) {
            const float *x = rec + p * step;
            const float R = x[D], lp = x[D + 1];
            float v[PER];
            load_row(x + lane * PER, v);
            if (lp == 0.0f) continue;                        // the piece has no token that the row sees
            const float f = R == -INFINITY ? 1.0f : fast_exp2(R - Rm);
            l += f * lp;
#pragma unroll
            for (int k = 0; k < PER; ++k) o[k] += f * v[k];
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T *dst = static_cast<T *>(a.out) + (int64_t)(row0 + i) * a.out_stride +
                 (int64_t)(kvh * P.g.group + head0 + h) * D + lane * PER;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const float y = o[k] * inv;
            if constexpr (sizeof(T) == 4) dst[k] = y;
            else if constexpr (std::is_same<T, __half>::value) dst[k] = __float2half_rn(y);
            else dst[k] = __float2bfloat16_rn(y);
        }
    }
}

// ---------------------------------------------------------------- launching

// 16-bit rows at head sizes 64 and 128 take pairs of row tiles, unless most
// sequences' rows fit in one.  (32 heads on 8, head size 128, 16 sequences of 4096
// tokens: 32 rows each, one tile, split 84 us, pairs 105; 48 rows 147 and 105; a
// prompt of 2048 rows 91 and 57.)
Mode mode_of(const PrefillArgs &a) {
    if (a.head_size == 256) return kSingle;
    if (a.dtype == PA_Q8_F32) return kSplit;
    return a.num_rows * (a.num_heads / a.num_kv_heads) > (int64_t)128 * a.num_seqs ? kPair : kSplit;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Geometry and workspace layout; returns the workspace's bytes.
size_t layout(const PrefillArgs &a, Params &P) {
    const int nt = mode_of(a) == kPair ? 2 : 1;
    Geometry &g = P.g;
    g.group = a.num_heads / a.num_kv_heads;
    g.heads = g.group < 128 ? g.group : 128;
    g.slices = (g.group + 127) / 128;
    g.over_heads = (65536u + g.heads - 1) / g.heads;
    g.tokens = 128 / g.heads;
    g.span = nt * g.tokens;
    g.groups = a.num_kv_heads * g.slices;
    P.rows = 128 * nt;
    P.tn = a.head_size == 256 ? kTN : 2 * kTN;           // tokens of a K/V tile: items are cut between tiles
    const int64_t least = (a.num_rows + g.span - 1) / g.span;        // items, at least and at most
    const int64_t most = a.num_rows / g.span + (a.num_seqs < a.num_rows ? a.num_seqs : a.num_rows);
    // places of the tokens that an item's rows see, at most
    const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;
    const int64_t room = a.window ? std::min<int64_t>(cap, (int64_t)a.window + a.sinks + g.span + 8) : cap;
    Plan &p = P.plan;
    p.cap_items = most;
    // Whether fine pieces can pay at all (fine_pays, solved for the largest share that the room
    // allows).  Where they cannot, no place is kept for them: a CTA per SM that the grid has too
    // many costs 1 us.
    const double ctas = (double)(most * g.groups), part = ctas / a.num_sms, share = part * ((room + P.tn - 1) / P.tn);
    P.fine = least * g.groups < kMaySplit * a.num_sms && room >= 2 * kMinPiece &&
             (part > 1.0 ? share > 36.0 : share * (part - 0.0625) > 16.0 || share * (part - 0.5) > 2.0);
    P.may_split = P.fine || (least * g.groups < a.num_sms && room >= 2 * kMinPiece);
    const int64_t ends = (int64_t)a.num_sms * (P.fine ? kFine : 1);
    // pieces of split items: tiles / piece of each, at most
    p.cap_slots = P.may_split ? std::min<int64_t>(ends / g.groups + 1, most * ((room + P.tn) / kMinPiece)) : 0;
    p.cap_entries = most + p.cap_slots;
    char *base = static_cast<char *>(a.workspace);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *q = base + at;
        at += up16(bytes);
        return q;
    };
    p.head = reinterpret_cast<uint32_t *>(take(16));
    p.first = reinterpret_cast<uint32_t *>(take((size_t)(a.num_seqs + 1) * 4));
    p.entries = reinterpret_cast<uint4 *>(take((size_t)p.cap_entries * 16));
    p.items = reinterpret_cast<uint4 *>(take(P.may_split ? (size_t)p.cap_items * 16 : 0));
    p.splits = reinterpret_cast<uint4 *>(take((size_t)p.cap_slots * 16));
    p.part = reinterpret_cast<float *>(take((size_t)p.cap_slots * g.groups * P.rows * (a.head_size + 4) * 4));
    p.places = reinterpret_cast<uint32_t *>(take((size_t)(a.num_sms + 31) / 32 * 4));
    // (16-bit rows never flush, nor does a context short of the shortest flush)
    const bool sums = a.dtype == PA_Q8_F32 && room > (a.window ? kWindowFlush : kFlush) * kTN;
    p.sums = reinterpret_cast<float *>(
        take(sums ? (size_t)a.num_sms * (a.head_size == 256 ? 1 : 2) * 128 * a.head_size * 4 : 0));
    return at;
}

template <typename... KArgs>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Params &P) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <typename T, typename C, bool WIN>
cudaError_t launch_cfg(const Params &P, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(prefill_kernel<T, C, WIN>), C::SMEM, done);
    if (e != cudaSuccess) return e;
    plan_kernel<WIN><<<1, kPlanThreads, 0, st>>>(P);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(prefill_kernel<T, C, WIN>, dim3((unsigned)(P.plan.cap_entries * P.g.groups)), C::THREADS, C::SMEM, st, P);
    if (e != cudaSuccess || !P.may_split) return e;
    const int64_t units = P.plan.cap_slots * P.g.groups * (C::ROWS / 8);
    return launch_after(join_kernel<T, C::D>, dim3((unsigned)std::min<int64_t>(units, P.a.num_sms * kJoinPerSm)), 256, 0,
                        st, P);
}

template <typename T, bool WIN>
cudaError_t launch_16bit(const Params &P, Mode mode, cudaStream_t st) {
    if (P.a.head_size == 64)
        return mode == kPair ? launch_cfg<T, Cfg<64, 1, kPair>, WIN>(P, st) : launch_cfg<T, Cfg<64, 1, kSplit>, WIN>(P, st);
    if (P.a.head_size == 128)
        return mode == kPair ? launch_cfg<T, Cfg<128, 1, kPair>, WIN>(P, st) : launch_cfg<T, Cfg<128, 1, kSplit>, WIN>(P, st);
    return launch_cfg<T, Cfg<256, 1, kSingle>, WIN>(P, st);
}

size_t workspace_of(const PrefillArgs &a) {
    Params P;
    P.a = a;
    return layout(a, P);
}

int64_t ctas_of(const PrefillArgs &a) {
    Params P;
    P.a = a;
    layout(a, P);
    return P.plan.cap_entries * P.g.groups;
}

template <bool WIN>
cudaError_t launch_rows(const PrefillArgs &a, cudaStream_t st) {
    Params P;
    P.a = a;
    layout(a, P);
    P.log2B = 0;
    while ((1 << P.log2B) < a.block_size) ++P.log2B;
    P.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    const Mode mode = mode_of(a);
    if (a.dtype == PA_Q8_F16) return launch_16bit<__half, WIN>(P, mode, st);
    if (a.dtype == PA_Q8_BF16) return launch_16bit<__nv_bfloat16, WIN>(P, mode, st);
    if (a.head_size == 64) return launch_cfg<float, Cfg<64, 2, kSplit>, WIN>(P, st);
    if (a.head_size == 128) return launch_cfg<float, Cfg<128, 2, kSplit>, WIN>(P, st);
    return launch_cfg<float, Cfg<256, 2, kSingle>, WIN>(P, st);
}

}  // namespace
}  // namespace pa_q8
