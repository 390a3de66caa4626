// Single-token attention under a sliding window with sinks over the paged int8
// caches (pa_q8_window_decode).
//
// out[s, h] = sum_t w_t V_t / sum_t w_t, w_t = 2^(z_t - m), z_t = log2(e) scale
// q . K_t, over the tokens t < c with t >= c - window or t < sinks; one pass with a
// running reference m, in f32, on mma.sync f16 tiles: the codes are exact in f16, q and
// the weights enter as hi + lo pairs (rows 0-7 of a tile the hi, rows 8-15 the lo parts
// of the same 8 heads).
//
// What it costs is the words of the visible tokens, read once: 2 (D + 4) bytes a token
// and kv head.  So the split is made for the memory.  The chunks (32 tokens) of all
// sequences stand in one row, cut into equal runs whatever the sequences' lengths; a run
// is walked by a team of streams, one for each kv head, which so read the same pages, whose
// heads lie side by side, at about the same time.  A stream is a warp; or, for 9 to 16 heads and
// at head size 256, a pair of warps, each with half of a chunk's tokens for the logits and half of
// the head dims for the sums, of all heads, so that a code is converted once.  (100 windows of
// 16,000 tokens, a pair with 8 heads each: 64 heads on 4, head size 128, 291 us for 249; 16 on 1,
// head size 256, 146 for 123.  100 windows of 4000, 16 heads on 8, head size 256, a warp alone:
// 211 us for 198.)  A stream's ring of chunk buffers runs on across the sequences' borders, so no
// memory pause comes with them.  Where the streams outnumber what there is to read, that
// crossing (lengths, table, q: one load behind another) costs as much as a few chunks, and
// each sequence is cut into pieces of its own instead, when that makes none much longer
// (1056 chunks on 608 streams: 23.2 -> 15.1 us).  A sequence that lies in one run is written
// by its streams; the pieces of the others are records in the workspace, joined by a second grid.
#include <type_traits>

#include <cuda_bf16.h>

#include "decode_common.cuh"
#include "launch.h"
#include "pa_q8.h"

namespace pa_q8 {
namespace {

constexpr int kStreams = 4;               // of a CTA

struct WindowParams {
    PrefillArgs a;
    int log2B, log2ptok;
    int group;                            // query heads of a kv head
    int head_groups;                      // of up to 8 HT heads
    int units;                            // of a sequence: kv heads x head groups
    int team;                             // streams of a team: units walked side by side
    int rounds;                           // in which a team walks all units of a sequence
    int teams;
    int cuts;                             // pieces of a unit, where runs end with their units (0: they never do)
    uint32_t page16;                      // of a page, in 16-byte units
    float scale_log2;
    float *part;                          // [2 streams][8 HT][D + 4]: A (fragment order), m, l
    uint4 *joins;                         // sequence, unit, pieces (0: nothing to join), first record: of every unit,
    int by_unit;                          // or of every stream, the unit whose first piece ends its run
    int join_log2;                        // of the warps that join a row
};

template <int D, int HT>
struct WinCfg {
    static constexpr int W = D / 4 + 1;
    static constexpr int RING = D == 64 ? 3 : 2;
    static constexpr int WHOLE_EXTRA = D == 256 ? 3 : 1;             // what passing on costs, in chunks
    static constexpr int HEADS = 8 * HT;
    static constexpr bool Q_SMEM = D == 256 || HT == 2;
    static constexpr int PER_SM = D == 256 ? 1 : HT == 2 ? 2 : 3;
    static constexpr int SPLIT = D == 256 || HT == 2 ? 2 : 1;       // warps of a stream
    static constexpr int THREADS = 32 * SPLIT * kStreams;
    static constexpr uint32_t SLOT = (2u * kChunk * W * 4 + 127) / 128 * 128;
    static constexpr uint32_t QF_OFF = 256;                         // q fragments [stream][HT][D / 16][32] uint4
    static constexpr uint32_t X_OFF = QF_OFF + (Q_SMEM ? kStreams * HT * (D / 16) * 512u : 0u);
    static constexpr uint32_t RING_OFF = X_OFF + (SPLIT == 2 ? kStreams * 2 * HT * 512u : 0u);    // weights [stream][half][HT][32] uint4
    static constexpr uint32_t SMEM = RING_OFF + kStreams * RING * SLOT;
};

// The visible tokens of a sequence of c cached ones, as chunks 0 .. n - 1: the sinks'
// first, then the window's; chunk i is tokens 32 (i + skip) from the ns-th on.  (An empty
// sequence has one chunk without tokens.)
struct Visible {
    int c, lo, sinks, ns, skip, n;
    __device__ Visible(const PrefillArgs &a, uint32_t len) {
        const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;
        c = (int)min((int64_t)len, cap);
        lo = max(0, c - a.window);
        sinks = min(a.sinks, lo);
        const int first = lo / kChunk;
        ns = min((sinks + kChunk - 1) / kChunk, first);
        skip = first - ns;
        n = max(1, (c + kChunk - 1) / kChunk - skip);
    }
    __device__ int token(int i) const { return (i < ns ? i : i + skip) * kChunk; }
};

__device__ __forceinline__ float4 load_q4(const void *q, int64_t i, int dtype) {
    if (dtype == PA_Q8_F32) return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(q) + i));
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(q) + i));
    if (dtype == PA_Q8_F16) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
        return make_float4(x.x, x.y, y.x, y.y);
    }
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store_out4(void *out, int64_t i, int dtype, float4 v) {
    if (dtype == PA_Q8_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + i) = v;
        return;
    }
    uint2 w;
    if (dtype == PA_Q8_F16) {
        const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + i) = w;
}

// What a stream copies next: a run of chunks whose tokens follow one another.  Its copying
// warp's alone; kept in shared memory, out of the registers of the loop.
struct Feed {
    const uint32_t *row;                  // the sequence's block table
    uint64_t head16;                      // of the kv head in a page, in 16-byte units
    int lo, hi;                           // tokens that are seen (and the sinks below hi)
    uint32_t seq, round;
    int next;                             // chunk behind the run
    unsigned long long left;              // chunks behind the run
    Visible v;
};

// What a warp computes on; in shared memory for the same reason.
struct Current {
    Visible v;
    uint32_t seq, round;
    unsigned long long left;              // chunks from this unit's on
    unsigned long long run;               // chunks of a run (of a whole piece)
    uint4 join;                           // of the unit whose first piece ends the run
};

// EXACT: f32 rows.
template <int D, int HT, bool EXACT>
__global__ void __launch_bounds__(WinCfg<D, HT>::THREADS, WinCfg<D, HT>::PER_SM) window_decode_kernel(WindowParams P) {
    using C = WinCfg<D, HT>;
    constexpr int W = C::W, RING = C::RING, NKS = D / 16, SPLIT = C::SPLIT;
    constexpr int JT = 4 / SPLIT;                    // token tiles of a warp
    constexpr int NJ = D / 32 / SPLIT;               // V word groups of a warp
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned long long scan_part[C::THREADS / 32], start_rest[kStreams];
    __shared__ uint32_t start_seq[kStreams], start_len[kStreams], scan_most[C::THREADS / 32];
    __shared__ uint32_t failed[kStreams];
    __shared__ float q_scale[kStreams][8 * HT];
    __shared__ float2 tops[kStreams][2][8 * HT];                       // a half's largest logits and V scale
    static_assert(sizeof(Current) % 16 == 0, "aligned places");
    __shared__ __align__(16) uint8_t feed_mem[kStreams * sizeof(Feed)], current_mem[kStreams * SPLIT * sizeof(Current)];
    const PrefillArgs &a = P.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int side = warp / kStreams, ts = warp % kStreams;
    const int gq = lane >> 2, cq = lane & 3;
    const uint32_t bars = smem_addr(smem) + 8 * RING * ts;
    const uint32_t ring = smem_addr(smem + C::RING_OFF) + RING * C::SLOT * ts;
    if (side == 0 && lane == 0) {
        for (int k = 0; k < RING; ++k) mbar_init(bars + 8 * k, 1);
        fence_mbar_init();
        failed[ts] = 0;
    }
    grid_dependents_launch();
    const uint32_t k = blockIdx.x * kStreams + ts;                     // this stream
    const uint32_t team = k / (uint32_t)P.team, member = k - team * (uint32_t)P.team;
    // where runs end with their units: this team's, and the sequence
    const uint32_t unit_at = P.cuts ? team / (uint32_t)P.cuts : 0u, cut = team - unit_at * P.cuts;
    const uint32_t cut_seq = P.rounds == 1 ? unit_at : unit_at / (uint32_t)P.rounds;
    // (the lengths too are read behind the kernel before this one, whose they may be)
    grid_dependency_wait();
    const uint32_t cut_len = P.cuts && cut_seq < (uint32_t)a.num_seqs ? __ldg(a.context_lens + cut_seq) : 0u;

    // ---- chunks before each sequence, and where this CTA's streams begin
    const int each = (a.num_seqs + C::THREADS - 1) / C::THREADS;
    const int s0 = (int)min((int64_t)tid * each, (int64_t)a.num_seqs), s1 = min(s0 + each, a.num_seqs);
    unsigned long long sum = 0;
    uint32_t len = 0;                                                  // of the thread's last sequence
    uint32_t most = 0;                                                 // chunks of a sequence
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        len = __ldg(a.context_lens + s);
        const uint32_t n = Visible(a, len).n;
        sum += n;
        most = max(most, n);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    unsigned long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) {
        scan_part[warp] = incl;
        scan_most[warp] = most;
    }
    __syncthreads();
    unsigned long long before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
        if (w < warp) before += scan_part[w];
        total += scan_part[w];
        most = max(most, scan_most[w]);
    }
    total *= (unsigned)P.rounds;
    // P.cuts pieces a unit, all that the teams allow (a chunk takes a stream 1.4 to 2.7 us, its record
    // less: with two chunks at least small windows take 7.1 us for 6.3), if the longest is no more than WHOLE_EXTRA
    // chunks longer than equal runs.  (12 sequences of 126 chunks at head size 256: 20.6 -> 18.3 us
    // with 3 for 0, nothing changes with 5, and 110 of them are 79 for 67.6 us with 8.)
    const bool whole = P.cuts && ((long long)((most + P.cuts - 1) / (uint32_t)P.cuts) - 1 - C::WHOLE_EXTRA) * P.teams <
                                     (long long)total;
    uint32_t seq0, len0;
    unsigned long long rest0, left0, run0;                             // chunks before the stream's own of the sequence's
    if (whole) {                                                       // units, its own, and of a run
        const uint32_t n = Visible(a, cut_len).n, r = (n + P.cuts - 1) / (uint32_t)P.cuts;
        const uint32_t at = cut * r;
        seq0 = cut_seq;
        len0 = cut_len;
        run0 = r;
        rest0 = (unsigned long long)(unit_at - cut_seq * P.rounds) * n + at;
        left0 = cut_seq < (uint32_t)a.num_seqs && at < n ? min(r, n - at) : 0u;
    } else {
        const unsigned long long per = (total + (unsigned)P.teams - 1) / (unsigned)P.teams;
#pragma unroll 1
        for (int j = 0; j < kStreams; ++j) {
            const uint32_t other = (blockIdx.x * kStreams + j) / (uint32_t)P.team;
            const unsigned long long f = other * per;
            unsigned long long at = before * (unsigned)P.rounds;
            if (other >= (uint32_t)P.teams || f < at || f >= at + sum * (unsigned)P.rounds) continue;
            for (int s = s0; s < s1; ++s) {
                if (s1 - s0 > 1) len = __ldg(a.context_lens + s);
                const unsigned long long n = (unsigned long long)Visible(a, len).n * (unsigned)P.rounds;
                if (f < at + n) {
                    start_seq[j] = s;
                    start_len[j] = len;
                    start_rest[j] = f - at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        const unsigned long long f0 = (unsigned long long)team * per;
        seq0 = start_seq[ts];
        len0 = start_len[ts];
        run0 = per;
        rest0 = start_rest[ts];
        left0 = team < (uint32_t)P.teams && f0 < total ? min(per, total - f0) : 0u;
    }
    if (left0 == 0) {
        if (side == 0 && lane == 0 && !P.by_unit) P.joins[k] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    Feed &feed = reinterpret_cast<Feed *>(feed_mem)[ts];
    Current &now = reinterpret_cast<Current *>(current_mem)[warp];
    const Visible v0(a, len0);
    const uint32_t round0 = P.rounds == 1 ? 0u : (uint32_t)(rest0 / (unsigned)v0.n);
    int chunk = (int)(rest0 - (unsigned long long)round0 * (unsigned)v0.n);
    if (lane == 0) {
        now.v = v0;
        now.seq = seq0;
        now.join = make_uint4(0u, 0u, 0u, 0u);
        now.left = left0;
        now.run = run0;
        now.round = round0;
        if (side == 0) {
            feed.v = v0;
            feed.seq = seq0;
            feed.left = left0;
            feed.round = round0;
            feed.next = chunk;
        }
    }
    __syncwarp();
    const uint64_t policy = l2_policy_evict_first();
    const int ptok = 1 << P.log2ptok;
    const int turn = lane >> (5 - P.log2ptok);                         // the lanes' pieces are those of 2^log2ptok chunks
    int t = 0;                                                         // this lane's piece: its first token
    uint32_t page = 0;                                                 // and its page
    int turns = 0;                                                     // chunks copied of those that the lanes have
    int run = 0;                                                       // chunks left of the run
    uint32_t issued = 0;                                               // chunks copied
    auto seen = [&]() { return t < feed.hi && (t + ptok > feed.lo || t < feed.v.sinks); };
    auto find = [&]() {
        turns = 0;
        if (seen()) page = __ldg(feed.row + (t >> P.log2B));
    };
    auto next_run = [&]() {
        if (lane == 0) {
            if (feed.next == feed.v.n) {
                feed.next = 0;
                if (++feed.round == (uint32_t)P.rounds) {
                    feed.round = 0;
                    feed.v = Visible(a, __ldg(a.context_lens + ++feed.seq));
                }
            }
        }
        __syncwarp();
        const int i = feed.next, end = i < feed.v.ns ? feed.v.ns : feed.v.n;
        run = (int)min((unsigned long long)(end - i), feed.left);
        t = feed.v.token(i) + (lane << P.log2ptok);
        const uint32_t unit = min(feed.round * P.team + member, (uint32_t)P.units - 1), g = unit / (uint32_t)P.head_groups;
        if (i == 0 && issued > 0) {
            // the next unit's q, on its way to L2
            const int first = (int)(unit - g * P.head_groups) * C::HEADS, size = a.dtype == PA_Q8_F32 ? 4 : 2;
            const char *row = static_cast<const char *>(a.q) +
                              ((int64_t)feed.seq * a.q_stride + ((int64_t)g * P.group + first) * D) * size;
            for (int x = lane * 128; x < min(C::HEADS, P.group - first) * D * size; x += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(row + x));
        }
        __syncwarp();
        if (lane == 0) {
            feed.lo = i < feed.v.ns ? 0 : feed.v.lo;
            feed.hi = i < feed.v.ns ? feed.v.sinks : feed.v.c;
            feed.row = a.block_tables + (int64_t)feed.seq * a.max_blocks_per_seq;
            feed.head16 = (uint64_t)g * (uint32_t)(a.block_size * W / 4);
            feed.next = i + run;
            feed.left -= (unsigned)run;
        }
        __syncwarp();
    };
    // Copy the next chunk into buffer b; tokens on a page that does not exist get zero scales.
    auto copy = [&](int b) {
        const uint32_t bar = bars + 8 * b, slot = ring + b * C::SLOT;
        const bool sees = turn == turns && seen(), exists = (int64_t)page < a.num_blocks;
        const uint32_t bytes = (uint32_t)W * 4 << P.log2ptok, dst = (lane & ((kChunk >> P.log2ptok) - 1)) * bytes;
        if (sees && !exists) {
            flag_error(a.status, kDevBadBlock);
            float *p = reinterpret_cast<float *>(smem + C::RING_OFF + (RING * ts + b) * C::SLOT + dst) + (W - 1);
            for (int x = 0; x < ptok; ++x) p[x * W] = p[(kChunk + x) * W] = 0.0f;
        }
        __syncwarp();                                                  // the zeros before the arrival
        const uint32_t pieces = __popc(__ballot_sync(0xFFFFFFFFu, sees && exists));
        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * pieces * bytes);
        const uint64_t at = ((uint64_t)page * P.page16 + feed.head16 + (uint32_t)(t & (a.block_size - 1)) * W / 4) * 16;
        __syncwarp();
        if (sees && exists) {
            fence_proxy_async_smem();
            bulk_copy_g2s(slot + dst, reinterpret_cast<const char *>(a.key_cache) + at, bytes, bar, policy);
            bulk_copy_g2s(slot + kChunk * W * 4 + dst, reinterpret_cast<const char *>(a.value_cache) + at, bytes, bar, policy);
        }
        ++issued;
        if (--run == 0) {
            if (feed.left == 0) return;
            next_run();
            find();
        } else if (++turns == ptok) {
            t += kChunk << P.log2ptok;
            find();
        }
    };
    if (side == 0) {
        next_run();
        find();
        for (int b = 0; b < RING && run; ++b) copy(b);
    }

    const F16Consts fk;
    uint4 *qf = reinterpret_cast<uint4 *>(smem + C::QF_OFF) + ts * HT * NKS * 32;
    uint4 *swap = reinterpret_cast<uint4 *>(smem + C::X_OFF) + ts * 2 * HT * 32;
    uint32_t aq[C::Q_SMEM ? 1 : NKS][4];
    uint32_t done = 0;                                                 // chunks consumed (a buffer's phase)
    bool at_start = true, ok = true;
#pragma unroll 1
    while (ok) {
        // ---- the next unit, or what of it is this stream's
        const uint32_t place = now.round * P.team + member;            // (the last round may have too few units)
        const uint32_t unit = min(place, (uint32_t)P.units - 1), g = unit / (uint32_t)P.head_groups;
        const int h0 = (int)(unit - g * P.head_groups) * C::HEADS;     // of the kv head's heads
        auto row_ok = [&](int u) { return place < (uint32_t)P.units && h0 + 8 * u + gq < P.group; };
        const uint32_t seq = now.seq;
        const int end = (int)min((unsigned long long)now.v.n, chunk + now.left), first = chunk;
        float qk2[HT];
        {
            // a warp's own tile of 8 heads; with up to 8, a pair's first warp has it
            if (side < HT) {
                float4 qraw[NKS];
                const int64_t row = (int64_t)seq * a.q_stride + ((int64_t)g * P.group + (row_ok(side) ? h0 + 8 * side + gq : 0)) * D;
                float mx = 0.0f;
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) qraw[ks] = load_q4(a.q, row + 4 * kword<D>(cq, ks), a.dtype);
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    if (!row_ok(side)) qraw[ks] = make_float4(0.f, 0.f, 0.f, 0.f);
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(qraw[ks].x), fabsf(qraw[ks].y)),
                                         fmaxf(fabsf(qraw[ks].z), fabsf(qraw[ks].w))));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                // q 2^-e with its largest value in [1, 2), as hi and lo f16 parts
                const int eq = mx > 0.0f ? max(-126, min(126, (int)(__float_as_uint(mx) >> 23) - 127)) : 0;
                const float down = __uint_as_float((uint32_t)(127 - eq) << 23);
                qk2[0] = P.scale_log2 * __uint_as_float((uint32_t)(127 + eq) << 23);
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    uint32_t f0, f1, f2, f3;
                    split_f16x2(qraw[ks].x * down, qraw[ks].y * down, f0, f1);
                    split_f16x2(qraw[ks].z * down, qraw[ks].w * down, f2, f3);
                    if constexpr (C::Q_SMEM) {
                        qf[(side * NKS + ks) * 32 + lane] = make_uint4(f0, f1, f2, f3);    // read by the same lanes
                    } else {
                        aq[ks][0] = f0; aq[ks][1] = f1; aq[ks][2] = f2; aq[ks][3] = f3;
                    }
                }
                if constexpr (SPLIT > 1)
                    if (cq == 0) q_scale[ts][8 * side + gq] = qk2[0];
            }
            if constexpr (SPLIT > 1) {
                named_barrier(1 + ts, SPLIT * 32);
#pragma unroll
                for (int u = 0; u < HT; ++u) qk2[u] = q_scale[ts][8 * u + gq];
            }
        }
        float acc[HT][4 * NJ][4];
        float m[HT];
        float2 l2[HT];
#pragma unroll
        for (int u = 0; u < HT; ++u) {
#pragma unroll
            for (int i = 0; i < 4 * NJ; ++i) acc[u][i][0] = acc[u][i][1] = acc[u][i][2] = acc[u][i][3] = 0.0f;
            m[u] = -INFINITY;
            l2[u] = make_float2(0.0f, 0.0f);
        }
        int E = 12;                       // running max biased exponent of V scales (>= 12)
        float wscale = __uint_as_float((uint32_t)(kVScaleBias + 127 - E) << 23);
#pragma unroll 1
        for (; chunk < end; ++chunk, ++done) {
            const int b = done % RING;
            const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(bars + 8 * b, (done / RING) & 1));
            if (!got) {
                if (lane == 0) flag_error(a.status, kDevWaitTimeout);
                if constexpr (SPLIT == 1) {
                    ok = false;
                    break;
                }
                if (lane == 0) failed[ts] = 1;                         // (the other warp learns it at the next barrier)
            }
            const uint32_t *sK = reinterpret_cast<const uint32_t *>(smem + C::RING_OFF) + (RING * ts + b) * (C::SLOT / 4);
            const uint32_t *sV = sK + kChunk * W;
            const int t0 = now.v.token(chunk), c = now.v.c, lo = now.v.lo, sinks = now.v.sinks;
            const bool full = t0 + kChunk <= c && (t0 >= lo || t0 + kChunk <= sinks);

            // ---- S = Q K^T (n-tile j holds tokens 8j .. 8j+7; those of a pair's warp are its own 16)
            float s[HT][JT][4];
#pragma unroll
            for (int u = 0; u < HT; ++u)
#pragma unroll
                for (int j = 0; j < JT; ++j) s[u][j][0] = s[u][j][1] = s[u][j][2] = s[u][j][3] = 0.0f;
            const uint32_t *kr = sK + (8 * JT * side + gq) * W;
#pragma unroll
            for (int ks = 0; ks < NKS; ++ks) {
                const int wd = kword<D>(cq, ks);
                uint32_t f[HT][4];
#pragma unroll
                for (int u = 0; u < HT; ++u) {
                    if constexpr (C::Q_SMEM) {
                        const uint4 x = qf[(u * NKS + ks) * 32 + lane];
                        f[u][0] = x.x; f[u][1] = x.y; f[u][2] = x.z; f[u][3] = x.w;
                    } else {
                        f[u][0] = aq[ks][0]; f[u][1] = aq[ks][1]; f[u][2] = aq[ks][2]; f[u][3] = aq[ks][3];
                    }
                }
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    uint32_t b0, b1;
                    codes4_to_f16x2(kr[8 * j * W + wd], b0, b1, fk);
#pragma unroll
                    for (int u = 0; u < HT; ++u) mma_16816(s[u][j], f[u], b0, b1);
                }
            }
            // ---- online softmax over this thread's tokens, 8j + 2cq + e of the warp's
            float2 z[HT][JT], vs[JT];
            float cmax[HT], vmax = 0.0f;
#pragma unroll
            for (int u = 0; u < HT; ++u) cmax[u] = -INFINITY;
#pragma unroll
            for (int j = 0; j < JT; ++j) {
                const int t = 8 * (JT * side + j) + 2 * cq;
                const float2 ks = make_float2(__uint_as_float(sK[t * W + D / 4]), __uint_as_float(sK[(t + 1) * W + D / 4]));
                vs[j] = make_float2(__uint_as_float(sV[t * W + D / 4]), __uint_as_float(sV[(t + 1) * W + D / 4]));
#pragma unroll
                for (int u = 0; u < HT; ++u)
                    z[u][j] = mul_f2(mul_f2(add_f2(make_float2(s[u][j][0], s[u][j][1]), make_float2(s[u][j][2], s[u][j][3])), ks),
                                     make_float2(qk2[u], qk2[u]));
                if (!full) {
                    auto valid = [&](int x) { return x < c && (x >= lo || x < sinks); };
                    const bool v0 = valid(t0 + t), v1 = valid(t0 + t + 1);
                    if (!v0) vs[j].x = 0.0f;
                    if (!v1) vs[j].y = 0.0f;
#pragma unroll
                    for (int u = 0; u < HT; ++u) {
                        if (!v0) z[u][j].x = -INFINITY;
                        if (!v1) z[u][j].y = -INFINITY;
                    }
                }
#pragma unroll
                for (int u = 0; u < HT; ++u) cmax[u] = max3f(cmax[u], z[u][j].x, z[u][j].y);
                vmax = max3f(vmax, fabsf(vs[j].x), fabsf(vs[j].y));
            }
            // Weights 2^(z - m) may reach 2^kLazy before the accumulators are rescaled;
            // kVScaleBias leaves room for that in f16.  The row's threads compare for
            // themselves, and share their maxima only where one of the stream's is passed.
            bool raise = (int)(__float_as_uint(vmax) >> 23) > E;
#pragma unroll
            for (int u = 0; u < HT; ++u) raise = raise || cmax[u] > m[u] + (float)kLazy;
            if constexpr (SPLIT > 1) raise = named_barrier_or(1 + ts, SPLIT * 32, raise || !got);
            if (__any_sync(0xFFFFFFFFu, raise)) {
                if constexpr (SPLIT > 1) {
                    if (failed[ts]) {                                  // set before the barrier: both warps see it
                        ok = false;
                        break;
                    }
                }
                vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, 1));
                vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, 2));
#pragma unroll
                for (int u = 0; u < HT; ++u) {
                    cmax[u] = fmaxf(cmax[u], __shfl_xor_sync(0xFFFFFFFFu, cmax[u], 1));
                    cmax[u] = fmaxf(cmax[u], __shfl_xor_sync(0xFFFFFFFFu, cmax[u], 2));
                    if constexpr (SPLIT > 1)
                        if (cq == 0) tops[ts][side][8 * u + gq] = make_float2(cmax[u], vmax);
                }
                if constexpr (SPLIT > 1) {
                    named_barrier(1 + ts, SPLIT * 32);
#pragma unroll
                    for (int u = 0; u < HT; ++u) {
                        const float2 x = tops[ts][side ^ 1][8 * u + gq];
                        cmax[u] = fmaxf(cmax[u], x.x);
                        vmax = fmaxf(vmax, x.y);
                    }
                }
                const int E_new = max(E, (int)(__float_as_uint(vmax) >> 23));
                const float ea = (E - E_new < -126) ? 0.0f : __uint_as_float((uint32_t)(127 + E - E_new) << 23);
#pragma unroll
                for (int u = 0; u < HT; ++u) {
                    const float m_new = fmaxf(m[u], cmax[u]);
                    const float alpha = (m[u] == -INFINITY) ? 0.0f : fast_exp2(m[u] - m_new);
                    const float fa = alpha * ea;
#pragma unroll
                    for (int n = 0; n < 4 * NJ; ++n) {
                        acc[u][n][0] *= fa; acc[u][n][1] *= fa; acc[u][n][2] *= fa; acc[u][n][3] *= fa;
                    }
                    l2[u] = mul_f2(l2[u], make_float2(alpha, alpha));
                    m[u] = m_new;
                }
                E = E_new;
                wscale = __uint_as_float((uint32_t)(kVScaleBias + 127 - E) << 23);
            }
            // The weights as f16 parts, for two k-steps of 16 tokens; a pair's warps swap theirs.
            uint32_t ap[2][HT][4];
#pragma unroll
            for (int u = 0; u < HT; ++u) {
                // a row that has seen no token yet keeps m = -inf; its z are all -inf
                const float m_ref = m[u] == -INFINITY ? 0.0f : m[u];
                const float2 back = make_float2(-m_ref, -m_ref), ws = make_float2(wscale, wscale);
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const float2 d = add_f2(z[u][j], back);
                    const float2 p = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                    l2[u] = add_f2(l2[u], p);
                    const float2 pw = mul_f2(mul_f2(p, vs[j]), ws);
                    split_f16x2_fma(pw.x, pw.y, ap[j / 2][u][2 * (j & 1)], ap[j / 2][u][2 * (j & 1) + 1]);
                }
                if constexpr (SPLIT > 1)
                    swap[(side * HT + u) * 32 + lane] = make_uint4(ap[0][u][0], ap[0][u][1], ap[0][u][2], ap[0][u][3]);
            }
            if constexpr (SPLIT > 1) {
                named_barrier(1 + ts, SPLIT * 32);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int u = 0; u < HT; ++u) {
                        const uint4 x = swap[(kk * HT + u) * 32 + lane];
                        ap[kk][u][0] = x.x; ap[kk][u][1] = x.y; ap[kk][u][2] = x.z; ap[kk][u][3] = x.w;
                    }
            }
            // ---- O += P V, a pair's warp for its half of the head dims.  A sum that the tensor cores
            // carry on loses 1e-7 of itself a step, toward zero; f32 rows take a chunk's products from
            // zero and are added to the accumulators in f32.
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj) {
                const uint32_t *r = sV + 2 * cq * W + vword<D>(gq, NJ * side + jj);
                uint32_t w[2][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    w[kk][0] = r[16 * kk * W]; w[kk][1] = r[(16 * kk + 1) * W];
                    w[kk][2] = r[(16 * kk + 8) * W]; w[kk][3] = r[(16 * kk + 9) * W];
                }
                auto tile = [&](auto xc) {
                    constexpr int x = decltype(xc)::value;
                    uint32_t v[2][2];
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        v[kk][0] = codes_pair_to_f16x2<x>(w[kk][0], w[kk][1], fk);
                        v[kk][1] = codes_pair_to_f16x2<x>(w[kk][2], w[kk][3], fk);
                    }
#pragma unroll
                    for (int u = 0; u < HT; ++u) {
                        float (&o)[4] = acc[u][4 * jj + x];
                        if constexpr (EXACT) {
                            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_16816(part, ap[0][u], v[0][0], v[0][1]);
                            mma_16816(part, ap[1][u], v[1][0], v[1][1]);
                            const float2 p = add_f2(make_float2(o[0], o[1]), make_float2(part[0], part[1]));
                            const float2 q = add_f2(make_float2(o[2], o[3]), make_float2(part[2], part[3]));
                            o[0] = p.x; o[1] = p.y; o[2] = q.x; o[3] = q.y;
                        } else {
                            mma_16816(o, ap[0][u], v[0][0], v[0][1]);
                            mma_16816(o, ap[1][u], v[1][0], v[1][1]);
                        }
                    }
                };
                tile(std::integral_constant<int, 0>());
                tile(std::integral_constant<int, 1>());
                tile(std::integral_constant<int, 2>());
                tile(std::integral_constant<int, 3>());
            }
            // ---- release the buffer, refill it
            if constexpr (SPLIT > 1) named_barrier(1 + ts, SPLIT * 32);
            else __syncwarp();
            if (side == 0 && run) copy(b);
        }
        if (!ok) break;
        // ---- the unit's rows, or this piece's record
        float lsum[HT];
#pragma unroll
        for (int u = 0; u < HT; ++u) {
            lsum[u] = l2[u].x + l2[u].y;
            lsum[u] += __shfl_xor_sync(0xFFFFFFFFu, lsum[u], 1);
            lsum[u] += __shfl_xor_sync(0xFFFFFFFFu, lsum[u], 2);
            if constexpr (SPLIT > 1)
                if (cq == 0) tops[ts][side][8 * u + gq].x = lsum[u];
        }
        if constexpr (SPLIT > 1) {
            named_barrier(1 + ts, SPLIT * 32);
#pragma unroll
            for (int u = 0; u < HT; ++u) lsum[u] = tops[ts][0][8 * u + gq].x + tops[ts][1][8 * u + gq].x;
        }
        const uint32_t rec_at = 2 * k + (at_start ? 0u : 1u);
        const bool begins = first == 0, ends = end == now.v.n, whole = begins && ends;
        const float f = ldexpf(1.0f, E - kVScaleBias);
#pragma unroll
        for (int u = 0; u < HT; ++u) {
            if (!row_ok(u)) continue;
            const float inv = whole ? (lsum[u] == 0.0f ? 0.0f : 1.0f / lsum[u]) : 1.0f;
            float *rec = P.part + ((int64_t)rec_at * C::HEADS + 8 * u + gq) * (D + 4);
            const int64_t row = (int64_t)seq * a.out_stride + ((int64_t)g * P.group + h0 + 8 * u + gq) * D;
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj) {
                const int y = NJ * side + jj;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4 o;
                    o.x = (acc[u][4 * jj + 0][e] + acc[u][4 * jj + 0][e + 2]) * f * inv;
                    o.y = (acc[u][4 * jj + 1][e] + acc[u][4 * jj + 1][e + 2]) * f * inv;
                    o.z = (acc[u][4 * jj + 2][e] + acc[u][4 * jj + 2][e + 2]) * f * inv;
                    o.w = (acc[u][4 * jj + 3][e] + acc[u][4 * jj + 3][e + 2]) * f * inv;
                    if (whole) store_out4(a.out, row + 4 * vword<D>(2 * cq + e, y), a.dtype, o);
                    else reinterpret_cast<float4 *>(rec)[(2 * y + e) * 4 + cq] = o;
                }
            }
            if (!whole && side == 0 && cq == 0) {
                rec[D] = m[u];
                rec[D + 1] = lsum[u];
            }
        }
        if (side == 0 && lane == 0 && place < (uint32_t)P.units && begins) {     // the unit may go on in the next teams' streams
            const unsigned long long rest = (unsigned)(now.v.n - end), per = now.run;
            const uint4 join =
                make_uint4(seq, unit, ends ? 0u : 1u + (uint32_t)((rest + per - 1) / per), rec_at);
            if (P.by_unit) P.joins[(int64_t)seq * P.units + unit] = join;
            else now.join = join;
        }
        if (now.left == (unsigned)(end - first)) break;
        at_start = false;
        chunk = 0;
        __syncwarp();
        if (lane == 0) {
            now.left -= (unsigned)(end - first);
            if (++now.round == (uint32_t)P.rounds) {
                now.round = 0;
                now.v = Visible(a, __ldg(a.context_lens + ++now.seq));
            }
        }
        __syncwarp();
    }
    if (side == 0 && lane == 0) {
        if (!P.by_unit) P.joins[k] = ok ? now.join : make_uint4(0u, 0u, 0u, 0u);
        // copies in flight end before their memory goes
        for (uint32_t i = done; !ok && i != issued; ++i)
            if (!mbar_wait(bars + 8 * (i % RING), (i / RING) & 1)) break;
    }
}

// ------------------------------------------------------------------- join
//
// out = sum_r A_r 2^(m_r - M) / sum_r l_r 2^(m_r - M), M = max m_r, over the records
// of a unit.  2^join_log2 warps share a row: warp w has records w, w + 2^join_log2, ...,
// and their sums are added in the order of the warps, so the schedule does not matter.
// With few sequences a unit has many records and there are few units, so rows are given
// more warps, 32 at most, and the list has the units; with many, two or three records, and
// the list has the streams, each of which cuts one unit.  (500 records by 8 warps: 24.8 us
// a call, by 16: 19.6, by 32: 16.5.)
constexpr int kJoinThreads = 1024;                // of a CTA at most

template <int D, int HT>
__global__ void __launch_bounds__(kJoinThreads) window_join_kernel(WindowParams P) {
    constexpr int N4 = D == 256 ? 2 : 1;          // float4 of the row per lane (head size 64: half the lanes)
    constexpr int RU = 4;                         // records' loads in flight
    constexpr int STEP = 8 * HT * (D + 4);        // floats of a stream's records are 2 STEP apart
    extern __shared__ __align__(16) float4 sums[];                  // [warps][N4][32]
    __shared__ float2 tops[kJoinThreads / 32];
    grid_dependents_launch();
    grid_dependency_wait();
    const PrefillArgs &a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t warps = 1u << P.join_log2;                        // of a row
    const uint4 j = P.joins[blockIdx.x];
    // (an entry that a stream which gave up has not written leads nowhere out of bounds)
    if (j.z == 0 || j.z > (uint32_t)P.teams || j.x >= (uint32_t)a.num_seqs || j.y >= (uint32_t)P.units ||
        (uint64_t)(j.w >> 1) + (uint64_t)(j.z - 1) * P.team >= (uint64_t)P.teams * P.team)
        return;
    const uint32_t g = P.head_groups == 1 ? j.y : j.y / (uint32_t)P.head_groups, h0 = (j.y - g * P.head_groups) * (8 * HT);
    const uint32_t w = warp & (warps - 1);
    const int h = (int)(blockIdx.y * (blockDim.x / 32) + warp) >> P.join_log2;
    const bool act = lane < D / 4, row_ok = h < min(8 * HT, P.group - (int)h0);
    // record r: the first one, or the first one of the stream r teams further
    const float *part = P.part + (row_ok ? h : 0) * (D + 4);
    auto record = [&](uint32_t r) {
        return part + (uint64_t)(r == 0 ? j.w : 2 * ((j.w >> 1) + r * P.team)) * STEP;
    };
    float M = -INFINITY, l = 0.0f;
    float4 o[N4];
#pragma unroll
    for (int x = 0; x < N4; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t r0 = w; r0 < j.z; r0 += RU * warps) {
        float4 v[RU][N4];
        float2 ml[RU];
        float top = M;
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            // (most units have two or three records: no loads for more)
            const uint32_t r = r0 + u * warps;
            ml[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int x = 0; x < N4; ++x) v[u][x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < j.z) {
                const float *rec = record(r);
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(rec + D));
#pragma unroll
                for (int x = 0; x < N4; ++x)
                    if (act) v[u][x] = __ldcg(reinterpret_cast<const float4 *>(rec) + lane + 32 * x);
            }
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) top = fmaxf(top, ml[u].x);
        const float f = M == -INFINITY ? 0.0f : fast_exp2(M - top), ref = top == -INFINITY ? 0.0f : top;
        M = top;
        l *= f;
#pragma unroll
        for (int x = 0; x < N4; ++x) o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            if (r0 + u * warps >= j.z) break;
            const float e = fast_exp2(ml[u].x - ref);
            l = fmaf(ml[u].y, e, l);
#pragma unroll
            for (int x = 0; x < N4; ++x) {
                o[x].x = fmaf(v[u][x].x, e, o[x].x);
                o[x].y = fmaf(v[u][x].y, e, o[x].y);
                o[x].z = fmaf(v[u][x].z, e, o[x].z);
                o[x].w = fmaf(v[u][x].w, e, o[x].w);
            }
        }
    }
    if (warps > 1) {
        if (lane == 0) tops[warp] = make_float2(M, l);
#pragma unroll
        for (int x = 0; x < N4; ++x) sums[(warp * N4 + x) * 32 + lane] = o[x];
        __syncthreads();
        if (w != 0) return;
        for (int y = warp + 1; y < warp + (int)warps; ++y) {
            const float2 ml = tops[y];
            const float top = fmaxf(M, ml.x), ref = top == -INFINITY ? 0.0f : top;
            const float f = fast_exp2(M - ref), e = fast_exp2(ml.x - ref);
            M = top;
            l = l * f + ml.y * e;
#pragma unroll
            for (int x = 0; x < N4; ++x) {
                const float4 v = sums[(y * N4 + x) * 32 + lane];
                o[x] = make_float4(o[x].x * f + v.x * e, o[x].y * f + v.y * e, o[x].z * f + v.z * e,
                                   o[x].w * f + v.w * e);
            }
        }
    }
    if (!act || !row_ok) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = (int64_t)j.x * a.out_stride + ((int64_t)g * P.group + h0 + h) * D;
#pragma unroll
    for (int x = 0; x < N4; ++x)
        store_out4(a.out, row + 4 * tc_record_dim4<D>(lane + 32 * x), a.dtype,
                   make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv));
}

// ---------------------------------------------------------------- launching

int per_sm(const PrefillArgs &a) {
    if (a.head_size == 256) return 1;
    return a.num_heads / a.num_kv_heads > 8 ? 2 : 3;
}

constexpr int kJoinLog2 = 5;
constexpr int kTeam = 32;                 // streams of a team, at most

size_t layout(const PrefillArgs &a, WindowParams &P, int64_t &ctas) {
    P.group = a.num_heads / a.num_kv_heads;
    const int heads = P.group > 8 ? 16 : 8;
    P.head_groups = (P.group + heads - 1) / heads;
    P.units = a.num_kv_heads * P.head_groups;
    P.rounds = (P.units + kTeam - 1) / kTeam;
    P.team = (P.units + P.rounds - 1) / P.rounds;
    // as many teams as fit on the SMs, or as the most chunks that the table allows are runs for
    const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;
    const int64_t seen = std::min<int64_t>(cap / kChunk + 1, ((int64_t)a.window + a.sinks) / kChunk + 4);
    const double runs = (double)a.num_seqs * P.rounds * (double)seen + 1.0;
    P.teams = (int)std::min<double>(a.num_sms * per_sm(a) * kStreams / P.team, runs);
    ctas = ((int64_t)P.teams * P.team + kStreams - 1) / kStreams;
    const int64_t streams = ctas * kStreams;
    P.cuts = (int)(P.teams / ((int64_t)a.num_seqs * P.rounds));
    // records of a unit, about: a row gets a warp for every two to four
    const int64_t pieces = std::min<int64_t>(P.teams / ((int64_t)a.num_seqs * P.rounds), seen);
    P.join_log2 = 0;
    while (P.join_log2 < kJoinLog2 && pieces > 4 << P.join_log2) ++P.join_log2;
    P.by_unit = (int64_t)a.num_seqs * P.units <= streams;
    char *p = static_cast<char *>(a.workspace);
    P.joins = reinterpret_cast<uint4 *>(p);
    P.part = reinterpret_cast<float *>(p + streams * sizeof(uint4));
    return (size_t)streams * (sizeof(uint4) + 2 * (size_t)heads * (a.head_size + 4) * sizeof(float));
}

template <int D, int HT, bool EXACT>
cudaError_t launch_typed(const WindowParams &P, int64_t ctas, cudaStream_t st) {
    using C = WinCfg<D, HT>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(window_decode_kernel<D, HT, EXACT>), C::SMEM, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, window_decode_kernel<D, HT, EXACT>, P)) != cudaSuccess) return e;
    const int64_t lists = P.by_unit ? (int64_t)P.a.num_seqs * P.units : ctas * kStreams;
    const int warps = std::max(8, 1 << P.join_log2), rows = warps >> P.join_log2, heads = std::min(C::HEADS, P.group);
    cfg.gridDim = dim3((unsigned)lists, (heads + rows - 1) / rows);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = P.join_log2 ? warps * (D == 256 ? 2 : 1) * 512 : 0;
    return cudaLaunchKernelEx(&cfg, window_join_kernel<D, HT>, P);
}

template <int D, int HT>
cudaError_t launch(const WindowParams &P, int64_t ctas, cudaStream_t st) {
    return P.a.dtype == PA_Q8_F32 ? launch_typed<D, HT, true>(P, ctas, st) : launch_typed<D, HT, false>(P, ctas, st);
}

}  // namespace

size_t window_decode_workspace_bytes(const PrefillArgs &a) {
    WindowParams P;
    int64_t ctas;
    return layout(a, P, ctas);
}

cudaError_t launch_window_decode(const PrefillArgs &a, cudaStream_t st) {
    WindowParams P;
    P.a = a;
    int64_t ctas;
    layout(a, P, ctas);
    P.log2B = 0;
    while ((1 << P.log2B) < a.block_size) ++P.log2B;
    P.page16 = (uint32_t)a.num_kv_heads * (uint32_t)(a.block_size * (a.head_size / 4 + 1) / 4);
    P.log2ptok = P.log2B < 5 ? P.log2B : 5;
    P.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    const bool wide = P.group > 8;
    if (a.head_size == 64) return wide ? launch<64, 2>(P, ctas, st) : launch<64, 1>(P, ctas, st);
    if (a.head_size == 128) return wide ? launch<128, 2>(P, ctas, st) : launch<128, 1>(P, ctas, st);
    return wide ? launch<256, 2>(P, ctas, st) : launch<256, 1>(P, ctas, st);
}

}  // namespace pa_q8
