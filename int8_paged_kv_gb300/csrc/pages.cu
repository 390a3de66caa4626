// Pages of a cache: copying them, and the pool that says who holds them
// (reference counts, a stack of free pages, the sequences' block tables).
//
// The pool operators are whole-number bookkeeping over a few hundred KB that
// sits in L2, so their time is launches and dependent loads, not bytes.  Each
// is two launches, the second queued so that it may begin while the first one
// drains: decisions that depend on other requests are scans (over the request
// index in one CTA, over the page numbers in a cluster of eight), and a CTA
// per row walks the block tables.  Results do not depend on the order in which
// CTAs run: the only atomics are whole-number sums, minima and exchanges.
//
// Replayed in a CUDA graph behind a copy that puts the tables back, for 256
// sequences of up to 8192 tokens in a pool of 52,000 pages of 16: fork of 128
// and the copy of their open pages 12.3 us, free and extend of 128 together
// 16.4 us; of one, among 64 sequences of up to 4096 tokens, 14.4 us.  (Both launches of an operator as one of a single
// cluster, tables walked by its 256 warps: 4-5 us less on the host for each
// operator, but 2-4 us more on the GPU for one request and 6-8 us for 128.)
#include <cooperative_groups.h>

#include "device_util.cuh"
#include "kernels.h"

namespace pa_q8 {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;                         // of a CTA that walks one row, four entries a thread
constexpr uint32_t kNone = 0xFFFFFFFFu;
// A page whose count reached zero in this call carries this mark until the
// stack takes it.  The mark and every correction are additions, so they
// commute: a second release of the same page (a caller error) takes the
// count below the mark or below zero, is seen as such (>= kOver) and adds
// back the one it took.
constexpr uint32_t kFreedMark = 0x40000000u;
constexpr uint32_t kOver = 0x20000000u;

// ------------------------------------------------------------ page copies

constexpr int kCopyPiece = 16384;                        // most bytes of one bulk copy
constexpr int kCopyStages = 4, kCopyAhead = 2;           // buffers of a CTA; loads it has under way
constexpr int kCopyPerSm = 3;                            // CTAs of one warp
constexpr int kCopyLists = 4;                            // list entries that a lane looks up at once

__device__ __forceinline__ void bulk_copy_s2g(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Pair p copies page src[p] to dst[p] of both caches.  A unit is one page of
// one cache, cut into equal pieces of at most kCopyPiece bytes that go through
// a ring of shared-memory buffers, in and out by bulk copies: no register
// holds a byte, and a CTA keeps kCopyAhead pieces under way.  Units go round
// the grid; a lane looks up four of them at a time, so that a list's padding
// costs one round of loads per 128 units of a CTA.
//
// Bound by HBM: 8192 pairs of 16,896-byte pages, 554 MB read and written, take
// 92 us (6.0 TB/s); in a list of 24,576 with the other entries empty, 92 us.
// (Through registers, four 16-byte loads per thread: 99 and 128 us.  Pieces of
// at most 4, 8, 16 and 32 KB: 95, 94, 92 and 92 us; one CTA per SM 94-134 us,
// two or three 92.)  Few pairs cost a launch: 4.1 us for five.
__global__ void __launch_bounds__(32)
copy_pages_kernel(char *key, char *value, const uint32_t *src, const uint32_t *dst, int64_t pairs,
                  int64_t page_bytes, uint32_t piece_bytes, int64_t num_blocks, uint32_t *status) {
    extern __shared__ __align__(128) char buffers[];
    __shared__ uint64_t bars[kCopyStages];
    __shared__ struct { char *to; uint32_t bytes; } place[kCopyStages];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kCopyStages; ++i) mbar_init(smem_addr(bars + i), 1);
        fence_mbar_init();
    }
    __syncwarp();
    const uint64_t policy = l2_policy_evict_first();
    uint32_t loads = 0, stores = 0;                      // lane 0's
    bool ok = true;
    auto store_next = [&]() {
        const uint32_t st = stores % kCopyStages;
        ok = ok && mbar_wait(smem_addr(bars + st), stores / kCopyStages & 1);
        if (ok) bulk_copy_s2g(place[st].to, smem_addr(buffers + st * piece_bytes), place[st].bytes);
        ++stores;
    };
    const int64_t units = 2 * pairs;
    for (int64_t u0 = blockIdx.x; u0 < units; u0 += (int64_t)gridDim.x * 32 * kCopyLists) {
        uint32_t s[kCopyLists], d[kCopyLists];
#pragma unroll
        for (int k = 0; k < kCopyLists; ++k) {
            const int64_t u = u0 + (int64_t)gridDim.x * (32 * k + lane);
            s[k] = u < units ? src[u >> 1] : kNone;
            d[k] = u < units ? dst[u >> 1] : kNone;
        }
#pragma unroll
        for (int k = 0; k < kCopyLists; ++k) {
            bool good = s[k] != kNone && d[k] != kNone;
            if (good && (s[k] >= num_blocks || d[k] >= num_blocks)) {
                flag_error(status, kDevBadBlock);
                good = false;
            }
            for (uint32_t left = __ballot_sync(0xFFFFFFFFu, good); left; left &= left - 1) {
                const int l = __ffs(left) - 1;
                const int64_t from = (int64_t)__shfl_sync(0xFFFFFFFFu, s[k], l) * page_bytes;
                const int64_t to = (int64_t)__shfl_sync(0xFFFFFFFFu, d[k], l) * page_bytes;
                if (lane != 0) continue;
                char *base = (u0 + (int64_t)gridDim.x * (32 * k + l)) & 1 ? value : key;
                for (int64_t at = 0; at < page_bytes && ok; at += piece_bytes) {
                    const uint32_t st = loads % kCopyStages, bar = smem_addr(bars + st);
                    const uint32_t bytes = (uint32_t)min((int64_t)piece_bytes, page_bytes - at);
                    // the buffer's last store, kCopyStages pieces ago, has read it
                    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kCopyStages - kCopyAhead - 1) : "memory");
                    place[st].to = base + to + at;
                    place[st].bytes = bytes;
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_copy_g2s(smem_addr(buffers + st * piece_bytes), base + from + at, bytes, bar, policy);
                    if (++loads - stores > kCopyAhead) store_next();
                }
            }
        }
    }
    if (lane == 0) {
        while (stores != loads) store_next();
        if (!ok) {
            flag_error(status, kDevWaitTimeout);
            for (int i = 0; i < kCopyStages; ++i)        // what is still under way writes to this CTA's memory
                if (loads > (uint32_t)i) mbar_wait(smem_addr(bars + i), (loads - 1 - i) / kCopyStages & 1);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// -------------------------------------------------------------- the pool

__device__ __forceinline__ uint32_t tokens_of(const PoolArgs &a, uint32_t seq) {
    return (uint32_t)min((int64_t)a.context_lens[seq], (int64_t)a.max_blocks_per_seq * a.block_size);
}
__device__ __forceinline__ uint32_t pages_of(const PoolArgs &a, uint32_t tokens) {
    return (tokens + a.block_size - 1) / a.block_size;
}

// f(j, get(j)) for the entries j < n of one row, by a CTA of kRowThreads with
// four loads in flight per thread.
template <typename G, typename F>
__device__ __forceinline__ void for_entries(uint32_t n, G get, F f) {
    for (uint32_t j0 = threadIdx.x; j0 < n; j0 += kRowThreads * 4) {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = j0 + kRowThreads * k < n ? get(j0 + kRowThreads * k) : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j0 + kRowThreads * k < n) f(j0 + kRowThreads * k, b[k]);
    }
}

// Exclusive sum of x over the CTA's kPlanThreads threads, and its total.
__device__ unsigned long long scan_cta(unsigned long long x, unsigned long long &total) {
    __shared__ unsigned long long part[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += y;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    unsigned long long w = part[lane];                   // kPlanThreads / 32 == 32 warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const unsigned long long before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0ull;
    __syncthreads();                                     // part is free again
    return before + sum - x;
}

__global__ void __launch_bounds__(kPlanThreads) pool_init_kernel(PoolArgs a) {
    for (int64_t i = blockIdx.x * (int64_t)kPlanThreads + threadIdx.x; i < a.num_blocks;
         i += (int64_t)gridDim.x * kPlanThreads) {
        a.ref_counts[i] = 0;
        a.free_blocks[i] = (uint32_t)(a.num_blocks - 1 - i);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.num_free = (uint32_t)a.num_blocks;
}

// claim[seq] = the first request that names the row (workspace)
__device__ void claim_rows(const PoolArgs &a, const uint32_t *rows, int n, uint32_t *claim) {
    for (int i = threadIdx.x; i < a.num_seqs; i += kPlanThreads) claim[i] = kNone;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (rows[i] < (uint32_t)a.num_seqs) atomicMin(claim + rows[i], (uint32_t)i);
    __syncthreads();
}

// ---- fork: the child's row gets the parent's whole pages and, when the
// parent's last page is part full, a fresh page to copy that one into.
// info[i]: the child's tokens (kNone: refused) and its fresh page.
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(PoolArgs a, const uint32_t *parents, const uint32_t *children, int n, uint32_t *copy_src,
                 uint32_t *copy_dst, uint32_t *claim, uint2 *info) {
    claim_rows(a, children, n, claim);
    const uint32_t top = (uint32_t)min((int64_t)*a.num_free, a.num_blocks);
    unsigned long long base = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        uint32_t tokens = 0, open = kNone;
        bool ok = false;
        if (i < n) {
            const uint32_t p = parents[i], c = children[i];
            ok = p < (uint32_t)a.num_seqs && c < (uint32_t)a.num_seqs && p != c && claim[c] == (uint32_t)i &&
                 a.context_lens[c] == 0;
            if (!ok) flag_error(a.status, kDevBadSeq);
            if (ok) {
                tokens = tokens_of(a, p);
                if (tokens % a.block_size) {
                    open = a.block_tables[(int64_t)p * a.max_blocks_per_seq + tokens / a.block_size];
                    if (open >= a.num_blocks) {
                        flag_error(a.status, kDevBadBlock);
                        ok = false;
                    }
                }
            }
        }
        const bool takes = ok && open != kNone;
        unsigned long long total;
        const unsigned long long rank = base + scan_cta(takes ? 1ull : 0ull, total);
        base += total;
        uint32_t fresh = kNone;
        if (takes) {
            if (rank >= top) {
                flag_error(a.status, kDevNoBlock);
                ok = false;
            } else {
                fresh = a.free_blocks[top - 1 - (uint32_t)rank];
            }
        }
        if (i < n) {
            copy_src[i] = ok && takes ? open : kNone;
            copy_dst[i] = fresh;
            info[i] = make_uint2(ok ? tokens : kNone, fresh);
        }
    }
    __syncthreads();            // every length that decides anything has been read
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (info[i].x != kNone) a.context_lens[children[i]] = info[i].x;
    if (threadIdx.x == 0) *a.num_free = top - (uint32_t)min(base, (unsigned long long)top);
}

__global__ void __launch_bounds__(kRowThreads)
fork_rows_kernel(PoolArgs a, const uint32_t *parents, const uint32_t *children, const uint2 *info) {
    grid_dependency_wait();
    const uint2 t = info[blockIdx.x];
    if (t.x == kNone) return;
    const uint32_t *from = a.block_tables + (int64_t)parents[blockIdx.x] * a.max_blocks_per_seq;
    uint32_t *to = a.block_tables + (int64_t)children[blockIdx.x] * a.max_blocks_per_seq;
    const uint32_t whole = t.x / a.block_size;
    for_entries(whole, [&](uint32_t j) { return from[j]; }, [&](uint32_t j, uint32_t b) {
        to[j] = b;
        if (b < a.num_blocks) atomicAdd(a.ref_counts + b, 1u);
        else flag_error(a.status, kDevBadBlock);
    });
    if (threadIdx.x == 0 && t.x % a.block_size) {
        to[whole] = t.y;
        if (t.y < a.num_blocks) a.ref_counts[t.y] = 1;
        else flag_error(a.status, kDevBadBlock);
    }
}

// ---- extend: pages for a sequence's tokens up to a new length, popped in
// request order; growth within the last page needs none, whatever was refused
// before.  info[i]: pages held, pages added, the stack's top for it.
__global__ void __launch_bounds__(kPlanThreads)
extend_plan_kernel(PoolArgs a, const uint32_t *seqs, const uint32_t *new_lens, int n, uint32_t *claim, uint4 *info) {
    claim_rows(a, seqs, n, claim);
    const uint32_t top = (uint32_t)min((int64_t)*a.num_free, a.num_blocks);
    unsigned long long base = 0, taken = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        uint32_t held = 0, need = 0, s = 0, len = 0;
        bool grows = false;
        if (i < n) {
            s = seqs[i];
            len = new_lens[i];
            const bool ok = s < (uint32_t)a.num_seqs && claim[s] == (uint32_t)i &&
                            (int64_t)len <= (int64_t)a.max_blocks_per_seq * a.block_size;
            if (!ok) {
                flag_error(a.status, kDevBadSeq);
            } else if (len > tokens_of(a, s)) {
                grows = true;
                held = pages_of(a, tokens_of(a, s));
                need = pages_of(a, len) - held;
            }
        }
        unsigned long long total;
        const unsigned long long start = base + scan_cta(need, total);
        base += total;
        const bool fits = need == 0 || start + need <= top;
        if (grows && !fits) {
            flag_error(a.status, kDevNoBlock);
            need = 0;
        }
        if (grows && fits) a.context_lens[s] = len;
        if (i < n) info[i] = make_uint4(held, need, (uint32_t)(top - min(start, (unsigned long long)top)), 0u);
        unsigned long long used;
        scan_cta(need, used);
        taken += used;
    }
    if (threadIdx.x == 0) *a.num_free = top - (uint32_t)taken;
}

__global__ void __launch_bounds__(kRowThreads)
extend_rows_kernel(PoolArgs a, const uint32_t *seqs, const uint4 *info) {
    grid_dependency_wait();
    const uint4 t = info[blockIdx.x];
    if (!t.y) return;
    uint32_t *row = a.block_tables + (int64_t)seqs[blockIdx.x] * a.max_blocks_per_seq + t.x;
    for_entries(t.y, [&](uint32_t k) { return a.free_blocks[t.z - 1 - k]; }, [&](uint32_t k, uint32_t b) {
        row[k] = b;
        if (b < a.num_blocks) a.ref_counts[b] = 1;
        else flag_error(a.status, kDevBadBlock);
    });
}

// ---- free: one count less per page held.  A row's length is exchanged for
// zero by the request that frees it: named twice, it has no pages the second
// time.
__global__ void __launch_bounds__(kRowThreads) free_rows_kernel(PoolArgs a, const uint32_t *seqs) {
    __shared__ uint32_t pages;
    const uint32_t s = seqs[blockIdx.x];
    grid_dependents_launch();
    if (s >= (uint32_t)a.num_seqs) {
        if (threadIdx.x == 0) flag_error(a.status, kDevBadSeq);
        return;
    }
    if (threadIdx.x == 0) {
        const uint32_t len = atomicExch(a.context_lens + s, 0u);
        pages = pages_of(a, (uint32_t)min((int64_t)len, (int64_t)a.max_blocks_per_seq * a.block_size));
    }
    __syncthreads();
    const uint32_t held = pages;
    const uint32_t *row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
    for_entries(held, [&](uint32_t j) { return row[j]; }, [&](uint32_t, uint32_t b) {
        if (b >= a.num_blocks) {
            flag_error(a.status, kDevBadBlock);
            return;
        }
        const uint32_t old = atomicSub(a.ref_counts + b, 1u);
        if (old == 0 || old >= kOver) {
            atomicAdd(a.ref_counts + b, 1u);
            flag_error(a.status, kDevBadBlock);
        } else if (old == 1) {
            atomicAdd(a.ref_counts + b, kFreedMark);
        }
    });
}

// The page numbers are cut into one run per warp of a cluster of eight CTAs.
// A warp counts its run with ballots, the counts of all go into a table in
// every CTA through distributed shared memory, and each warp adds up the ones
// before its own: one exchange, and no barrier inside a run.  (Sweeps of a
// whole CTA with a scan after each: 12.5 us against 6.3 for
// what a free puts back and 20 against 11 for a compaction's plan, in a pool of
// 52,000 pages.)
constexpr int kCluster = 8;
constexpr int kRuns = kCluster * kPlanThreads / 32;

struct Run {
    int id;
    int64_t lo, hi, per;
};
__device__ __forceinline__ Run run_of(const cg::cluster_group &cl, int64_t num_blocks) {
    Run r;
    r.id = (int)cl.block_rank() * (kPlanThreads / 32) + (threadIdx.x >> 5);
    r.per = (num_blocks + kRuns * 32 - 1) / (kRuns * 32) * 32;
    r.lo = min(num_blocks, r.per * r.id);
    r.hi = min(num_blocks, r.lo + r.per);
    return r;
}

// f(page, its count, warp-wide) for the pages [lo, hi) in steps of 32, four
// loads in flight; lanes behind hi get count 0 and page >= hi.
template <typename F>
__device__ __forceinline__ void for_pages(const uint32_t *ref_counts, int64_t lo, int64_t hi, F f) {
    for (int64_t b0 = lo + (threadIdx.x & 31); b0 - (threadIdx.x & 31) < hi; b0 += 128) {
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = b0 + 32 * k < hi ? ref_counts[b0 + 32 * k] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) f(b0 + 32 * k, c[k]);
    }
}

// Puts a run's count into the table of every CTA.  The cluster's CTAs have all
// arrived at its barrier once before.
__device__ __forceinline__ void share_count(cg::cluster_group &cl, uint32_t *counts, int id, uint32_t mine) {
    const int lane = threadIdx.x & 31;
    cl.barrier_wait();                                   // every CTA runs
    if (lane < kCluster) *cl.map_shared_rank(&counts[id], lane) = mine;
    cl.sync();
}

// The sum of the counts of the runs before run `id`.
__device__ __forceinline__ uint32_t count_before(const uint32_t *counts, int id) {
    uint32_t sum = 0;
    for (int r = threadIdx.x & 31; r < id; r += 32) sum += counts[r];
    return __reduce_add_sync(0xFFFFFFFFu, sum);
}

// The pages freed in this call go onto the stack, lowest number first.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kPlanThreads) free_push_kernel(PoolArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();
    const Run run = run_of(cl, a.num_blocks);
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
    grid_dependency_wait();
    const uint32_t top = (uint32_t)min((int64_t)*a.num_free, a.num_blocks);
    __shared__ uint32_t counts[kRuns];
    uint32_t mine = 0;
    for_pages(a.ref_counts, run.lo, run.hi, [&](int64_t, uint32_t c) {
        mine += __popc(__ballot_sync(0xFFFFFFFFu, c == kFreedMark));
    });
    share_count(cl, counts, run.id, mine);               // (and every CTA has read the top)
    uint32_t at = top + count_before(counts, run.id);
    if (mine)
        for_pages(a.ref_counts, run.lo, run.hi, [&](int64_t b, uint32_t c) {
            const uint32_t freed = __ballot_sync(0xFFFFFFFFu, c == kFreedMark);
            const uint32_t to = at + __popc(freed & below);
            if (c == kFreedMark) {
                a.ref_counts[b] = 0;
                if (to < a.num_blocks) a.free_blocks[to] = (uint32_t)b;
                else flag_error(a.status, kDevBadBlock);      // more free pages than the pool has
            }
            at += __popc(freed);
        });
    if (run.id == 0) {
        const uint32_t total = count_before(counts, kRuns);
        if (threadIdx.x == 0) *a.num_free = (uint32_t)min((int64_t)top + total, a.num_blocks);
    }
}

// ---- compact: with L pages held, the k-th held page >= L moves to the k-th
// free page < L.  remap[b] for every b >= L: where it went, or b itself.
//
// Below L a run's first free page has rank lo - (pages held before the run);
// above L its first held page has rank (held before the run) - (held below L),
// and the last term needs a count of only the run that L falls into, which
// every warp makes for itself.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kPlanThreads)
compact_plan_kernel(PoolArgs a, uint32_t *move_src, uint32_t *move_dst, int64_t capacity, uint32_t *remap) {
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_arrive();
    const Run run = run_of(cl, a.num_blocks);
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
    __shared__ uint32_t counts[kRuns];
    uint32_t mine = 0;
    for_pages(a.ref_counts, run.lo, run.hi, [&](int64_t, uint32_t c) {
        mine += __popc(__ballot_sync(0xFFFFFFFFu, c != 0));
    });
    share_count(cl, counts, run.id, mine);
    const uint32_t live = count_before(counts, kRuns), held_before = count_before(counts, run.id);
    const int split = (int)(live / run.per);             // run.per >= 32; kRuns when the pool is full
    uint32_t held_below = count_before(counts, split);
    for_pages(a.ref_counts, min(a.num_blocks, run.per * split), (int64_t)live, [&](int64_t, uint32_t c) {
        held_below += __popc(__ballot_sync(0xFFFFFFFFu, c != 0));
    });
    const uint32_t moves = live - held_below;
    uint32_t at_hole = (uint32_t)run.lo - held_before, at_mover = max(held_before, held_below) - held_below;
    for_pages(a.ref_counts, run.lo, run.hi, [&](int64_t b, uint32_t c) {
        const bool hole = c == 0 && b < min((int64_t)live, run.hi), mover = c != 0 && b >= live;
        const uint32_t holes = __ballot_sync(0xFFFFFFFFu, hole), movers = __ballot_sync(0xFFFFFFFFu, mover);
        if (hole) move_dst[at_hole + __popc(holes & below)] = (uint32_t)b;
        if (mover) move_src[at_mover + __popc(movers & below)] = (uint32_t)b;
        if (b >= live && b < run.hi) remap[b] = (uint32_t)b;
        at_hole += __popc(holes);
        at_mover += __popc(movers);
    });
    cl.sync();                                           // both lists and remap stand
    const int64_t step = (int64_t)kCluster * kPlanThreads;
    for (int64_t k = (int64_t)cl.block_rank() * kPlanThreads + threadIdx.x; k < max(capacity, a.num_blocks); k += step) {
        if (k < moves) {
            const uint32_t s = move_src[k], d = move_dst[k];
            remap[s] = d;
            a.ref_counts[d] = a.ref_counts[s];
            a.ref_counts[s] = 0;
        } else if (k < capacity) {
            move_src[k] = move_dst[k] = kNone;
        }
        if (k < a.num_blocks) a.free_blocks[k] = k < a.num_blocks - live ? (uint32_t)(a.num_blocks - 1 - k) : kNone;
    }
    if (cl.block_rank() == 0 && threadIdx.x == 0) *a.num_free = (uint32_t)(a.num_blocks - live);
}

__global__ void __launch_bounds__(kRowThreads) compact_rows_kernel(PoolArgs a, const uint32_t *remap) {
    grid_dependency_wait();
    const uint32_t live = (uint32_t)a.num_blocks - *a.num_free;
    for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        uint32_t *row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
        const uint32_t held = pages_of(a, tokens_of(a, s));
        for_entries(held, [&](uint32_t j) { return row[j]; }, [&](uint32_t j, uint32_t b) {
            if (b >= a.num_blocks) flag_error(a.status, kDevBadBlock);
            else if (b >= live) row[j] = remap[b];
        });
    }
}

// The second launch of an operator may begin while the first one drains.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

size_t pool_workspace_bytes(int num_seqs, int64_t num_blocks, int num_requests) {
    const size_t requests = up16((size_t)num_requests * sizeof(uint4)) + up16((size_t)num_seqs * 4);
    const size_t pages = up16((size_t)num_blocks * 4);
    return requests > pages ? requests : pages;
}

cudaError_t launch_copy_pages(uint32_t *key, uint32_t *value, const uint32_t *src, const uint32_t *dst, int64_t pairs,
                              int64_t page_bytes, int64_t num_blocks, int num_sms, uint32_t *status,
                              cudaStream_t st) {
    const int64_t pieces = (page_bytes + kCopyPiece - 1) / kCopyPiece;
    const uint32_t piece = (uint32_t)(((page_bytes + pieces - 1) / pieces + 15) / 16 * 16);
    const int64_t most = (int64_t)num_sms * kCopyPerSm;
    const unsigned grid = (unsigned)(pairs * 2 < most ? pairs * 2 : most);
    const int smem = (int)(piece * kCopyStages);
    cudaError_t e = cudaFuncSetAttribute(copy_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kCopyPiece * kCopyStages);
    if (e != cudaSuccess) return e;
    copy_pages_kernel<<<grid, 32, smem, st>>>(reinterpret_cast<char *>(key), reinterpret_cast<char *>(value), src, dst,
                                              pairs, page_bytes, piece, num_blocks, status);
    return cudaGetLastError();
}

cudaError_t launch_pool_init(const PoolArgs &a, cudaStream_t st) {
    const int64_t grid = (a.num_blocks + kPlanThreads - 1) / kPlanThreads;
    pool_init_kernel<<<(unsigned)(grid < 256 ? grid : 256), kPlanThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_fork(const PoolArgs &a, const uint32_t *parents, const uint32_t *children, int n, uint32_t *copy_src,
                        uint32_t *copy_dst, void *workspace, cudaStream_t st) {
    uint2 *info = static_cast<uint2 *>(workspace);
    uint32_t *claim = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + up16((size_t)n * sizeof(uint4)));
    fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, parents, children, n, copy_src, copy_dst, claim, info);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(fork_rows_kernel, dim3(n), kRowThreads, st, a, parents, children,
                                               static_cast<const uint2 *>(info));
}

cudaError_t launch_extend(const PoolArgs &a, const uint32_t *seqs, const uint32_t *new_lens, int n, void *workspace,
                          cudaStream_t st) {
    uint4 *info = static_cast<uint4 *>(workspace);
    uint32_t *claim = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + up16((size_t)n * sizeof(uint4)));
    extend_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, seqs, new_lens, n, claim, info);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(extend_rows_kernel, dim3(n), kRowThreads, st, a, seqs,
                                               static_cast<const uint4 *>(info));
}

cudaError_t launch_free(const PoolArgs &a, const uint32_t *seqs, int n, cudaStream_t st) {
    free_rows_kernel<<<n, kRowThreads, 0, st>>>(a, seqs);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(free_push_kernel, dim3(kCluster), kPlanThreads, st, a);
}

cudaError_t launch_compact(const PoolArgs &a, uint32_t *move_src, uint32_t *move_dst, int64_t capacity,
                           void *workspace, cudaStream_t st) {
    uint32_t *remap = static_cast<uint32_t *>(workspace);
    compact_plan_kernel<<<kCluster, kPlanThreads, 0, st>>>(a, move_src, move_dst, capacity, remap);
    const cudaError_t e = cudaGetLastError();
    const int grid = a.num_seqs < 1024 ? a.num_seqs : 1024;
    return e != cudaSuccess ? e : launch_after(compact_rows_kernel, dim3(grid), kRowThreads, st, a,
                                               static_cast<const uint32_t *>(remap));
}

}  // namespace pa_q8
