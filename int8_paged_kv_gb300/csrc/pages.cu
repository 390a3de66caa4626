// Pages of a cache: copying them, and the pool that says who holds them
// (reference counts, a stack of free pages, the sequences' block tables).
//
// The pool operators are whole-number bookkeeping over a few hundred KB that
// sits in L2, so their time is launches and dependent loads, not bytes.  Each
// is one or two launches: a planning CTA that decides for all requests in
// order (a scan), then a CTA per request that touches the tables.  Results do
// not depend on the order in which CTAs run: every decision that depends on
// other requests is a scan over the request index or the page number, and
// the only atomics are whole-number sums and minima.
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
// request order.  info[i]: pages held, pages added, the stack's top for it.
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
        const bool fits = start + need <= top;
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

// The exclusive sum over a cluster's CTAs of per-CTA counts, and the total:
// every CTA writes its count into rank 0..7's table through shared memory.
constexpr int kCluster = 8;
__device__ uint32_t scan_cluster(cg::cluster_group &cl, uint32_t mine, uint32_t &total) {
    __shared__ uint32_t counts[kCluster];
    cl.sync();                                           // the table is free in every CTA
    if (threadIdx.x < kCluster) *cl.map_shared_rank(&counts[cl.block_rank()], threadIdx.x) = mine;
    cl.sync();
    uint32_t before = 0;
    total = 0;
    for (int r = 0; r < kCluster; ++r) {
        if (r < (int)cl.block_rank()) before += counts[r];
        total += counts[r];
    }
    return before;
}

// A CTA's share of the pages, in whole sweeps of its threads.
__device__ __forceinline__ void share_of(int64_t num_blocks, int rank, int64_t &lo, int64_t &hi) {
    const int64_t per = (num_blocks + kCluster * (int64_t)kPlanThreads - 1) / (kCluster * (int64_t)kPlanThreads) *
                        kPlanThreads;
    lo = min(num_blocks, per * rank);
    hi = min(num_blocks, lo + per);
}

// The pages freed in this call go onto the stack, lowest number first.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kPlanThreads) free_push_kernel(PoolArgs a) {
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    int64_t lo, hi;
    share_of(a.num_blocks, cl.block_rank(), lo, hi);
    const uint32_t top = (uint32_t)min((int64_t)*a.num_free, a.num_blocks);
    uint32_t n = 0;
    for (int64_t b = lo + threadIdx.x; b < hi; b += kPlanThreads) n += a.ref_counts[b] == kFreedMark;
    unsigned long long mine;
    scan_cta(n, mine);
    uint32_t total;
    uint32_t at = top + scan_cluster(cl, (uint32_t)mine, total);
    for (int64_t b0 = lo; b0 < hi; b0 += kPlanThreads) {
        const int64_t b = b0 + threadIdx.x;
        const bool freed = b < hi && a.ref_counts[b] == kFreedMark;
        unsigned long long here;
        const unsigned long long k = scan_cta(freed, here);
        if (freed) {
            a.ref_counts[b] = 0;
            if (at + k < a.num_blocks) a.free_blocks[at + k] = (uint32_t)b;
            else flag_error(a.status, kDevBadBlock);     // more free pages than the pool has
        }
        at += (uint32_t)here;
    }
    cl.sync();                                           // every CTA has read the top
    if (cl.block_rank() == 0 && threadIdx.x == 0) *a.num_free = (uint32_t)min((int64_t)top + total, a.num_blocks);
}

// ---- compact: with L pages held, the k-th held page >= L moves to the k-th
// free page < L.  remap[b] for every b >= L: where it went, or b itself.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kPlanThreads)
compact_plan_kernel(PoolArgs a, uint32_t *move_src, uint32_t *move_dst, int64_t capacity, uint32_t *remap) {
    cg::cluster_group cl = cg::this_cluster();
    int64_t lo, hi;
    share_of(a.num_blocks, cl.block_rank(), lo, hi);
    uint32_t n = 0;
    for (int64_t b = lo + threadIdx.x; b < hi; b += kPlanThreads) n += a.ref_counts[b] != 0;
    unsigned long long mine;
    scan_cta(n, mine);
    uint32_t live;
    scan_cluster(cl, (uint32_t)mine, live);
    uint32_t holes = 0, movers = 0;
    for (int64_t b = lo + threadIdx.x; b < hi; b += kPlanThreads) {
        const bool used = a.ref_counts[b] != 0;
        holes += !used && b < live;
        movers += used && b >= live;
    }
    unsigned long long both;
    scan_cta((unsigned long long)holes << 32 | movers, both);
    uint32_t moves, same;
    uint32_t at_hole = scan_cluster(cl, (uint32_t)(both >> 32), moves);
    uint32_t at_mover = scan_cluster(cl, (uint32_t)both, same);
    for (int64_t b0 = lo; b0 < hi; b0 += kPlanThreads) {
        const int64_t b = b0 + threadIdx.x;
        const bool in = b < hi;
        const bool used = in && a.ref_counts[b] != 0;
        const bool hole = in && !used && b < live, mover = used && b >= live;
        unsigned long long here;
        const unsigned long long k = scan_cta((unsigned long long)hole << 32 | (mover ? 1u : 0u), here);
        if (hole) move_dst[at_hole + (uint32_t)(k >> 32)] = (uint32_t)b;
        if (mover) move_src[at_mover + (uint32_t)k] = (uint32_t)b;
        if (in && b >= live) remap[b] = (uint32_t)b;
        at_hole += (uint32_t)(here >> 32);
        at_mover += (uint32_t)here;
    }
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
