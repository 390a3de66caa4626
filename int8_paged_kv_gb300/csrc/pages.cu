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
constexpr uint32_t kNone = 0xFFFFFFFFu;
// A page whose count reached zero in this call carries this mark until the
// stack takes it.  The mark and every correction are additions, so they
// commute: a second release of the same page (a caller error) takes the
// count below the mark or below zero, is seen as such (>= kOver) and adds
// back the one it took.
constexpr uint32_t kFreedMark = 0x40000000u;
constexpr uint32_t kOver = 0x20000000u;

// ------------------------------------------------------------ page copies

constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 4;                            // 16-byte loads in flight per thread

// Pair p copies page src[p] to dst[p] of both caches.  Units of
// kCopyThreads * kCopyBatch * 16 bytes (16 KB) go round the grid.
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(uint4 *key, uint4 *value, const uint32_t *src, const uint32_t *dst, int64_t pairs,
                  int64_t page_vecs, int64_t num_blocks, uint32_t *status) {
    constexpr int kUnit = kCopyThreads * kCopyBatch;
    const int64_t pieces = (page_vecs + kUnit - 1) / kUnit;
    const int64_t units = pairs * 2 * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t p = u / (2 * pieces);
        const int64_t r = u - p * 2 * pieces;
        const uint32_t s = src[p], d = dst[p];
        if (s == kNone || d == kNone) continue;
        if (s >= num_blocks || d >= num_blocks) {
            if (threadIdx.x == 0) flag_error(status, kDevBadBlock);
            continue;
        }
        uint4 *base = r < pieces ? key : value;
        const int64_t v0 = (r < pieces ? r : r - pieces) * kUnit + threadIdx.x;
        const uint4 *from = base + (int64_t)s * page_vecs;
        uint4 *to = base + (int64_t)d * page_vecs;
        uint4 x[kCopyBatch];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (v0 + k * kCopyThreads < page_vecs) x[k] = from[v0 + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (v0 + k * kCopyThreads < page_vecs) to[v0 + k * kCopyThreads] = x[k];
    }
}

// -------------------------------------------------------------- the pool

__device__ __forceinline__ uint32_t tokens_of(const PoolArgs &a, uint32_t seq) {
    return (uint32_t)min((int64_t)a.context_lens[seq], (int64_t)a.max_blocks_per_seq * a.block_size);
}
__device__ __forceinline__ uint32_t pages_of(const PoolArgs &a, uint32_t tokens) {
    return (tokens + a.block_size - 1) / a.block_size;
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

__global__ void __launch_bounds__(128)
fork_rows_kernel(PoolArgs a, const uint32_t *parents, const uint32_t *children, const uint2 *info) {
    grid_dependency_wait();
    const uint2 t = info[blockIdx.x];
    if (t.x == kNone) return;
    const uint32_t *from = a.block_tables + (int64_t)parents[blockIdx.x] * a.max_blocks_per_seq;
    uint32_t *to = a.block_tables + (int64_t)children[blockIdx.x] * a.max_blocks_per_seq;
    const uint32_t whole = t.x / a.block_size;
    for (uint32_t j = threadIdx.x; j < whole; j += blockDim.x) {
        const uint32_t b = from[j];
        to[j] = b;
        if (b < a.num_blocks) atomicAdd(a.ref_counts + b, 1u);
        else flag_error(a.status, kDevBadBlock);
    }
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

__global__ void __launch_bounds__(128)
extend_rows_kernel(PoolArgs a, const uint32_t *seqs, const uint4 *info) {
    grid_dependency_wait();
    const uint4 t = info[blockIdx.x];
    if (!t.y) return;
    uint32_t *row = a.block_tables + (int64_t)seqs[blockIdx.x] * a.max_blocks_per_seq + t.x;
    for (uint32_t k = threadIdx.x; k < t.y; k += blockDim.x) {
        const uint32_t b = a.free_blocks[t.z - 1 - k];
        row[k] = b;
        if (b < a.num_blocks) a.ref_counts[b] = 1;
        else flag_error(a.status, kDevBadBlock);
    }
}

// ---- free: one count less per page held; a row named twice is freed once.
__global__ void __launch_bounds__(256) free_rows_kernel(PoolArgs a, const uint32_t *seqs, int n) {
    const int i = blockIdx.x;
    const uint32_t s = seqs[i];
    grid_dependents_launch();
    if (s >= (uint32_t)a.num_seqs) {
        if (threadIdx.x == 0) flag_error(a.status, kDevBadSeq);
        return;
    }
    bool again = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) again |= seqs[j] == s;
    if (__syncthreads_or(again)) return;
    const uint32_t held = pages_of(a, tokens_of(a, s));
    const uint32_t *row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
    for (uint32_t j = threadIdx.x; j < held; j += blockDim.x) {
        const uint32_t b = row[j];
        if (b >= a.num_blocks) {
            flag_error(a.status, kDevBadBlock);
            continue;
        }
        const uint32_t old = atomicSub(a.ref_counts + b, 1u);
        if (old == 0 || old >= kOver) {
            atomicAdd(a.ref_counts + b, 1u);
            flag_error(a.status, kDevBadBlock);
        } else if (old == 1) {
            atomicAdd(a.ref_counts + b, kFreedMark);
        }
    }
    __syncthreads();                                     // the length was read
    if (threadIdx.x == 0) a.context_lens[s] = 0;
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

__global__ void __launch_bounds__(256) compact_rows_kernel(PoolArgs a, const uint32_t *remap) {
    grid_dependency_wait();
    const uint32_t live = (uint32_t)a.num_blocks - *a.num_free;
    for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        uint32_t *row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
        const uint32_t held = pages_of(a, tokens_of(a, s));
        for (uint32_t j = threadIdx.x; j < held; j += blockDim.x) {
            const uint32_t b = row[j];
            if (b >= a.num_blocks) flag_error(a.status, kDevBadBlock);
            else if (b >= live) row[j] = remap[b];
        }
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
    const int64_t vecs = page_bytes / 16, unit = kCopyThreads * kCopyBatch;
    const int64_t units = pairs * 2 * ((vecs + unit - 1) / unit);
    const int64_t grid = units < num_sms * 8 ? units : num_sms * 8;
    copy_pages_kernel<<<(unsigned)grid, kCopyThreads, 0, st>>>(reinterpret_cast<uint4 *>(key),
                                                               reinterpret_cast<uint4 *>(value), src, dst, pairs,
                                                               vecs, num_blocks, status);
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
    return e != cudaSuccess ? e : launch_after(fork_rows_kernel, dim3(n), 128, st, a, parents, children,
                                               static_cast<const uint2 *>(info));
}

cudaError_t launch_extend(const PoolArgs &a, const uint32_t *seqs, const uint32_t *new_lens, int n, void *workspace,
                          cudaStream_t st) {
    uint4 *info = static_cast<uint4 *>(workspace);
    uint32_t *claim = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + up16((size_t)n * sizeof(uint4)));
    extend_plan_kernel<<<1, kPlanThreads, 0, st>>>(a, seqs, new_lens, n, claim, info);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(extend_rows_kernel, dim3(n), 128, st, a, seqs,
                                               static_cast<const uint4 *>(info));
}

cudaError_t launch_free(const PoolArgs &a, const uint32_t *seqs, int n, cudaStream_t st) {
    free_rows_kernel<<<n, 256, 0, st>>>(a, seqs, n);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_after(free_push_kernel, dim3(kCluster), kPlanThreads, st, a);
}

cudaError_t launch_compact(const PoolArgs &a, uint32_t *move_src, uint32_t *move_dst, int64_t capacity,
                           void *workspace, cudaStream_t st) {
    uint32_t *remap = static_cast<uint32_t *>(workspace);
    compact_plan_kernel<<<kCluster, kPlanThreads, 0, st>>>(a, move_src, move_dst, capacity, remap);
    const cudaError_t e = cudaGetLastError();
    const int grid = a.num_seqs < 1024 ? a.num_seqs : 1024;
    return e != cudaSuccess ? e : launch_after(compact_rows_kernel, dim3(grid), 256, st, a,
                                               static_cast<const uint32_t *>(remap));
}

}  // namespace pa_q8
