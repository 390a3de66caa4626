// Prompt attention over the paged int8 caches (pa_q8_prefill).
//
// A warp per (row, head): the row's visible tokens one after the other, the
// head's dimensions spread over the lanes, running maximum and sum of the
// softmax in f32.
#include <cuda_bf16.h>

#include "device_util.cuh"
#include "kernels.h"
#include "pa_q8.h"

namespace pa_q8 {
namespace {

template <typename T> __device__ float to_f32(T x);
template <> __device__ float to_f32(float x) { return x; }
template <> __device__ float to_f32(__half x) { return __half2float(x); }
template <> __device__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ T from_f32(float x);
template <> __device__ float from_f32(float x) { return x; }
template <> __device__ __half from_f32(float x) { return __float2half_rn(x); }
template <> __device__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(128) prefill_rows_kernel(PrefillArgs a) {
    constexpr int W = D / 4 + 1, PER = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (item >= a.num_rows * a.num_heads) return;
    const int64_t row = item / a.num_heads;
    const int head = (int)(item % a.num_heads), g = head / (a.num_heads / a.num_kv_heads);
    // the sequence whose bounds hold this row
    for (int s = 0; s < a.num_seqs; ++s) {
        const uint32_t lo = a.query_starts[s], hi = a.query_starts[s + 1];
        if (hi < lo || hi > a.num_rows) {
            if (lane == 0) flag_error(a.status, kDevBadRows);
            continue;
        }
        if (row < lo || row >= hi) continue;
        const int64_t c = min((int64_t)a.context_lens[s], (int64_t)a.max_blocks_per_seq * a.block_size);
        const int64_t sees = c - (hi - 1 - row);
        float q[PER], o[PER], m = -INFINITY, l = 0.0f;
        for (int k = 0; k < PER; ++k) {
            q[k] = to_f32(static_cast<const T *>(a.q)[row * a.q_stride + head * D + lane * PER + k]);
            o[k] = 0.0f;
        }
        for (int64_t t = 0; t < sees; ++t) {
            const uint32_t b = a.block_tables[(int64_t)s * a.max_blocks_per_seq + t / a.block_size];
            if (b >= a.num_blocks) {
                if (lane == 0) flag_error(a.status, kDevBadBlock);
                continue;
            }
            const int64_t at = (((int64_t)b * a.num_kv_heads + g) * a.block_size + t % a.block_size) * W;
            const int8_t *k8 = reinterpret_cast<const int8_t *>(a.key_cache + at) + lane * PER;
            const int8_t *v8 = reinterpret_cast<const int8_t *>(a.value_cache + at) + lane * PER;
            float z = 0.0f;
            for (int k = 0; k < PER; ++k) z += q[k] * (float)k8[k];
            for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
            z *= __uint_as_float(a.key_cache[at + W - 1]) * a.scale;
            const float m2 = fmaxf(m, z), f = m == -INFINITY ? 0.0f : expf(m - m2), p = expf(z - m2);
            const float vs = __uint_as_float(a.value_cache[at + W - 1]);
            l = l * f + p;
            for (int k = 0; k < PER; ++k) o[k] = o[k] * f + p * vs * (float)v8[k];
            m = m2;
        }
        for (int k = 0; k < PER; ++k)
            static_cast<T *>(a.out)[row * a.out_stride + head * D + lane * PER + k] =
                from_f32<T>(l == 0.0f ? 0.0f : o[k] / l);
        return;
    }
}

template <typename T>
cudaError_t launch_typed(const PrefillArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.num_rows * a.num_heads + 3) / 4);
    if (a.head_size == 64) prefill_rows_kernel<T, 64><<<grid, 128, 0, st>>>(a);
    else if (a.head_size == 128) prefill_rows_kernel<T, 128><<<grid, 128, 0, st>>>(a);
    else prefill_rows_kernel<T, 256><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t prefill_workspace_bytes(const PrefillArgs &) { return 16; }

cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t st) {
    if (a.dtype == PA_Q8_F32) return launch_typed<float>(a, st);
    if (a.dtype == PA_Q8_F16) return launch_typed<__half>(a, st);
    return launch_typed<__nv_bfloat16>(a, st);
}

}  // namespace pa_q8
