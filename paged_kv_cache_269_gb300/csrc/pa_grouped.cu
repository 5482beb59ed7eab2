// pa_grouped.cu -- attention of query heads that share K/V heads over the
// paged cache, with capped scores, a bias by distance, a window and a prefix.
//
// One warp per (query row, query head): lanes share the head's dims, keys are
// visited in order with an fp32 running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ __forceinline__ float widen(uint16_t u, bool bf16) {
    if (bf16) return __uint_as_float(static_cast<uint32_t>(u) << 16);
    return __half2float(*reinterpret_cast<const __half *>(&u));
}
__device__ __forceinline__ uint16_t narrow(float x, bool bf16) {
    if (bf16) {
        const __nv_bfloat16 b = __float2bfloat16_rn(x);
        return *reinterpret_cast<const uint16_t *>(&b);
    }
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t *>(&h);
}

template <int D>
__global__ void __launch_bounds__(128) attend_rows_kernel(const GroupedArgs a, bool bf16) {
    allow_dependents_to_launch();
    grid_dependency_wait();
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int s = blockIdx.x / a.num_q_heads, h = blockIdx.x % a.num_q_heads;
    const int hk = h / (a.num_q_heads / a.num_kv_heads);
    int ctx = a.context_lens[s];
    int first = s, count = 1;
    const bool ctx_bad = ctx < 0 || ctx > a.max_blocks_per_seq * a.block_size;
    if (a.query_start) {
        first = a.query_start[s];
        const int end = a.query_start[s + 1];
        const bool rows_bad = first < 0 || end < first || end > a.total_q;
        count = rows_bad ? 0 : end - first;
        if (rows_bad || (count > 0 && (ctx_bad || count > ctx || count > a.max_q))) {
            if (h == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_CONTEXT);
            return;
        }
    } else if (ctx_bad) {
        if (h == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_CONTEXT);
        ctx = 0;
    }
    const int pre = a.prefix_lens ? max(0, min(a.prefix_lens[s], ctx)) : 0;
    const float slope = a.alibi_slopes ? a.alibi_slopes[h] : 0.f;
    for (int i = blockIdx.y * 4 + warp; i < count; i += gridDim.y * 4) {
        const int p = ctx - count + i;
        const int lo = a.window ? max(0, p - a.window + 1) : 0;
        const size_t row = (static_cast<size_t>(first + i) * a.num_q_heads + h) * D;
        float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[e] = widen(a.q[row + lane * E + e], bf16);
            acc[e] = 0.f;
        }
        const int stop = max(p + 1, pre);
        for (int j = pre > 0 ? 0 : lo; j < stop; ++j) {
            if (j >= pre && j < lo) j = lo;
            if (j >= pre && j > p) break;
            const int blk = a.block_tables[static_cast<size_t>(s) * a.max_blocks_per_seq + j / a.block_size];
            if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.num_blocks)) {
                if (lane == 0) atomicOr(a.err, PA_DEVERR_TABLE);
                continue;
            }
            const size_t kv = ((static_cast<size_t>(blk) * a.num_kv_heads + hk) * a.block_size +
                               j % a.block_size) * D + lane * E;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x += q[e] * widen(a.k_cache[kv + e], bf16);
#pragma unroll
            for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
            x *= a.scale;
            if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
            x -= slope * fabsf(static_cast<float>(p - j));
            const float mn = fmaxf(m, x), r = m == -INFINITY ? 0.f : expf(m - mn), w = expf(x - mn);
            m = mn;
            l = l * r + w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = acc[e] * r + w * widen(a.v_cache[kv + e], bf16);
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            a.out[row + lane * E + e] = narrow(l > 0.f ? acc[e] / l : 0.f, bf16);
    }
}

cudaError_t launch_rows(const GroupedArgs &a, int dtype, int head_dim, int rows, cudaStream_t s) {
    void (*kernel)(GroupedArgs, bool) = head_dim == 64    ? attend_rows_kernel<64>
                                        : head_dim == 128 ? attend_rows_kernel<128>
                                                          : attend_rows_kernel<256>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int y = (rows + 3) / 4;
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs * a.num_q_heads), y < 1024 ? y : 1024);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, dtype == PA_DTYPE_BF16);
}

}  // namespace

bool prefill_grouped_supported(int dtype, int head_dim, int block_size, int group) {
    return decode_variant_supported(dtype, head_dim, block_size) && head_dim != 256 && group <= 128;
}
size_t prefill_grouped_workspace_bytes(int, int, int, int, int) { return 0; }
size_t prefill_grouped_counters_bytes() { return 256; }

cudaError_t launch_prefill_grouped(const GroupedArgs &args, int dtype, int head_dim, int,
                                   cudaStream_t stream) {
    return launch_rows(args, dtype, head_dim, args.max_q, stream);
}

}  // namespace pa
