// pa_gather.cu -- gather_cache_q8: tokens of an 8-bit paged cache read back as
// 16-bit rows.
//
// out[i, h] = code(slot_i, h) * scale_h for K and V, the product in fp32 and
// rounded once.  1 byte in and 2 out per element, one flop: bound by HBM.
//
// One thread moves 16 codes (one 16-byte load, two 16-byte stores); the chunks
// of a token's K then V rows lie side by side in its index, so the stores of a
// warp are whole rows of the output.  A CTA takes kTokens neighbouring tokens,
// which usually share a block, and asks for several chunks before it stores the
// first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <bool kBf16>
__device__ __forceinline__ uint32_t scaled(uint32_t f16x2, float scale) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&f16x2));
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(f.x * scale, f.y * scale);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) gather_q8_kernel(const GatherArgs a, int chunks, long long total) {
    allow_dependents_to_launch();
    grid_dependency_wait();
    // chunk index: ((token * 2 + matrix) * H + head) * chunks + chunk
    const int per_matrix = a.num_kv_heads * chunks;
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    uint4 codes[kUnroll];
    float scale[kUnroll];
    uint4 *dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long long i = first + u * kThreads;
        dst[u] = nullptr;
        if (i >= total) continue;
        const int token = static_cast<int>(i / (2 * per_matrix));
        int rest = static_cast<int>(i - static_cast<long long>(token) * (2 * per_matrix));
        const bool is_v = rest >= per_matrix;
        if (is_v) rest -= per_matrix;
        const int slot = __ldg(a.slots + token);
        if (slot < 0) continue;
        if (slot >= a.pool_slots) {
            if (rest == 0 && !is_v) atomicOr(a.err, PA_DEVERR_SLOT);
            continue;
        }
        const int h = rest / chunks, c = rest - h * chunks;
        const size_t row = (static_cast<size_t>(slot / a.block_size) * a.num_kv_heads + h) * a.block_size +
                           slot % a.block_size;
        codes[u] = __ldg(reinterpret_cast<const uint4 *>(is_v ? a.v_cache : a.k_cache) + row * chunks + c);
        scale[u] = __ldg((is_v ? a.v_scales : a.k_scales) + h);
        dst[u] = reinterpret_cast<uint4 *>(is_v ? a.v_out : a.k_out) +
                 2 * (static_cast<size_t>(token) * per_matrix + rest);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (!dst[u]) continue;
        const uint32_t w[4] = {codes[u].x, codes[u].y, codes[u].z, codes[u].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = scaled<kBf16>(e4m3x2_to_f16x2(w[i]), scale[u]);
            o[2 * i + 1] = scaled<kBf16>(e4m3x2_to_f16x2_high(w[i]), scale[u]);
        }
        dst[u][0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[u][1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

cudaError_t launch_gather_q8(const GatherArgs &args, int dtype, cudaStream_t stream) {
    const int chunks = args.head_dim / 16;
    const long long total = static_cast<long long>(args.num_tokens) * 2 * args.num_kv_heads * chunks;
    const long long blocks = (total + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dtype == PA_DTYPE_BF16 ? gather_q8_kernel<true> : gather_q8_kernel<false>, args,
                              chunks, total);
}

}  // namespace pa
