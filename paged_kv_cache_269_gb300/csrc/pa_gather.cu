// pa_gather.cu -- gather_cache_q8: tokens of an 8-bit paged cache read back as
// 16-bit rows.
//
// out[i, h] = code(slot_i, h) * scale_h for K and V, the product in fp32 and
// rounded once.  1 byte in and 2 out per element, one flop: bound by HBM.
//
// One thread moves 16 codes (one 16-byte load, one 32-byte store), one or four times; the
// chunks of a token's K then V rows lie side by side in its index, so the stores of a
// warp are whole rows of the output.  64 sequences of 256 to 2048 tokens, 8 heads of 128,
// bf16 (403 MB): 62 us, 6.5 TB/s, 0.97 of this GPU's copy rate; a persistent grid, with
// the next slots asked for while numbers are on their way, took 71 us, and all of a
// thread's slots asked for before its first number 66.  1000 tokens: 2.1 us, what a launch
// costs and two round trips.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

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

// 32 bytes in one store; dst 32-byte aligned.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <bool kBf16, int kUnroll>
__global__ void __launch_bounds__(kThreads) gather_q8_kernel(const GatherArgs a, int chunk_shift) {
    allow_dependents_to_launch();
    // chunk `rest` of token `token`: its K rows, then its V rows; the thread's chunks are
    // kThreads apart.  (All of it is reckoned while the kernel before still runs.)
    const int per_matrix = a.num_kv_heads << chunk_shift, per_token = 2 * per_matrix;
    const int step_tokens = kThreads / per_token, step_rest = kThreads - step_tokens * per_token;
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    int token[kUnroll], rest[kUnroll];
    token[0] = static_cast<int>(first / per_token);
    rest[0] = static_cast<int>(first - static_cast<long long>(token[0]) * per_token);
#pragma unroll
    for (int u = 1; u < kUnroll; ++u) {
        token[u] = token[u - 1] + step_tokens;
        rest[u] = rest[u - 1] + step_rest;
        if (rest[u] >= per_token) rest[u] -= per_token, ++token[u];
    }
    grid_dependency_wait();
    uint4 codes[kUnroll];
    float scale[kUnroll];
    uint8_t *dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        dst[u] = nullptr;
        const int slot = token[u] < a.num_tokens ? a.slots[token[u]] : -1;
        const bool is_v = rest[u] >= per_matrix;
        scale[u] = (is_v ? a.v_scales : a.k_scales)[(is_v ? rest[u] - per_matrix : rest[u]) >> chunk_shift];
        if (slot >= 0 && slot < a.pool_slots) {
            const int c = is_v ? rest[u] - per_matrix : rest[u], h = c >> chunk_shift;
            const int block = slot >> a.block_shift, off = slot - (block << a.block_shift);
            const size_t row = ((static_cast<size_t>(block) * a.num_kv_heads + h) << a.block_shift) + off;
            codes[u] = __ldcg(reinterpret_cast<const uint4 *>(is_v ? a.v_cache : a.k_cache) +
                              ((row - h) << chunk_shift) + c);
            dst[u] = reinterpret_cast<uint8_t *>(is_v ? a.v_out : a.k_out) +
                     32 * (static_cast<size_t>(token[u]) * per_matrix + c);
        } else if (slot >= 0 && rest[u] == 0) {
            atomicOr(a.err, PA_DEVERR_SLOT);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (!dst[u]) continue;
        const uint32_t n[4] = {codes[u].x, codes[u].y, codes[u].z, codes[u].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = scaled<kBf16>(e4m3x2_to_f16x2(n[j]), scale[u]);
            o[2 * j + 1] = scaled<kBf16>(e4m3x2_to_f16x2_high(n[j]), scale[u]);
        }
        if (a.wide_stores) {
            store32(dst[u], o);
        } else {
            reinterpret_cast<uint4 *>(dst[u])[0] = make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint4 *>(dst[u])[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace

cudaError_t launch_gather_q8(const GatherArgs &args, int dtype, int num_sms, cudaStream_t stream) {
    const int chunk_shift = args.head_dim == 64 ? 2 : (args.head_dim == 128 ? 3 : 4);
    const long long total = (2LL * args.num_kv_heads << chunk_shift) * args.num_tokens;
    // Four chunks a thread where the device is full of them (403 MB: 62 us, 72 with one);
    // one where it is not, and the two round trips of a thread are all there is (1000
    // tokens in a graph: 2.1 us, 3.6 with four).
    const int unroll = total > 8LL * kThreads * num_sms ? 4 : 1;
    const long long ctas = (total + kThreads * unroll - 1) / (kThreads * unroll);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool bf16 = dtype == PA_DTYPE_BF16;
    const auto kernel = unroll == 4 ? (bf16 ? gather_q8_kernel<true, 4> : gather_q8_kernel<false, 4>)
                                    : (bf16 ? gather_q8_kernel<true, 1> : gather_q8_kernel<false, 1>);
    return cudaLaunchKernelEx(&cfg, kernel, args, chunk_shift);
}

}  // namespace pa
