// pa_rope.cu -- rope_and_cache: rotate q and k by the tokens' positions and
// append k and v to the paged cache in the same pass.
//
// Per token, every head row of q, k and v is read once and written once; the
// rotation is 3 flops per element, so the call is bound by HBM (large batches)
// or by its launch (a decode step's few tokens).
//
// One thread handles 16 elements of a row: for the half-split order the two
// 16-byte chunks that hold each other's partners (chunk p and chunk
// p + rotary_dim / 16), for the interleaved order two neighbouring chunks.
// Both need the same 8 cosines and 8 sines (8 p .. 8 p + 7 of the token's
// table row), which the thread keeps in registers while it walks over head
// rows, so the table costs its bytes once per token, not once per head.  Dims
// past rotary_dim, and all of v, are copied by the same threads.
//
// Launched with programmatic dependent launch, like reshape_and_cache: it
// waits for the previous kernel on the stream before it touches memory.
//
// Measured, bf16, 32 + 8 + 8 heads of 128: 16384 tokens 63.3 us, 6.5 TB/s of
// its 411 MB, 0.96 of this GPU's copy rate; 256 tokens 3.8 us, a launch and two
// round trips to HBM (positions and slots, then the rows and the table); one token
// 1.8 us, which is what a launch costs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 128;

struct RopeF16 {
    __device__ static __forceinline__ float2 widen(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    __device__ static __forceinline__ uint32_t round(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
struct RopeBF16 {
    __device__ static __forceinline__ float2 widen(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    __device__ static __forceinline__ uint32_t round(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Rotate the 8 pairs held by two chunks: half-split order pairs element e of
// `a` with element e of `b`; interleaved order pairs neighbours, a first.
template <typename E, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float (&c)[8],
                                       const float (&s)[8]) {
    uint32_t *ua = reinterpret_cast<uint32_t *>(&a), *ub = reinterpret_cast<uint32_t *>(&b);
    if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = E::widen(ua[i]), y = E::widen(ub[i]);
            ua[i] = E::round(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
            ub[i] = E::round(y.x * c[i + 4] - y.y * s[i + 4], y.y * c[i + 4] + y.x * s[i + 4]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = E::widen(ua[i]), y = E::widen(ub[i]);
            const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
            ua[i] = E::round(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
            ub[i] = E::round(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
        }
    }
}

template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a, int lanes,
                                                                  int row_splits) {
    allow_dependents_to_launch();
    grid_dependency_wait();
    // `lanes` = D / 16 threads share a head row
    const int p = threadIdx.x % lanes, r0 = threadIdx.x / lanes, rows_per_pass = kThreads / lanes;
    const int split = blockIdx.x % row_splits;
    const int token = blockIdx.x / row_splits;
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    const int pos = __ldg(a.positions + token);
    if (pos < 0) return;   // a padding row
    if (pos >= a.max_positions) {
        if (split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_POSITION);
        return;
    }
    const int slot = __ldg(a.slot_mapping + token);
    const bool store_kv = slot >= 0 && slot < a.pool_slots;
    if (slot >= a.pool_slots && split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_SLOT);

    const int pairs = a.rotary_dim / 16;   // threads of a row whose chunks are rotated
    const bool rotated = p < pairs;
    // the thread's two chunks, in units of 8 elements
    int c0, c1;
    if (!rotated || kInterleaved) {
        c0 = 2 * p;
        c1 = 2 * p + 1;
    } else {
        c0 = p;
        c1 = p + pairs;
    }
    float cs[8], sn[8];
    if (rotated) {
        const float4 *t = reinterpret_cast<const float4 *>(
            a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 8 * p);
        const float4 x0 = __ldg(t), x1 = __ldg(t + 1);
        const float4 y0 = __ldg(t + 2 * pairs), y1 = __ldg(t + 2 * pairs + 1);
        cs[0] = x0.x, cs[1] = x0.y, cs[2] = x0.z, cs[3] = x0.w;
        cs[4] = x1.x, cs[5] = x1.y, cs[6] = x1.z, cs[7] = x1.w;
        sn[0] = y0.x, sn[1] = y0.y, sn[2] = y0.z, sn[3] = y0.w;
        sn[4] = y1.x, sn[5] = y1.y, sn[6] = y1.z, sn[7] = y1.w;
    }
    const int chunks = 2 * lanes;          // of 8 elements, per row
    const int rows = store_kv ? Hq + 2 * Hk : Hq;
    size_t cache_row = 0;                  // row of (block, head 0, offset); heads are B rows apart
    if (store_kv)
        cache_row = (static_cast<size_t>(slot / a.block_size) * Hk) * a.block_size +
                    slot % a.block_size;
    for (int r = split * rows_per_pass + r0; r < rows; r += row_splits * rows_per_pass) {
        const uint4 *src;
        uint4 *dst;
        if (r < Hq) {
            src = reinterpret_cast<const uint4 *>(a.q + token * a.q_stride) + static_cast<size_t>(r) * chunks;
            dst = reinterpret_cast<uint4 *>(a.q_out + token * a.q_out_stride) + static_cast<size_t>(r) * chunks;
        } else {
            const bool is_k = r < Hq + Hk;
            const int h = r - Hq - (is_k ? 0 : Hk);
            src = reinterpret_cast<const uint4 *>(is_k ? a.k + token * a.k_stride
                                                       : a.v + token * a.v_stride) +
                  static_cast<size_t>(h) * chunks;
            dst = reinterpret_cast<uint4 *>(is_k ? a.k_cache : a.v_cache) +
                  (cache_row + static_cast<size_t>(h) * a.block_size) * chunks;
        }
        uint4 x = src[c0], y = src[c1];
        if (rotated && r < Hq + Hk) rotate<E, kInterleaved>(x, y, cs, sn);
        dst[c0] = x;
        dst[c1] = y;
    }
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs &args, int dtype, bool interleaved, int num_sms,
                                  cudaStream_t stream) {
    const int lanes = args.head_dim / 16;
    const int rows = args.num_q_heads + 2 * args.num_kv_heads;
    const int rows_per_pass = kThreads / lanes;
    // few tokens: a row per thread; many: a block walks over all rows of its
    // token, so that the token's cosines and sines are loaded once
    const int passes = (rows + rows_per_pass - 1) / rows_per_pass;
    const int row_splits = args.num_tokens >= 8 * num_sms ? 1 : passes;
    const long long blocks = static_cast<long long>(args.num_tokens) * row_splits;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    void (*kernel)(RopeArgs, int, int) =
        dtype == PA_DTYPE_BF16
            ? (interleaved ? rope_and_cache_kernel<RopeBF16, true> : rope_and_cache_kernel<RopeBF16, false>)
            : (interleaved ? rope_and_cache_kernel<RopeF16, true> : rope_and_cache_kernel<RopeF16, false>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args, lanes, row_splits);
}

}  // namespace pa
