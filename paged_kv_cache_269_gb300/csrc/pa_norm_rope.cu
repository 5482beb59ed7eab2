// pa_norm_rope.cu -- norm_rope_and_cache: norm each head of q and k, rotate them
// by the tokens' positions and append k and v to a paged cache of 16-bit or of
// e4m3 elements, in one pass.
//
// Per head row: y_i = x_i w_i / sqrt(mean x^2 + eps) (where weights are given),
// the rotation of rope_and_cache, and one rounding: to the element type, or for
// an 8-bit cache to e4m3 of x / scale.  4 flops an element for the norm and 3
// for the rotation, so the call is bound by HBM, or by its launch and two round
// trips to HBM where tokens are few.
//
// As in rope_and_cache a row is shared by D / 16 threads of 16 elements each
// (two chunks of 8, which hold each other's partners), so the mean square is a
// sum of 16 products and 2 to 4 shuffles, and the row stays in registers from
// its load to its store.  The token's cosines and sines and the weights of the
// thread's 16 dims stay in registers while it walks over head rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 128;

template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4 &c, float *x) {
    const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBf16) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}
template <bool kBf16>
__device__ __forceinline__ uint4 round8(const float *x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint2 quantise8(const float *x, float scale, float inv) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = f32x2_to_e4m3x2(divide_by_scale(x[2 * i], scale, inv), divide_by_scale(x[2 * i + 1], scale, inv));
    return make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
}
__device__ __forceinline__ void load8(const float *p, float *x) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <bool kBf16, bool kInterleaved, bool kNorm, bool kQ8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const AppendArgs a, int lanes, int row_splits) {
    allow_dependents_to_launch();
    grid_dependency_wait();
    // `lanes` = D / 16 threads share a head row
    const int p = threadIdx.x % lanes, r0 = threadIdx.x / lanes, rows_per_pass = kThreads / lanes;
    const int split = blockIdx.x % row_splits;
    const int token = blockIdx.x / row_splits;
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    const int pos = a.positions ? __ldg(a.positions + token) : 0;
    const int slot = __ldg(a.slot_mapping + token);

    const int pairs = a.rotary_dim / 16;   // threads of a row whose chunks are rotated
    const bool rotated = p < pairs;
    // the thread's two chunks, in units of 8 elements
    const int c0 = !rotated || kInterleaved ? 2 * p : p;
    const int c1 = !rotated || kInterleaved ? 2 * p + 1 : p + pairs;
    auto row_of = [&](int r) -> const uint4 * {
        const uint16_t *src = r < Hq ? a.q + token * a.q_stride + static_cast<size_t>(r) * a.head_dim
                              : r < Hq + Hk
                                  ? a.k + token * a.k_stride + static_cast<size_t>(r - Hq) * a.head_dim
                                  : a.v + token * a.v_stride + static_cast<size_t>(r - Hq - Hk) * a.head_dim;
        return reinterpret_cast<const uint4 *>(src);
    };
    // the first row is asked for together with the position and the slot
    int r = split * rows_per_pass + r0;
    const int step = row_splits * rows_per_pass;
    uint4 d0 = make_uint4(0, 0, 0, 0), d1 = d0;
    if (r < Hq + 2 * Hk) {
        const uint4 *src = row_of(r);
        d0 = src[c0], d1 = src[c1];
    }
    if (pos < 0) return;   // a padding row
    if (a.positions && pos >= a.max_positions) {
        if (split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_POSITION);
        return;
    }
    const bool store_kv = slot >= 0 && slot < a.pool_slots;
    if (slot >= a.pool_slots && split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_SLOT);

    float cs[8], sn[8];
    if (rotated) {
        const float *t = a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 8 * p;
        load8(t, cs);
        load8(t + 8 * pairs, sn);
    }
    const int rows = store_kv ? Hq + 2 * Hk : Hq;
    size_t cache_row = 0;                  // row of (block, head 0, offset); heads are B rows apart
    if (store_kv)
        cache_row = (static_cast<size_t>(slot / a.block_size) * Hk) * a.block_size + slot % a.block_size;
    // threads of one row: they meet in the norm's shuffles, whatever the warp's others do
    const unsigned mates = (lanes == 32 ? ~0u : (1u << lanes) - 1u) << ((threadIdx.x % 32) / lanes * lanes);
    float w[16];
    const float *weight = nullptr;         // whose dims w holds
    for (; r < rows; r += step) {
        float x[16];
        widen8<kBf16>(d0, x);
        widen8<kBf16>(d1, x + 8);
        const bool is_q = r < Hq, is_v = r >= Hq + Hk;
        const int h = is_q ? r : (is_v ? r - Hq - Hk : r - Hq);
        if (r + step < rows) {             // the next row is on its way while this one is worked on
            const uint4 *src = row_of(r + step);
            d0 = src[c0], d1 = src[c1];
        }
        if constexpr (kNorm) {
            const float *now = is_v ? nullptr : (is_q ? a.q_weight : a.k_weight);
            if (now) {
                if (now != weight) {
                    weight = now;
                    load8(weight + 8 * c0, w);
                    load8(weight + 8 * c1, w + 8);
                }
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
                for (int o = lanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(mates, sum, o);
                const float f = rsqrtf(fmaf(sum, a.inv_dim, a.eps));
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = x[i] * f * w[i];
            }
        }
        if (rotated && !is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : i + 8;
                const float y = x[ia] * cs[i] - x[ib] * sn[i];
                x[ib] = x[ib] * cs[i] + x[ia] * sn[i];
                x[ia] = y;
            }
        }
        if (is_q) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + token * a.q_out_stride + static_cast<size_t>(h) * a.head_dim);
            dst[c0] = round8<kBf16>(x);
            dst[c1] = round8<kBf16>(x + 8);
            continue;
        }
        const size_t row = (cache_row + static_cast<size_t>(h) * a.block_size) * (2 * lanes);   // in chunks
        void *cache = is_v ? a.v_cache : a.k_cache;
        if constexpr (kQ8) {
            const float scale = __ldg((is_v ? a.v_scales : a.k_scales) + h), inv = 1.f / scale;
            uint2 *dst = static_cast<uint2 *>(cache) + row;
            dst[c0] = quantise8(x, scale, inv);
            dst[c1] = quantise8(x + 8, scale, inv);
        } else {
            uint4 *dst = static_cast<uint4 *>(cache) + row;
            dst[c0] = round8<kBf16>(x);
            dst[c1] = round8<kBf16>(x + 8);
        }
    }
}

using Kernel = void (*)(AppendArgs, int, int);
template <bool kBf16, bool kInterleaved>
Kernel pick(bool norm, bool q8) {
    return norm ? (q8 ? norm_rope_kernel<kBf16, kInterleaved, true, true>
                      : norm_rope_kernel<kBf16, kInterleaved, true, false>)
                : (q8 ? norm_rope_kernel<kBf16, kInterleaved, false, true>
                      : norm_rope_kernel<kBf16, kInterleaved, false, false>);
}

}  // namespace

cudaError_t launch_norm_rope(const AppendArgs &args, int dtype, bool interleaved, int num_sms, cudaStream_t stream) {
    const int lanes = args.head_dim / 16;
    const int rows = args.num_q_heads + 2 * args.num_kv_heads;
    const int rows_per_pass = kThreads / lanes;
    // few tokens: a row per thread; many: a block walks over all rows of its
    // token, so that the token's cosines and sines are loaded once
    const int passes = (rows + rows_per_pass - 1) / rows_per_pass;
    const int row_splits = args.num_tokens >= 8 * num_sms ? 1 : passes;
    const long long blocks = static_cast<long long>(args.num_tokens) * row_splits;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool norm = args.q_weight || args.k_weight, q8 = args.k_scales != nullptr;
    const Kernel kernel = dtype == PA_DTYPE_BF16 ? (interleaved ? pick<true, true>(norm, q8) : pick<true, false>(norm, q8))
                                                 : (interleaved ? pick<false, true>(norm, q8) : pick<false, false>(norm, q8));
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
