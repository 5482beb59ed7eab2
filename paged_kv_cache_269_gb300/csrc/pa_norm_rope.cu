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
// its load to its store; elements are worked on in packed pairs.
//
// Two kernels: few tokens are bound by the round trips, so a thread loads its row
// itself, at once; many (8 a processor and more) are streamed through shared memory.
// 16384 tokens of 32 + 8 + 8 heads of 128, bf16, norms, 8-bit cache (378 MB): 66 us,
// 5.7 TB/s, 0.86 of this GPU's copy rate; the first kernel takes 70 us there (84 with
// the weights kept in registers, which cost it occupancy), and 91 us without packed
// pairs.  The schedulers issue 2.1 instructions a cycle then: it is the arithmetic, 220
// instructions for 512 elements, beside the loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <mutex>

#include "pa_device.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_tensor.cuh"

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
__device__ __forceinline__ void load8(const float *p, float *x) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Neighbouring elements are worked on as packed pairs (one instruction for two).
struct Pairs {
    uint64_t v[8];
};
__device__ __forceinline__ Pairs load_pairs(const float *lo, const float *hi) {
    Pairs r;
    float x[16];
    load8(lo, x);
    load8(hi, x + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = make_pair(x[2 * i], x[2 * i + 1]);
    return r;
}

// The same from shared memory.
__device__ __forceinline__ Pairs shared_pairs(const float *lo, const float *hi) {
    Pairs r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 t = reinterpret_cast<const ulonglong2 *>(i < 2 ? lo : hi)[i % 2];
        r.v[2 * i] = t.x, r.v[2 * i + 1] = t.y;
    }
    return r;
}

template <bool kBf16>
__device__ __forceinline__ void widen_pairs(const uint4 &d0, const uint4 &d1, uint64_t (&x)[8]) {
    float f[16];
    widen8<kBf16>(d0, f);
    widen8<kBf16>(d1, f + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_pair(f[2 * i], f[2 * i + 1]);
}
// What a row's elements are multiplied by before the weights; the row's threads call
// it together (`mates`).
template <int D>
__device__ __forceinline__ float norm_factor(const uint64_t (&x)[8], unsigned mates, float eps) {
    uint64_t s2 = mul_pair(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s2 = fma_pair(x[i], x[i], s2);
    float sum, other;
    split_pair(s2, sum, other);
    sum += other;
#pragma unroll
    for (int o = D / 32; o > 0; o /= 2) sum += __shfl_xor_sync(mates, sum, o);
    return rsqrtf(fmaf(sum, 1.f / D, eps));
}
__device__ __forceinline__ void apply_norm(uint64_t (&x)[8], float f, const Pairs &w) {
    const uint64_t f2 = make_pair(f, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mul_pair(mul_pair(x[i], f2), w.v[i]);
}
// The rotation of the thread's 8 pairs: turn holds their cosines, then their sines.
template <bool kInterleaved>
__device__ __forceinline__ void rotate(uint64_t (&x)[8], const Pairs &turn) {
    if constexpr (kInterleaved) {
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            split_pair(turn.v[i], cs[2 * i], cs[2 * i + 1]);
            split_pair(turn.v[i + 4], sn[2 * i], sn[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float xa, xb;
            split_pair(x[i], xa, xb);
            x[i] = make_pair(fmaf(-xb, sn[i], xa * cs[i]), fmaf(xa, sn[i], xb * cs[i]));
        }
    } else {
        const uint64_t minus = make_pair(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t xa = x[i], xb = x[i + 4], c = turn.v[i], s = turn.v[i + 4];
            x[i] = fma_pair(mul_pair(xb, minus), s, mul_pair(xa, c));
            x[i + 4] = fma_pair(xa, s, mul_pair(xb, c));
        }
    }
}
// Row r of token `token` to where it belongs; cache_row: row of (block, head 0, offset)
// in the caches, whose heads are a block apart.
template <bool kBf16, int D, bool kQ8>
__device__ __forceinline__ void store_row(const AppendArgs &a, const uint64_t (&x)[8], int token, int r,
                                          size_t cache_row, int e0, int e1) {
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    float y[16];
    if (!kQ8 || r < Hq) {
#pragma unroll
        for (int i = 0; i < 8; ++i) split_pair(x[i], y[2 * i], y[2 * i + 1]);
    }
    if (r < Hq) {
        uint16_t *dst = a.q_out + token * a.q_out_stride + static_cast<ptrdiff_t>(r) * D;
        *reinterpret_cast<uint4 *>(dst + e0) = round8<kBf16>(y);
        *reinterpret_cast<uint4 *>(dst + e1) = round8<kBf16>(y + 8);
        return;
    }
    const bool is_v = r >= Hq + Hk;
    const int h = r - (is_v ? Hq + Hk : Hq);
    const size_t at = (cache_row + (static_cast<size_t>(h) << a.block_shift)) * D;
    void *cache = is_v ? a.v_cache : a.k_cache;
    if constexpr (kQ8) {
        const float scale = (is_v ? a.v_scales : a.k_scales)[h], inv = fast_rcp(scale);
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = quantise_pair(x[i], make_pair(-scale, -scale), make_pair(inv, inv));
        uint8_t *dst = static_cast<uint8_t *>(cache) + at;
        *reinterpret_cast<uint2 *>(dst + e0) =
            make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
        *reinterpret_cast<uint2 *>(dst + e1) =
            make_uint2(__byte_perm(c[4], c[5], 0x5410), __byte_perm(c[6], c[7], 0x5410));
    } else {
        uint16_t *dst = static_cast<uint16_t *>(cache) + at;
        *reinterpret_cast<uint4 *>(dst + e0) = round8<kBf16>(y);
        *reinterpret_cast<uint4 *>(dst + e1) = round8<kBf16>(y + 8);
    }
}
__device__ __forceinline__ size_t cache_row_of(const AppendArgs &a, int slot) {
    const int block = slot >> a.block_shift;
    return ((static_cast<size_t>(block) * a.num_kv_heads) << a.block_shift) + (slot - (block << a.block_shift));
}

// Few tokens: a thread loads its row itself.
template <bool kBf16, int D, bool kInterleaved, bool kNorm, bool kQ8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const AppendArgs a, int row_splits) {
    constexpr int kLanes = D / 16;         // threads that share a head row
    constexpr int kRows = kThreads / kLanes;
    allow_dependents_to_launch();
    // (what needs no memory is reckoned while the kernel before still runs)
    const int p = threadIdx.x % kLanes;
    const int token = row_splits == 1 ? blockIdx.x : blockIdx.x / row_splits;
    const int split = row_splits == 1 ? 0 : blockIdx.x - token * row_splits;
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    const int pairs = a.rotary_dim / 16;   // threads of a row whose chunks are rotated
    const bool rotated = p < pairs;
    // the thread's two chunks of 8, at these elements of the row
    const int e0 = !rotated || kInterleaved ? 16 * p : 8 * p;
    const int e1 = !rotated || kInterleaved ? 16 * p + 8 : 8 * (p + pairs);
    const uint16_t *q = a.q + token * a.q_stride, *k = a.k + token * a.k_stride - static_cast<ptrdiff_t>(Hq) * D;
    const uint16_t *v = a.v + token * a.v_stride - static_cast<ptrdiff_t>(Hq + Hk) * D;
    auto row_of = [&](int r) { return (r < Hq ? q : (r < Hq + Hk ? k : v)) + static_cast<ptrdiff_t>(r) * D; };
    int r = split * kRows + threadIdx.x / kLanes;
    const int step = row_splits * kRows;
    grid_dependency_wait();
    // the first row is asked for together with the position and the slot
    const int pos = a.positions ? a.positions[token] : 0;
    const int slot = a.slot_mapping[token];
    uint4 d0 = make_uint4(0, 0, 0, 0), d1 = d0;
    if (r < Hq + 2 * Hk) {
        const uint16_t *src = row_of(r);
        d0 = *reinterpret_cast<const uint4 *>(src + e0);
        d1 = *reinterpret_cast<const uint4 *>(src + e1);
    }
    if (pos < 0) return;   // a padding row
    if (a.positions && pos >= a.max_positions) {
        if (split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_POSITION);
        return;
    }
    const bool store_kv = slot >= 0 && slot < a.pool_slots;
    if (slot >= a.pool_slots && split == 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_SLOT);

    Pairs turn;
    if (rotated) {
        const float *t = a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 8 * p;
        turn = load_pairs(t, t + 8 * pairs);
    }
    const int rows = store_kv ? Hq + 2 * Hk : Hq;
    const size_t cache_row = store_kv ? cache_row_of(a, slot) : 0;
    // threads of one row: they meet in the norm's shuffles, whatever the warp's others do
    const unsigned mates = ((1u << kLanes) - 1u) << (threadIdx.x % 32 / kLanes * kLanes);
    for (; r < rows; r += step) {
        uint64_t x[8];                     // the chunk at e0, then the one at e1
        widen_pairs<kBf16>(d0, d1, x);
        if (r + step < rows) {             // the next row is on its way while this one is worked on
            const uint16_t *src = row_of(r + step);
            d0 = *reinterpret_cast<const uint4 *>(src + e0);
            d1 = *reinterpret_cast<const uint4 *>(src + e1);
        }
        if constexpr (kNorm) {
            const float *now = r >= Hq + Hk ? nullptr : (r < Hq ? a.q_weight : a.k_weight);
            if (now) {
                apply_norm(x, norm_factor<D>(x, mates, a.eps), load_pairs(now + e0, now + e1));
            }
        }
        if (rotated && r < Hq + Hk) rotate<kInterleaved>(x, turn);
        store_row<kBf16, D, kQ8>(a, x, token, r, cache_row, e0, e1);
    }
}

// Many tokens: a persistent CTA streams them.  A producer warp brings each token's q, k
// and v rows and its row of the table by bulk copies into a ring of stages, so that the
// bytes on their way do not depend on how many registers and warps there are; four warps
// take the stages' rows in turn (the count of rows goes on from token to token, so that
// no warp has more of them than the others).
constexpr int kWarps = 4;
constexpr int kMostCtas = 5;               // an SM; with at least kLeastStages stages each
constexpr int kLeastStages = 2;
constexpr int kStreamThreads = (kWarps + 1) * 32;
constexpr int kMaxStages = 6;
struct StreamPlan {
    int stages, stage_bytes;               // 0 stages: rows too long for two of them
    int smem, ctas_per_sm;
};
constexpr int kStreamHead = 256;           // barriers, tokens and slots of the stages, flag

template <bool kBf16, int D, bool kInterleaved, bool kNorm, bool kQ8>
__global__ void __launch_bounds__(kStreamThreads, kMostCtas) norm_rope_stream_kernel(const AppendArgs a, int stages,
                                                                          int stage_bytes) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + kMaxStages;
    volatile int *tokens = reinterpret_cast<volatile int *>(empty + kMaxStages), *slots = tokens + kMaxStages;
    volatile int *abort_flag = slots + kMaxStages;
    float *weights = reinterpret_cast<float *>(smem + kStreamHead);   // of q, then of k
    uint8_t *ring = smem + kStreamHead + (kNorm ? 2 * D * 4 : 0);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int Hq = a.num_q_heads, Hk = a.num_kv_heads;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kWarps);
        *abort_flag = 0;
        mbar_init_fence();
    }
    allow_dependents_to_launch();
    grid_dependency_wait();
    if constexpr (kNorm) {
        for (int i = threadIdx.x; i < 2 * D; i += kStreamThreads) {
            const float *src = i < D ? a.q_weight : a.k_weight;
            weights[i] = src ? src[i % D] : 0.f;
        }
    }
    __syncthreads();
    const int q_bytes = Hq * D * 2, kv_bytes = Hk * D * 2, table_bytes = a.rotary_dim * 4;
    if (warp == kWarps) {
        int n = 0;                         // stages filled
        bool ok = true;
        // 32 tokens' positions and slots at a time, the next ones on their way
        auto load = [&](long long i, int &pos, int &slot) {
            const long long t = blockIdx.x + (i + lane) * gridDim.x;
            pos = -1, slot = -1;
            if (t < a.num_tokens) {
                pos = a.positions ? a.positions[t] : 0;
                slot = a.slot_mapping[t];
            }
        };
        int next_pos, next_slot;
        load(0, next_pos, next_slot);
        for (long long i = 0; ok && blockIdx.x + i * gridDim.x < a.num_tokens; i += 32) {
            const int pos_l = next_pos, slot_l = next_slot;
            load(i + 32, next_pos, next_slot);
            for (int j = 0; ok && j < 32; ++j) {
                const int pos = __shfl_sync(0xffffffffu, pos_l, j);
                int slot = __shfl_sync(0xffffffffu, slot_l, j);
                if (pos < 0) continue;     // a padding row, or past the last token
                if (a.positions && pos >= a.max_positions) {
                    if (lane == 0) atomicOr(a.err, PA_DEVERR_POSITION);
                    continue;
                }
                if (slot >= a.pool_slots) {
                    if (lane == 0) atomicOr(a.err, PA_DEVERR_SLOT);
                    slot = -1;
                }
                if (slot < 0 && Hq == 0) continue;
                const int st = n % stages;
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / stages) & 1) ^ 1, abort_flag, a.err));
                if (!ok) break;
                if (lane == 0) {
                    const int token = static_cast<int>(blockIdx.x + (i + j) * gridDim.x);
                    uint8_t *dst = ring + st * stage_bytes;
                    tokens[st] = token;
                    slots[st] = slot;
                    mbar_arrive_expect_tx(&full[st], q_bytes + (slot >= 0 ? 2 * kv_bytes : 0) + table_bytes);
                    if (Hq > 0) bulk_copy_g2s(dst, a.q + token * a.q_stride, q_bytes, &full[st]);
                    dst += q_bytes;
                    if (slot >= 0) {
                        bulk_copy_g2s(dst, a.k + token * a.k_stride, kv_bytes, &full[st]);
                        bulk_copy_g2s(dst + kv_bytes, a.v + token * a.v_stride, kv_bytes, &full[st]);
                    }
                    if (table_bytes > 0)
                        bulk_copy_g2s(dst + 2 * kv_bytes, a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim, table_bytes,
                                      &full[st]);
                }
                __syncwarp();
                ++n;
            }
        }
        if (ok) {   // the last stage says that there are no more
            const int st = n % stages;
            ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / stages) & 1) ^ 1, abort_flag, a.err));
            if (ok && lane == 0) {
                tokens[st] = -1;
                mbar_arrive(&full[st]);
            }
        }
        if (!ok && lane == 0)   // let every copy already issued land
            for (int i = max(0, n - stages); i < n; ++i) mbar_wait_drain(&full[i % stages], (i / stages) & 1);
        return;
    }
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int p = lane % kLanes;
    const int pairs = a.rotary_dim / 16;
    const bool rotated = p < pairs;
    const int e0 = !rotated || kInterleaved ? 16 * p : 8 * p;
    const int e1 = !rotated || kInterleaved ? 16 * p + 8 : 8 * (p + pairs);
    const int all_groups = (Hq + 2 * Hk + kRows - 1) / kRows;
    int first = warp;                      // the warp's first group of rows of the stage
    for (int n = 0;; ++n) {
        const int st = n % stages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (n / stages) & 1, abort_flag, a.err))) return;
        const int token = tokens[st], slot = slots[st];
        if (token < 0) return;
        const uint8_t *stage = ring + st * stage_bytes;
        const int rows = slot >= 0 ? Hq + 2 * Hk : Hq;
        const size_t cache_row = slot >= 0 ? cache_row_of(a, slot) : 0;
        const float *table = reinterpret_cast<const float *>(stage + q_bytes + 2 * kv_bytes) + 8 * p;
        Pairs turn;
        if (rotated) turn = shared_pairs(table, table + 8 * pairs);
        for (int g = first; g * kRows < rows; g += kWarps) {
            const int r = g * kRows + lane / kLanes;
            // (rows past the last stand in for it and are not stored)
            const uint16_t *src = reinterpret_cast<const uint16_t *>(stage) + min(r, rows - 1) * D;
            uint64_t x[8];
            widen_pairs<kBf16>(*reinterpret_cast<const uint4 *>(src + e0), *reinterpret_cast<const uint4 *>(src + e1), x);
            if constexpr (kNorm) {
                if (g * kRows < Hq + Hk) {
                    const float f = norm_factor<D>(x, 0xffffffffu, a.eps);
                    const bool is_q = r < Hq;
                    if (r < Hq + Hk && (is_q ? a.q_weight : a.k_weight)) {
                        const float *now = weights + (is_q ? 0 : D);
                        apply_norm(x, f, shared_pairs(now + e0, now + e1));
                    }
                }
            }
            if (rotated && r < Hq + Hk) rotate<kInterleaved>(x, turn);
            if (r < rows) store_row<kBf16, D, kQ8>(a, x, token, r, cache_row, e0, e1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        // the count of groups goes on with the next token
        first = (first - all_groups) % kWarps;
        if (first < 0) first += kWarps;
    }
}

using Kernel = void (*)(AppendArgs, int);
using StreamKernel = void (*)(AppendArgs, int, int);
struct Variant {
    Kernel direct;
    StreamKernel stream;
};
template <bool kBf16, int D, bool kInterleaved, bool kNorm>
Variant pick(bool q8) {
    return q8 ? Variant{norm_rope_kernel<kBf16, D, kInterleaved, kNorm, true>,
                        norm_rope_stream_kernel<kBf16, D, kInterleaved, kNorm, true>}
              : Variant{norm_rope_kernel<kBf16, D, kInterleaved, kNorm, false>,
                        norm_rope_stream_kernel<kBf16, D, kInterleaved, kNorm, false>};
}
template <bool kBf16, int D>
Variant pick(bool interleaved, bool norm, bool q8) {
    return interleaved ? (norm ? pick<kBf16, D, true, true>(q8) : pick<kBf16, D, true, false>(q8))
                       : (norm ? pick<kBf16, D, false, true>(q8) : pick<kBf16, D, false, false>(q8));
}
template <bool kBf16>
Variant pick(int D, bool interleaved, bool norm, bool q8) {
    return D == 64 ? pick<kBf16, 64>(interleaved, norm, q8)
                   : (D == 128 ? pick<kBf16, 128>(interleaved, norm, q8) : pick<kBf16, 256>(interleaved, norm, q8));
}

StreamPlan stream_plan(const AppendArgs &a, bool norm) {
    StreamPlan p = {};
    const long long bytes = (static_cast<long long>(a.num_q_heads) + 2LL * a.num_kv_heads) * a.head_dim * 2 + a.rotary_dim * 4LL;
    const int head = kStreamHead + (norm ? 2 * a.head_dim * 4 : 0);
    for (int ctas = kMostCtas; ctas >= 1; --ctas) {
        const long long room = 232448 / ctas - 1024 - head;
        if (bytes * kLeastStages > room) continue;
        p.stages = static_cast<int>(room / bytes < kMaxStages ? room / bytes : kMaxStages);
        p.stage_bytes = static_cast<int>(bytes);
        p.smem = head + p.stages * p.stage_bytes;
        p.ctas_per_sm = ctas;
        return p;
    }
    return p;
}

}  // namespace

cudaError_t launch_norm_rope(const AppendArgs &args, int dtype, bool interleaved, int num_sms, cudaStream_t stream) {
    const bool norm = args.q_weight || args.k_weight, q8 = args.k_scales != nullptr, bf16 = dtype == PA_DTYPE_BF16;
    const Variant v = bf16 ? pick<true>(args.head_dim, interleaved, norm, q8)
                           : pick<false>(args.head_dim, interleaved, norm, q8);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool many = args.num_tokens >= 8 * num_sms;
    const StreamPlan plan = many ? stream_plan(args, norm) : StreamPlan{};
    if (plan.stages) {
        // the kernel's shared-memory limit, once per device and variant
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
        {
            static std::mutex mu;
            static bool ready[64][48] = {};
            const int which = (args.head_dim == 64 ? 0 : (args.head_dim == 128 ? 1 : 2)) * 16 + (bf16 ? 8 : 0) +
                              (interleaved ? 4 : 0) + (norm ? 2 : 0) + (q8 ? 1 : 0);
            std::lock_guard<std::mutex> lock(mu);
            if (!ready[device][which]) {
                e = cudaFuncSetAttribute(reinterpret_cast<const void *>(v.stream),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
                if (e != cudaSuccess) return e;
                ready[device][which] = true;
            }
        }
        cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas_per_sm * num_sms));
        cfg.blockDim = dim3(kStreamThreads);
        cfg.dynamicSmemBytes = plan.smem;
        return cudaLaunchKernelEx(&cfg, v.stream, args, plan.stages, plan.stage_bytes);
    }
    const int rows = args.num_q_heads + 2 * args.num_kv_heads;
    const int rows_per_pass = kThreads / (args.head_dim / 16);
    // few tokens: a row per thread; many: a block walks over all rows of its
    // token, so that the token's cosines and sines are loaded once
    const int passes = (rows + rows_per_pass - 1) / rows_per_pass;
    const int row_splits = many ? 1 : passes;
    const long long blocks = static_cast<long long>(args.num_tokens) * row_splits;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    return cudaLaunchKernelEx(&cfg, v.direct, args, row_splits);
}

}  // namespace pa
