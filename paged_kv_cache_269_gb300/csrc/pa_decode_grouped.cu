// pa_decode_grouped.cu -- attention of one new token per sequence over the
// paged cache, with query heads that share K/V heads (sm_103a).
//
// Mathematics: for the G = Hq / Hkv query heads of one K/V head,
//   s_gj = f(scale q_g . k_j),  o_g = sum_j 2^(x_gj - m_g) v_j / sum_j 2^(x_gj - m_g)
// with x = s log2(e) (f: the optional tanh cap and distance bias), one pass
// over the keys with a running reference m_g that every weight and the sum
// share, so the result does not depend on it.
//
// What bounds it: each K and V element is read once for up to 16 query heads (8
// at head_dim 256; wider groups are taken in chunks, and each chunk reads the
// context again), 2 flops for each of them, so the call is bound by HBM as long
// as the products are cheaper than the loads.  On the FMA pipe they are not from
// G = 4 on, so both products run as mma.sync m16n8k16 with the 16 rows on the
// keys (then the head dims) and the 8 columns on the query heads: a group of 8
// heads fills the shape, where tcgen05's 128-row tiles would be 1/16 used.
//
// How:
//  * Work is cut evenly, not by sequence: all sequences' visible key tiles,
//    laid end to end per (sequence, K/V head, chunk of query heads), form one
//    line; CTA i takes the i-th equal piece of it.  A piece may end inside a
//    context: it then leaves a partial (max, sum, unnormalised output) in one
//    of its two slots, and the last piece of the context to finish (a ticket
//    per context) joins all of them, in order, so the result does not depend
//    on which came last.
//  * No roles: each warp owns a ring of stages and is its own producer.  It
//    takes the next tile of its CTA's piece, waits for the tile's TMA boxes,
//    computes, and refills the stage it just read; the table entry of the
//    refill was loaded one tile earlier.  Warps meet only where a context
//    ends, to merge their (max, sum, output) through shared memory, while
//    their rings keep filling.
//  * S^T = K Q^T (rows: keys, columns: heads), so a lane holds the scores of
//    two heads; the weights become the second product's B operand with one
//    movmatrix, and O^T = V^T P^T accumulates in registers.
//  * The weights enter P V as a 16-bit pair P_hi + P_lo (about 22 bits; 16 in
//    bf16), so the output is as exact as fp32 weights make it.  With G <= 4
//    the two halves share one product: columns 4-7 repeat the heads and carry
//    P_lo.
//  * The reference m is raised only when a score exceeds it by about 8
//    (weights stay below 2^(8 + 6), inside fp16), so most tiles need no
//    maximum across lanes and no rescaling.
//  * Keys that are not visible get weight 0 and their V values are cleared in
//    registers, so nothing they hold reaches the output.
//
// Shape: 4 warps a CTA and 2 CTAs an SM, as many as 181 to 251 registers a thread
// leave, with as many stages a warp as shared memory holds.  A third stage at
// head_dim 128 (in exchange for a smaller merge area) cost 4 % (59.5 us against
// 57.1 on the first batch below), at 256 nothing changed.  Work cut into small
// pieces from a queue, instead of one equal piece a CTA, took 78 us there: the
// partials to join are many.
//
// Measured: 64 sequences of 256 to 2048 tokens, 32 heads on 8 of 128, bf16:
// 57 us, 5.3 TB/s; 256 sequences of 1000 to 4000 tokens 386 us, 6.8 TB/s,
// the rate of a copy.  4 documents of 20001 to 32768 tokens, 64 heads on 8,
// distance bias: 74 us, 5.6 TB/s (HBM busy, the tensor pipe 12 %).  96
// sequences, window 1024, head_dim 256, capped: 134 us, 6.0 TB/s.  What is not
// streaming is the start until all rings are full (lengths, table entry, first
// tiles, one after another) and the end (merge, ticket, join), about 12 us of
// such calls together; a sequence of 1000 tokens is nothing else, and takes
// 8.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tensor.cuh"

namespace pa {
namespace {

constexpr int kW = 4;                  // warps per CTA
constexpr int kThreads = kW * 32;
constexpr int kChunks = 512;           // entries of the CTA's prefix over the sequences
constexpr int kMaxCtas = 640;          // bounds the partial slots (2 per CTA)
// The reference is raised by scores more than this above it.  The sum is rounded
// down: past 2^26 fp32's step is 8 and the bias below becomes 8 too, so a score one
// step above the reference would have a weight of 2^16, past fp16.
constexpr float kRaise = 7.9f;
constexpr float kBias = 6.f;           // weights are 2^(x - m + 6)

struct DecodeGroupedArgs {
    GroupedArgs g;
    float scale_log2;                  // plain scores: x = scale_log2 (q . k)
    float cap_log2, cap_in;            // capped: x = cap_log2 tanh(...), 2^(cap_in q.k) = e^(2 s / cap)
    float cap_v, tanh_k[5];            // as a polynomial (fill_tanh), where |s / cap| < 0.75
    int group, chunks;                 // heads per K/V head; chunks of heads per K/V head
    int chunk_shift;                   // sequences per prefix entry: 2^chunk_shift
    float *partials;                   // [2 * kMaxCtas][heads * (D + 2)]
};

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (kBf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float fast_rcp(float x) {   // 1 ulp; 1 / inf = 0
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two weights as packed 16-bit values, and the packed remainders.
template <bool kBf16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(hi << 16),
                                                       b - __uint_as_float(hi & 0xFFFF0000u));
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// A sequence's visible keys as tiles of TK keys: tile i covers keys from
// TK * (i < na ? i : i + skip); [lo, ctx) and [0, pre) are visible.
// `len` is what a unit takes of the line: its tiles, and what its end costs a
// CTA (kCost, in tiles' time).
struct Geo {
    int ctx, lo, pre, na, skip, nt, len;
};
template <int TK, int kCost>
__device__ __forceinline__ Geo make_geo(const GroupedArgs &a, int ctx, int pre_raw) {
    Geo g;
    g.ctx = ctx;
    g.lo = a.window > 0 ? max(0, ctx - a.window) : 0;
    g.pre = max(0, min(pre_raw, ctx));
    const int total = (ctx + TK - 1) / TK, first = g.lo / TK;
    g.na = (g.pre + TK - 1) / TK;
    if (first <= g.na && g.pre > 0) {
        g.na = 0, g.skip = 0, g.nt = total;
    } else {
        g.skip = first - g.na;
        g.nt = g.na + total - first;
    }
    g.len = g.nt > 0 ? g.nt + kCost : 0;
    return g;
}

// Context length of sequence s (0 for one outside its bounds) and prefix.
__device__ __forceinline__ int load_ctx(const GroupedArgs &a, int s) {
    if (s >= a.num_seqs) return 0;
    const int c = __ldg(a.context_lens + s);
    return (c < 0 || c > a.max_blocks_per_seq * a.block_size) ? 0 : c;
}
__device__ __forceinline__ int load_pre(const GroupedArgs &a, int s) {
    return a.prefix_lens && s < a.num_seqs ? __ldg(a.prefix_lens + s) : 0;
}

// A position on the line: tile `idx` of unit `unit` of sequence s.  A unit is
// one (K/V head, chunk of query heads); the lanes hold the lengths of 32
// sequences.
template <int TK, int kCost>
struct Cursor {
    int s, unit, idx;
    Geo g;
    int base, ctx_l, pre_l;
    __device__ __forceinline__ void load_group(const GroupedArgs &a, int lane) {
        base = s & ~31;
        ctx_l = load_ctx(a, base + lane);
        pre_l = load_pre(a, base + lane);
    }
    __device__ __forceinline__ void set_geo(const GroupedArgs &a) {
        g = make_geo<TK, kCost>(a, __shfl_sync(0xffffffffu, ctx_l, s & 31),
                         __shfl_sync(0xffffffffu, pre_l, s & 31));
    }
    // The next sequence with tiles (or s = num_seqs, nt = 0).
    __device__ __forceinline__ void next_seq(const GroupedArgs &a, int lane) {
        ++s;
        unit = 0;
        for (;;) {
            if (s >= a.num_seqs) {
                s = a.num_seqs;
                g.nt = g.len = 0;
                return;
            }
            if ((s & ~31) != base) load_group(a, lane);
            const unsigned rest = __ballot_sync(0xffffffffu, ctx_l > 0) >> (s & 31);
            if (rest) {
                s += __ffs(rest) - 1;
                set_geo(a);
                return;
            }
            s = base + 32;
        }
    }
    __device__ __forceinline__ void advance(const GroupedArgs &a, int units, int by, int lane) {
        idx += by;
        while (idx >= g.len && s < a.num_seqs) {
            idx -= g.len;
            if (++unit == units) next_seq(a, lane);
        }
    }
};

template <int D, int NT>
struct Cfg {
    static constexpr int TK = D == 64 ? 32 : 16;       // keys per tile
    static constexpr int MT = TK / 16;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kMat = TK * D * 2;            // bytes of a K (or V) tile
    static constexpr int kStage = 2 * kMat;
    // more bytes in flight do not help (a third stage for D = 128 made 256 long
    // sequences 7 % slower); for D = 64 there is room for one
    static constexpr int kStages = D == 64 && NT == 1 ? 3 : 2;
    // what a unit's end (merging the warps, a partial's ticket; 1.5 us) costs in
    // tiles' time: 64 sequences 61.3 us uncounted, 57.1 at 4; 16 heads 69.5 at 4,
    // 66.0 at 8
    static constexpr int kCost = 4 * NT;
    static constexpr int kRow = D + 4;                 // floats of a merge row (no bank conflicts)
    static constexpr int OFF_O = kW * kStages * kStage;
    static constexpr int OFF_ML = OFF_O + kW * kHeads * kRow * 4;
    static constexpr int OFF_PREFIX = OFF_ML + kW * kHeads * 8;
    static constexpr int OFF_BAR = OFF_PREFIX + (kChunks + 1 + kW) * 8;
    static constexpr int OFF_MASK = OFF_BAR + (kW * kStages + 1) * 8;   // rings, partial written
    static constexpr int OFF_FLAG = OFF_MASK + kW * kStages * 4;
    static constexpr int kBytes = OFF_FLAG + 16 + 1024;  // + alignment slack
    static constexpr int kCtasPerSm = 2 * (kBytes + 1024) <= 233472 ? 2 : 1;
};

// Takes the ticket of a partial that the CTA left (one warp; the partial's
// writes happen before the call at CTA scope): whether it was the unit's last.
__device__ __forceinline__ bool take_ticket(const DecodeGroupedArgs &p, int s, int units, int unit,
                                            int others, int lane) {
    uint32_t last = 0;
    if (lane == 0) {
        uint32_t *ticket = p.g.counters + static_cast<size_t>(s) * units + unit;   // a word a unit
        last = ticket_add(ticket, 1u) == static_cast<uint32_t>(others);
        if (last) atomicExch(ticket, 0u);
    }
    return __shfl_sync(0xffffffffu, last, 0) != 0;
}

// Joins the partials of a unit, which pieces i0 .. i1 left, and writes its
// output rows.  tid of n threads.
template <bool kBf16, int D, int kHeads>
__device__ __forceinline__ void join_unit(const DecodeGroupedArgs &p, int s, int unit, int i0, int i1,
                                          int tid, int n) {
    constexpr int kVec = D / 4;
    const GroupedArgs &a = p.g;
    const int hk = unit / p.chunks, h0 = (unit % p.chunks) * kHeads;
    const int heads = min(kHeads, p.group - h0);
    // slot of piece i: 2 i + 1 for the one the unit starts in, else 2 i
    auto part = [&](int i) {
        return p.partials + static_cast<size_t>(2 * i + (i == i0 ? 1 : 0)) * (kHeads * (D + 2));
    };
    for (int i = tid; i < heads * kVec; i += n) {
        const int h = i / kVec, d4 = i % kVec;
        // batches of partials, each one round trip to L2
        constexpr int kBatch = 8;
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = i0; c0 <= i1; c0 += kBatch) {
            float2 w[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const float *src = part(min(c0 + c, i1));
                w[c] = __ldcg(reinterpret_cast<const float2 *>(src + kHeads * D + 2 * h));
                v[c] = __ldcg(reinterpret_cast<const float4 *>(src + h * D + d4 * 4));
            }
            float t2 = top;
#pragma unroll
            for (int c = 0; c < kBatch; ++c) t2 = fmaxf(t2, w[c].x);
            const float f0_ = top == -INFINITY ? 0.f : fast_exp2(top - t2);
            sum *= f0_, acc.x *= f0_, acc.y *= f0_, acc.z *= f0_, acc.w *= f0_;
            top = t2;
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const float f = w[c].x == -INFINITY || c0 + c > i1 ? 0.f : fast_exp2(w[c].x - top);
                sum += f * w[c].y;
                acc.x += f * v[c].x, acc.y += f * v[c].y, acc.z += f * v[c].z, acc.w += f * v[c].w;
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint2 r = make_uint2(pack_pair<kBf16>(acc.x * inv, acc.y * inv),
                             pack_pair<kBf16>(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2 *>(
            a.out + (static_cast<size_t>(s) * a.num_q_heads + hk * p.group + h0 + h) * D + d4 * 4) = r;
    }
}

template <bool kBf16, int D, int NT, bool kDup>
__global__ void __launch_bounds__(kThreads, 1)
    decode_grouped_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ DecodeGroupedArgs p) {
    using C = Cfg<D, NT>;
    constexpr int TK = C::TK, kCost = C::kCost, MT = C::MT, KS = D / 16, kHeads = C::kHeads;
    const GroupedArgs &a = p.g;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float *obuf = reinterpret_cast<float *>(smem + C::OFF_O);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    long long *prefix = reinterpret_cast<long long *>(smem + C::OFF_PREFIX);
    long long *warp_sum = prefix + kChunks + 1;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    volatile int *last_flag = abort_flag + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * C::kStages;
    uint64_t *part_bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + kW * C::kStages;
    volatile uint32_t *stage_mask =
        reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MASK) + warp * C::kStages;
    uint8_t *ring = smem + warp * C::kStages * C::kStage;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        uint64_t *all = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
        for (int i = 0; i < kW * C::kStages; ++i) mbar_init(&all[i], 1);
        mbar_init(&all[kW * C::kStages], kW);
        mbar_init_fence();
    }
    allow_dependents_to_launch();
    grid_dependency_wait();

    const int units = a.num_kv_heads * p.chunks;
    // rows of sequences without keys are zero; bad lengths are reported
    auto zero_rows = [&]() {
        for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
            const int c = __ldg(a.context_lens + s);
            if (c > 0 && c <= a.max_blocks_per_seq * a.block_size) continue;
            if (c != 0 && threadIdx.x == 0) atomicOr(a.err, PA_DEVERR_CONTEXT);
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + static_cast<size_t>(s) * a.num_q_heads * D);
            for (int i = threadIdx.x; i < a.num_q_heads * (D / 8); i += kThreads)
                dst[i] = make_uint4(0, 0, 0, 0);
        }
    };

    // The line's length, and prefix[c], the tiles of the sequences before chunk
    // c.  Up to 32 sequences need no prefix: a warp's lanes hold them.
    Cursor<TK, kCost> cons;
    cons.base = -1;
    const bool small = a.num_seqs <= 32;
    long long total;
    if (small) {
        cons.s = 0;
        cons.load_group(a, lane);
        total = static_cast<long long>(make_geo<TK, kCost>(a, cons.ctx_l, cons.pre_l).len) * units;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) total += __shfl_xor_sync(0xffffffffu, total, o);
        __syncthreads();                              // the barriers are set up
    } else {
        constexpr int kPer = kChunks / kThreads;      // neighbouring entries per thread
        const int nchunks = (a.num_seqs + (1 << p.chunk_shift) - 1) >> p.chunk_shift;
        long long v[kPer], sum = 0;
        if (p.chunk_shift == 0) {     // an entry is a sequence: all loads at once
            int ctx[kPer], pre[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                ctx[i] = load_ctx(a, threadIdx.x * kPer + i);
                pre[i] = load_pre(a, threadIdx.x * kPer + i);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                v[i] = static_cast<long long>(make_geo<TK, kCost>(a, ctx[i], pre[i]).len) * units;
        } else
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = threadIdx.x * kPer + i;
            long long n = 0;
            if (c < nchunks) {
                const int s0 = c << p.chunk_shift;
                const int s1 = min(a.num_seqs, (c + 1) << p.chunk_shift);
                for (int s = s0; s < s1; ++s)
                    n += make_geo<TK, kCost>(a, load_ctx(a, s), load_pre(a, s)).len;
            }
            v[i] = n * units;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            sum += v[i];
            v[i] = sum;
        }
        long long run = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long t = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += t;
        }
        if (lane == 31) warp_sum[warp] = run;
        __syncthreads();
        run -= sum;
        for (int w = 0; w < warp; ++w) run += warp_sum[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) prefix[threadIdx.x * kPer + i + 1] = run + v[i];
        if (threadIdx.x == 0) prefix[0] = 0;
        __syncthreads();
        total = prefix[kChunks];
    }

    // Equal pieces.  Few tiles go to fewer CTAs: a context of n tiles is not
    // cut finer than about sqrt(n / 2) tiles, where one CTA's streaming of a
    // piece and its joining of the other pieces' partials take equally long.
    const float mean = static_cast<float>(total) / (static_cast<float>(a.num_seqs) * units);
    const int least = max(kW, static_cast<int>(sqrtf(mean * 0.5f)));
    const long long ctas = min(static_cast<long long>(gridDim.x), (total + least - 1) / least);
    if (blockIdx.x >= ctas) {
        zero_rows();
        return;
    }
    const long long f0 = blockIdx.x * total / ctas, f1 = (blockIdx.x + 1) * total / ctas;
    const int mine = static_cast<int>(f1 - f0);       // tiles of this CTA

    // the piece's start: its prefix entry, then its sequence within the entry
    {
        long long r = f0;
        int s = 0;
        if (!small) {
            int below = 0;
            for (int c = lane; c < kChunks; c += 32) below += prefix[c + 1] <= f0;
            const int c = __reduce_add_sync(0xffffffffu, below);
            r -= prefix[c];
            s = c << p.chunk_shift;
        }
        for (;;) {
            cons.s = s;
            if ((s & ~31) != cons.base) cons.load_group(a, lane);
            const long long n = lane >= (s & 31)
                                    ? static_cast<long long>(make_geo<TK, kCost>(a, cons.ctx_l, cons.pre_l).len) * units
                                    : 0;
            long long run = n;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const long long t = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += t;
            }
            const unsigned past = __ballot_sync(0xffffffffu, run > r);
            if (past) {
                const int l = __ffs(past) - 1;
                r -= __shfl_sync(0xffffffffu, run - n, l);
                cons.s = cons.base + l;
                cons.set_geo(a);
                cons.unit = static_cast<int>(r / cons.g.len);
                cons.idx = static_cast<int>(r - static_cast<long long>(cons.unit) * cons.g.len);
                break;
            }
            r -= __shfl_sync(0xffffffffu, run, 31);
            s = cons.base + 32;
            if (s >= a.num_seqs) return;   // cannot happen: f0 < total
        }
    }

    // ---------------------------------------------------------- producer side
    // A tile arrives as boxes of RB rows (8 for 8-token blocks, else 16): lane
    // i < TK / RB owns box i, its table entry and its two copies.
    const int B = a.block_size;
    const int RB = B == 8 ? 8 : 16;
    const int rb_shift = B == 8 ? 3 : 4;
    const int boxes = TK / RB;
    Cursor<TK, kCost> prod = cons;
    int at = 0;                              // tile of the piece `prod` is at
    // the lane's box of tile `at`: physical block (-1: not needed, -2: needed
    // but its entry is bad) and row within the block
    int box_blk = -1, box_row = 0;
    auto look_up = [&](int tile) {           // moves to the warp's first tile from `tile` on
        while (tile < mine) {
            prod.advance(a, units, tile - at, lane);
            at = tile;
            if (prod.idx < prod.g.nt) break;
            tile += kW;
        }
        at = tile;
        box_blk = -1;
        if (lane < boxes && tile < mine) {
            const int i = prod.idx;
            const int k = TK * (i < prod.g.na ? i : i + prod.g.skip) + lane * RB;
            if (k < prod.g.ctx && (k < prod.g.pre || k + RB > prod.g.lo)) {
                const int e = __ldg(a.block_tables + static_cast<size_t>(prod.s) * a.max_blocks_per_seq + k / B);
                box_blk = static_cast<unsigned>(e) < static_cast<unsigned>(a.num_blocks) ? e : -2;
                box_row = k % B;
            }
        }
    };
    auto issue = [&](int stage, int blk, int box_y, int unit) {
        // every lane has read the stage's last tile (the caller's __syncwarp)
        if (blk == -2) atomicOr(a.err, PA_DEVERR_TABLE);
        const unsigned have = __ballot_sync(0xffffffffu, blk >= 0);
        if (lane == 0) {
            stage_mask[stage] = have;
            mbar_arrive_expect_tx(&bar[stage], __popc(have) * 2u * RB * D * 2u);
        }
        __syncwarp();
        if (blk >= 0) {
            const int y = (blk * a.num_kv_heads + unit / p.chunks) * B + box_y;
            uint8_t *dst = ring + stage * C::kStage + lane * (RB * D * 2);
            tma_load_3d(dst, &tm_k, 0, y, 0, &bar[stage]);
            tma_load_3d(dst + C::kMat, &tm_v, 0, y, 0, &bar[stage]);
        }
    };
    int queue[C::kStages];                   // tiles issued and not yet taken
    int issued = 0;
    {
        int blk[C::kStages], y[C::kStages], un[C::kStages];
#pragma unroll
        for (int st = 0; st < C::kStages; ++st) {   // all entries before the first wait
            look_up(st == 0 ? warp : at + kW);
            queue[st] = at;
            blk[st] = box_blk, y[st] = box_row, un[st] = prod.unit;
        }
#pragma unroll
        for (int st = 0; st < C::kStages; ++st)
            if (queue[st] < mine) {
                issue(st, blk[st], y[st], un[st]);
                ++issued;
            }
    }
    look_up(at + kW);

    // ---------------------------------------------------------- consumer side
    // shared-memory layout of 16 keys: [D / 64 halves][16 rows][128 bytes],
    // or per 8-token box, [halves][8 rows][128 bytes]; 128-byte swizzle
    const uint32_t row_group = B == 8 ? 8 * D * 2 : 1024;   // rows 8-15 of 16
    const uint32_t half_step = B == 8 ? 1024 : 2048;        // dims 64 apart
    const uint32_t ring_addr = smem_addr(ring);
    // ldmatrix rows: K (a0: keys 0-7, a1: keys 8-15, a2, a3: next 8 dims);
    // V transposed (a0, a1: dims 0-7, 8-15 of keys 0-7; a2, a3: keys 8-15)
    const int krow = (lane & 7), kgrp = (lane >> 3) & 1, kchunk = lane >> 4;
    const int vgrp = lane >> 4, vchunk = (lane >> 3) & 1;
    const uint32_t k_lane = kgrp * row_group + krow * 128;
    const uint32_t v_lane = vgrp * row_group + krow * 128;
    const int col = 2 * (lane & 3);          // the lane's two head columns
    const int row = lane >> 2;               // its key row (and row + 8)

    uint32_t qf[KS][NT][2];
    float m[NT][2], l[NT][2], o[KS][NT][4], slope[NT][2];
    bool ok = true;
    int n_done = 0;                          // tiles taken
    int seg_start = 0;                       // CTA tile at which the segment starts

    auto load_q = [&]() {
        const int hk = cons.unit / p.chunks, h0 = (cons.unit % p.chunks) * kHeads;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(
            a.q + (static_cast<size_t>(cons.s) * a.num_q_heads + hk * p.group) * D);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int hq = h0 + nt * 8 + (kDup ? (lane >> 2) % 4 : lane >> 2);
            const bool live = hq < p.group;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[ks][nt][0] = live ? __ldg(src + (hq * D + ks * 16) / 2 + (lane & 3)) : 0u;
                qf[ks][nt][1] = live ? __ldg(src + (hq * D + ks * 16 + 8) / 2 + (lane & 3)) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = h0 + nt * 8 + (kDup ? (col + e) % 4 : col + e);
                slope[nt][e] = a.alibi_slopes && h < p.group
                                   ? __ldg(a.alibi_slopes + hk * p.group + h) * 1.4426950408889634f
                                   : 0.f;
            }
        }
    };

    load_q();
    while (seg_start < mine) {
        const Geo g = cons.g;
        const int seg_len = min(g.len - cons.idx, mine - seg_start);
        const int idx0 = cons.idx;
        if (idx0 >= g.nt) {   // the piece starts past the unit's tiles
            seg_start += seg_len;
            cons.idx += seg_len;
            if (seg_start < mine) {
                cons.advance(a, units, 0, lane);
                load_q();
            }
            continue;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[ks][nt][e] = 0.f;
        }
        // key k0 + i of a tile whose loaded boxes are `have`
        auto visible = [&](int k0, int i, unsigned have) {
            const int key = k0 + i;
            return (key < g.pre || key >= g.lo) && key < g.ctx && ((have >> (i >> rb_shift)) & 1);
        };
        while (queue[0] < seg_start + seg_len) {
            const int t = queue[0];
#pragma unroll
            for (int i = 0; i + 1 < C::kStages; ++i) queue[i] = queue[i + 1];
            queue[C::kStages - 1] = 0x7fffffff;
            const int st = n_done % C::kStages;
            const uint32_t ph = (n_done / C::kStages) & 1;
            ++n_done;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&bar[st], ph, abort_flag, a.err));
            if (!ok) continue;
            const int ti = idx0 + (t - seg_start);
            const int k0 = TK * (ti < g.na ? ti : ti + g.skip);
            const uint32_t kb = ring_addr + st * C::kStage, vb = kb + C::kMat;
            float sc[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t c16 = ks * 2 + kchunk;   // 16-byte chunk of the row
                const uint32_t off = (ks / 4) * half_step + (((c16 & 7) ^ krow) << 4);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t kf[4];
                    ldsm4(kf, kb + mt * (16 * D * 2) + k_lane + off);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<kBf16>(sc[mt][nt], kf, qf[ks][nt][0], qf[ks][nt][1]);
                }
            }
            // scores in the log2 domain
            const unsigned have = stage_mask[st];
            const bool partial = have != (1u << boxes) - 1 || k0 + TK > g.ctx ||
                                 (k0 < g.lo && k0 + TK > g.pre);
            bool raise = false;
            if (a.softcap > 0.f) {
                // Each score by the form that its own size asks for: the polynomial where it
                // holds (small scores would lose their low bits in 1 - 2 / (1 + e^(2u))).
                // So no score depends on another's, which may be of a key that is not
                // visible or of a box that was not loaded; a tile without far ones skips
                // the second form.
                bool far = false;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = sc[mt][nt][e] * p.cap_v;
                            far |= !(v * v < 2.f);
                        }
                far = __any_sync(0xffffffffu, far);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &x = sc[mt][nt][e];
                            const float s = x, v = x * p.cap_v, w = v * v;
                            float y = p.tanh_k[4];
#pragma unroll
                            for (int i = 3; i >= 0; --i) y = fmaf(y, w, p.tanh_k[i]);
                            x = v * y;
                            if (far && !(w < 2.f))
                                x = p.cap_log2 - 2.f * p.cap_log2 * fast_rcp(1.f + fast_exp2(s * p.cap_in));
                        }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[mt][nt][e] *= p.scale_log2;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = sc[mt][nt][e];
                        const int key = k0 + mt * 16 + row + (e >= 2 ? 8 : 0);
                        if (a.alibi_slopes) x -= slope[nt][e & 1] * static_cast<float>(g.ctx - 1 - key);
                        if (partial) x = visible(k0, key - k0, have) ? x : -INFINITY;
                        sc[mt][nt][e] = x;
                        raise |= x > __fadd_rd(m[nt][e & 1], kRaise);
                    }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = -INFINITY;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            x = fmaxf(x, fmaxf(sc[mt][nt][e], sc[mt][nt][e + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d *= 2)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if (x > __fadd_rd(m[nt][e], kRaise)) {
                            const float r = m[nt][e] == -INFINITY ? 0.f : fast_exp2(m[nt][e] - x);
                            m[nt][e] = x;
                            l[nt][e] *= r;
#pragma unroll
                            for (int ks = 0; ks < KS; ++ks) {
                                o[ks][nt][e] *= r;
                                o[ks][nt][e + 2] *= r;
                            }
                        }
                    }
            }
            uint32_t ph_[MT][NT][2], pl_[MT][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float b0 = m[nt][0] == -INFINITY ? 0.f : kBias - m[nt][0];
                const float b1 = m[nt][1] == -INFINITY ? 0.f : kBias - m[nt][1];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float w0 = fast_exp2(sc[mt][nt][2 * hf] + b0);
                        const float w1 = fast_exp2(sc[mt][nt][2 * hf + 1] + b1);
                        l[nt][0] += w0;
                        l[nt][1] += w1;
                        uint32_t hi, lo;
                        split_pair<kBf16>(w0, w1, hi, lo);
                        if constexpr (kDup) {
                            // columns 4-7 (lanes with col >= 4) carry the remainders
                            ph_[mt][nt][hf] = transpose8x8(col >= 4 ? lo : hi);
                            pl_[mt][nt][hf] = 0;
                        } else {
                            ph_[mt][nt][hf] = transpose8x8(hi);
                            pl_[mt][nt][hf] = transpose8x8(lo);
                        }
                    }
            }
            // O^T += V^T P^T
            auto pv = [&](auto masked) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
                    if constexpr (decltype(masked)::value) {
                        keep0 = keep1 = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool vis = visible(k0, mt * 16 + col + (e & 1) + (e >= 2 ? 8 : 0), have);
                            const uint32_t bits = vis ? ((e & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
                            if (e < 2)
                                keep0 |= bits;
                            else
                                keep1 |= bits;
                        }
                    }
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const uint32_t c16 = ks * 2 + vchunk;
                        const uint32_t off = (ks / 4) * half_step + (((c16 & 7) ^ krow) << 4);
                        uint32_t vf[4];
                        ldsm4_trans(vf, vb + mt * (16 * D * 2) + v_lane + off);
                        if constexpr (decltype(masked)::value) {
                            vf[0] &= keep0, vf[1] &= keep0, vf[2] &= keep1, vf[3] &= keep1;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<kBf16>(o[ks][nt], vf, ph_[mt][nt][0], ph_[mt][nt][1]);
                            if constexpr (!kDup)
                                mma16816<kBf16>(o[ks][nt], vf, pl_[mt][nt][0], pl_[mt][nt][1]);
                        }
                    }
                }
            };
            if (partial)
                pv(std::true_type{});
            else
                pv(std::false_type{});
            __syncwarp();
            if (at < mine) {
                issue(st, box_blk, box_row, prod.unit);
                ++issued;
                queue[C::kStages - 1] = at;
                look_up(at + kW);
            }
        }

        // ------------------------------------------------ end of the segment
        const int s = cons.s, unit = cons.unit;
        const int hk = unit / p.chunks, h0 = (unit % p.chunks) * kHeads;
        const int heads = min(kHeads, p.group - h0);
        // the unit's place on the line, and whether this piece covers it whole
        const bool from_start = idx0 == 0, to_end = idx0 + seg_len >= g.nt;
        const long long u0 = f0 + seg_start - idx0, u1 = u0 + g.nt;   // its tiles
        // the next unit's q is loaded while this one is merged
        seg_start += seg_len;
        cons.idx += seg_len;
        if (seg_start < mine) {
            cons.advance(a, units, 0, lane);
            load_q();
        }
        __syncthreads();   // everyone has read the previous merge
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
                const int h = nt * 8 + col + e;
                if (row == 0) ml[warp * kHeads + h] = make_float2(m[nt][e], x);
                float *dst = obuf + (warp * kHeads + h) * C::kRow + row;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    dst[ks * 16] = o[ks][nt][e];
                    dst[ks * 16 + 8] = o[ks][nt][e + 2];
                }
            }
        __syncthreads();
        constexpr int kVec = D / 4;            // float4s per head
        const bool whole = from_start && to_end;
        float *slot = p.partials + static_cast<size_t>(2 * blockIdx.x + (from_start ? 1 : 0)) *
                                       (kHeads * (D + 2));
        for (int i = threadIdx.x; i < heads * kVec; i += kThreads) {
            const int h = i / kVec, d4 = i % kVec;
            float mw[kW], top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                mw[w] = ml[w * kHeads + h].x;
                top = fmaxf(top, mw[w]);
            }
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float f = mw[w] == -INFINITY ? 0.f : fast_exp2(mw[w] - top);
                sum += f * ml[w * kHeads + h].y;
                float4 v = *reinterpret_cast<const float4 *>(obuf + (w * kHeads + h) * C::kRow + d4 * 4);
                if constexpr (kDup) {
                    const float4 r = *reinterpret_cast<const float4 *>(
                        obuf + (w * kHeads + h + 4) * C::kRow + d4 * 4);
                    v.x += r.x, v.y += r.y, v.z += r.z, v.w += r.w;
                }
                acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
            }
            if (whole) {
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                uint2 r = make_uint2(pack_pair<kBf16>(acc.x * inv, acc.y * inv),
                                     pack_pair<kBf16>(acc.z * inv, acc.w * inv));
                *reinterpret_cast<uint2 *>(
                    a.out + (static_cast<size_t>(s) * a.num_q_heads + hk * p.group + h0 + h) * D + d4 * 4) = r;
            } else {
                *reinterpret_cast<float4 *>(slot + h * D + d4 * 4) = acc;
                if (d4 == 0)
                    *reinterpret_cast<float2 *>(slot + kHeads * D + 2 * h) = make_float2(top, sum);
            }
        }
        if (!whole) {
            // pieces that hold part of the unit: the CTAs of its first and last tile
            const int i0 = static_cast<int>(((u0 + 1) * ctas - 1) / total);
            const int i1 = static_cast<int>((u1 * ctas - 1) / total);
            if (seg_start < mine) {
                // the warps go on; one of them sees to the ticket (a piece has at
                // most one such segment, its first)
                __syncwarp();
                if (lane == 0) mbar_arrive(part_bar);
                if (warp == kW - 1) {
                    ok = ok && __all_sync(0xffffffffu, mbar_wait(part_bar, 0, abort_flag, a.err));
                    if (ok && take_ticket(p, s, units, unit, i1 - i0, lane)) {
                        join_unit<kBf16, D, kHeads>(p, s, unit, i0, i1, lane, 32);
                    }
                }
            } else {
                __syncthreads();
                if (warp == 0) {
                    const bool last = take_ticket(p, s, units, unit, i1 - i0, lane);
                    if (lane == 0) *last_flag = last;
                }
                __syncthreads();
                if (*last_flag) join_unit<kBf16, D, kHeads>(p, s, unit, i0, i1, threadIdx.x, kThreads);
            }
        }
    }
    zero_rows();
    if (!ok) {   // let every copy already issued land before the CTA leaves
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
            mbar_wait_drain(&bar[i % C::kStages], (i / C::kStages) & 1);
    }
}

int heads_per_chunk(int head_dim, int group) { return group > 8 && head_dim != 256 ? 16 : 8; }

using Kernel = void (*)(CUtensorMap, CUtensorMap, DecodeGroupedArgs);
struct Variant {
    Kernel kernel;
    int smem, ctas_per_sm;
};
template <bool kBf16, int D>
Variant variant_of(int group) {
    if (D != 256 && group > 8)
        return {decode_grouped_kernel<kBf16, D, D == 256 ? 1 : 2, false>, Cfg<D, D == 256 ? 1 : 2>::kBytes,
                Cfg<D, D == 256 ? 1 : 2>::kCtasPerSm};
    if (group > 4)
        return {decode_grouped_kernel<kBf16, D, 1, false>, Cfg<D, 1>::kBytes, Cfg<D, 1>::kCtasPerSm};
    return {decode_grouped_kernel<kBf16, D, 1, true>, Cfg<D, 1>::kBytes, Cfg<D, 1>::kCtasPerSm};
}

}  // namespace

size_t decode_grouped_workspace_bytes(int head_dim, int group) {
    return static_cast<size_t>(2 * kMaxCtas) * heads_per_chunk(head_dim, group) * (head_dim + 2) * 4;
}
// A ticket for every unit, and nothing else (take_ticket); never 0, which says
// that the sizes are invalid.
size_t decode_grouped_counters_bytes(int num_seqs, int num_kv_heads, int group, int head_dim) {
    const int per = heads_per_chunk(head_dim, group);
    const size_t tickets = static_cast<size_t>(num_seqs) * num_kv_heads * ((group + per - 1) / per);
    return (tickets < 1 ? 1 : (tickets + 63) / 64) * 256;
}

cudaError_t launch_decode_grouped(const GroupedArgs &args, int dtype, int head_dim, int num_sms,
                                  cudaStream_t stream) {
    const bool bf16 = dtype == PA_DTYPE_BF16;
    const int B = args.block_size, Hk = args.num_kv_heads;
    DecodeGroupedArgs p;
    p.g = args;
    const double log2e = 1.4426950408889634;
    p.scale_log2 = static_cast<float>(args.scale * log2e);
    p.cap_log2 = static_cast<float>(args.softcap * log2e);
    p.cap_in = args.softcap > 0.f ? static_cast<float>(2.0 * args.scale / args.softcap * log2e) : 0.f;
    fill_tanh(args.scale, args.softcap, &p.cap_v, p.tanh_k);
    p.group = args.num_q_heads / Hk;
    const int per = heads_per_chunk(head_dim, p.group);
    p.chunks = (p.group + per - 1) / per;
    p.chunk_shift = 0;
    while (((static_cast<long long>(args.num_seqs) - 1) >> p.chunk_shift) >= kChunks) ++p.chunk_shift;
    p.partials = static_cast<float *>(args.workspace);

    // [D / 64 halves] x [all cache rows] x 64 dims: one box is a block's rows
    // (or 16 of them) of one head, each half in the 128-byte swizzle
    CUtensorMap tm_k, tm_v;
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(args.num_blocks) * Hk * B,
                                static_cast<cuuint64_t>(head_dim / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(B == 8 ? 8 : 16),
                               static_cast<cuuint32_t>(head_dim / 64)};
    if (!encode(&tm_k, bf16, args.k_cache, 3, dims, strides, box) ||
        !encode(&tm_v, bf16, args.v_cache, 3, dims, strides, box))
        return cudaErrorInvalidValue;

    Variant v;
    if (bf16)
        v = head_dim == 64 ? variant_of<true, 64>(p.group)
                           : (head_dim == 128 ? variant_of<true, 128>(p.group) : variant_of<true, 256>(p.group));
    else
        v = head_dim == 64 ? variant_of<false, 64>(p.group)
                           : (head_dim == 128 ? variant_of<false, 128>(p.group) : variant_of<false, 256>(p.group));
    // the kernel's shared-memory limit, once per device and variant
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    {
        static std::mutex mu;
        static bool ready[64][18] = {};
        const int which = (bf16 ? 9 : 0) + (head_dim == 64 ? 0 : head_dim == 128 ? 3 : 6) + (p.group <= 4 ? 0 : p.group <= 8 ? 1 : 2);
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[device][which]) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(v.kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
            if (e != cudaSuccess) return e;
            ready[device][which] = true;
        }
    }
    const int ctas = v.ctas_per_sm * num_sms;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < kMaxCtas ? ctas : kMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = v.smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *params[] = {&tm_k, &tm_v, &p};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(v.kernel), params);
}

}  // namespace pa
