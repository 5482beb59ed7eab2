// pa_prefill_grouped.cu -- many queries of each sequence over the paged cache,
// with query heads that share K/V heads, on the tcgen05 tensor cores (sm_103a).
//
// Mathematics: for query row (token at position p, head g of K/V head h) and
// key j, x_j = log2(e) f(scale q . k_j) with f the optional tanh cap and
// distance bias, and o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m) over the
// visible keys, in one pass over tiles of keys with a reference m that is only
// raised when a tile's maximum exceeds it by about 8 (a common factor of
// weights and sum cancels, so m need not be the maximum).
//
// What bounds it: 4 D flops per (row, key) pair on the tensor cores; beside
// them the softmax warps spend an ex2 a pair on the special-function unit, and
// with the cap a polynomial of 7 products on the FMA pipe.
//
// Measured (32 heads on 4, one prompt of 8192 tokens, bf16): head_dim 128 330 us,
// 1660 TFLOP/s, 0.87 of this GPU's largest library product, the products bound;
// with distance biases 362 us; with the cap 503 us, 1093 TFLOP/s, the latency of
// the softmax warps' longer chains, two warps a scheduler (no pipe is busier than
// 46 %: tensor 46, FMA 45, special functions 39; an instruction in 0.58 of the
// cycles); head_dim 64 327 us, 841 TFLOP/s, the softmax again, with half the
// products a pair.  16 prompts of 333 to 1024 tokens, 32 heads on 8: 79 us, 840
// TFLOP/s (118 capped): the first key tile of an item and its output cost as much
// as several tiles.
//
// How (persistent, one CTA per SM, 512 threads):
//  * A tile is 128 rows of (token, head) pairs: 128 / G tokens x the G heads of
//    one K/V head, gathered by one tensor-map box of Q, so K and V are loaded
//    and multiplied once for all heads that share them.  A work item is two
//    such tiles, one K/V head, one sequence, and a range of key tiles.
//  * Warp 8 takes items from a queue, heaviest first, describes each to the
//    other roles through a two-slot ring, and streams Q and tiles of 64 keys of
//    K; warp 13 streams V.  One copy brings a block of one head, in groups of 8
//    keys x (64 dims, 64 dims), the operand layout of both products.  Issuing a
//    copy takes about 100 cycles: with one warp for both and a copy per 64-dim
//    half, 16 copies a tile took 1600 of its 2400 cycles.
//  * Warps 9, 10 issue S = Q K^T of query tile 0 and 1 into the next of two S/P
//    buffers of tensor memory (three at head_dim 64, where there is room), ahead of the softmax, once the P V product that
//    last read the buffer is complete; warps 11, 12 issue O += P V (P read from
//    tensor memory) once the softmax has stored P.  A thread's stream of
//    tcgen05.mma is bound by its own issue and waits, so the four streams have
//    warps of their own: with S and P V of a tile issued by one thread, a step
//    of 64 keys took 2600 cycles, all of them the thread's.  The issuing lane
//    is an elected one (at first 1552 TFLOP/s on that prompt, 1416 under
//    `lane == 0`, where every operand is moved to a uniform register first).
//  * Warps 0-3 / 4-7 (softmax of tile 0 / 1): thread = row = tensor-memory
//    lane.  Loads its 64 scores, exponentiates, and stores the weights as
//    16-bit values over the scores.  Weights are first taken against the
//    running reference as it is: a small enough row sum proves that all of them
//    fit the type, and no maximum is needed.  (One load of all 64: taken in
//    halves, the second under the first's weights, 8192 tokens took 351 us
//    instead of 332.)  Otherwise (always on a tile's
//    first keys) the scores are loaded again, which P has not overwritten yet,
//    and the maximum comes first.  With a distance bias the key tiles are taken
//    from the row's own position backwards, so that scores fall along the way
//    and the reference need not be raised at every tile.
//  * tanh: an odd polynomial on the FMA pipe (degree 9, |u| <= 0.75, within
//    5e-7); a tile with visible scores past that is taken again with 1 - 2 /
//    (1 + e^(2u)) for these, whose two special-function operations per score
//    cost 3400 cycles per 128 keys where a polynomial of degree 11 cost 1300.
//  * The weights are rounded to 16 bits (the element type) before P V, the sum
//    is taken before the rounding, in fp32.  A weight is then off by half a
//    step of the type, independently of its neighbours, so the output's error
//    grows to about 1.4 times that of its own final rounding; carrying a
//    second 16-bit term would cost half as much tensor work again.
//  * V rows that no query may see (past the context, or of blocks that are not
//    loaded) are cleared, since a zero weight times a NaN is NaN.
//  * Masks: tiles that every row of a warp sees whole take no mask; the causal
//    diagonal is one bound per key under a minimum; windows, prefixes and blocks
//    that are missing take a bit mask and a select a key.  A row without a query
//    stands where its warp's last one does, so that it adds no mask (5 prompts
//    of 517 to 2500 tokens, three heads to one: 67 us, and 49 so).
//  * Few rows over long contexts: while there are fewer items than SMs, an
//    item's key tiles are split over several CTAs, which leave partial (max,
//    sum, output) and take a ticket; the last one joins them in order.
//  * Q has two buffers, so that the next item's is there when its turn comes.
//    The output rows are staged in their item's Q, whose products are complete,
//    and leave as one tensor copy per warp and 64 dims, while the softmax goes
//    on with the next item (row by row they cost 6400 cycles an item, by
//    coalesced stores 3800).  Rows that are not 32 of whole tokens (a ragged
//    end, or G that does not divide 32) take the coalesced stores.
//  * Every wait is bounded; tensor memory is released on every path.
//
// Over an 8-bit cache (kQ8): the same kernel with fp16 operands for both types outside.
// K and V blocks arrive by untiled copies in the upper half of their tile's slot, and warps
// 14 and 15 widen each tile where it lies (widen_tile), so the ring has as many tiles as
// that of 16 bits and the products see no difference. A key tile of 64 x 128 costs its warp
// 128 conversions of pairs a lane; with bf16 operands, three instructions more for each pair, the
// two warps set the pace (chunks of 512 tokens over 4097 to 8192 keys, 32 heads on 8: 313
// us, and 174 so; a 16-bit cache 152). A bf16 Q is made fp16 by its softmax threads, row by
// row with a scale of its own, while the item before waits for its last product.
// Measured: those chunks 161 us, 1165 TFLOP/s (fp16 150), with the items by falling numbers
// of keys (ByLength); 8191 tokens of head_dim 64, 32 heads on 4, distance biases 373 us
// (fp16 359, the 16-bit cache's time).
// What bounds it at head_dim 128 is shared memory: the products' operands take 87 of its 128
// bytes a cycle, and a step's tiles are written as bytes, read, and written widened (1060
// cycles a tile of a step's 1500, half of them waiting for the stores to drain). Between
// items nothing makes up for it: one prompt of 8192 tokens, 32 heads on 4, takes 368 us in
// fp16 (335 over 16 bits), 16 prompts of 333 to 1024 tokens 90 (81); and a bf16 Q costs
// another 3500 cycles an item, for the same reason: 400 and 108 us. Bytes loaded to registers
// by three warps instead of staged took 632 us (latency), half a tile ahead in registers 409.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_tensor.cuh"

namespace pa {
namespace {

constexpr int kBM = 128;               // rows per tile (MMA M)
constexpr int kBN = 64;                // keys per tile
constexpr int kThreads = 512;          // 2 x 4 softmax warps, 2 TMA warps, 4 MMA warps, 2 that widen
constexpr int kTmaWarp = 8;            // items, Q, K
constexpr int kVWarp = 13;
constexpr int kSWarp0 = 9;
constexpr int kPvWarp0 = 11;
constexpr int kWidenWarp0 = 14;        // 8-bit caches: K, then V; idle otherwise
// Register split: launched at 128 per thread; the warpgroups of the TMA and
// MMA warps give registers up to the softmax warps: 2 x 168 + 2 x 88 = 4 x 128.
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
constexpr uint32_t kTmemCols = 512;
// Where a maximum is taken, the reference is kept if it is this near.  The sum is
// rounded down: past 2^26 fp32's step is 8 and the bias below may become 8, so a
// score one step above the reference would have a weight of 2^16, past fp16.
constexpr float kRaise = 7.9f;
// Weights are 2^(x - m + bias).  fp16 holds at most 2^16: a row sum of up to
// 2^15 proves every weight fits; bf16 has the exponent range of fp32, and its
// reference hardly ever has to be raised.
constexpr float kBias = 4.f;
template <bool kBf16> constexpr float kMostSum = kBf16 ? 1.1529215e18f : 32768.f;   // 2^60, 2^15
constexpr float kFar = 1e30f;
// Up to this cap one score in four may be taken by 1 - 2 / (1 + e^(2u)) whatever
// its size, which is off by up to 2^-20 of the cap: a quarter of what the weights'
// rounding to the type moves.  Past it every score is taken by the form of its own
// size, off by 2^-20 of itself, in the second form of the weights (one prompt of
// 8192 tokens 504 us at a cap of 30, 686 past the limit).
template <bool kBf16> constexpr float kShareCap = kBf16 ? 1024.f : 128.f;
constexpr int kMaskRing = 32;         // key tiles whose blocks are known; see Cfg
// Work is split over keys while there are fewer items than SMs (152).
constexpr int kSplitTarget = 152;
constexpr int kCounters = 2 + 2 * kSplitTarget;   // queue head, CTAs done, a ticket per (item, tile)

struct PrefillGroupedArgs {
    GroupedArgs g;
    float scale_log2, cap_log2, cap_in;
    float cap_v;                       // v = cap_v (q . k) has v^2 < 2 iff |s / cap| < 0.75
    float tanh_k[5];                   // there, x = v (k0 + k1 v^2 + ... + k4 v^8)
    int group, tpt;                    // heads per K/V head; tokens per tile
    int num_pairs, splits;
    int store_boxes;                   // a warp's 32 rows are whole tokens: tm_out applies
    int num_items;                     // num_pairs * splits * S * Hkv
    float *partials;                   // [item without split][split][tile][D + 2][128]
};

// Everything the roles need to know of an item (the TMA warp writes it).
struct Item {
    int done;                          // 1: the queue is empty
    int hk, q_first, tok0, q_len, ctx, pre;
    int first_pos;                     // position of the pair's first token
    int na, skip;                      // key tile of list entry i: i < na ? i : i + skip
    int j0, nkt;                       // list entries of this split
    int nk0, nk1;                      // of which tile 0 / 1 needs the first nk
    int split, splits;                 // this split, of how many
    int slot;                          // item without its split (partials, tickets)
    int joins;                         // bit t: parity of tile t's split items so far
    int s;
};

template <int D, bool kQ8>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfQ = kBM * 128;
    static constexpr int kTileQ = kHalves * kHalfQ;
    static constexpr int kGroup = kHalves * 1024;  // 8 keys of a K or V tile
    static constexpr int kTileKV = kBN / 8 * kGroup;
    static constexpr int kSlots = D == 64 ? 8 : 3;  // tiles of K, and of V
    // tensor memory: S/P buffer b of tile t at columns 64 (kBufs t + b), then O.
    // A third buffer (head_dim 64 leaves room) takes P V out of the next S's way.
    static constexpr uint32_t kBufs = D == 64 ? 3 : 2;
    static constexpr uint32_t TM_O = 2 * kBufs * 64;
    static_assert(TM_O + 2 * D <= kTmemCols, "tensor memory");
    static constexpr int OFF_Q = 0;                              // [item parity][tile]
    static constexpr int OFF_K = 4 * kTileQ;
    static constexpr int OFF_V = OFF_K + kSlots * kTileKV;
    static constexpr int OFF_BAR = OFF_V + kSlots * kTileKV;
    static constexpr int Q_FULL = 0, V_LAND = 2;                 // Q_FULL: [item parity]
    static constexpr int S_FULL = 3, P_FULL = 9, PV_DONE = 15;   // [tile][buffer]
    static constexpr int MMA_DONE = 21;                          // [issuing thread]
    static constexpr int ITEM_FULL = 25, ITEM_EMPTY = 27;
    static constexpr int PARTS = 29, TICKET = 31;                // [tile]
    static constexpr int K_FULL = 33, V_FULL = K_FULL + kSlots;
    static constexpr int K_EMPTY = V_FULL + kSlots, V_EMPTY = K_EMPTY + kSlots;
    // 8-bit caches: a tile's bytes are there (K, then V), to be widened
    static constexpr int K_BYTES = V_EMPTY + kSlots, V_BYTES = K_BYTES + (kQ8 ? kSlots : 0);
    // a bf16 Q is there as fp16: [item parity][tile]
    static constexpr int Q_READY = V_BYTES + (kQ8 ? kSlots : 0);
    static constexpr int kNumBars = Q_READY + (kQ8 ? 4 : 0);
    static constexpr int OFF_TMEM = OFF_BAR + kNumBars * 8;
    static constexpr int OFF_FLAG = OFF_TMEM + 4;
    static constexpr int OFF_LAST = OFF_FLAG + 4;                   // int[2]
    static constexpr int OFF_MASK = OFF_LAST + 8;                   // uint32[kMaskRing]
    static constexpr int OFF_ITEM = OFF_MASK + kMaskRing * 4;       // Item[2]
    static constexpr int OFF_INFO = OFF_ITEM + 2 * static_cast<int>(sizeof(Item));   // uint32[kSlots]: V's rows
    static constexpr int kSmemBytes = OFF_INFO + (kQ8 ? kSlots * 4 : 0) + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory");
    // A tile's entry in the mask ring is read by the softmax before its P and is
    // rewritten without a wait, so the ring is longer than the K warp can get
    // ahead of a softmax that stands at tile a: V is loaded up to a + kSlots - 1
    // (P V of tile a holds its slot), the other query tile's S goes kBufs products
    // past that and over the kBufs - 1 tiles for which the first one has S ahead,
    // and K is loaded kSlots further.  With 16 entries a context's last key tile
    // could stand in for another at head_dim 64.
    static_assert(2 * kSlots + 2 * static_cast<int>(kBufs) - 2 < kMaskRing, "mask ring");
};

// kind::f16 instruction descriptor: fp32 accumulate, A and B fp16 or bf16, A
// K-major, B K-major or MN-major, M = 128.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool b_mn, int n) {
    return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kBM >> 4) << 24);
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
// The low n bits set (none for n <= 0, all from n = 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
// Keys 32 q .. 32 q + 31 of a tile that lie in blocks with their bit in `have`.
__device__ __forceinline__ uint32_t present(unsigned have, int q, int block_size) {
    if (block_size == 32) return (have >> q) & 1 ? 0xffffffffu : 0u;
    if (block_size == 16)
        return ((have >> (2 * q)) & 1 ? 0xffffu : 0u) | ((have >> (2 * q + 1)) & 1 ? 0xffff0000u : 0u);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m |= (have >> (4 * q + i)) & 1 ? 0xffu << (8 * i) : 0u;
    return m;
}
__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// The item of a pair of tiles, a sequence and a K/V head.  False for an empty item, or
// for a sequence whose lengths are inconsistent (reported once).
__device__ __forceinline__ bool item_geometry(const PrefillGroupedArgs &p, int s, int hk, int pair, int split,
                                              bool report, Item &it) {
    const GroupedArgs &a = p.g;
    const int q_first = __ldg(a.query_start + s), q_end = __ldg(a.query_start + s + 1);
    const int ctx = __ldg(a.context_lens + s);
    const int pre_raw = a.prefix_lens ? __ldg(a.prefix_lens + s) : 0;
    const bool rows_bad = q_first < 0 || q_end < q_first || q_end > a.total_q;
    const int q_len = rows_bad ? 0 : q_end - q_first;
    const int tok0 = pair * 2 * p.tpt;
    if (rows_bad || (q_len > 0 && (q_len > ctx || ctx > a.max_blocks_per_seq * a.block_size ||
                                   q_len > a.max_q))) {
        if (report && hk == 0 && pair == 0 && split == 0) atomicOr(a.err, PA_DEVERR_CONTEXT);
        return false;
    }
    if (tok0 >= q_len) return false;
    it.done = 0;
    it.s = s;
    it.hk = hk;
    it.q_first = q_first;
    it.tok0 = tok0;
    it.q_len = q_len;
    it.ctx = ctx;
    it.pre = max(0, min(pre_raw, ctx));
    it.first_pos = ctx - q_len + tok0;
    // keys: [0, pre) and [lo, up), as a list of key tiles
    const int last_tok = min(tok0 + 2 * p.tpt, q_len) - 1;
    const int up = max(ctx - q_len + last_tok + 1, it.pre);
    const int lo = a.window > 0 ? max(0, it.first_pos - a.window + 1) : 0;
    const int total = (up + kBN - 1) / kBN, first = lo / kBN;
    int count;
    it.na = (it.pre + kBN - 1) / kBN;
    if (first <= it.na && it.pre > 0) {
        it.na = 0, it.skip = 0, count = total;
    } else {
        it.skip = first - it.na;
        count = it.na + max(total - first, 0);
    }
    // tile 0 ends earlier: its last token's key, or the prefix
    const int up0 = max(min(it.first_pos + p.tpt, ctx), it.pre);
    const int end0 = (up0 + kBN - 1) / kBN;
    const int need0 = min(count, end0 <= it.na ? end0 : max(it.na, end0 - it.skip));
    // one split per about sqrt(count / 2) tiles of 128 keys: there, streaming a
    // part and joining the others' partials take about equally long
    int parts = 1;
    if (p.splits > 1) {
        constexpr float kUnit = 128.f / kBN;
        const int per = static_cast<int>(ceilf(kUnit * fmaxf(2.f, sqrtf(0.5f * count / kUnit))));
        parts = min(p.splits, (count + per - 1) / per);
    }
    if (split >= parts) return false;
    const int j1 = static_cast<int>(static_cast<long long>(count) * (split + 1) / parts);
    it.j0 = static_cast<int>(static_cast<long long>(count) * split / parts);
    it.nkt = j1 - it.j0;
    it.nk0 = max(0, min(need0, j1) - it.j0);
    it.nk1 = tok0 + p.tpt < q_len ? it.nkt : -1;   // -1: tile 1 has no rows
    it.split = split;
    it.splits = parts;
    it.slot = (pair * a.num_seqs + s) * a.num_kv_heads + hk;
    return true;
}
// Work item w: (pair level, split, sequence, K/V head), latest pairs first.
__device__ __forceinline__ bool item_geometry(const PrefillGroupedArgs &p, int w, bool report,
                                              Item &it) {
    const GroupedArgs &a = p.g;
    const int sh = a.num_seqs * a.num_kv_heads;
    const int level = w / (sh * p.splits);
    int rem = w - level * (sh * p.splits);
    const int split = rem / sh;
    rem -= split * sh;
    const int s = rem / a.num_kv_heads;
    return item_geometry(p, s, rem - s * a.num_kv_heads, p.num_pairs - 1 - level, split, report, it);
}

// The same work by falling numbers of keys whatever sequence they are of, for up to 32
// sequences (a lane has one) and one to four rounds of CTAs (with more the rest evens out
// by itself: 16 prompts of 333 to 1024 tokens, fp16, 101 us so, 90 by levels): a chunk of
// a long context that starts last would run alone at the end (four chunks of 512 tokens
// over 4097 to 8192 keys, bf16: 174 us by levels of pairs, 158 so).  A sequence's pairs end
// `step` keys apart, so how many of them end at T or later is a division, and the r-th place
// is found by halving the range of T.  Calls with distance biases keep the levels: their
// loop pays for the code beside it (8191 tokens of head_dim 64 359 us, 381 with it).
constexpr unsigned kOrderedRounds = 4;
struct ByLength {
    int end, n, step, total, most;         // end of the last pair's keys; pairs; sums over the lanes
    __device__ __forceinline__ void load(const PrefillGroupedArgs &p, int lane) {
        const GroupedArgs &a = p.g;
        step = 2 * p.tpt;
        end = n = 0;
        if (lane < a.num_seqs) {
            const int q0 = __ldg(a.query_start + lane), q1 = __ldg(a.query_start + lane + 1);
            const int ctx = __ldg(a.context_lens + lane), q = q1 - q0;
            const bool rows_bad = q0 < 0 || q1 < q0 || q1 > a.total_q;
            const bool bad = rows_bad || (q > 0 && (q > ctx || ctx > a.max_blocks_per_seq * a.block_size || q > a.max_q));
            if (bad && blockIdx.x == 0) atomicOr(a.err, PA_DEVERR_CONTEXT);
            if (!bad && q > 0) {
                n = (q - 1) / step + 1;
                end = ctx - q + n * step;
            }
        }
        total = __reduce_add_sync(0xffffffffu, n);
        most = __reduce_max_sync(0xffffffffu, end);
    }
};
// Place r < total: its sequence (low 5 bits) and pair.  A call of its own: inlined, its
// registers cost the loop around it (one prompt of 8192 tokens, which has no use for it,
// 382 -> 397 us).
__device__ __noinline__ int find_place(int end, int n, int step, int most, int r) {
    auto at_least = [&](int t) { return __reduce_add_sync(0xffffffffu, end < t ? 0 : min(n, (end - t) / step + 1)); };
    int lo = 1, hi = most;                 // the largest T that r + 1 pairs reach
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (at_least(mid) > r)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int back = end < lo ? 0 : (end - lo) / step;
    const bool here = end >= lo && back < n && end - back * step == lo;
    const unsigned mask = __ballot_sync(0xffffffffu, here);
    const int s = static_cast<int>(__fns(mask, 0, r - at_least(lo + 1) + 1)) & 31;
    return __shfl_sync(0xffffffffu, n - 1 - back, s) << 5 | s;
}

// A sequence's blocks of one K/V head, as the copies of K and V take them:
// lane i holds block i of a key tile.  Only blocks that some query of the
// sequence sees are read.
struct KeyBlocks {
    const int32_t *table;
    int ctx, pre, lo_seq, num_blocks, heads, hk, b_shift, lane;
    bool descending;
    __device__ __forceinline__ KeyBlocks(const GroupedArgs &a, int s, int hk_, int ctx_, int pre_, int q_len,
                                         int shift, int lane_, bool desc)
        : table(a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq), ctx(ctx_), pre(pre_),
          lo_seq(a.window > 0 ? max(0, ctx_ - q_len - a.window + 1) : 0), num_blocks(a.num_blocks),
          heads(a.num_kv_heads), hk(hk_), b_shift(shift), lane(lane_), descending(desc) {}
    __device__ __forceinline__ int first_key(const Item &it, int j) const {
        const int i = it.j0 + (descending ? it.nkt - 1 - j : j);
        return kBN * (i < it.na ? i : i + it.skip);
    }
    // The lane's physical block of list entry j: -1 if it is not needed, -2 if
    // its entry is bad.
    __device__ __forceinline__ int entry(const Item &it, int j) const {
        const int key = first_key(it, j) + (lane << b_shift);
        if (lane >= (kBN >> b_shift) || key >= ctx || (key >= pre && key + (1 << b_shift) <= lo_seq)) return -1;
        const int e = __ldg(table + (key >> b_shift));
        return static_cast<unsigned>(e) < static_cast<unsigned>(num_blocks) ? e : -2;
    }
    // The block's first group of 8 keys in the cache.
    __device__ __forceinline__ int group(int blk) const { return (blk * heads + hk) << (b_shift - 3); }
};

// A tile of kBN keys of an 8-bit cache, widened where it lies: its bytes are in the
// upper half of the slot, key after key, and become the slot's 16-bit operand
// layout.  Groups of 8 keys in order, each read before the one ahead of it is
// written: a group's output ends where the bytes of the next one start, or before.
// valid(key): keys to keep, the others become 0.
//
// A lane's chunk of 16 numbers: lanes 8 q .. 8 q + 7 take keys 2 q and 2 q + 1, half a
// row of each and not the same half, so that neither the loads nor the stores (every
// other 16-byte chunk of a line, even ones of one key and odd ones of the next) meet
// in a bank.
template <int D, typename Valid>
__device__ __forceinline__ void widen_tile(uint8_t *slot, int lane, Valid &&valid) {
    constexpr int kGroup = D * 16, kIn = D * 8, kPer = D / 64;   // bytes out and in a group; chunks a lane
    const uint8_t *in = slot + kBN * D;
    const int y = D == 64 ? lane / 4 : lane / 8 * 2 + (lane >> 2 & 1);   // key within the group
    auto chunk_of = [&](int u) { return (lane & 3) + (D == 64 ? 0 : 4 * ((lane >> 2 & 1) ^ u)); };
    uint4 next[kPer];
    auto fetch = [&](int g) {
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            next[u] = *reinterpret_cast<const uint4 *>(in + g * kIn + y * D + chunk_of(u) * 16);
    };
    fetch(0);
#pragma unroll
    for (int g = 0; g < kBN / 8; ++g) {
        uint4 now[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) now[u] = valid(g * 8 + y) ? next[u] : make_uint4(0, 0, 0, 0);
        if (g + 1 < kBN / 8) fetch(g + 1);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t w[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = e4m3x2_to_f16x2(w[i]);
                o[2 * i + 1] = e4m3x2_to_f16x2_high(w[i]);
            }
            const int c = chunk_of(u), c16 = 2 * (c & 3);
            uint8_t *line = slot + g * kGroup + (c >> 2) * 1024 + y * 128;
            *reinterpret_cast<uint4 *>(line + ((c16 ^ y) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(line + (((c16 + 1) ^ y) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// kSplit: the call has key splits.  A call without them runs a kernel that leaves
// out the code that writes and joins partials, which the softmax warps' loop pays
// for although it does not run (one prompt of 8192 tokens: 348 us with it, 333
// without).
template <bool kBf16, bool kQ8, int D, bool kCap, bool kAlibi, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_grouped_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_out,
                           const __grid_constant__ PrefillGroupedArgs p) {
    using C = Cfg<D, kQ8>;
    // over an 8-bit cache the products are fp16's whatever the type outside is
    constexpr bool kMmaBf16 = kBf16 && !kQ8, kScaleQ = kBf16 && kQ8;
    const GroupedArgs &a = p.g;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    volatile int *last_flag = reinterpret_cast<volatile int *>(smem + C::OFF_LAST);
    volatile uint32_t *mask_ring = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MASK);
    Item *items = reinterpret_cast<Item *>(smem + C::OFF_ITEM);
    [[maybe_unused]] volatile uint32_t *v_rows = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_INFO);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int B = a.block_size, b_shift = B == 8 ? 3 : (B == 16 ? 4 : 5);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            uint32_t count = 1;
            if ((i >= C::P_FULL && i < C::P_FULL + 6) || i == C::PARTS || i == C::PARTS + 1 ||
                (kQ8 && i >= C::Q_READY))
                count = 4;                                    // softmax warps
            if (i == C::ITEM_EMPTY || i == C::ITEM_EMPTY + 1) count = kQ8 ? 15 : 13;     // 4 MMA threads, 8 softmax warps, V, 2 that widen
            if (i >= C::K_EMPTY && i < C::V_EMPTY + C::kSlots) count = 2;               // both tiles' threads
            mbar_init(&bar[i], count);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(const_cast<uint32_t *>(tmem_slot))),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    allow_dependents_to_launch();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kTmaWarp) {
            // -------------------------------------------------------- items, Q, K
            uint32_t g = 0;                        // K tiles issued, over all items
            bool first_item = true;
            int k = 0, q_loads = 0;                // items whose K is issued, Q loads issued
            int joins = 0;                         // bit t: parity of tile t's split items
            bool ok = true;
            const bool by_length = kQ8 && !kAlibi && a.num_seqs <= 32 && a.num_seqs > 1 && p.splits == 1 &&
                                   static_cast<unsigned>(p.num_items) > gridDim.x &&
                                   static_cast<unsigned>(p.num_items) <= kOrderedRounds * gridDim.x;
            ByLength order = {};
            if (by_length) order.load(p, lane);
            for (;;) {
                int w = 0;
                Item it;
                for (;;) {
                    // the first item by the CTA's index, the rest from the queue
                    if (first_item) {
                        w = blockIdx.x;
                        first_item = false;
                    } else {
                        if (lane == 0) w = static_cast<int>(gridDim.x + atomicAdd(a.counters, 1u));
                        w = __shfl_sync(0xffffffffu, w, 0);
                    }
                    if (static_cast<unsigned>(w) >= static_cast<unsigned>(p.num_items)) break;
                    if (by_length) {
                        const int r = w / a.num_kv_heads;
                        if (r >= order.total) {    // the rest are empty
                            w = p.num_items;
                            break;
                        }
                        const int at = find_place(order.end, order.n, order.step, order.most, r);
                        if (item_geometry(p, at & 31, w - r * a.num_kv_heads, at >> 5, 0, false, it)) break;
                        continue;
                    }
                    if (item_geometry(p, w, lane == 0, it)) break;
                }
                const bool done = static_cast<unsigned>(w) >= static_cast<unsigned>(p.num_items);
                const int slot = k % 2;
                it.joins = joins;
                if (!done && it.splits > 1) joins ^= it.nk1 >= 0 ? 3 : 1;
                ok = warp_all(mbar_wait(&bar[C::ITEM_EMPTY + slot], ((k / 2) & 1) ^ 1, abort_flag, a.err));
                if (!ok) break;
                if (lane == 0) {
                    if (done)
                        items[slot].done = 1;
                    else
                        items[slot] = it;
                    mbar_arrive(&bar[C::ITEM_FULL + slot]);
                }
                if (done) break;
                // Q into the buffer of the item before the last, whose roles are done
                if (lane == 0) {
                    const int nt = it.nk1 >= 0 ? 2 : 1;
                    mbar_arrive_expect_tx(&bar[C::Q_FULL + slot],
                                          static_cast<uint32_t>(nt * p.tpt * p.group * D * 2));
                    for (int t = 0; t < nt; ++t)
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            tma_load_3d(smem + C::OFF_Q + (slot * 2 + t) * C::kTileQ + hf * C::kHalfQ, &tm_q,
                                        hf * 64, it.hk * p.group, it.q_first + it.tok0 + t * p.tpt,
                                        &bar[C::Q_FULL + slot]);
                }
                ++q_loads;
                __syncwarp();
                KeyBlocks blocks(a, it.s, it.hk, it.ctx, it.pre, it.q_len, b_shift, lane, kAlibi);
                int blk = blocks.entry(it, 0);
                for (int j = 0; j < it.nkt; ++j) {
                    const int next = j + 1 < it.nkt ? blocks.entry(it, j + 1) : -1;
                    if (blk == -2) atomicOr(a.err, PA_DEVERR_TABLE);
                    const unsigned have = __ballot_sync(0xffffffffu, blk >= 0);
                    const int st = g % C::kSlots;
                    ok = warp_all(mbar_wait(&bar[C::K_EMPTY + st], ((g / C::kSlots) & 1) ^ 1, abort_flag, a.err));
                    if (!ok) break;
                    if (lane == 0) {
                        mask_ring[g % kMaskRing] = have;
                        mbar_arrive_expect_tx(&bar[kQ8 ? C::K_BYTES + st : C::K_FULL + st],
                                              __popc(have) * static_cast<uint32_t>(kQ8 ? B * D : B * D * 2));
                    }
                    __syncwarp();
                    if (blk >= 0) {
                        if constexpr (kQ8)
                            bulk_copy_g2s(smem + C::OFF_K + st * C::kTileKV + kBN * D + lane * (B * D),
                                          reinterpret_cast<const uint8_t *>(a.k_cache) +
                                              static_cast<size_t>(blocks.group(blk)) * (8 * D),
                                          B * D, &bar[C::K_BYTES + st]);
                        else
                            tma_load_4d(smem + C::OFF_K + st * C::kTileKV + lane * (B / 8) * C::kGroup, &tm_k, 0, 0, 0,
                                        blocks.group(blk), &bar[C::K_FULL + st]);
                    }
                    ++g;
                    blk = next;
                }
                if (!ok) break;
                ++k;
            }
            if (lane == 0) {
                if (!ok) {   // let every copy already issued land
                    for (int i = max(0, k - 1); i <= k; ++i)   // item k's Q may be on its way
                        if (i < q_loads) mbar_wait_drain(&bar[C::Q_FULL + (i & 1)], (i >> 1) & 1);
                    for (uint32_t i = g > C::kSlots ? g - C::kSlots : 0; i < g; ++i)
                        mbar_wait_drain(&bar[(kQ8 ? C::K_BYTES : C::K_FULL) + i % C::kSlots], (i / C::kSlots) & 1);
                }
                __threadfence();
                if (atomicAdd(a.counters + 1, 1u) == gridDim.x - 1) {
                    atomicExch(a.counters, 0u);
                    atomicExch(a.counters + 1, 0u);
                }
            }
            __syncwarp();
        } else if (warp == kVWarp) {
            // -------------------------------------------------------- V
            uint32_t g = 0, lands = 0;             // V tiles issued; of these, landed on V_LAND
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int slot = k % 2;
                ok = warp_all(mbar_wait(&bar[C::ITEM_FULL + slot], (k / 2) & 1, abort_flag, a.err));
                if (!ok) break;
                const Item it = items[slot];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[C::ITEM_EMPTY + slot]);
                if (it.done) break;
                KeyBlocks blocks(a, it.s, it.hk, it.ctx, it.pre, it.q_len, b_shift, lane, kAlibi);
                int blk = blocks.entry(it, 0);
                for (int j = 0; j < it.nkt; ++j) {
                    const int next = j + 1 < it.nkt ? blocks.entry(it, j + 1) : -1;
                    const unsigned have = __ballot_sync(0xffffffffu, blk >= 0);
                    const uint32_t bytes = __popc(have) * static_cast<uint32_t>(B * D * 2);
                    const int st = g % C::kSlots;
                    ok = warp_all(mbar_wait(&bar[C::V_EMPTY + st], ((g / C::kSlots) & 1) ^ 1, abort_flag, a.err));
                    if (!ok) break;
                    uint8_t *vt = smem + C::OFF_V + st * C::kTileKV;
                    if constexpr (kQ8) {   // what is not seen is cleared as the rest is widened
                        if (lane == 0) {
                            const int tail = max(0, min(kBN, it.ctx - blocks.first_key(it, j)));
                            v_rows[st] = have | static_cast<uint32_t>(tail) << 16;
                            mbar_arrive_expect_tx(&bar[C::V_BYTES + st], __popc(have) * static_cast<uint32_t>(B * D));
                        }
                        __syncwarp();
                        if (blk >= 0)
                            bulk_copy_g2s(vt + kBN * D + lane * (B * D),
                                          reinterpret_cast<const uint8_t *>(a.v_cache) +
                                              static_cast<size_t>(blocks.group(blk)) * (8 * D),
                                          B * D, &bar[C::V_BYTES + st]);
                        ++g;
                        blk = next;
                        continue;
                    }
                    auto clear_row = [&](int r) {
                        for (int c = lane; c < C::kHalves * 8; c += 32)
                            *reinterpret_cast<uint4 *>(vt + (r / 8) * C::kGroup + (c / 8) * 1024 + (r % 8) * 128 +
                                                       (c % 8) * 16) = make_uint4(0, 0, 0, 0);
                    };
                    if (have != (1u << (kBN >> b_shift)) - 1) {   // blocks that are not loaded: cleared up front
                        for (int r = 0; r < kBN; ++r)
                            if (!((have >> (r >> b_shift)) & 1)) clear_row(r);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    // rows of the context's last block past its end are cleared
                    // once the copies have landed
                    const int tail = it.ctx - blocks.first_key(it, j);          // valid rows, if < kBN
                    const bool land = tail < kBN && tail % B != 0 && ((have >> (tail >> b_shift)) & 1);
                    uint64_t *vbar = land ? &bar[C::V_LAND] : &bar[C::V_FULL + st];
                    if (lane == 0) mbar_arrive_expect_tx(vbar, bytes);
                    __syncwarp();
                    if (blk >= 0)
                        tma_load_4d(vt + lane * (B / 8) * C::kGroup, &tm_v, 0, 0, 0, blocks.group(blk), vbar);
                    if (land) {
                        ok = warp_all(mbar_wait(&bar[C::V_LAND], lands & 1, abort_flag, a.err));
                        if (!ok) {
                            mbar_wait_drain(&bar[C::V_LAND], lands & 1);
                            break;   // nothing will signal this slot's FULL barrier
                        }
                        ++lands;
                        for (int r = tail; r < ((tail >> b_shift) + 1) * B; ++r) clear_row(r);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[C::V_FULL + st]);
                    }
                    ++g;
                    blk = next;
                }
            }
            if (!ok && lane == 0)   // let every copy already issued land
                for (uint32_t i = g > C::kSlots ? g - C::kSlots : 0; i < g; ++i)
                    mbar_wait_drain(&bar[(kQ8 ? C::V_BYTES : C::V_FULL) + i % C::kSlots], (i / C::kSlots) & 1);
            __syncwarp();
        } else if (kQ8 && warp >= kWidenWarp0) {
            // -------------------------------------------------------- 8 bits to 16
            if constexpr (kQ8) {
                const bool is_k = warp == kWidenWarp0;
                uint64_t *bytes = &bar[is_k ? C::K_BYTES : C::V_BYTES], *full = &bar[is_k ? C::K_FULL : C::V_FULL];
                uint8_t *slots = smem + (is_k ? C::OFF_K : C::OFF_V);
                uint32_t g = 0;                    // tiles widened, over all items
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int slot = k % 2;
                    ok = warp_all(mbar_wait(&bar[C::ITEM_FULL + slot], (k / 2) & 1, abort_flag, a.err));
                    if (!ok) break;
                    const bool done = static_cast<const volatile Item *>(items + slot)->done;
                    const int nkt = static_cast<const volatile Item *>(items + slot)->nkt;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[C::ITEM_EMPTY + slot]);
                    if (done) break;
                    for (int j = 0; j < nkt; ++j, ++g) {
                        const uint32_t st = g % C::kSlots;
                        ok = warp_all(mbar_wait(bytes + st, (g / C::kSlots) & 1, abort_flag, a.err));
                        if (!ok) break;
                        uint8_t *tile = slots + st * C::kTileKV;
                        if (is_k) {
                            widen_tile<D>(tile, lane, [](int) { return true; });
                        } else {
                            const uint32_t rows = v_rows[st];
                            const int tail = static_cast<int>(rows >> 16);
                            if (tail == kBN && (rows & 0xffffu) == (1u << (kBN >> b_shift)) - 1)
                                widen_tile<D>(tile, lane, [](int) { return true; });
                            else
                                widen_tile<D>(tile, lane, [&](int r) {
                                    return r < tail && ((rows >> (r >> b_shift)) & 1);
                                });
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full + st);
                    }
                }
            }
            __syncwarp();
        } else if (warp >= kSWarp0 && warp < kPvWarp0 + 2) {
            // -------------------------------------------------------- products
            if (elect_one()) {
                const bool is_s = warp < kPvWarp0;
                const int t = warp - (is_s ? kSWarp0 : kPvWarp0);
                constexpr uint32_t idesc_s = instr_desc(kMmaBf16, false, kBN);
                constexpr uint32_t idesc_pv = instr_desc(kMmaBf16, true, D);
                const uint32_t kv_addr = smem_addr(smem + (is_s ? C::OFF_K : C::OFF_V));
                uint64_t *kv_full = &bar[is_s ? C::K_FULL : C::V_FULL], *kv_empty = &bar[is_s ? C::K_EMPTY : C::V_EMPTY];
                const uint32_t tm_s = tmem + t * C::kBufs * 64, tm_o = tmem + C::TM_O + t * D;
                uint32_t g = 0;              // K (V) tiles seen
                uint32_t n = 0;              // products of this thread, over all items
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int slot = k % 2;
                    ok = mbar_wait(&bar[C::ITEM_FULL + slot], (k / 2) & 1, abort_flag, a.err);
                    if (!ok) break;
                    const volatile Item *it = items + slot;
                    const bool done = it->done;
                    const int nkt = it->nkt, nk = max(0, t == 0 ? it->nk0 : it->nk1);
                    mbar_arrive(&bar[C::ITEM_EMPTY + slot]);
                    if (done) break;
                    if (is_s) {
                        ok = mbar_wait(&bar[kScaleQ ? C::Q_READY + slot * 2 + t : C::Q_FULL + slot], (k / 2) & 1,
                                       abort_flag, a.err);
                        if (!ok) break;
                    }
                    const uint32_t q_addr = smem_addr(smem + C::OFF_Q) + (slot * 2 + t) * C::kTileQ;
                    for (int j = 0; j < nkt; ++j, ++g) {
                        const uint32_t st = g % C::kSlots;
                        ok = mbar_wait(kv_full + st, (g / C::kSlots) & 1, abort_flag, a.err);
                        if (!ok) break;
                        // the entries this query tile needs: the first nk in key order
                        const int jj = kAlibi ? nkt - 1 - j : j;
                        if (jj >= nk) {   // not this one: hand the slot back
                            mbar_arrive(kv_empty + st);
                            continue;
                        }
                        const uint32_t buf = n % C::kBufs, ph = (n / C::kBufs) & 1;
                        const uint32_t kv = kv_addr + st * C::kTileKV;
                        if (is_s) {
                            // the product that last read the buffer's P
                            if (n >= C::kBufs) ok = mbar_wait(&bar[C::PV_DONE + t * 3 + buf], ph ^ 1, abort_flag, a.err);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                const int half = ks / 4, kk = ks % 4;
                                mma_ss(tm_s + buf * 64, smem_desc(q_addr + half * C::kHalfQ + kk * 32, 16, 1024),
                                       smem_desc(kv + half * 1024 + kk * 32, 16, C::kGroup), idesc_s, ks > 0);
                            }
                            mma_commit(&bar[C::S_FULL + t * 3 + buf]);
                        } else {
                            ok = mbar_wait(&bar[C::P_FULL + t * 3 + buf], ph, abort_flag, a.err);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < kBN / 16; ++ks)
                                mma_ts(tm_o, tm_s + buf * 64 + ks * 8, smem_desc(kv + ks * 2 * C::kGroup, 1024, C::kGroup),
                                       idesc_pv, (kAlibi ? jj < nk - 1 : jj > 0) || ks > 0);
                            mma_commit(&bar[C::PV_DONE + t * 3 + buf]);
                        }
                        mma_commit(kv_empty + st);
                        ++n;
                    }
                }
                mma_commit(&bar[C::MMA_DONE + warp - kSWarp0]);
                mbar_wait_drain(&bar[C::MMA_DONE + warp - kSWarp0], 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax
        const int t = warp / 4;
        const int r = (warp % 4) * 32 + lane;
        const int tok = r / p.group, head = r - tok * p.group;   // within the tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
        const uint32_t s_cols = lane_base + t * C::kBufs * 64;
        const uint32_t o_col = lane_base + C::TM_O + t * D;
        float c = p.scale_log2;            // 8-bit caches: times the head's scale, for each item
        const unsigned full = (1u << (kBN >> b_shift)) - 1;
        // the polynomial's coefficients as pairs, kept in registers (volatile: not
        // built again at each use, which took as many moves as products)
        uint64_t tanh2[5], cap_v2;
        if constexpr (kCap) {
#pragma unroll
            for (int i = 0; i < 5; ++i) tanh2[i] = keep_pair(p.tanh_k[i]);
            cap_v2 = keep_pair(p.cap_v);
        }
        float cap_v = p.cap_v, cap_in = p.cap_in;   // as c
        // The item before: its slot and its Q buffer, which holds the staged rows,
        // are handed back once the copies out of it have read them.
        int pending = -1;
        auto release = [&]() {
            if (pending >= 0 && lane == 0) {
                bulk_wait_read();
                mbar_arrive(&bar[C::ITEM_EMPTY + pending]);
            }
            pending = -1;
        };
        // Item k's Q, where it has to be made fp16, each row by a power of two of its own
        // (fp16_row_exponent).  A thread takes its own row: while the item before waits for its last
        // product, if Q is there by then, and else after that item's output (waiting for it
        // first cost 16 prompts of 333 to 1024 tokens 114 us instead of 108).  The row is
        // 2^q_exponent times what its buffer holds.
        int q_exponent = 0;
        int q_ready = -1;          // the last item whose Q is ready
        auto ready_q = [&](int k) {
            const int slot = k % 2;
            if (!warp_all(mbar_wait(&bar[C::ITEM_FULL + slot], (k / 2) & 1, abort_flag, a.err))) return false;
            const volatile Item *it = items + slot;
            if (it->done) return true;
            if ((t == 0 ? it->nk0 : it->nk1) >= 0) {
                if (!warp_all(mbar_wait(&bar[C::Q_FULL + slot], (k / 2) & 1, abort_flag, a.err))) return false;
                uint8_t *row = smem + C::OFF_Q + (slot * 2 + t) * C::kTileQ + r * 128;
                auto chunk = [&](int i) {
                    return reinterpret_cast<uint4 *>(row + i / 8 * C::kHalfQ + (((i & 7) ^ (r & 7)) << 4));
                };
                uint4 v[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) v[i] = *chunk(i);
                __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        most = __hmax2(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u[z])));
                }
                const float top = fmaxf(__low2float(most), __high2float(most));
                q_exponent = fp16_row_exponent(top);
                const float down = power_of_two(-q_exponent);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        u[z] = pack_pair<false>(__uint_as_float(u[z] << 16) * down,
                                                __uint_as_float(u[z] & 0xFFFF0000u) * down);
                    *chunk(i) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::Q_READY + slot * 2 + t]);
            q_ready = k;
            return true;
        };
        uint32_t n = 0;            // S tiles consumed
        uint32_t tiles = 0;        // key tiles of all items (mask ring)
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int slot = k % 2;
            ok = warp_all(mbar_wait(&bar[C::ITEM_FULL + slot], (k / 2) & 1, abort_flag, a.err));
            if (!ok) break;
            // the slot stays held until the item's rows are written, so that its
            // fields can be read when they are needed
            const volatile Item *it = items + slot;
            const bool done = it->done;
            const int nk = t == 0 ? it->nk0 : it->nk1;
            if (done) break;
            if constexpr (kScaleQ) {
                if (q_ready < k) ok = ready_q(k);
                if (!ok) break;
            }
            // the tile's Q is done with when its last S is: then the warp's output
            // rows are staged there
            uint8_t *staging = smem + C::OFF_Q + (slot * 2 + t) * C::kTileQ + (warp % 4) * (C::kTileQ / 4);
            // descending: a tile that needs fewer entries skips the first ones
            const uint32_t tile_base = tiles + (kAlibi ? it->nkt - max(nk, 0) : 0);
            tiles += it->nkt;
            if (nk < 0) {
                release();
                pending = slot;
                continue;
            }
            // The row's position.  A row without a query stands where the warp's last
            // query does, so that it costs the warp no mask; in a warp without any,
            // every row is at -1 and sees nothing.  Its Q is another sequence's, or what
            // an earlier item's output has left there, so it is not written and has no
            // say in what the warp does.
            const bool live = tok < min(p.tpt, it->q_len - it->tok0 - t * p.tpt);
            const int own = live ? it->first_pos + t * p.tpt + tok : -1;
            const int wmax = __reduce_max_sync(0xffffffffu, own);
            const int pos = live ? own : wmax;
            const int wmin = __reduce_min_sync(0xffffffffu, pos);
            const int pre_all = it->pre, na = it->na, skip = it->skip, j0 = it->j0;
            const int last = j0 + max(nk, 0) - 1;
            if constexpr (kQ8) {
                const float f = __ldg(a.k_scales + it->hk);
                const int e = kScaleQ ? q_exponent : 0;
                c = score_factor(f, p.scale_log2, e);
                if constexpr (kCap) {
                    cap_v = score_factor(f, p.cap_v, e);
                    cap_in = kCapInPerV * cap_v;
                    cap_v2 = keep_pair(cap_v);
                }
            }
            float slope = 0.f;
            if constexpr (kAlibi)
                slope = pos >= 0 ? __ldg(a.alibi_slopes + it->hk * p.group + head) * 1.4426950408889634f : 0.f;
            // (m = 0 in rows without a query: no maximum is missing)
            float m = live ? -INFINITY : 0.f, l = 0.f;
            for (int j = 0; j < nk; ++j, ++n) {
                const uint32_t buf = n % C::kBufs;
                ok = warp_all(mbar_wait(&bar[C::S_FULL + t * 3 + buf], (n / C::kBufs) & 1, abort_flag, a.err));
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_col = s_cols + buf * 64;
                const int i = kAlibi ? last - j : j0 + j;   // list entry
                const int k0 = kBN * (i < na ? i : i + skip);
                const unsigned have = mask_ring[(tile_base + j) % kMaskRing];
                const bool all_visible = have == full &&
                                         (k0 + kBN <= pre_all ? wmin >= 0
                                                              : k0 + kBN - 1 <= wmin &&
                                                                    (a.window == 0 || k0 > wmax - a.window));
                // The scores as they are in tensor memory.
                float x[kBN];
                auto load_raw = [&]() {
                    uint32_t u[kBN];
#pragma unroll
                    for (int q = 0; q < kBN / 32; ++q)
                        tmem_ld32_nowait(s_col + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[q * 32]));
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < kBN; ++e) x[e] = __uint_as_float(u[e]);
                };
                // tanh's polynomial: v = cap_v x and its value over v, w = v^2
                auto cap_poly = [&](float x0, float x1, uint64_t &v, uint64_t &y, uint32_t &any) {
                    v = mul_pair(make_pair(x0, x1), cap_v2);
                    const uint64_t w2 = mul_pair(v, v);
                    any |= static_cast<uint32_t>(w2) | static_cast<uint32_t>(w2 >> 32);
                    y = fma_pair(tanh2[4], w2, tanh2[3]);
#pragma unroll
                    for (int i = 2; i >= 0; --i) y = fma_pair(y, w2, tanh2[i]);
                };
                // cap tanh(s / cap) + bias by 1 - 2 / (1 + e^(2 s / cap)), in log2 units
                auto cap_mufu = [&](float s, float b) {
                    return fmaf(-2.f * p.cap_log2, fast_rcp(1.f + fast_exp2(s * (kQ8 ? cap_in : p.cap_in))), p.cap_log2 + b);
                };
                // One bit per key: keys before pr, and from lw up to h (none for a row
                // without a query), in blocks that are there.
                auto visible = [&](uint32_t (&vis)[kBN / 32]) {
                    const int h = pos + 1 - k0, pr = pos < 0 ? 0 : pre_all - k0;
                    const int lw = a.window > 0 ? h - a.window : 0;
#pragma unroll
                    for (int q = 0; q < kBN / 32; ++q) {
                        vis[q] = bits_below(pr - 32 * q) | (bits_below(h - 32 * q) & ~bits_below(lw - 32 * q));
                        if (have != full) vis[q] &= present(have, q, B);
                    }
                };
                uint32_t w[kBN / 2];       // the weights, packed
                float sum = 0.f;
                load_raw();
                // First against the reference as it is (with the distance bias: if no
                // visible key is ahead of the row).
                bool done_fast = false;
                const bool fast = (!kAlibi || pre_all <= k0 || k0 + kBN - 1 <= wmin) && warp_all(m != -INFINITY) &&
                                  (!kCap || a.softcap <= kShareCap<kMmaBf16>);
                uint32_t any = 0;
                auto weights = [&](auto masked) {
                    uint32_t vis[kBN / 32];
                    if constexpr (decltype(masked)::value == 2) visible(vis);
                    const float edge = (static_cast<float>(pos - k0) + 0.5f) * kFar;
                    float sums[4] = {0.f, 0.f, 0.f, 0.f};
                    // exponent of key e: score + bias, the distance bias being
                    // slope (k0 + e - pos), rising along the tile
                    const float bias = kBias - m + (kAlibi ? slope * static_cast<float>(k0 - pos) : 0.f);
#pragma unroll
                    for (int z = 0; z < kBN / 2; ++z) {
                        // pairs 8 apart in turn (in their order: capped 511 us instead
                        // of 503, head_dim 64 327 instead of 324, at 8192 tokens)
                        const int e = z / 8 * 16 + z % 2 * 8 + z / 2 % 4 * 2;
                        float y0, y1;
                        float b0 = bias, b1 = bias;
                        if constexpr (kAlibi) {
                            b0 = fmaf(slope, static_cast<float>(e), bias);
                            b1 = fmaf(slope, static_cast<float>(e + 1), bias);
                        }
                        if constexpr (kCap) {
                            // what is not visible has no say in the form of tanh
                            float x0 = x[e], x1 = x[e + 1];
                            if constexpr (decltype(masked)::value == 2) {
                                x0 = (vis[e / 32] >> (e % 32)) & 1 ? x0 : 0.f;
                                x1 = (vis[e / 32] >> (e % 32 + 1)) & 1 ? x1 : 0.f;
                            }
                            if (e % 8 == 0) {
                                // one pair in four by the special-function unit, which
                                // has time left (8192 tokens: none 540 us, one in eight
                                // 543, in four 503, in three 516, 3 in 8 521)
                                y0 = cap_mufu(x0, b0);
                                y1 = cap_mufu(x1, b1);
                            } else {
                                uint64_t v, y;
                                cap_poly(x0, x1, v, y, any);
                                split_pair(fma_pair(v, y, make_pair(b0, b1)), y0, y1);
                            }
                        } else {
                            fma2(y0, y1, x[e], x[e + 1], c, c, b0, b1);
                        }
                        if constexpr (decltype(masked)::value == 1) {
                            // keys up to the row's own: kFar (pos + 1/2 - key) is far above
                            // every exponent for them, and far below for the rest
                            y0 = fminf(y0, edge - static_cast<float>(e) * kFar);
                            y1 = fminf(y1, edge - static_cast<float>(e + 1) * kFar);
                        }
                        if constexpr (decltype(masked)::value == 2) {
                            y0 = (vis[e / 32] >> (e % 32)) & 1 ? y0 : -INFINITY;
                            y1 = (vis[e / 32] >> (e % 32 + 1)) & 1 ? y1 : -INFINITY;
                        }
                        y0 = fast_exp2(y0);
                        y1 = fast_exp2(y1);
                        add2(sums[e & 2], sums[(e & 2) + 1], sums[e & 2], sums[(e & 2) + 1], y0, y1);
                        w[e / 2] = pack_pair<kMmaBf16>(y0, y1);
                    }
                    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                };
                if (fast) {
                    if (all_visible)
                        weights(std::integral_constant<int, 0>{});
                    else if (!kCap && have == full && a.window == 0 && pre_all <= k0)
                        weights(std::integral_constant<int, 1>{});
                    else
                        weights(std::integral_constant<int, 2>{});
                    // the sum bounds every weight; v^2 < 2
                    // that the polynomial holds (no bit pattern reaches that of 2)
                    done_fast = warp_all((sum <= kMostSum<kMmaBf16> && any < 0x40000000u) || !live);
                    if (!kCap && !done_fast) load_raw();
                }
                if (!done_fast) {
                    // scores to the log2 domain
                    if constexpr (kCap) {
                        // in tensor memory, 16 at a time: each by the form that its own size
                        // asks for, so that no score depends on another's, seen or not.
                        // (Unrolled in registers over the tile, or 32 at a time, this took
                        // the loop's other tiles 4 to 8 % longer: 8192 tokens 521 to 540 us
                        // instead of 503.)
#pragma unroll 1
                        for (int q = 0; q < kBN / 16; ++q) {
                            uint32_t u[16], far = 0;
                            tmem_ld16_nowait(s_col + q * 16, u);
                            tmem_ld_wait();
                            float z[16];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                uint64_t v, y;
                                cap_poly(__uint_as_float(u[e]), __uint_as_float(u[e + 1]), v, y, far);
                                split_pair(mul_pair(v, y), z[e], z[e + 1]);
                            }
                            if (!warp_all(far < 0x40000000u)) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float v = __uint_as_float(u[e]) * (kQ8 ? cap_v : p.cap_v);
                                    if (!(v * v < 2.f)) z[e] = cap_mufu(__uint_as_float(u[e]), 0.f);
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(z[e]);
                            tmem_st16(s_col + q * 16, u);
                        }
                        tmem_st_wait();
                        load_raw();
                    } else {
#pragma unroll
                        for (int e = 0; e < kBN; ++e) x[e] *= c;
                    }
                    if constexpr (kAlibi) {
                        const float d0 = static_cast<float>(pos - k0);
#pragma unroll
                        for (int e = 0; e < kBN; ++e) x[e] -= slope * fabsf(d0 - static_cast<float>(e));
                    }
                    if (!all_visible) {
                        uint32_t vis[kBN / 32];
                        visible(vis);
#pragma unroll
                        for (int e = 0; e < kBN; ++e)
                            x[e] = (vis[e / 32] >> (e % 32)) & 1 ? x[e] : -INFINITY;
                    }
                    float mx[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) mx[q] = fmaxf(x[q], x[q + 8]);
#pragma unroll
                    for (int e = 16; e < kBN; e += 8)
#pragma unroll
                        for (int q = 0; q < 8; ++q) mx[q] = fmaxf(mx[q], x[e + q]);
                    const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                            fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                    const bool raise = top > __fadd_rd(m, kRaise);
                    if (__any_sync(0xffffffffu, raise && live)) {
                        const float m_new = raise ? top : m;
                        const float alpha = m == m_new ? 1.f : fast_exp2(m - m_new);
                        m = m_new;
                        l *= alpha;
                        if (j > 0) {   // O, once the product before is complete
                            ok = warp_all(mbar_wait(&bar[C::PV_DONE + t * 3 + (n - 1) % C::kBufs],
                                                    ((n - 1) / C::kBufs) & 1, abort_flag, a.err));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t ov[16];
                                tmem_ld16_nowait(o_col + q * 16, ov);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                tmem_st16(o_col + q * 16, ov);
                            }
                        }
                    }
                    const float bias = m == -INFINITY ? 0.f : kBias - m;
                    float sums[2] = {0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < kBN; e += 2) {
                        const float y0 = fast_exp2(x[e] + bias), y1 = fast_exp2(x[e + 1] + bias);
                        add2(sums[0], sums[1], sums[0], sums[1], y0, y1);
                        w[e / 2] = pack_pair<kMmaBf16>(y0, y1);
                    }
                    sum = sums[0] + sums[1];
                }
                l += sum;
                tmem_st32(s_col, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[C::P_FULL + t * 3 + buf]);
                if (j == 0) release();
            }
            if (!ok) break;
            if constexpr (kScaleQ) {
                const int after = (k + 1) % 2, wrap = ((k + 1) / 2) & 1;
                if (nk > 0 && warp_all(mbar_test(&bar[C::ITEM_FULL + after], wrap) &&
                                       mbar_test(&bar[C::Q_FULL + after], wrap))) {
                    ok = ready_q(k + 1);
                    if (!ok) break;
                }
            }
            if (nk > 0) {
                ok = warp_all(mbar_wait(&bar[C::PV_DONE + t * 3 + (n - 1) % C::kBufs], ((n - 1) / C::kBufs) & 1, abort_flag,
                                        a.err));
                if (!ok) break;
                tc_fence_after();
            }
            const int splits = kSplit ? it->splits : 1;
            if (!kSplit || splits == 1) {
                float inv = l > 0.f ? 1.f / l : 0.f;
                if constexpr (kQ8) inv *= __ldg(a.v_scales + it->hk);
                const bool whole = p.store_boxes && warp_all(live);
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf) {
                    uint32_t ov[64];
                    tmem_ld32_nowait(o_col + hf * 64, *reinterpret_cast<uint32_t(*)[32]>(&ov[0]));
                    tmem_ld32_nowait(o_col + hf * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[32]));
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint4 v;
                        uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            u[z] = pack_pair<kBf16>(__uint_as_float(ov[e * 8 + 2 * z]) * inv,
                                                    __uint_as_float(ov[e * 8 + 2 * z + 1]) * inv);
                        *reinterpret_cast<uint4 *>(staging + hf * 4096 + lane * 128 + ((e ^ (lane & 7)) << 4)) = v;
                    }
                }
                tc_fence_before();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (whole) {   // 32 rows of whole tokens leave as tensor copies
                    if (lane == 0) {
                        const int z = it->q_first + it->tok0 + t * p.tpt + tok;   // lane 0 holds the first row
                        for (int hf = 0; hf < C::kHalves; ++hf)
                            tma_store_3d(&tm_out, hf * 64, it->hk * p.group, z, staging + hf * 4096);
                    }
                } else {
                    // rows of the tile's output, from its first token's first head
                    uint16_t *base = a.out + (static_cast<size_t>(it->q_first + it->tok0 + t * p.tpt) * a.num_q_heads +
                                              it->hk * p.group) * D;
                    const int my_row = live ? tok * a.num_q_heads + head : -1;
#pragma unroll 1
                    for (int hf = 0; hf < C::kHalves; ++hf) {
                        // four rows a step, 128 bytes of each; all loads before the
                        // stores, which the compiler cannot tell apart from them
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int rr = i * 4 + lane / 8;
                            v[i] = *reinterpret_cast<const uint4 *>(staging + hf * 4096 + rr * 128 +
                                                                    (((lane % 8) ^ (rr & 7)) << 4));
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int row_at = __shfl_sync(0xffffffffu, my_row, i * 4 + lane / 8);
                            if (row_at >= 0)
                                *reinterpret_cast<uint4 *>(base + static_cast<size_t>(row_at) * D + hf * 64 +
                                                           (lane % 8) * 8) = v[i];
                        }
                    }
                }
            } else if constexpr (kSplit) {
                // The thread's place, at head_dim 128 read again: kept from the kernel's start,
                // what is reckoned from it for this part holds registers in the loop above (4
                // tokens over 32000 keys, 16 bits: 42.6 us so kept, 41.3 so; spills too).
                int tid = threadIdx.x;
                if constexpr (D == 128) asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
                const int place = tid % 32, quarter = tid / 32 % 4;
                // a partial: [split][tile][D + 2][128 rows]
                constexpr size_t kPart = static_cast<size_t>(D + 2) * kBM;
                float *base = p.partials + (static_cast<size_t>(it->slot) * p.splits * 2 + t) * kPart + quarter * 32 + place;
                float *mine = base + static_cast<size_t>(it->split) * 2 * kPart;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t ov[32];
                    tmem_ld32_nowait(o_col + q * 32, ov);
                    tmem_ld_wait();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            mine[(q * 32 + e) * kBM] = nk > 0 ? __uint_as_float(ov[e]) : 0.f;
                    }
                }
                tc_fence_before();
                if (live) {
                    mine[D * kBM] = m;
                    mine[(D + 1) * kBM] = l;
                }
                // The tile's four warps take one ticket, and those of the last split
                // join all of them, a quarter of the dims each (each its own 32 rows,
                // a few rows kept one warp: 4 tokens of 8 heads took 44 us over 32000
                // keys, and take 30).
                __syncwarp();
                if (place == 0) mbar_arrive(&bar[C::PARTS + t]);
                if (quarter == 0) {
                    ok = warp_all(mbar_wait(&bar[C::PARTS + t], (it->joins >> t) & 1, abort_flag, a.err));
                    if (!ok) break;
                    if (place == 0) {
                        uint32_t *ticket = a.counters + 2 + it->slot * 2 + t;
                        const bool last = ticket_add(ticket, 1u) == static_cast<uint32_t>(splits - 1);
                        if (last) atomicExch(ticket, 0u);
                        last_flag[t] = last;
                        mbar_arrive(&bar[C::TICKET + t]);
                    }
                }
                ok = warp_all(mbar_wait(&bar[C::TICKET + t], (it->joins >> t) & 1, abort_flag, a.err));
                if (!ok) break;
                const int ntok = min(p.tpt, it->q_len - it->tok0 - t * p.tpt);
                for (int r0 = 0; last_flag[t] && r0 < ntok * p.group; r0 += 32) {
                    const int rr = min(r0 + place, ntok * p.group - 1);
                    const float *rows = base - (quarter * 32 + place) + rr;
                    uint16_t *dst = a.out + (static_cast<size_t>(it->q_first + it->tok0 + t * p.tpt + rr / p.group) *
                                                 a.num_q_heads + it->hk * p.group + rr % p.group) * D;
                    // four splits at a time, so that their loads share a round trip
                    // (one by one, joining three took 13000 cycles)
                    constexpr int kZ = 4;
                    auto part = [&](int z) {
                        return rows + static_cast<size_t>(min(z, splits - 1)) * 2 * kPart;
                    };
                    // Up to kZ splits: everything a row needs in one round trip, in the order of
                    // the loop below (3 chunks of up to 17 tokens of 4 heads over 640 keys: 15.4 us
                    // so, 16.9 by the loop; over 8 bits 16.3 and 17.9, at head_dim 64 12.9 and 14.4,
                    // but over 16 bits 14.0 and 13.6, so not there).
                    if ((kQ8 || D == 128) && splits <= kZ) {
                        constexpr int kDims = D / 4;
                        const int d0 = quarter * kDims;
                        float mz[kZ], lz[kZ], v[kZ][kDims];
#pragma unroll
                        for (int z = 0; z < kZ; ++z) {
                            mz[z] = __ldcg(part(z) + D * kBM);
                            lz[z] = __ldcg(part(z) + (D + 1) * kBM);
#pragma unroll
                            for (int e = 0; e < kDims; ++e) v[z][e] = __ldcg(part(z) + (d0 + e) * kBM);
                        }
                        float top = -INFINITY, total = 0.f;
#pragma unroll
                        for (int z = 0; z < kZ; ++z) top = fmaxf(top, mz[z]);
#pragma unroll
                        for (int z = 0; z < kZ; ++z) {
                            mz[z] = z < splits && mz[z] != -INFINITY ? fast_exp2(mz[z] - top) : 0.f;
                            if (mz[z] > 0.f) total += mz[z] * lz[z];
                        }
                        float inv = total > 0.f ? 1.f / total : 0.f;
                        if constexpr (kQ8) inv *= __ldg(a.v_scales + it->hk);
                        if (r0 + place < ntok * p.group) {
#pragma unroll
                            for (int e = 0; e < kDims; e += 8) {
                                uint4 out;
                                uint32_t *u = reinterpret_cast<uint32_t *>(&out);
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    float acc[2] = {0.f, 0.f};
#pragma unroll
                                    for (int z = 0; z < kZ; ++z) {
                                        acc[0] += mz[z] * v[z][e + 2 * y];
                                        acc[1] += mz[z] * v[z][e + 2 * y + 1];
                                    }
                                    u[y] = pack_pair<kBf16>(acc[0] * inv, acc[1] * inv);
                                }
                                *reinterpret_cast<uint4 *>(dst + d0 + e) = out;
                            }
                        }
                        continue;
                    }
                    float top = -INFINITY, total = 0.f;
                    for (int z0 = 0; z0 < splits; z0 += kZ) {
                        float mz[kZ], lz[kZ], t2 = top;
#pragma unroll
                        for (int z = 0; z < kZ; ++z) {
                            mz[z] = __ldcg(part(z0 + z) + D * kBM);
                            lz[z] = __ldcg(part(z0 + z) + (D + 1) * kBM);
                        }
#pragma unroll
                        for (int z = 0; z < kZ; ++z) t2 = fmaxf(t2, mz[z]);
                        if (top != -INFINITY) total *= fast_exp2(top - t2);
                        top = t2;
#pragma unroll
                        for (int z = 0; z < kZ; ++z)
                            if (z0 + z < splits && mz[z] != -INFINITY) total += fast_exp2(mz[z] - top) * lz[z];
                    }
                    float inv = total > 0.f ? 1.f / total : 0.f;
                    if constexpr (kQ8) inv *= __ldg(a.v_scales + it->hk);
#pragma unroll 1
                    for (int d0 = quarter * (D / 4); d0 < (quarter + 1) * (D / 4); d0 += 16) {
                        float acc[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 1
                        for (int z0 = 0; z0 < splits; z0 += kZ) {
                            float v[kZ][16], f[kZ];
#pragma unroll
                            for (int z = 0; z < kZ; ++z) {
                                f[z] = __ldcg(part(z0 + z) + D * kBM);
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[z][e] = __ldcg(part(z0 + z) + (d0 + e) * kBM);
                            }
#pragma unroll
                            for (int z = 0; z < kZ; ++z) {
                                f[z] = z0 + z < splits && f[z] != -INFINITY ? fast_exp2(f[z] - top) : 0.f;
#pragma unroll
                                for (int e = 0; e < 16; ++e) acc[e] += f[z] * v[z][e];
                            }
                        }
                        if (r0 + place < ntok * p.group) {
#pragma unroll
                            for (int e = 0; e < 16; e += 8) {
                                uint4 v;
                                uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    u[z] = pack_pair<kBf16>(acc[e + 2 * z] * inv, acc[e + 2 * z + 1] * inv);
                                *reinterpret_cast<uint4 *>(dst + d0 + e) = v;
                            }
                        }
                    }
                }
            }
            __syncwarp();
            release();             // (an item without key tiles)
            pending = slot;
        }
        if (lane == 0) bulk_wait_all();   // copies out of shared memory that this CTA still holds
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols));
}

// Query tiles (pairs) and key splits of a call.
struct Plan {
    long long pairs, base;    // base: items without splits
    int splits;
};
inline Plan make_plan(int num_seqs, int num_kv_heads, int group, int max_q) {
    Plan pl;
    const int tpt = kBM / group;
    pl.pairs = (static_cast<long long>(max_q) + 2 * tpt - 1) / (2 * tpt);
    pl.base = pl.pairs * num_seqs * num_kv_heads;
    pl.splits = pl.base > 0 && pl.base < kSplitTarget ? static_cast<int>(kSplitTarget / pl.base) : 1;
    return pl;
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, PrefillGroupedArgs);
template <bool kBf16, bool kQ8, int D, bool kSplit>
Kernel pick(bool cap, bool alibi) {
    return cap ? (alibi ? prefill_grouped_kernel<kBf16, kQ8, D, true, true, kSplit>
                        : prefill_grouped_kernel<kBf16, kQ8, D, true, false, kSplit>)
               : (alibi ? prefill_grouped_kernel<kBf16, kQ8, D, false, true, kSplit>
                        : prefill_grouped_kernel<kBf16, kQ8, D, false, false, kSplit>);
}
template <bool kQ8, bool kSplit>
Kernel pick(bool bf16, int D, bool cap, bool alibi) {
    return bf16 ? (D == 64 ? pick<true, kQ8, 64, kSplit>(cap, alibi) : pick<true, kQ8, 128, kSplit>(cap, alibi))
                : (D == 64 ? pick<false, kQ8, 64, kSplit>(cap, alibi) : pick<false, kQ8, 128, kSplit>(cap, alibi));
}

// The launch over a cache of 16 bits, or with kQ8 of 8.
template <bool kQ8>
cudaError_t launch_prefill_kind(const GroupedArgs &args, int dtype, int head_dim, int num_sms, cudaStream_t stream) {
    const bool bf16 = dtype == PA_DTYPE_BF16;
    const int Hk = args.num_kv_heads, Hq = args.num_q_heads, B = args.block_size, D = head_dim;
    PrefillGroupedArgs p;
    p.g = args;
    const double log2e = 1.4426950408889634;
    p.scale_log2 = static_cast<float>(args.scale * log2e);
    p.cap_log2 = static_cast<float>(args.softcap * log2e);
    p.cap_in = args.softcap > 0.f ? static_cast<float>(2.0 * args.scale / args.softcap * log2e) : 0.f;
    p.group = Hq / Hk;
    fill_tanh(args.scale, args.softcap, &p.cap_v, p.tanh_k);
    p.tpt = kBM / p.group;
    const Plan pl = make_plan(args.num_seqs, Hk, p.group, args.max_q);
    const long long items = pl.base * pl.splits;   // fits an int (the caller checks), with room past the end
    p.num_pairs = static_cast<int>(pl.pairs);
    p.splits = pl.splits;
    p.num_items = static_cast<int>(items);
    p.partials = static_cast<float *>(args.workspace);

    p.store_boxes = 32 % p.group == 0;
    CUtensorMap tm_q, tm_k, tm_v, tm_out;
    const cuuint64_t q_dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                                  static_cast<cuuint64_t>(args.total_q)};
    const cuuint64_t q_strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2};
    const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tpt)};
    const cuuint32_t out_box[3] = {64, static_cast<cuuint32_t>(p.store_boxes ? p.group : 1),
                                   static_cast<cuuint32_t>(p.store_boxes ? 32 / p.group : 1)};
    // groups of 8 keys x 64-dim halves x keys x dims: a box is one block of a head
    const cuuint64_t kv_dims[4] = {64, 8, static_cast<cuuint64_t>(D / 64),
                                   static_cast<cuuint64_t>(args.num_blocks) * Hk * (B / 8)};
    const cuuint64_t kv_strides[3] = {static_cast<cuuint64_t>(D) * 2, 128, static_cast<cuuint64_t>(D) * 16};
    const cuuint32_t kv_box[4] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(B / 8)};
    if (!encode(&tm_q, bf16, args.q, 3, q_dims, q_strides, q_box) ||
        !encode(&tm_out, bf16, args.out, 3, q_dims, q_strides, out_box))
        return cudaErrorInvalidValue;
    // (bytes of an 8-bit cache are fetched by untiled copies)
    if constexpr (kQ8)
        tm_k = tm_v = tm_q;
    else if (!encode(&tm_k, bf16, args.k_cache, 4, kv_dims, kv_strides, kv_box) ||
        !encode(&tm_v, bf16, args.v_cache, 4, kv_dims, kv_strides, kv_box))
        return cudaErrorInvalidValue;
    const bool cap = args.softcap > 0.f, alibi = args.alibi_slopes != nullptr;
    const bool split = pl.splits > 1;
    const Kernel kernel = split ? pick<kQ8, true>(bf16, D, cap, alibi) : pick<kQ8, false>(bf16, D, cap, alibi);
    const int smem = D == 64 ? Cfg<64, kQ8>::kSmemBytes : Cfg<128, kQ8>::kSmemBytes;
    // the kernel's shared-memory limit, once per device and variant
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    {
        static std::mutex mu;
        static bool ready[64][32] = {};
        const int which = (bf16 ? 8 : 0) + (D == 64 ? 0 : 4) + (cap ? 2 : 0) + (alibi ? 1 : 0) + (split ? 16 : 0);
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[device][which]) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            ready[device][which] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items < num_sms ? items : num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *params[] = {&tm_q, &tm_k, &tm_v, &tm_out, &p};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), params);
}

}  // namespace

#ifndef PA_Q8_LAUNCHES   // pa_prefill_q8.cu takes the kernel alone

bool prefill_grouped_supported(int dtype, int head_dim, int block_size, int group) {
    return decode_variant_supported(dtype, head_dim, block_size) && head_dim != 256 && group <= kBM;
}

size_t prefill_grouped_workspace_bytes(int num_seqs, int num_kv_heads, int group, int head_dim,
                                       int max_query_len) {
    const Plan pl = make_plan(num_seqs, num_kv_heads, group, max_query_len);
    if (pl.splits <= 1) return 0;
    return static_cast<size_t>(pl.base) * pl.splits * 2 * (head_dim + 2) * kBM * sizeof(float);
}

long long prefill_grouped_items(int num_seqs, int num_kv_heads, int group, int max_query_len) {
    const Plan pl = make_plan(num_seqs, num_kv_heads, group, max_query_len);
    return pl.base * pl.splits;
}

size_t prefill_grouped_counters_bytes() { return (kCounters * 4 + 255) / 256 * 256; }

cudaError_t launch_prefill_grouped(const GroupedArgs &args, int dtype, int head_dim, int num_sms,
                                   cudaStream_t stream) {
    return launch_prefill_kind<false>(args, dtype, head_dim, num_sms, stream);
}

#endif  // PA_Q8_LAUNCHES

}  // namespace pa
