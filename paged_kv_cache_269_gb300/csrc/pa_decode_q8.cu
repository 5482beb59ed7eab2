// pa_decode_q8.cu -- the launches of the grouped decode over an 8-bit cache (the
// kernel: pa_decode_grouped.cu), in a translation unit of their own.
#define PA_Q8_LAUNCHES
#include "pa_decode_grouped.cu"

namespace pa {

cudaError_t launch_decode_grouped_q8(const GroupedArgs &args, int dtype, int head_dim, int num_sms,
                                     cudaStream_t stream) {
    DecodeGroupedArgs p = prepare_args(args, head_dim);
    p.io_bf16 = dtype == PA_DTYPE_BF16;
    const int D = head_dim, B = args.block_size;

    // [D / 128 halves] x [all cache rows] x 128 bytes: one box is a block's rows of
    // one head, or as many of them as a tile holds
    const int tile_keys = 4096 / D;
    const int line = D < 128 ? D : 128, halves = D / line;
    CUtensorMap tm_k, tm_v;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(line),
                                static_cast<cuuint64_t>(args.num_blocks) * args.num_kv_heads * B,
                                static_cast<cuuint64_t>(halves)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(line)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(line), static_cast<cuuint32_t>(B < tile_keys ? B : tile_keys),
                               static_cast<cuuint32_t>(halves)};
    if (!encode_bytes(&tm_k, args.k_cache, 3, dims, strides, box, line) ||
        !encode_bytes(&tm_v, args.v_cache, 3, dims, strides, box, line))
        return cudaErrorInvalidValue;

    const Variant v = D == 64 ? variant_of<false, true, 64>(p.group)
                              : (D == 128 ? variant_of<false, true, 128>(p.group) : variant_of<false, true, 256>(p.group));
    const int which = (D == 64 ? 0 : D == 128 ? 3 : 6) + (p.group <= 4 ? 0 : p.group <= 8 ? 1 : 2);
    return launch_variant(v, which, tm_k, tm_v, p, num_sms, stream);
}

}  // namespace pa
