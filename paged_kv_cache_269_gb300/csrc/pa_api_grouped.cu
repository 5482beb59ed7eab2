// pa_api_grouped.cu -- C ABI entry points for rotary cache appends and
// grouped-query attention (declared in include/pa.h): argument checks and
// launches.  Nothing here throws, aborts or synchronises.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa.h"
#include "pa_internal.h"

namespace pa {
namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks of pa_dims and the query heads that every grouped call shares.
int check_grouped_dims(const pa_dims *dims, int32_t num_q_heads, bool need_seqs) {
    if (!dims) return PA_ERR_NULL;
    if (dims->num_heads <= 0 || dims->head_dim <= 0 || dims->block_size <= 0 ||
        dims->num_blocks <= 0 || num_q_heads <= 0)
        return PA_ERR_SHAPE;
    if (need_seqs && (dims->num_seqs < 0 || num_q_heads % dims->num_heads != 0)) return PA_ERR_SHAPE;
    if (!decode_variant_supported(dims->dtype, dims->head_dim, dims->block_size))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// The scale and the score options.  The kernels hold scale log2(e), softcap
// log2(e) and scale / softcap in fp32, so these have to be numbers that fp32
// holds with room on both sides (scale 0 is one: every score is 0).
int check_scores(float scale, const pa_attn_opts *o) {
    const double wide = 1.2676506002282294e30;   // 2^100
    if (!isfinite(scale) || fabs(scale) > wide) return PA_ERR_SHAPE;
    if (!o) return PA_OK;
    if (!isfinite(o->softcap) || o->softcap < 0.f || o->window < 0) return PA_ERR_SHAPE;
    if (o->softcap > 0.f) {
        const double turn = fabs(static_cast<double>(scale)) / o->softcap;
        if (o->softcap > wide || o->softcap < 1. / wide || turn > wide || (scale != 0.f && turn < 1. / wide))
            return PA_ERR_SHAPE;
    }
    return PA_OK;
}

// Products that the kernels hold in 32 bits (positions and counts of
// sequences with room for a tile past the end).
int check_ranges(const pa_dims *dims, int32_t num_q_heads, int32_t max_blocks_per_seq) {
    const long long lim = 0x7fffffffLL;
    const long long slots = static_cast<long long>(dims->num_blocks) * dims->block_size;
    if (max_blocks_per_seq <= 0 || slots > lim || slots * dims->num_heads > lim ||
        static_cast<long long>(max_blocks_per_seq) * dims->block_size > (1LL << 30) ||
        dims->num_seqs > (1 << 28) || static_cast<long long>(dims->num_seqs) * num_q_heads > lim)
        return PA_ERR_SHAPE;
    return PA_OK;
}

GroupedArgs make_args(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, const int32_t *context_lens, float scale,
                      int32_t max_blocks_per_seq, const pa_dims *dims, int32_t num_q_heads,
                      const pa_attn_opts *opts, void *workspace, uint32_t *counters) {
    GroupedArgs a = {};
    a.out = static_cast<uint16_t *>(out);
    a.q = static_cast<const uint16_t *>(q);
    a.k_cache = static_cast<const uint16_t *>(k_cache);
    a.v_cache = static_cast<const uint16_t *>(v_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.alibi_slopes = opts ? opts->alibi_slopes : nullptr;
    a.prefix_lens = opts ? opts->prefix_lens : nullptr;
    a.scale = scale;
    a.softcap = opts ? opts->softcap : 0.f;
    // a window as long as any context limits nothing
    a.window = opts && opts->window < max_blocks_per_seq * dims->block_size ? opts->window : 0;
    a.num_seqs = dims->num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = dims->num_heads;
    a.num_blocks = dims->num_blocks;
    a.block_size = dims->block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.workspace = workspace;
    a.counters = counters;
    return a;
}

int finish(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return PA_ERR_UNSUPPORTED;  // tensor maps could not be made
    if (e == cudaErrorInvalidConfiguration) return PA_ERR_SHAPE;  // too many work items
    return e == cudaSuccess ? PA_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

int pa_rope_and_cache(void *q_out, const void *q, const void *k, const void *v, void *k_cache,
                      void *v_cache, const int32_t *positions, const float *cos_sin,
                      const int32_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t q_out_stride,
                      int32_t rotary_dim, int32_t max_positions, int32_t interleaved,
                      const pa_dims *dims, void *stream) {
    int rc = check_grouped_dims(dims, num_q_heads, false);
    if (rc != PA_OK) return rc;
    const int D = dims->head_dim;
    const long long slots = static_cast<long long>(dims->num_blocks) * dims->block_size;
    if (num_tokens < 0 || max_positions <= 0 || q_stride < 0 || k_stride < 0 || v_stride < 0 ||
        slots > 0x7fffffffLL ||
        static_cast<long long>(num_q_heads) + 2LL * dims->num_heads > 0x3fffffLL)
        return PA_ERR_SHAPE;
    if (rotary_dim <= 0 || rotary_dim > D) return PA_ERR_SHAPE;
    if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (q_out_stride < static_cast<long long>(num_q_heads) * D) return PA_ERR_SHAPE;
    if (!q_out || !q || !k || !v || !k_cache || !v_cache || !positions || !cos_sin || !slot_mapping)
        return PA_ERR_NULL;
    for (const void *p : {static_cast<const void *>(q_out), q, k, v,
                          static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(cos_sin)})
        if (!aligned(p, 16)) return PA_ERR_ALIGN;
    if (!aligned(positions, 4) || !aligned(slot_mapping, 4) || q_stride % 8 || k_stride % 8 ||
        v_stride % 8 || q_out_stride % 8)
        return PA_ERR_ALIGN;
    unsigned int *err = nullptr;
    int sms = 0;
    rc = current_device_info(&err, &sms);
    if (rc != PA_OK) return rc;
    RopeArgs a = {};
    a.q_out = static_cast<uint16_t *>(q_out);
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.k_cache = static_cast<uint16_t *>(k_cache);
    a.v_cache = static_cast<uint16_t *>(v_cache);
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.slot_mapping = slot_mapping;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = dims->num_heads;
    a.head_dim = D;
    a.block_size = dims->block_size;
    a.rotary_dim = rotary_dim;
    a.max_positions = max_positions;
    a.pool_slots = slots;
    a.err = err;
    const cudaError_t e = launch_rope_and_cache(a, dims->dtype, interleaved != 0, sms,
                                                static_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration) return PA_ERR_SHAPE;   // too many tokens x rows
    return e == cudaSuccess ? PA_OK : record_cuda_error(e);
}

size_t pa_decode_grouped_workspace_bytes(const pa_dims *dims, int32_t num_q_heads) {
    if (check_grouped_dims(dims, num_q_heads, true) != PA_OK) return static_cast<size_t>(-1);
    return decode_grouped_workspace_bytes(dims->head_dim, num_q_heads / dims->num_heads);
}

size_t pa_decode_grouped_counters_bytes(const pa_dims *dims, int32_t num_q_heads) {
    if (check_grouped_dims(dims, num_q_heads, true) != PA_OK) return 0;
    return decode_grouped_counters_bytes(dims->num_seqs, dims->num_heads,
                                         num_q_heads / dims->num_heads, dims->head_dim);
}

int pa_decode_grouped(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, const int32_t *context_lens, float scale,
                      int32_t max_blocks_per_seq, const pa_dims *dims, int32_t num_q_heads,
                      const pa_attn_opts *opts, void *workspace, size_t workspace_bytes,
                      uint32_t *counters, size_t counters_bytes, void *stream) {
    int rc = check_grouped_dims(dims, num_q_heads, true);
    if (rc != PA_OK) return rc;
    rc = check_scores(scale, opts);
    if (rc != PA_OK) return rc;
    rc = check_ranges(dims, num_q_heads, max_blocks_per_seq);
    if (rc != PA_OK) return rc;
    if (dims->num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        (opts && (!aligned(opts->alibi_slopes, 4) || !aligned(opts->prefix_lens, 4))))
        return PA_ERR_ALIGN;
    if (!counters || !aligned(counters, 4) ||
        counters_bytes < pa_decode_grouped_counters_bytes(dims, num_q_heads))
        return PA_ERR_WORKSPACE;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pa_decode_grouped_workspace_bytes(dims, num_q_heads))
        return PA_ERR_WORKSPACE;
    GroupedArgs a = make_args(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                              max_blocks_per_seq, dims, num_q_heads, opts, workspace, counters);
    int sms = 0;
    rc = current_device_info(&a.err, &sms);
    if (rc != PA_OK) return rc;
    return finish(launch_decode_grouped(a, dims->dtype, dims->head_dim, sms,
                                        static_cast<cudaStream_t>(stream)));
}

size_t pa_prefill_grouped_workspace_bytes(const pa_dims *dims, int32_t num_q_heads,
                                          int32_t max_query_len) {
    if (check_grouped_dims(dims, num_q_heads, true) != PA_OK || max_query_len < 0 ||
        !prefill_grouped_supported(dims->dtype, dims->head_dim, dims->block_size,
                                   num_q_heads / dims->num_heads))
        return static_cast<size_t>(-1);
    return prefill_grouped_workspace_bytes(dims->num_seqs, dims->num_heads,
                                           num_q_heads / dims->num_heads, dims->head_dim,
                                           max_query_len);
}

size_t pa_prefill_grouped_counters_bytes(const pa_dims *dims, int32_t num_q_heads) {
    if (check_grouped_dims(dims, num_q_heads, true) != PA_OK) return 0;
    return prefill_grouped_counters_bytes();
}

int pa_prefill_grouped(void *out, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_tables, const int32_t *context_lens,
                       const int32_t *query_start, int32_t total_query_tokens,
                       int32_t max_query_len, float scale, int32_t max_blocks_per_seq,
                       const pa_dims *dims, int32_t num_q_heads, const pa_attn_opts *opts,
                       void *workspace, size_t workspace_bytes, uint32_t *counters,
                       size_t counters_bytes, void *stream) {
    int rc = check_grouped_dims(dims, num_q_heads, true);
    if (rc != PA_OK) return rc;
    if (!prefill_grouped_supported(dims->dtype, dims->head_dim, dims->block_size,
                                   num_q_heads / dims->num_heads))
        return PA_ERR_UNSUPPORTED;
    rc = check_scores(scale, opts);
    if (rc != PA_OK) return rc;
    rc = check_ranges(dims, num_q_heads, max_blocks_per_seq);
    if (rc != PA_OK) return rc;
    if (total_query_tokens < 0 || max_query_len < 0) return PA_ERR_SHAPE;
    // work items (query tiles x sequences x K/V heads) are counted in 32 bits
    if (prefill_grouped_items(dims->num_seqs, dims->num_heads, num_q_heads / dims->num_heads, max_query_len) >
        0x7fffffffLL - 4096)
        return PA_ERR_SHAPE;
    if (dims->num_seqs == 0 || total_query_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start)
        return PA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) ||
        (opts && (!aligned(opts->alibi_slopes, 4) || !aligned(opts->prefix_lens, 4))))
        return PA_ERR_ALIGN;
    if (!counters || !aligned(counters, 4) || counters_bytes < prefill_grouped_counters_bytes())
        return PA_ERR_WORKSPACE;
    const size_t need = pa_prefill_grouped_workspace_bytes(dims, num_q_heads, max_query_len);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
        return PA_ERR_WORKSPACE;
    GroupedArgs a = make_args(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                              max_blocks_per_seq, dims, num_q_heads, opts, workspace, counters);
    a.query_start = query_start;
    a.total_q = total_query_tokens;
    a.max_q = max_query_len;
    int sms = 0;
    rc = current_device_info(&a.err, &sms);
    if (rc != PA_OK) return rc;
    return finish(launch_prefill_grouped(a, dims->dtype, dims->head_dim, sms,
                                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
