// pa_prefill_q8.cu -- the launches of the grouped prefill over an 8-bit cache (the
// kernel: pa_prefill_grouped.cu), in a translation unit of their own.
#define PA_Q8_LAUNCHES
#include "pa_prefill_grouped.cu"

namespace pa {

cudaError_t launch_prefill_grouped_q8(const GroupedArgs &args, int dtype, int head_dim, int num_sms,
                                      cudaStream_t stream) {
    return launch_prefill_kind<true>(args, dtype, head_dim, num_sms, stream);
}

}  // namespace pa
