// bpw_attention_d256.hip - the attention kernels of bpw_attention.h for head sizes padded to 256.
#include "bpw_attention.h"

namespace bpw {

int launch_attn_d256(const AttnArgs &a, int32_t dtype, int32_t mp, int32_t ms, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == 1) return run_attn_tiles<__bf16, 256>(a, mp, ms, s);
    return run_attn_tiles<_Float16, 256>(a, mp, ms, s);
}

}  // namespace bpw
