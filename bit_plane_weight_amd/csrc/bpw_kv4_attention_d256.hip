// bpw_kv4_attention_d256.hip - the attention kernels of bpw_kv4_attention.h for head sizes padded to 256.
#include "bpw_kv4_attention.h"

namespace bpw {

int launch_attn4_d256(const Attn4Args &a, int32_t dtype, bool one_launch, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == 1) return run_attn4<__bf16, 256>(a, one_launch, s);
    return run_attn4<_Float16, 256>(a, one_launch, s);
}

}  // namespace bpw
