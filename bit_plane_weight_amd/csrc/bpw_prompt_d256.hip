// bpw_prompt_d256.hip - the attention kernels of bpw_prompt.h for head sizes padded to 256.
#include "bpw_prompt.h"

namespace bpw {

int launch_prompt_d256(const PromptArgs &a, int32_t dtype, bool many, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == 1) return run_prompt<__bf16, 256>(a, many, s);
    return run_prompt<_Float16, 256>(a, many, s);
}

}  // namespace bpw
