// Attention of whole prompts, heads of 128 channels.
#include "prompt_attn.h"

namespace sv {

hipError_t launch_prompt_128(const PromptAttn& p, int dtype, hipStream_t s) { return launch_prompt<128>(p, dtype, s); }

}  // namespace sv
