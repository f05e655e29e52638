// Attention of whole prompts, heads of 256 channels.
#include "prompt_attn.h"

namespace sv {

hipError_t launch_prompt_256(const PromptAttn& p, int dtype, hipStream_t s) { return launch_prompt<256>(p, dtype, s); }

}  // namespace sv
