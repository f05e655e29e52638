// Attention of whole prompts, heads of 96 channels.
#include "prompt_attn.h"

namespace sv {

hipError_t launch_prompt_96(const PromptAttn& p, int dtype, hipStream_t s) { return launch_prompt<96>(p, dtype, s); }

}  // namespace sv
