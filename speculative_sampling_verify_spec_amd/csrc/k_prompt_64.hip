// Attention of whole prompts, heads of 64 channels.
#include "prompt_attn.h"

namespace sv {

hipError_t launch_prompt_64(const PromptAttn& p, int dtype, hipStream_t s) { return launch_prompt<64>(p, dtype, s); }

}  // namespace sv
