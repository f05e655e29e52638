// Attention of whole prompts and the weights they give, heads of 64 channels.
#include "prompt_attn.h"
#include "prompt_weights.h"

namespace sv {

hipError_t launch_prompt_64(const PromptAttn& p, int dtype, hipStream_t s) { return launch_prompt<64>(p, dtype, s); }

hipError_t launch_prompt_weights_64(const PromptWeights& p, int dtype, hipStream_t s) {
  return launch_weights<64>(p, dtype, s);
}

}  // namespace sv
