// Cache attention for heads of 96 channels.
#include "kv_attn.h"

namespace sv {

hipError_t launch_kv_attn_96(const KvAttn& p, int dtype, int fmt, hipStream_t st) {
  return launch_dim<96>(p, dtype, fmt, st);
}

}  // namespace sv
