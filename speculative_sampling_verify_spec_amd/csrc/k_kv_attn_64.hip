// Cache attention for heads of 64 channels.
#include "kv_attn.h"

namespace sv {

hipError_t launch_kv_attn_64(const KvAttn& p, int dtype, int fmt, hipStream_t st) {
  return launch_dim<64>(p, dtype, fmt, st);
}

}  // namespace sv
