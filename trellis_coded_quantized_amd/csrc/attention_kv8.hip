// attention_kv8.hip -- attention over the cache held in 8 bits.
#include "attention_kernels.hpp"

namespace trellis {

hipError_t launch_attention_kv8(Attn8Args a, void* workspace, hipStream_t stream) {
  return launch_store<Kv8>(a, workspace, stream);
}

}  // namespace trellis
