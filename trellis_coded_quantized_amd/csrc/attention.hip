// attention.hip -- attention over the cache of the queries' own type.
#include "attention_kernels.hpp"

namespace trellis {

size_t attention_workspace_bytes(const AttnArgs& a) {
  const Parts p = part_bytes(a);
  return p.o + p.ml + p.notes;
}

hipError_t launch_attention(AttnArgs a, void* workspace, hipStream_t stream) {
  return launch_store<Kv16>(a, workspace, stream);
}

}  // namespace trellis
