// Instantiations of the attention kernel for trees of drafts: per-token INT8 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* tree_kernel_i8t(int D, bool bf) {
  if (D == 64)
    return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8T, true, true>)
              : reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8T, false, true>);
  return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8T, true, true>)
            : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8T, false, true>);
}

}  // namespace pkv
