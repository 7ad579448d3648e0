// Instantiations of the attention kernel for trees of drafts: bf16 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* tree_kernel_bf16(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_BF16, true, true>)
                 : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_BF16, true, true>);
}

}  // namespace pkv
