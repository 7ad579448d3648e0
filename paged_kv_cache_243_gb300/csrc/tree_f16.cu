// Instantiations of the attention kernel for trees of drafts: fp16 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* tree_kernel_f16(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_F16, false, true>)
                 : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_F16, false, true>);
}

}  // namespace pkv
