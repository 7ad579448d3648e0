// Instantiations of the shared-prefix attention kernel: bf16 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_bf16(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_BF16, true, kPrefixes>)
                 : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_BF16, true, kPrefixes>);
}

}  // namespace pkv
