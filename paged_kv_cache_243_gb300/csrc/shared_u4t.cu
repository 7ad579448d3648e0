// Instantiations of the shared-prefix attention kernel: 4-bit caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_u4t(int D, bool bf) {
  if (D == 64)
    return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_U4T, true>)
              : reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_U4T, false>);
  return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_U4T, true>)
            : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_U4T, false>);
}

}  // namespace pkv
