// Instantiations of the shared-prefix attention kernel: per-group INT8 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_i8g(int D, bool bf) {
  if (D == 64)
    return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8G, true>)
              : reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8G, false>);
  return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8G, true>)
            : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8G, false>);
}

}  // namespace pkv
