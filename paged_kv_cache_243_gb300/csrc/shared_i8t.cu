// Instantiations of the shared-prefix attention kernel: per-token INT8 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_i8t(int D, bool bf) {
  if (D == 64)
    return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8T, true>)
              : reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_I8T, false>);
  return bf ? reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8T, true>)
            : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_I8T, false>);
}

}  // namespace pkv
