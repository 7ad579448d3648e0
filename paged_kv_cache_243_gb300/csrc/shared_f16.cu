// Instantiations of the shared-prefix attention kernel: fp16 caches.
#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_f16(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&shared_attention_kernel<64, KV_F16, false, kPrefixes>)
                 : reinterpret_cast<const void*>(&shared_attention_kernel<128, KV_F16, false, kPrefixes>);
}

}  // namespace pkv
