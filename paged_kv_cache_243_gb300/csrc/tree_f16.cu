// Instantiations of the attention kernel for trees of drafts: fp16 caches.
#include "shared_kernel.cuh"

namespace pkv {

template <int D>
static const void* of(bool few) {
  return few ? reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_F16, false, kFewDrafts>)
             : reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_F16, false, kDraftRows>);
}

const void* tree_kernel_f16(int D, bool few) { return D == 64 ? of<64>(few) : of<128>(few); }

}  // namespace pkv
