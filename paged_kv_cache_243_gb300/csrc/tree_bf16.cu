// Instantiations of the attention kernel for trees of drafts: bf16 caches.
#include "shared_kernel.cuh"

namespace pkv {

template <int D>
static const void* of(bool few) {
  return few ? reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_BF16, true, kFewDrafts>)
             : reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_BF16, true, kDraftRows>);
}

const void* tree_kernel_bf16(int D, bool few) { return D == 64 ? of<64>(few) : of<128>(few); }

}  // namespace pkv
