// attention_tree_f16.cu -- attention_tree_16.cuh for fp16 caches.
#include "attention_tree_16.cuh"

namespace gpt2 {
namespace tree {

int launch_mma_f16(const TreeArgs& a, int hs, int* ctas, cudaStream_t s) { return mma_heads<__half>(a, hs, ctas, s); }

}  // namespace tree
}  // namespace gpt2
