// attention_tree_bf16.cu -- attention_tree_16.cuh for bf16 caches.
#include "attention_tree_16.cuh"

namespace gpt2 {
namespace tree {

int launch_mma_bf16(const TreeArgs& a, int hs, int* ctas, cudaStream_t s) { return mma_heads<__nv_bfloat16>(a, hs, ctas, s); }

}  // namespace tree
}  // namespace gpt2
