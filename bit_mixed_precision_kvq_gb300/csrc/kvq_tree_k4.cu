// Instantiations of the tree-attention kernel for K bit-width 4 (all V
// widths); one translation unit per K width so that they compile in parallel.
#include "kvq_tree.cuh"

namespace kvq {
namespace tree {
const void* tree_kernel_k4(int vb) {
  switch (vb) {
    case 2: return reinterpret_cast<const void*>(&tree_kernel<4, 2>);
    case 4: return reinterpret_cast<const void*>(&tree_kernel<4, 4>);
    case 8: return reinterpret_cast<const void*>(&tree_kernel<4, 8>);
    case 16: return reinterpret_cast<const void*>(&tree_kernel<4, 16>);
  }
  return nullptr;
}
}  // namespace tree
}  // namespace kvq
