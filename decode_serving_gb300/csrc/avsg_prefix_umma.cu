// The parts of an attention over common prefixes on the 5th-generation tensor cores (a file of its
// own: the kernels compile beside the tree attention's).
#include "avsg_tree_umma.cuh"

namespace avsg {
cudaError_t launch_prefix_umma(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st) {
  return tree::launch_umma_any<true>(a, dtype, D, dev, st);
}
}  // namespace avsg
