// Tree attention on the 5th-generation tensor cores: its kernels (avsg_tree_umma.cuh).
#include "avsg_tree_umma.cuh"

namespace avsg {
cudaError_t launch_tree_umma(const TreeArgs& a, int dtype, int D, int dev, cudaStream_t st) {
  return tree::launch_umma_any<false>(a, dtype, D, dev, st);
}
}  // namespace avsg
