// Tree attention for heads of 64 values (a file of its own: the widths compile in parallel).
#include "avsg_tree_attn.cuh"

namespace avsg {
cudaError_t launch_tree_d64(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st) {
  return tree::launch_width<64>(a, dtype, wm, dev, st);
}
}  // namespace avsg
