// Tree attention for heads of 128 values (a file of its own: the widths compile in parallel).
#include "avsg_tree_attn.cuh"

namespace avsg {
cudaError_t launch_tree_d128(const TreeArgs& a, int dtype, int wm, int dev, cudaStream_t st) {
  return tree::launch_width<128>(a, dtype, wm, dev, st);
}
}  // namespace avsg
