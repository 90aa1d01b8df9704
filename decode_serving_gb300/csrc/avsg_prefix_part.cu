// The parts of an attention over common prefixes for few rows, small pages or short contexts (a file
// of its own: the kernels compile beside the tree attention's).
#include "avsg_tree_attn.cuh"

namespace avsg {
cudaError_t launch_prefix_part(const TreeArgs& a, int dtype, int D, int wm, int dev, cudaStream_t st) {
  return D == 64    ? tree::launch_width<64, true>(a, dtype, wm, dev, st)
         : D == 128 ? tree::launch_width<128, true>(a, dtype, wm, dev, st)
                    : tree::launch_width<256, true>(a, dtype, wm, dev, st);
}
}  // namespace avsg
