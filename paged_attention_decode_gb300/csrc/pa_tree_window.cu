// pa_tree_window.cu -- the tree attention's kernels for a sliding window (pa_tree_body.cuh).
#include "pa_tree_body.cuh"

namespace pa {

TreeKernel tree_kernel_window(bool f16, int D, bool tma) { return pick_tree<kWindow>(f16, D, tma); }

}  // namespace pa
