// pa_tree_sinks.cu -- the tree attention's kernels for a sliding window with sinks (pa_tree_body.cuh).
#include "pa_tree_body.cuh"

namespace pa {

TreeKernel tree_kernel_sinks(bool f16, int D, bool tma) { return pick_tree<kSinks>(f16, D, tma); }

}  // namespace pa
