// Attention of a tree of drafted tokens (include/mk.h, mk_tree_attention): the
// instantiations of the kernel for many rows.
#include "mk_tree_attention_tc.cuh"

namespace mk {

int launch_tree_attention_tc(const AttnParams& p, int head_dim, int type, cudaStream_t st) {
  return launch_tc(p, p.groups * p.row_tiles, head_dim, type, "mk_tree_attention", st);
}

}  // namespace mk
