// The split kernel of tree_attention.h for heads of 64 elements.
#include "tree_attention.h"

namespace dspark {
namespace attn {

void launch_dim64(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  launch_dim<64>(a, ws, dt, s);
}

}  // namespace attn
}  // namespace dspark
