// The split kernel of tree_attention.h for heads of 256 elements.
#include "tree_attention.h"

namespace dspark {
namespace attn {

void launch_dim256(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  launch_dim<256>(a, ws, dt, s);
}

}  // namespace attn
}  // namespace dspark
