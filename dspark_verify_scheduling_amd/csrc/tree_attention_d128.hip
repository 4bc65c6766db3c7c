// The split kernel of tree_attention.h for heads of 128 elements.
#include "tree_attention.h"

namespace dspark {
namespace attn {

void launch_dim128(const AttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  launch_dim<128>(a, ws, dt, s);
}

}  // namespace attn
}  // namespace dspark
