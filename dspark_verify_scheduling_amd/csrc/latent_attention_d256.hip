// The split kernel of latent_attention.h for latents of 256 elements.
#include "latent_attention.h"

namespace dspark {
namespace lattn {

void launch_dim256(const LatentAttnArgs& a, const Parts& ws, dspark_dtype dt, hipStream_t s) {
  launch_split<256>(a, ws, dt, s);
}

}  // namespace lattn
}  // namespace dspark
