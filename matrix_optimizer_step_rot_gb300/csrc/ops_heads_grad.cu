// The norm's backward pass (ops_heads.cuh).
#include "ops_heads.cuh"

namespace rot {
namespace ops {

int heads_norm_grad(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  return launch_heads_type<kNormGrad>(type, q, tokens, il, s);
}

}  // namespace ops
}  // namespace rot
