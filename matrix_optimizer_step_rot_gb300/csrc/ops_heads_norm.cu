// The norm of queries and keys, with the rotation (ops_heads.cuh).
#include "ops_heads.cuh"

namespace rot {
namespace ops {

int heads_norm(int32_t type, HeadArgs& q, int64_t tokens, bool il, cudaStream_t s) {
  return launch_heads_type<kNorm>(type, q, tokens, il, s);
}

}  // namespace ops
}  // namespace rot
