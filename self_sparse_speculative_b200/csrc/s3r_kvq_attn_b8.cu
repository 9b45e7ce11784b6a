// The quantised attention kernel over a cache held in 8 bits.
#include "s3r_kvq_attn_tok.cuh"

namespace s3r {

cudaError_t launch_kvq_attn_tok8(int head_dim, const KvqAttnParams& p, cudaStream_t st) {
  if (head_dim == 64) return p.P == 16 ? kvq::launch_rows<64, 16, 8>(p, st) : kvq::launch_rows<64, 64, 8>(p, st);
  return p.P == 16 ? kvq::launch_rows<128, 16, 8>(p, st) : kvq::launch_rows<128, 64, 8>(p, st);
}

}  // namespace s3r
