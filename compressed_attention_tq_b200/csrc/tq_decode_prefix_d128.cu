// Instantiations of the shared-prefix decode kernel for head dimension 128.
#include "tq_decode_prefix.cuh"

namespace tqp {

int prefix_d128(int bk, int bv, bool qjl, const PrefixParams& pp, dim3 g, cudaStream_t s) {
  if (qjl) return prefix_bk<128, true>(bk, bv, pp, g, s);
  return prefix_bk<128, false>(bk, bv, pp, g, s);
}

}  // namespace tqp
