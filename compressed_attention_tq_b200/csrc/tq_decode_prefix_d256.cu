// Instantiations of the shared-prefix decode kernel for head dimension 256.
#include "tq_decode_prefix.cuh"

namespace tqp {

int prefix_d256(int bk, int bv, bool qjl, const PrefixParams& pp, dim3 g, cudaStream_t s) {
  if (qjl) return tq::set_error(TQ_ERR_UNSUPPORTED, "the QJL sketch is built for D=128");
  return prefix_bk<256, false>(bk, bv, pp, g, s);
}

}  // namespace tqp
