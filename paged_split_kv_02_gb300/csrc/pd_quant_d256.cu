// Decode attention over an 8-bit cache, head size 256.
#include "pd_quant_attn.cuh"

namespace pd {

cudaError_t launch_quant_d256(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream) {
  switch (nt) {
    case 1: return bf16 ? launch_quant_t<256, 1, true>(p, l, stream) : launch_quant_t<256, 1, false>(p, l, stream);
    case 2: return bf16 ? launch_quant_t<256, 2, true>(p, l, stream) : launch_quant_t<256, 2, false>(p, l, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
