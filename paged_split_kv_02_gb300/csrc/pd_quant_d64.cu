// Decode attention over an 8-bit cache, head size 64.
#include "pd_quant_attn.cuh"

namespace pd {

cudaError_t launch_quant_d64(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream) {
  switch (nt) {
    case 1: return bf16 ? launch_quant_t<64, 1, true>(p, l, stream) : launch_quant_t<64, 1, false>(p, l, stream);
    case 2: return bf16 ? launch_quant_t<64, 2, true>(p, l, stream) : launch_quant_t<64, 2, false>(p, l, stream);
    case 4: return bf16 ? launch_quant_t<64, 4, true>(p, l, stream) : launch_quant_t<64, 4, false>(p, l, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
