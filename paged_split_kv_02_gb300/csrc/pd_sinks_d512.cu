// Window with sinks, head size 512: decode and prefill on mma.sync.
#include "pd_kernel.cuh"

namespace pd {

cudaError_t launch_sinks_d512(bool bf16, int path, const CUtensorMap &tk, const CUtensorMap &tv,
                              const Params &p, const Launch &l, cudaStream_t stream) {
  if (path != 1) return cudaErrorInvalidValue;
  return bf16 ? launch_mma_t<512, true, false, false, false, false, true>(tk, tv, p, l, stream)
              : launch_mma_t<512, false, false, false, false, false, true>(tk, tv, p, l, stream);
}

}  // namespace pd
