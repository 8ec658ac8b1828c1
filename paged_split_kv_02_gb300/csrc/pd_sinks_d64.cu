// Window with sinks, head size 64: decode (mma.sync) and prefill tiles with the rows on the M side.
#include "pd_window.cuh"
#include "pd_window_prefill.cuh"

namespace pd {

cudaError_t launch_sinks_d64(bool bf16, int path, const CUtensorMap &tk, const CUtensorMap &tv,
                              const Params &p, const Launch &l, cudaStream_t stream) {
  if (path == 4)
    return bf16 ? launch_mma_t<64, true, false, false, true, false, true>(tk, tv, p, l, stream)
                : launch_mma_t<64, false, false, false, true, false, true>(tk, tv, p, l, stream);
  if (path == 6)
    return bf16 ? launch_window_t<64, true>(tk, tv, p, l, stream)
                : launch_window_t<64, false>(tk, tv, p, l, stream);
  if (path != 1) return cudaErrorInvalidValue;
  return bf16 ? launch_mma_t<64, true, false, false, false, false, true>(tk, tv, p, l, stream)
              : launch_mma_t<64, false, false, false, false, false, true>(tk, tv, p, l, stream);
}

cudaError_t launch_window_prefill_d64(bool bf16, const CUtensorMap &tk, const CUtensorMap &tv,
                                       const CUtensorMap &tq, const Params &p, const Launch &l,
                                       cudaStream_t stream) {
  return bf16 ? launch_window_prefill_t<64, true>(tk, tv, tq, p, l, stream)
              : launch_window_prefill_t<64, false>(tk, tv, tq, p, l, stream);
}

}  // namespace pd
