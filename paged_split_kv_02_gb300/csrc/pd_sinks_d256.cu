// Window with sinks, head size 256: decode and split prefill (mma.sync) and
// tensor-memory prefill tiles.
#include "pd_window.cuh"
#include "pd_window_prefill.cuh"

namespace pd {

cudaError_t launch_sinks_d256(bool bf16, int path, const CUtensorMap &tk, const CUtensorMap &tv,
                              const Params &p, const Launch &l, cudaStream_t stream) {
  if (path == 6)
    return bf16 ? launch_window_t<256, true>(tk, tv, p, l, stream)
                : launch_window_t<256, false>(tk, tv, p, l, stream);
  if (path != 1) return cudaErrorInvalidValue;
  return bf16 ? launch_mma_t<256, true, false, false, false, false, true>(tk, tv, p, l, stream)
              : launch_mma_t<256, false, false, false, false, false, true>(tk, tv, p, l, stream);
}

cudaError_t launch_window_prefill_d256(bool bf16, const CUtensorMap &tk, const CUtensorMap &tv,
                                        const CUtensorMap &tq, const Params &p, const Launch &l,
                                        cudaStream_t stream) {
  return bf16 ? launch_window_prefill_t<256, true>(tk, tv, tq, p, l, stream)
              : launch_window_prefill_t<256, false>(tk, tv, tq, p, l, stream);
}

}  // namespace pd
