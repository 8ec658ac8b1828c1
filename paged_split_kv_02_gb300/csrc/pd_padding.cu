// Rows past the last request of a batch (padding of a captured step) see no key
// and are written as zeros.  The attention kernels do it beside their own rows;
// a batch without any (every request empty, or no request) has no such launch,
// only this one.  Bound by the launch: a captured batch pads a few rows.
#include "pd_internal.h"
#include "pd_ptx.cuh"

namespace pd {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    pd_zero_padding(const int32_t *query_start, int num_seqs, int num_tokens, int heads, int D,
                    unsigned short *out, int64_t o_s0, int64_t o_s1) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int t0 = min(max(__ldg(query_start + num_seqs), 0), num_tokens);
  const int per_head = D / 8;
  const int64_t per_row = (int64_t)heads * per_head, n = (num_tokens - t0) * per_row;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / per_row;
    const int rem = (int)(i - t * per_row), h = rem / per_head, c = rem - h * per_head;
    *reinterpret_cast<uint4 *>(out + (t0 + t) * o_s0 + h * o_s1 + c * 8) = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace

int zero_padding(const pd_tensor *out, const int32_t *query_start, int num_seqs, int num_sms,
                 void *stream) {
  const int64_t chunks = out->shape[0] * out->shape[1] * (out->shape[2] / 8);
  cudaLaunchConfig_t cfg = {};
  // (a few CTAs on an SM stream zeros as fast as more)
  const int64_t most = 4LL * num_sms, need = (chunks + kThreads - 1) / kThreads;
  cfg.gridDim = dim3((unsigned)(need < most ? need : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, pd_zero_padding, query_start, num_seqs, (int)out->shape[0], (int)out->shape[1],
      (int)out->shape[2], static_cast<unsigned short *>(out->data), out->stride[0], out->stride[1]);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}

}  // namespace pd
