// Device status words: every source file with bounded waits has its own (device
// globals are not shared between files), and vlaq_check reads them all in one
// round trip.
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace vlaq {

namespace {

constexpr int kWords = 4;
struct StatusWords {
  unsigned int* word[kWords];
};

__device__ unsigned int g_vlaq_all_status = 0;

// The words of all files into one, or all of them back to zero.
__global__ void status_kernel(const StatusWords s, bool clear) {
  griddep_wait();
  unsigned int all = 0;
  for (int i = 0; i < kWords; ++i) {
    if (clear)
      atomicExch(s.word[i], 0u);
    else
      all |= *static_cast<volatile unsigned int*>(s.word[i]);
  }
  if (!clear) g_vlaq_all_status = all;
}

}  // namespace

// The words stay as they are until one of them is seen set, so calls of several
// host threads lose no timeout.  One launch, one copy and one synchronization:
// 17 us (a copy, a store and two synchronizations for each word took 78).
cudaError_t read_and_clear_status(unsigned int* out, cudaStream_t s) {
  StatusWords w;
  cudaError_t e;
  if ((e = gemm_status_word(&w.word[0])) || (e = quant_status_word(&w.word[1])) ||
      (e = block_linear_status_word(&w.word[2])) || (e = block_quant_status_word(&w.word[3])))
    return e;
  if ((e = launch_pdl(status_kernel, dim3(1), dim3(1), 0, s, w, false))) return e;
  if ((e = cudaMemcpyFromSymbolAsync(out, g_vlaq_all_status, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, s)))
    return e;
  if ((e = cudaStreamSynchronize(s)) || *out == 0) return e;
  if ((e = launch_pdl(status_kernel, dim3(1), dim3(1), 0, s, w, true))) return e;
  return cudaStreamSynchronize(s);
}

}  // namespace vlaq
