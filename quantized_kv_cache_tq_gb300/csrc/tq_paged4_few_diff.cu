// The few-row kernel for two softmax maps (see tq_paged4_few.cuh).
#include "tq_paged4_few.cuh"

namespace tq {
namespace p4 {

cudaError_t launch_few_diff(const AttnArgs &a, cudaStream_t s) {
  if (a.wk == 64 && a.wv == 64) return launch_few_t<64, 64, 1, 2>(a, s);
  if (a.wk == 64 && a.wv == 128) return launch_few_t<64, 128, 1, 2>(a, s);
  if (a.wk == 128 && a.wv == 128) return launch_few_t<128, 128, 1, 2>(a, s);
  if (a.wk == 128 && a.wv == 256) return launch_few_t<128, 256, 1, 2>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace p4
}  // namespace tq
