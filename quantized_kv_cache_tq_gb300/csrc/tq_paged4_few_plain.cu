// The few-row kernel for one softmax map (see tq_paged4_few.cuh).
#include "tq_paged4_few.cuh"

namespace tq {
namespace p4 {

cudaError_t launch_few_plain(const AttnArgs &a, int columns, cudaStream_t s) {
  const int nt = columns > 8 ? 2 : 1;
  if (a.wk == 64 && a.wv == 64) return nt == 1 ? launch_few_t<64, 64, 1, 1>(a, s) : launch_few_t<64, 64, 2, 1>(a, s);
  if (a.wk == 128 && a.wv == 128)
    return nt == 1 ? launch_few_t<128, 128, 1, 1>(a, s) : launch_few_t<128, 128, 2, 1>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace p4
}  // namespace tq
