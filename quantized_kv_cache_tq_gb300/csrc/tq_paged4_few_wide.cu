// The few-row kernel for head dims above 128 (see tq_paged4_few.cuh).
#include "tq_paged4_few.cuh"

namespace tq {
namespace p4 {

cudaError_t launch_few_wide(const AttnArgs &a, int columns, cudaStream_t s) {
  const int nt = columns > 8 ? 2 : 1;
  if (a.wk == 256 && a.wv == 128)
    return nt == 1 ? launch_few_t<256, 128, 1, 1>(a, s) : launch_few_t<256, 128, 2, 1>(a, s);
  if (a.wk == 256 && a.wv == 256)
    return nt == 1 ? launch_few_t<256, 256, 1, 1>(a, s) : launch_few_t<256, 256, 2, 1>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace p4
}  // namespace tq
