// Prompt attention over the paged 4-bit cache (see tq_paged4_prefill.cuh).
#include "tq_paged4_prefill.cuh"

namespace tq {
namespace p4 {

bool prefill_supported(int wk, int wv) { return (wk == 64 && wv <= 128) || (wk == 128 && wv == 128); }

cudaError_t launch_prefill(const AttnArgs &a, cudaStream_t s) {
  if (a.wk == 64) return a.wv == 64 ? launch_prefill_t<64, 64>(a, s) : launch_prefill_t<64, 128>(a, s);
  return launch_prefill_t<128, 128>(a, s);
}

}  // namespace p4
}  // namespace tq
