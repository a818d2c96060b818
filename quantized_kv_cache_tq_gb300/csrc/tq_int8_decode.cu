// Single-token attention over int8 cells: rows of 64 and 128 codes, and the choice of kernel.
#include "tq_int8_decode.cuh"

namespace tq {
namespace i8 {

cudaError_t launch_decode_between(const p4::AttnArgs &a, cudaStream_t s);
cudaError_t launch_decode_wide(const p4::AttnArgs &a, cudaStream_t s);

cudaError_t launch_decode(const p4::AttnArgs &a, cudaStream_t s) {
  if (a.wk == 256 && (a.dk > 192 || a.wv == 256)) return launch_decode_wide(a, s);
  if (a.wk == 256 || (a.wk == 128 && a.dk <= 96 && a.dv <= 96)) return launch_decode_between(a, s);
  return a.wk == 64 ? launch_w<64, 64>(a, s) : launch_w<128, 128>(a, s);
}

}  // namespace i8
}  // namespace tq
