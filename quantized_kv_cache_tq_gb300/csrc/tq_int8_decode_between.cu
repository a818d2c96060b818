// Single-token attention over int8 cells: rows between the powers of two, of 80 and 96 codes, and K rows of 192.
#include "tq_int8_decode.cuh"

namespace tq {
namespace i8 {

cudaError_t launch_decode_between(const p4::AttnArgs &a, cudaStream_t s) {
  if (a.wk == 256) return launch_w<192, 128>(a, s);
  return a.dk <= 80 && a.dv <= 80 ? launch_w<80, 80>(a, s) : launch_w<96, 96>(a, s);
}

}  // namespace i8
}  // namespace tq
