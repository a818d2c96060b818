// Single-token attention over int8 cells: K rows of 256 codes.
#include "tq_int8_decode.cuh"

namespace tq {
namespace i8 {

cudaError_t launch_decode_wide(const p4::AttnArgs &a, cudaStream_t s) {
  return a.wv == 128 ? launch_w<256, 128>(a, s) : launch_w<256, 256>(a, s);
}

}  // namespace i8
}  // namespace tq
