// The attention of one new token per sequence under a window (decode.cuh).
#include "decode.cuh"

namespace qkvp {

cudaError_t launch_decode_window(DecodeParams& p, bool fp8, int grid, DevStatus st, cudaStream_t s) {
  switch (p.c.d) {
    case 64: return fp8 ? launch_decode<64, true, true>(p, grid, st, s) : launch_decode<64, false, true>(p, grid, st, s);
    case 96: return fp8 ? launch_decode<96, true, true>(p, grid, st, s) : launch_decode<96, false, true>(p, grid, st, s);
    default: return fp8 ? launch_decode<128, true, true>(p, grid, st, s) : launch_decode<128, false, true>(p, grid, st, s);
  }
}

}  // namespace qkvp
