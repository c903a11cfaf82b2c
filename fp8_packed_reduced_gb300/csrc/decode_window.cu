// The attention of one new token per sequence under a window (decode.cuh).  Bound
// by the fixed cost of that kernel, since a window leaves little to read: 64
// sequences of up to 8192 slots, 6 heads, E4M3, window 1024 and 16 sinks, weights:
// 28.7 us, 74 MB (10.9 us at a copy's rate); one of 131072 slots, bf16, window 4096:
// 18.6 us, of which the host takes all (16 us on the GPU with cold caches).
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
