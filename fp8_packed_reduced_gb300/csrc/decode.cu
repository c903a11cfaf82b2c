// The entry points of the attention of one new token per sequence (decode.cuh
// has the kernels), and its kernels without a window.
#include "decode.cuh"

namespace qkvp {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_heads(const CacheArgs& a, int Hq) {
  if (Hq < 1) return QKVP_ERR_INVALID_ARGUMENT;
  return Hq % a.H || Hq > 1024 ? QKVP_ERR_UNSUPPORTED : QKVP_OK;
}

// Parts of the workspace after its header: lse2, records, scores.
struct DecodeLayout {
  size_t lse2, records, scores, bytes;
};
// Query heads of one K/V head that share a read: up to 16, or 8 where the
// list of very many sequences takes the shared memory that their q needs.
int head_chunks(const CacheArgs& a, int Hq) {
  const int most = a.B <= 2048 ? 16 : 8;
  return (Hq / a.H + most - 1) / most;
}
int heads_per_chunk(const CacheArgs& a, int Hq) {
  const int G = Hq / a.H, n = head_chunks(a, Hq);
  return (G + n - 1) / n;
}
// Blocks for the units of `slots` slots a sequence, and one for every piece, up to a block
// per SM.
int most_blocks(const CacheArgs& a, int Hq, int slots) {
  const int64_t pieces = static_cast<int64_t>(a.B) * a.H * head_chunks(a, Hq);
  return static_cast<int>(std::min<int64_t>(kMaxBlocks, std::max(pieces, (pieces * (slots / 16) + 7) / 8)));
}
// Slots that one sequence can see: those below `sinks` and the last `window`
// lie in as many units of 32 and two that they share with others.
int most_seen(const CacheArgs& a, int window, int sinks) {
  return static_cast<int>(std::min<int64_t>(a.capacity(), static_cast<int64_t>(window) + sinks + 3 * 32));
}
DecodeLayout decode_layout(const CacheArgs& a, int Hq, int accumulate) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  DecodeLayout w;
  w.lse2 = kCacheHeaderBytes;
  w.records = w.lse2 + up(static_cast<size_t>(a.B) * Hq * sizeof(float));
  w.scores = w.records + up(static_cast<size_t>(most_blocks(a, Hq, a.capacity())) * (2 + kMaxWarps) * record_floats(heads_per_chunk(a, Hq)) * sizeof(float));
  w.bytes = w.scores + (accumulate ? static_cast<size_t>(a.B) * Hq * a.capacity() * sizeof(float) : 0);
  return w;
}

// window 0: none.
int decode_attention(const qkvp_cache* cache, int Hq, int window, int sinks, float scale, const uint16_t* q, uint16_t* out,
                     float* lse, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  DecodeParams p;
  int rc = check_cache(cache, &p.c);
  if (rc != QKVP_OK) return rc;
  rc = check_heads(p.c, Hq);
  if (rc != QKVP_OK) return rc;
  if (!q || !out || !ws || !(fabsf(scale) < INFINITY)) return QKVP_ERR_INVALID_ARGUMENT;
  if (accumulate && !p.c.weight) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, out, lse, ws};
  for (const void* x : ptrs)
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  const DecodeLayout w = decode_layout(p.c, Hq, accumulate);
  if (ws_bytes < w.bytes) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sms();
  if (sms <= 0) return QKVP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const DevStatus st{static_cast<int*>(ws), 0};
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  p.G = Hq / p.c.H;
  p.chunks = head_chunks(p.c, Hq);
  p.nh = heads_per_chunk(p.c, Hq);
  p.scale_log2 = scale * kLog2e;
  p.q = q;
  p.a = out;
  p.arrived = reinterpret_cast<unsigned int*>(wsb + kDecodeCounters);
  p.lse2 = reinterpret_cast<float*>(wsb + w.lse2);
  p.lse = lse;
  p.records = reinterpret_cast<float*>(wsb + w.records);
  p.scores = accumulate ? reinterpret_cast<float*>(wsb + w.scores) : nullptr;
  const bool windowed = window && window < p.c.capacity();   // else every sequence is seen whole
  const int seen = windowed ? most_seen(p.c, window, sinks) : p.c.capacity();
  p.window = std::min(window, p.c.capacity());
  p.sinks = std::min(sinks, p.c.capacity());
  const int grid = std::min(sms, most_blocks(p.c, Hq, seen));
  mark(s);
  cudaError_t e;
  if (windowed) {
    e = launch_decode_window(p, cache->fp8, grid, st, s);
  } else {
    switch (p.c.d) {
      case 64: e = cache->fp8 ? launch_decode<64, true, false>(p, grid, st, s) : launch_decode<64, false, false>(p, grid, st, s); break;
      case 96: e = cache->fp8 ? launch_decode<96, true, false>(p, grid, st, s) : launch_decode<96, false, false>(p, grid, st, s); break;
      default: e = cache->fp8 ? launch_decode<128, true, false>(p, grid, st, s) : launch_decode<128, false, false>(p, grid, st, s);
    }
  }
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  if (accumulate) {
    // Four slots a thread, up to two rounds of the blocks that the GPU holds: a
    // sequence may be far shorter than its pages allow (64 x 8 heads with 100 of
    // 131072 slots: 23 us for the call, 116 with blocks for them all).
    const int threads = std::min(kWeightThreads, (seen / 4 + 31) / 32 * 32);
    const int64_t pieces = static_cast<int64_t>(p.c.B) * p.c.H, full = (16 * sms + pieces - 1) / pieces;
    const int64_t blocks = std::min<int64_t>((seen + 4 * threads - 1) / (4 * threads), full);
    const dim3 wgrid(static_cast<unsigned>(blocks), p.c.H, p.c.B);
    if (launch_dependent(windowed ? decode_weight_kernel<true> : decode_weight_kernel<false>, wgrid, threads, 0, s, p, st) != cudaSuccess) return QKVP_ERR_CUDA;
    mark(s);
  }
  return QKVP_OK;
}

}  // namespace
}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_decode_attention_workspace_bytes(const qkvp_cache* cache, int Hq, int accumulate) {
  CacheArgs a;
  if (check_cache(cache, &a) != QKVP_OK || check_heads(a, Hq) != QKVP_OK) return 0;
  return decode_layout(a, Hq, accumulate).bytes;
}

int qkvp_decode_attention(const qkvp_cache* cache, int Hq, float scale, const uint16_t* q, uint16_t* out, float* lse,
                          int accumulate, void* ws, size_t ws_bytes, void* stream) {
  return decode_attention(cache, Hq, 0, 0, scale, q, out, lse, accumulate, ws, ws_bytes, stream);
}

int qkvp_decode_window_attention(const qkvp_cache* cache, int Hq, int window, int sinks, float scale, const uint16_t* q,
                                 uint16_t* out, float* lse, int accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (window < 1 || sinks < 0) return QKVP_ERR_INVALID_ARGUMENT;
  return decode_attention(cache, Hq, window, sinks, scale, q, out, lse, accumulate, ws, ws_bytes, stream);
}

}  // extern "C"
