// Attention of one new token per sequence over the paged cache.
//   s_i = scale * q . k_i,  a = sum_i e^(s_i) v_i / sum_i e^(s_i)
#include <cmath>

#include "cache.cuh"
#include "kernels.cuh"

namespace qkvp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

// One block per (query head, sequence).  Warp w takes slots w, w + 8, ... with
// a running maximum and sum of its own; the warps are joined at the end.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(CacheArgs c, int G, float scale, const uint16_t* __restrict__ q, uint16_t* __restrict__ a,
                  float* __restrict__ lse, float* __restrict__ scores, DevStatus st) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = blockIdx.x, b = blockIdx.y, Hq = gridDim.x, h = hq / G;
  const int n = checked_length(c, b, st, KID_DECODE);
  float qv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    qv[i] = __uint_as_float(static_cast<uint32_t>(q[(static_cast<int64_t>(hq) * c.B + b) * D + 32 * i + lane]) << 16);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (scores) scores += (static_cast<int64_t>(b) * Hq + hq) * c.capacity();
  for (int i = warp; i < n; i += kWarps) {
    const int64_t row = cache_row(c, b, h, i, st, KID_DECODE);
    float s = -INFINITY;
    if (row >= 0) {
      s = 0.f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const int64_t at = row * D + 32 * j + lane;
        s += qv[j] * (FP8 ? e4m3_value(c.k[at])
                          : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(c.k)[at]) << 16));
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= FP8 ? scale * c.k_scale[row] : scale;
    }
    if (scores && lane == 0) scores[i] = s;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
    const float pv = FP8 ? p * c.v_scale[row] : p;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = row * kDv + 32 * j + lane;
      o[j] = o[j] * f + pv * (FP8 ? e4m3_value(c.v[at])
                                  : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(c.v)[at]) << 16));
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kDv];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) so[warp][32 * j + lane] = o[j];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f, oo = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = sm[w] == -INFINITY ? 0.f : expf(sm[w] - mm);
    ll += f * sl[w];
    oo += f * so[w][threadIdx.x & 127];
  }
  const bool none = ll == 0.f;
  if (threadIdx.x < kDv)
    a[(static_cast<int64_t>(b) * Hq + hq) * kDv + threadIdx.x] =
        __bfloat16_as_ushort(__float2bfloat16_rn(none ? 0.f : oo / ll));
  if (threadIdx.x == 0) lse[static_cast<int64_t>(b) * Hq + hq] = none ? -INFINITY : mm + logf(ll);
}

// weight += the probabilities of the head's query heads
__global__ void __launch_bounds__(kThreads)
    decode_weight_kernel(CacheArgs c, int G, const float* __restrict__ lse, const float* __restrict__ scores,
                         DevStatus st) {
  const int h = blockIdx.y, b = blockIdx.z, Hq = c.H * G, i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= checked_length(c, b, st, KID_DECODE_WEIGHT)) return;
  const int64_t row = cache_row(c, b, h, i, st, KID_DECODE_WEIGHT);
  if (row < 0) return;
  float p = 0.f;
  for (int g = 0; g < G; ++g) {
    const int64_t at = static_cast<int64_t>(b) * Hq + h * G + g;
    const float s = scores[at * c.capacity() + i];
    if (s != -INFINITY) p += expf(s - lse[at]);
  }
  c.weight[row] += p;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_heads(const CacheArgs& a, int Hq) {
  if (Hq < 1) return QKVP_ERR_INVALID_ARGUMENT;
  return Hq % a.H || Hq > 1024 ? QKVP_ERR_UNSUPPORTED : QKVP_OK;
}
size_t lse_bytes(const CacheArgs& a, int Hq) { return (static_cast<size_t>(a.B) * Hq * sizeof(float) + 255) / 256 * 256; }

}  // namespace
}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_decode_attention_workspace_bytes(const qkvp_cache* cache, int Hq, int accumulate) {
  CacheArgs a;
  if (check_cache(cache, &a) != QKVP_OK || check_heads(a, Hq) != QKVP_OK) return 0;
  return kCacheStatusBytes + lse_bytes(a, Hq) +
         (accumulate ? static_cast<size_t>(a.B) * Hq * a.capacity() * sizeof(float) : 0);
}

int qkvp_decode_attention(const qkvp_cache* cache, int Hq, float scale, const uint16_t* q, uint16_t* out, float* lse,
                          int accumulate, void* ws, size_t ws_bytes, void* stream) {
  CacheArgs a;
  int rc = check_cache(cache, &a);
  if (rc != QKVP_OK) return rc;
  rc = check_heads(a, Hq);
  if (rc != QKVP_OK) return rc;
  if (!q || !out || !ws || !(fabsf(scale) < INFINITY)) return QKVP_ERR_INVALID_ARGUMENT;
  if (accumulate && !a.weight) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, out, lse, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return QKVP_ERR_MISALIGNED;
  if (ws_bytes < qkvp_decode_attention_workspace_bytes(cache, Hq, accumulate)) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const DevStatus st{static_cast<int*>(ws), 0};
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  if (!lse) lse = reinterpret_cast<float*>(wsb + kCacheStatusBytes);
  float* scores = accumulate ? reinterpret_cast<float*>(wsb + kCacheStatusBytes + lse_bytes(a, Hq)) : nullptr;
  const int G = Hq / a.H;
  const dim3 grid(Hq, a.B);
  mark(s);
#define QKVP_DECODE(D)                                                                                \
  (cache->fp8 ? decode_kernel<D, true><<<grid, kThreads, 0, s>>>(a, G, scale, q, out, lse, scores, st) \
              : decode_kernel<D, false><<<grid, kThreads, 0, s>>>(a, G, scale, q, out, lse, scores, st))
  if (a.d == 64) QKVP_DECODE(64);
  else if (a.d == 96) QKVP_DECODE(96);
  else QKVP_DECODE(128);
#undef QKVP_DECODE
  if (cudaGetLastError() != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  if (accumulate) {
    decode_weight_kernel<<<dim3((a.capacity() + kThreads - 1) / kThreads, a.H, a.B), kThreads, 0, s>>>(a, G, lse, scores,
                                                                                                    st);
    if (cudaGetLastError() != cudaSuccess) return QKVP_ERR_CUDA;
    mark(s);
  }
  return QKVP_OK;
}

}  // extern "C"
