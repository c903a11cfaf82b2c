// Causal attention over packed sequences, forward and backward (attn.cuh has
// the formulas): one warp a row on the CUDA cores.
#include <cmath>

#include "attn.cuh"

namespace qkvp {
namespace {

constexpr int kWarps = 8;

// delta = da . a of every row and head.
__global__ void __launch_bounds__(32 * kWarps) delta_kernel(const __grid_constant__ AttnArgs p, DevStatus st) {
  wait_for_previous();
  if (blockIdx.x == 0) check_offsets(p, st, KID_ATTN_DELTA);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);   // row * Hq + head
  if (r >= static_cast<int64_t>(p.T) * p.Hq) return;
  const int lane = threadIdx.x & 31;
  const uint2 x = __ldg(reinterpret_cast<const uint2*>(p.da + r * kDv) + lane), y = __ldg(reinterpret_cast<const uint2*>(p.a + r * kDv) + lane);
  const float s = warp_add(bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x) + bf16_lo(x.y) * bf16_lo(y.y) + bf16_hi(x.y) * bf16_hi(y.y));
  if (lane == 0) p.delta[(r % p.Hq) * p.T + r / p.Hq] = s;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) dq_kernel(const __grid_constant__ AttnArgs p) {
  wait_for_previous();
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row < p.T) dq_row<D>(p, row, blockIdx.y);
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) dkv_kernel(const __grid_constant__ AttnArgs p) {
  wait_for_previous();
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row < p.T) dkv_row<D>(p, row, blockIdx.y);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t delta_bytes(const AttnArgs& a) { return (static_cast<size_t>(a.Hq) * a.T * sizeof(float) + 255) / 256 * 256; }

template <int D>
cudaError_t backward(const AttnArgs& a, DevStatus st, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
  cudaError_t e = launch_dependent(delta_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)), 32 * kWarps, 0, s, a, st);
  if (e == cudaSuccess) e = launch_dependent(dq_kernel<D>, dim3((a.T + kWarps - 1) / kWarps, a.Hq), 32 * kWarps, 0, s, a);
  if (e == cudaSuccess) e = launch_dependent(dkv_kernel<D>, dim3((a.T + kWarps - 1) / kWarps, a.H), 32 * kWarps, 0, s, a);
  return e;
}

}  // namespace

int check_attention(const qkvp_attention* at, AttnArgs* a) {
  if (!at) return QKVP_ERR_INVALID_ARGUMENT;
  if (at->T < 0 || at->Hq < 1 || at->H < 1 || at->d_qk < 1 || at->d_v < 1 || at->B < 1 || at->window < 0 || at->sinks < 0)
    return QKVP_ERR_INVALID_ARGUMENT;
  if (!(at->scale > 0.f) || !(at->scale < INFINITY)) return QKVP_ERR_INVALID_ARGUMENT;
  if (!at->cu && at->B != 1) return QKVP_ERR_INVALID_ARGUMENT;
  if (at->T > (1 << 24) || at->H > 128 || at->Hq > 1024 || at->Hq % at->H || at->B > (1 << 20)) return QKVP_ERR_UNSUPPORTED;
  if (at->d_qk != 64 && at->d_qk != 96 && at->d_qk != 128) return QKVP_ERR_UNSUPPORTED;
  if (at->d_v != kDv) return QKVP_ERR_UNSUPPORTED;
  if (!aligned16(at->cu)) return QKVP_ERR_MISALIGNED;
  *a = AttnArgs{};
  a->T = at->T;
  a->Hq = at->Hq;
  a->H = at->H;
  a->G = at->Hq / at->H;
  a->d = at->d_qk;
  a->B = at->B;
  a->window = at->window ? at->window : (1 << 24);   // no sequence is longer
  a->sinks = at->sinks;
  a->scale = at->scale;
  a->scale_log2 = at->scale * 1.4426950408889634f;
  a->cu = at->cu;
  return QKVP_OK;
}

}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_attention_workspace_bytes(const qkvp_attention* at) {
  AttnArgs a;
  if (check_attention(at, &a) != QKVP_OK) return 0;
  return kAttnHeaderBytes + delta_bytes(a);
}

int qkvp_attention_forward(const qkvp_attention* at, const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* a,
                           float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttnArgs p;
  const int rc = check_attention(at, &p);
  if (rc != QKVP_OK) return rc;
  if (!ws) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, k, v, a, lse, ws};
  for (const void* x : ptrs) {
    if (!x && p.T) return QKVP_ERR_INVALID_ARGUMENT;
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  }
  if (ws_bytes < kAttnHeaderBytes) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  if (p.T == 0) return QKVP_OK;
  p.q = q;
  p.k = k;
  p.v = v;
  p.a = a;
  p.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mark(s);
  if (launch_attention_forward(p, dev_status(ws), s) != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

int qkvp_attention_backward(const qkvp_attention* at, const uint16_t* da, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, const uint16_t* a, const float* lse, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                            void* ws, size_t ws_bytes, void* stream) {
  AttnArgs p;
  const int rc = check_attention(at, &p);
  if (rc != QKVP_OK) return rc;
  if (!ws) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {da, q, k, v, a, lse, dq, dk, dv, ws};
  for (const void* x : ptrs) {
    if (!x && p.T) return QKVP_ERR_INVALID_ARGUMENT;
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  }
  if (ws_bytes < kAttnHeaderBytes + delta_bytes(p)) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  if (p.T == 0) return QKVP_OK;
  p.q = q;
  p.k = k;
  p.v = v;
  p.a = const_cast<uint16_t*>(a);
  p.lse = const_cast<float*>(lse);
  p.da = da;
  p.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnHeaderBytes);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  const DevStatus st{static_cast<int*>(ws), 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mark(s);
  const cudaError_t e = p.d == 64 ? backward<64>(p, st, s) : p.d == 96 ? backward<96>(p, st, s) : backward<128>(p, st, s);
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

}  // extern "C"
