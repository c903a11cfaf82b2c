// Rows of a packed projection, y [T, N] = q heads, k heads, v heads side by
// side, into head-major q, k and v, and back:
//   forward   r = (mean x^2 + eps)^-1/2,  q, k = R(x r gain),  v = x
//   backward  g = R^T(dq),  dgain = sum g x r,
//             dx = r (g gain - x r mean(g gain x r)),  dv as it is
// with R the rotation of the pairs (i, i + d / 2) by their angles.  Each value
// is read once and written once; a token's cosines and sines are read once for
// all its heads.
#include <algorithm>
#include <cmath>

#include "cache.cuh"
#include "kernels.cuh"

namespace qkvp {
namespace {

enum NormKernelId : int { KID_NORM_FWD = 22, KID_NORM_BWD = 23 };

struct NormArgs {
  int T, Hq, H, axes, max_pos;
  int bound[2];             // entries of the table from which on the second, the third axis turns
  int64_t ldy;              // elements between rows of y
  float eps;
  const float* table;       // [d / 4][max_pos][4]
  const int32_t* pos;       // [axes][T]
  const float *q_gain, *k_gain;   // [d] or null
  const uint16_t* y;
  uint16_t *q, *k, *v;      // [Hq, T, d], [H, T, d], [H, T, 128]
  float* rstd;              // [Hq + H, T]
  const uint16_t *dq, *dk, *dv;
  uint16_t* dy;             // [T, N]
  float* partial;           // [blocks][2][d] of the gains' gradients, or null
  float *dq_gain, *dk_gain;
};

constexpr int kThreads = 256;
constexpr int kNormHeader = 1024;   // of the workspace: the status word
constexpr int kMaxNormBlocks = 2048;

// A token takes GROUP lanes; lane c < d / 16 has columns 8 c .. 8 c + 7 and the
// same of the second half, that is, eight pairs.
template <int D>
struct Lanes {
  static constexpr int GROUP = D == 64 ? 4 : 8, USED = D / 16;
  static constexpr int TOKENS = kThreads / GROUP;   // of a block
};

__device__ __forceinline__ void unpack8(float (&x)[8], uint4 w) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
template <int GROUP>
__device__ __forceinline__ float group_add(float v) {
#pragma unroll
  for (int o = 1; o < GROUP; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosines and sines of the lane's eight pairs.
__device__ __forceinline__ void load_turn(const NormArgs& p, int t, int c, float (&cs)[8], float (&sn)[8], const DevStatus& st, int kid) {
  int at[3];
  bool bad = false;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    at[a] = a < p.axes ? __ldg(p.pos + static_cast<int64_t>(a) * p.T + t) : 0;
    bad |= at[a] < 0 || at[a] >= p.max_pos;
    at[a] = min(max(at[a], 0), p.max_pos - 1);
  }
  if (bad) record_error(st, QKVP_ERR_DEVICE_INPUT, kid);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * c + i, x = j < p.bound[0] ? at[0] : j < p.bound[1] ? at[1] : at[2];
    const float4 e = __ldg(reinterpret_cast<const float4*>(p.table) + static_cast<int64_t>(j) * p.max_pos + x);
    cs[2 * i] = e.x, cs[2 * i + 1] = e.y, sn[2 * i] = e.z, sn[2 * i + 1] = e.w;
  }
}

__device__ __forceinline__ void load_gain(const float* gain, int D, int c, float (&lo)[8], float (&hi)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = gain ? __ldg(gain + 8 * c + i) : 1.f;
    hi[i] = gain ? __ldg(gain + D / 2 + 8 * c + i) : 1.f;
  }
}

// Copies the rows of v between y's form and the head-major one.
template <int D, bool BACK>
__device__ __forceinline__ void copy_v(const NormArgs& p, int t, int c, int64_t N, int first, int last) {
  constexpr int GROUP = Lanes<D>::GROUP;
  const int64_t col = static_cast<int64_t>(p.Hq + p.H) * D;
#pragma unroll 2
  for (int h = first; h < last; ++h) {
    const uint4* from = reinterpret_cast<const uint4*>(BACK ? p.dv + (static_cast<int64_t>(h) * p.T + t) * kDv : p.y + t * p.ldy + col + h * kDv);
    uint4* to = reinterpret_cast<uint4*>(BACK ? p.dy + t * N + col + h * kDv : p.v + (static_cast<int64_t>(h) * p.T + t) * kDv);
    uint4 w[16 / GROUP];
#pragma unroll
    for (int i = 0; i < 16 / GROUP; ++i) w[i] = __ldg(from + i * GROUP + c);
#pragma unroll
    for (int i = 0; i < 16 / GROUP; ++i) to[i * GROUP + c] = w[i];
  }
}

// Heads are cut into gridDim.y parts where the tokens alone do not fill the GPU.
__device__ __forceinline__ void head_part(const NormArgs& p, int& first, int& last) {
  const int rows = p.Hq + 2 * p.H, each = (rows + gridDim.y - 1) / gridDim.y;
  first = min(rows, static_cast<int>(blockIdx.y) * each);
  last = min(rows, first + each);
}

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormArgs p, DevStatus st) {
  using L = Lanes<D>;
  wait_for_previous();
  const int c = threadIdx.x % L::GROUP;
  const int t = blockIdx.x * L::TOKENS + threadIdx.x / L::GROUP;
  const bool real = t < p.T, used = real && c < L::USED;
  const int64_t N = static_cast<int64_t>(p.Hq + p.H) * D + static_cast<int64_t>(p.H) * kDv;
  int first, last;
  head_part(p, first, last);
  float cs[8], sn[8];
  if (used && first < p.Hq + p.H) load_turn(p, t, c, cs, sn, st, KID_NORM_FWD);
  const auto heads = [&](int h0, int h1, const float* gain, uint16_t* out, int base) {
    if (h0 >= h1) return;
    float glo[8], ghi[8];
    if (used) load_gain(gain, D, c, glo, ghi);
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
      float lo[8], hi[8], sum = 0.f;
      if (used) {
        const uint4* x = reinterpret_cast<const uint4*>(p.y + t * p.ldy + static_cast<int64_t>(h) * D);
        unpack8(lo, __ldg(x + c));
        unpack8(hi, __ldg(x + D / 16 + c));
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += lo[i] * lo[i] + hi[i] * hi[i];
      }
      const float r = 1.f / sqrtf(group_add<L::GROUP>(sum) * (1.f / D) + p.eps);
      if (!used) continue;
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = lo[i] * r * glo[i], w = hi[i] * r * ghi[i];
        a[i] = u * cs[i] - w * sn[i];
        b[i] = w * cs[i] + u * sn[i];
      }
      uint4* to = reinterpret_cast<uint4*>(out + (static_cast<int64_t>(h - base) * p.T + t) * D);
      to[c] = pack8(a);
      to[D / 16 + c] = pack8(b);
      if (c == 0) p.rstd[static_cast<int64_t>(h) * p.T + t] = r;
    }
  };
  heads(first, min(last, p.Hq), p.q_gain, p.q, 0);
  heads(max(first, p.Hq), min(last, p.Hq + p.H), p.k_gain, p.k, p.Hq);
  if (real) copy_v<D, false>(p, t, c, N, max(first, p.Hq + p.H) - p.Hq - p.H, last - p.Hq - p.H);
}

template <int D, bool GAIN>
__global__ void __launch_bounds__(kThreads) norm_rope_back_kernel(const __grid_constant__ NormArgs p, DevStatus st) {
  using L = Lanes<D>;
  wait_for_previous();
  const int c = threadIdx.x % L::GROUP;
  const int64_t N = static_cast<int64_t>(p.Hq + p.H) * D + static_cast<int64_t>(p.H) * kDv;
  int first, last;
  head_part(p, first, last);
  float sums[2][16] = {};   // of q's gain, of k's
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * L::TOKENS; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * L::TOKENS) {
    const int64_t at = t0 + threadIdx.x / L::GROUP;
    const bool real = at < p.T, used = real && c < L::USED;
    const int t = static_cast<int>(at);
    float cs[8], sn[8];
    if (used && first < p.Hq + p.H) load_turn(p, t, c, cs, sn, st, KID_NORM_BWD);
    const auto heads = [&](int h0, int h1, const float* gain, const uint16_t* grad, int base, float (&sum)[16]) {
      if (h0 >= h1) return;
      float glo[8], ghi[8];
      if (used) load_gain(gain, D, c, glo, ghi);
#pragma unroll 2
      for (int h = h0; h < h1; ++h) {
        float lo[8], hi[8], a[8], b[8], dot = 0.f, r = 0.f;
        if (used) {
          const uint4* x = reinterpret_cast<const uint4*>(p.y + t * p.ldy + static_cast<int64_t>(h) * D);
          const uint4* g = reinterpret_cast<const uint4*>(grad + (static_cast<int64_t>(h - base) * p.T + t) * D);
          unpack8(lo, __ldg(x + c));
          unpack8(hi, __ldg(x + D / 16 + c));
          unpack8(a, __ldg(g + c));
          unpack8(b, __ldg(g + D / 16 + c));
          r = __ldg(p.rstd + static_cast<int64_t>(h) * p.T + t);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float u = a[i] * cs[i] + b[i] * sn[i], w = b[i] * cs[i] - a[i] * sn[i];
            lo[i] *= r;
            hi[i] *= r;
            if (GAIN) {
              sum[i] += u * lo[i];
              sum[8 + i] += w * hi[i];
            }
            a[i] = u * glo[i];
            b[i] = w * ghi[i];
            dot += a[i] * lo[i] + b[i] * hi[i];
          }
        }
        dot = group_add<L::GROUP>(dot) * (1.f / D);
        if (!used) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = r * (a[i] - lo[i] * dot);
          b[i] = r * (b[i] - hi[i] * dot);
        }
        uint4* to = reinterpret_cast<uint4*>(p.dy + t * N + static_cast<int64_t>(h) * D);
        to[c] = pack8(a);
        to[D / 16 + c] = pack8(b);
      }
    };
    heads(first, min(last, p.Hq), p.q_gain, p.dq, 0, sums[0]);
    heads(max(first, p.Hq), min(last, p.Hq + p.H), p.k_gain, p.dk, p.Hq, sums[1]);
    if (real) copy_v<D, true>(p, t, c, N, max(first, p.Hq + p.H) - p.Hq - p.H, last - p.Hq - p.H);
  }
  if (GAIN) {
    // lanes with the same columns, warps, and then (by another kernel) blocks, in a fixed order
    __shared__ float part[kThreads / 32][2][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = sums[w][i];
#pragma unroll
        for (int o = L::GROUP; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane < L::USED) part[warp][w][(i >> 3) * (D / 2) + 8 * lane + (i & 7)] = x;
      }
    __syncthreads();
    float* to = p.partial + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * (2 * D);
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) x += part[w][i / D][i % D];
      to[i] = x;
    }
  }
}

// Sums `blocks` partials of each of 2 d columns: 32 columns a block, its warps
// take the partials in turn.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const __grid_constant__ NormArgs p, int d, int blocks) {
  __shared__ float part[32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float x = 0.f;
#pragma unroll 4
  for (int b = warp; b < blocks; b += 32) x += __ldcg(p.partial + static_cast<int64_t>(b) * 2 * d + col);
  part[warp][lane] = x;
  __syncthreads();
  x = part[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int c = blockIdx.x * 32 + warp;
  if (lane == 0) (c < d ? p.dq_gain : p.dk_gain)[c < d ? c : c - d] = x;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_norm(const qkvp_norm_rope* n, NormArgs* a) {
  if (!n) return QKVP_ERR_INVALID_ARGUMENT;
  if (n->T < 0 || n->Hq < 1 || n->H < 1 || n->d_qk < 1 || n->d_v < 1 || n->max_pos < 1 || n->axes < 1 || !(n->eps >= 0.f) ||
      !(n->eps < INFINITY))
    return QKVP_ERR_INVALID_ARGUMENT;
  if (n->T > (1 << 24) || n->H > 128 || n->Hq > 1024 || n->Hq % n->H || n->axes > 3) return QKVP_ERR_UNSUPPORTED;
  if (n->d_qk != 64 && n->d_qk != 96 && n->d_qk != 128) return QKVP_ERR_UNSUPPORTED;
  if (n->d_v != kDv) return QKVP_ERR_UNSUPPORTED;
  if (!n->rope_table || (n->T && !n->pos)) return QKVP_ERR_INVALID_ARGUMENT;
  if (static_cast<int64_t>(n->max_pos) * n->d_qk > (int64_t(1) << 31)) return QKVP_ERR_UNSUPPORTED;
  if (!n->q_gain != !n->k_gain) return QKVP_ERR_INVALID_ARGUMENT;
  const int64_t N = static_cast<int64_t>(n->Hq + n->H) * n->d_qk + static_cast<int64_t>(n->H) * n->d_v;
  if (n->ldy < N) return QKVP_ERR_INVALID_ARGUMENT;
  if (n->ldy % 8) return QKVP_ERR_MISALIGNED;
  *a = NormArgs{};
  int entries = 0;
  for (int i = 0; i < n->axes; ++i) {
    const int s = n->axes == 1 ? n->d_qk / 2 : n->sections[i];
    if (s < 0 || s > n->d_qk / 2 || s % 2) return QKVP_ERR_INVALID_ARGUMENT;
    entries += s / 2;
    if (i < 2) a->bound[i] = entries;
  }
  if (entries != n->d_qk / 4) return QKVP_ERR_INVALID_ARGUMENT;
  if (n->axes == 1) a->bound[1] = entries;
  const void* ptrs[] = {n->rope_table, n->pos, n->q_gain, n->k_gain};
  for (const void* x : ptrs)
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  a->T = n->T;
  a->Hq = n->Hq;
  a->H = n->H;
  a->axes = n->axes;
  a->max_pos = n->max_pos;
  a->ldy = n->ldy;
  a->eps = n->eps;
  a->table = n->rope_table;
  a->pos = n->pos;
  a->q_gain = n->q_gain;
  a->k_gain = n->k_gain;
  return QKVP_OK;
}

// Parts of the heads: as many as bring the blocks to two a multiprocessor.
int head_parts(int64_t token_blocks, int rows, int sms) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, 2 * sms / std::max<int64_t>(1, token_blocks))));
}

template <int D>
cudaError_t forward(const NormArgs& a, int sms, DevStatus st, cudaStream_t s) {
  const int blocks = (a.T + Lanes<D>::TOKENS - 1) / Lanes<D>::TOKENS;
  return launch_dependent(norm_rope_kernel<D>, dim3(blocks, head_parts(blocks, a.Hq + 2 * a.H, sms)), kThreads, 0, s, a, st);
}

template <int D>
cudaError_t backward(const NormArgs& a, int sms, DevStatus st, cudaStream_t s) {
  // Two or three blocks fit a multiprocessor: more would only leave more partials.
  const int blocks = std::min((a.T + Lanes<D>::TOKENS - 1) / Lanes<D>::TOKENS, std::min(3 * sms, kMaxNormBlocks / 2));
  const int parts = std::min(head_parts(blocks, a.Hq + 2 * a.H, sms), kMaxNormBlocks / blocks);
  const dim3 grid(blocks, parts);
  if (!a.partial) return launch_dependent(norm_rope_back_kernel<D, false>, grid, kThreads, 0, s, a, st);
  const cudaError_t e = launch_dependent(norm_rope_back_kernel<D, true>, grid, kThreads, 0, s, a, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(gain_sum_kernel, dim3(2 * D / 32), 1024, 0, s, a, D, blocks * parts);
}

}  // namespace
}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_norm_rope_workspace_bytes(const qkvp_norm_rope* n) {
  NormArgs a;
  if (check_norm(n, &a) != QKVP_OK) return 0;
  return kNormHeader + (a.q_gain ? static_cast<size_t>(kMaxNormBlocks) * 2 * n->d_qk * sizeof(float) : 0);
}

int qkvp_norm_rope_forward(const qkvp_norm_rope* n, const uint16_t* y, uint16_t* q, uint16_t* k, uint16_t* v, float* rstd,
                           void* ws, size_t ws_bytes, void* stream) {
  NormArgs a;
  const int rc = check_norm(n, &a);
  if (rc != QKVP_OK) return rc;
  if (!ws) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {y, q, k, v, rstd, ws};
  for (const void* x : ptrs) {
    if (!x && a.T) return QKVP_ERR_INVALID_ARGUMENT;
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  }
  if (ws_bytes < kNormHeader) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  if (a.T == 0) return QKVP_OK;
  const int sms = device_sms();
  if (sms <= 0) return QKVP_ERR_CUDA;
  a.y = y;
  a.q = q;
  a.k = k;
  a.v = v;
  a.rstd = rstd;
  const DevStatus st{static_cast<int*>(ws), 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mark(s);
  const cudaError_t e = n->d_qk == 64   ? forward<64>(a, sms, st, s)
                        : n->d_qk == 96 ? forward<96>(a, sms, st, s)
                                        : forward<128>(a, sms, st, s);
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

int qkvp_norm_rope_backward(const qkvp_norm_rope* n, const uint16_t* dq, const uint16_t* dk, const uint16_t* dv,
                            const uint16_t* y, const float* rstd, uint16_t* dy, float* dq_gain, float* dk_gain, void* ws,
                            size_t ws_bytes, void* stream) {
  NormArgs a;
  const int rc = check_norm(n, &a);
  if (rc != QKVP_OK) return rc;
  if (!ws || (a.q_gain && (!dq_gain || !dk_gain))) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {dq, dk, dv, y, rstd, dy, ws};
  for (const void* x : ptrs) {
    if (!x && a.T) return QKVP_ERR_INVALID_ARGUMENT;
    if (!aligned16(x)) return QKVP_ERR_MISALIGNED;
  }
  if (!aligned16(dq_gain) || !aligned16(dk_gain)) return QKVP_ERR_MISALIGNED;
  if (ws_bytes < qkvp_norm_rope_workspace_bytes(n)) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.T == 0) {   // no token: no gradient
    if (a.q_gain && (cudaMemsetAsync(dq_gain, 0, n->d_qk * sizeof(float), s) != cudaSuccess ||
                     cudaMemsetAsync(dk_gain, 0, n->d_qk * sizeof(float), s) != cudaSuccess))
      return QKVP_ERR_CUDA;
    return QKVP_OK;
  }
  const int sms = device_sms();
  if (sms <= 0) return QKVP_ERR_CUDA;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.y = y;
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dq_gain = dq_gain;
  a.dk_gain = dk_gain;
  a.partial = a.q_gain ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kNormHeader) : nullptr;
  const DevStatus st{static_cast<int*>(ws), 0};
  mark(s);
  const cudaError_t e = n->d_qk == 64   ? backward<64>(a, sms, st, s)
                        : n->d_qk == 96 ? backward<96>(a, sms, st, s)
                                        : backward<128>(a, sms, st, s);
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

}  // extern "C"
