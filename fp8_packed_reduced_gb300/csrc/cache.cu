// The paged key-value cache: argument checks, append and eviction.
#include <algorithm>
#include <climits>

#include "cache.cuh"
#include "kernels.cuh"

namespace qkvp {

namespace {
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
}  // namespace

int check_cache(const qkvp_cache* c, CacheArgs* a) {
  if (!c) return QKVP_ERR_INVALID_ARGUMENT;
  if (c->P < 1 || c->page < 1 || c->H < 1 || c->d_qk < 1 || c->d_v < 1 || c->B < 1 || c->max_pages < 1)
    return QKVP_ERR_INVALID_ARGUMENT;
  if (c->fp8 != 0 && c->fp8 != 1) return QKVP_ERR_INVALID_ARGUMENT;
  if (c->H > 128 || c->B > kMaxSeqs) return QKVP_ERR_UNSUPPORTED;
  if (c->page < 16 || c->page > kMaxPage || (c->page & (c->page - 1))) return QKVP_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * c->page > (1 << 24)) return QKVP_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * c->page * c->B > (int64_t(1) << 34)) return QKVP_ERR_UNSUPPORTED;
  // rows are counted in 32 bits (2^31 of the smallest rows are 412 GB)
  if (static_cast<int64_t>(c->P) * c->H * c->page > (int64_t(1) << 31) - 1) return QKVP_ERR_UNSUPPORTED;
  if (c->d_qk != 64 && c->d_qk != 96 && c->d_qk != 128) return QKVP_ERR_UNSUPPORTED;
  if (c->d_v != kDv) return QKVP_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->table || !c->lengths) return QKVP_ERR_INVALID_ARGUMENT;
  if (c->fp8 && (!c->k_scale || !c->v_scale)) return QKVP_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {c->k, c->v, c->k_scale, c->v_scale, c->weight, c->pos, c->table, c->lengths};
  for (const void* p : ptrs)
    if (!aligned16(p)) return QKVP_ERR_MISALIGNED;
  a->k = static_cast<uint8_t*>(c->k);
  a->v = static_cast<uint8_t*>(c->v);
  a->k_scale = c->fp8 ? c->k_scale : nullptr;
  a->v_scale = c->fp8 ? c->v_scale : nullptr;
  a->weight = c->weight;
  a->pos = c->pos;
  a->table = c->table;
  a->lengths = c->lengths;
  a->P = c->P;
  a->H = c->H;
  a->B = c->B;
  a->max_pages = c->max_pages;
  a->page_shift = 0;
  while ((1 << a->page_shift) < c->page) ++a->page_shift;
  a->d = c->d_qk;
  return QKVP_OK;
}

namespace {

// ---------------------------------------------------------------------------
// Append.  Reads every new row once and writes it once, so it is bound by
// memory (by latency for one token per sequence).  A half-warp holds one row
// of k (D / 8 lanes) and of v (16 lanes), 16 bytes a lane, which puts the row
// maximum of the E4M3 form into four shuffles; a warp takes 2 R consecutive
// tokens of one head, whose rows are contiguous in k and v and, within a
// page, in the pools.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

// The number of entries of cu[0 .. n) that are <= t (cu non-decreasing),
// by the whole warp: 32 probes a step.
__device__ __forceinline__ int warp_upper_bound(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + step * (lane + 1) - 1;   // the last entry of the lane's part
    const bool le = i < hi && __ldg(cu + i) <= t;
    const int parts = __popc(__ballot_sync(0xffffffffu, le));
    hi = min(hi, lo + step * (parts + 1) - 1);
    lo = min(lo + step * parts, hi);
  }
  return lo;
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float absmax8(uint4 w) {
  float m = 0.f;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
  return m;
}

// Eight codes of the bf16 values w at scale s.  Below 2^-100 the scale's
// reciprocal may overflow, so the products that bracket the quotient cannot
// be formed and the division itself decides.
__device__ __forceinline__ uint2 codes8(uint4 w, float s) {
  const f2 x[4] = {f2_from_bf16x2(w.x), f2_from_bf16x2(w.y), f2_from_bf16x2(w.z), f2_from_bf16x2(w.w)};
  if (s < 7.888609e-31f) return quant8_exact(x[0], x[1], x[2], x[3], s);
  return quant8(x, make_bracket2(s));
}

template <int D, bool FP8, int R>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(CacheArgs c, int T, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                  const int32_t* __restrict__ pos, const int32_t* __restrict__ cu, int32_t* lengths_out, int in_place,
                  unsigned int* arrived, DevStatus st) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int h = blockIdx.y;
  const int t0 = (blockIdx.x * (kAppendThreads / 32) + warp) * 2 * R;
  constexpr int KL = D / 8;   // lanes of a k row

  uint4 kx[R], vx[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = t0 + 2 * r + half;
    kx[r] = vx[r] = make_uint4(0, 0, 0, 0);
    if (t < T) {
      const int64_t row = static_cast<int64_t>(h) * T + t;
      if (l < KL) kx[r] = __ldg(reinterpret_cast<const uint4*>(k) + row * KL + l);
      vx[r] = __ldg(reinterpret_cast<const uint4*>(v) + row * 16 + l);
    }
  }

  // lane j < 2 R finds the place of token t0 + j
  int64_t dst = -1;
  if (t0 < T) {
    const int t = t0 + (lane % (2 * R));
    int b = t, start = t;
    if (cu != nullptr) {
      b = warp_upper_bound(cu, c.B + 1, t0) - 1;
      while (b < c.B && t < T && __ldg(cu + b + 1) <= t) ++b;   // the warp's later tokens, past empty sequences
      start = b >= 0 && b < c.B ? __ldg(cu + b) : 0;
    }
    if (t < T && lane < 2 * R) {
      if (b < 0 || b >= c.B) {
        record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
      } else {
        const int64_t slot = static_cast<int64_t>(checked_length(c, b, st, KID_CACHE_APPEND)) + (t - start);
        if (slot < 0 || slot >= c.capacity())
          record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
        else
          dst = cache_row(c, b, h, static_cast<int>(slot), st, KID_CACHE_APPEND);
      }
      if (dst >= 0) {
        if (c.weight) c.weight[dst] = 0.f;
        if (c.pos) c.pos[dst] = __ldg(pos + t);
      }
    }
  }

#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = __shfl_sync(0xffffffffu, dst, 2 * r + half);
    if (FP8) {
      const float sk = scale_from_amax(half_warp_max(absmax8(kx[r])));
      const float sv = scale_from_amax(half_warp_max(absmax8(vx[r])));
      if (row >= 0) {
        if (l < KL) reinterpret_cast<uint2*>(c.k)[row * KL + l] = codes8(kx[r], sk);
        reinterpret_cast<uint2*>(c.v)[row * 16 + l] = codes8(vx[r], sv);
        if (l == 0) {
          c.k_scale[row] = sk;
          c.v_scale[row] = sv;
        }
      }
    } else if (row >= 0) {
      if (l < KL) reinterpret_cast<uint4*>(c.k)[row * KL + l] = kx[r];
      reinterpret_cast<uint4*>(c.v)[row * 16 + l] = vx[r];
    }
  }

  // The lengths after the append.  In place they may change only once every
  // block has read the old ones: the last block to arrive writes them.
  __shared__ bool writes;
  __syncthreads();
  if (threadIdx.x == 0) {
    if (in_place) {
      const unsigned int blocks = gridDim.x * gridDim.y;
      __threadfence();
      writes = atomicAdd(arrived, 1u) == blocks - 1;
      if (writes) *arrived = 0;
      __threadfence();
    } else {
      writes = blockIdx.x == 0 && blockIdx.y == 0;
    }
  }
  __syncthreads();
  if (!writes) return;
  for (int b = threadIdx.x; b < c.B; b += kAppendThreads) {
    const int n = __ldcg(c.lengths + b), cap = c.capacity();
    int64_t add = cu != nullptr ? static_cast<int64_t>(__ldg(cu + b + 1)) - __ldg(cu + b) : 1;
    if (add < 0 || n < 0 || n + add > cap) record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
    if (add < 0) add = 0;
    const int64_t m = static_cast<int64_t>(n < 0 ? 0 : n) + add;
    lengths_out[b] = static_cast<int32_t>(m > cap ? cap : m);
  }
}

template <int D, bool FP8>
cudaError_t launch_append(const CacheArgs& c, int T, const uint16_t* k, const uint16_t* v, const int32_t* pos,
                          const int32_t* cu, int32_t* lengths_out, unsigned int* arrived, DevStatus st,
                          cudaStream_t s) {
  const int in_place = lengths_out == c.lengths;
  const auto blocks = [&](int r) { return std::max(1, (T + 16 * r - 1) / (16 * r)); };
  append_kernel<D, FP8, 1><<<dim3(blocks(1), c.H), kAppendThreads, 0, s>>>(c, T, k, v, pos, cu, lengths_out, in_place,
                                                                           arrived, st);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_append_d(const CacheArgs& c, int T, const uint16_t* k, const uint16_t* v, const int32_t* pos,
                            const int32_t* cu, int32_t* lengths_out, unsigned int* arrived, DevStatus st,
                            cudaStream_t s) {
  switch (c.d) {
    case 64: return launch_append<64, FP8>(c, T, k, v, pos, cu, lengths_out, arrived, st, s);
    case 96: return launch_append<96, FP8>(c, T, k, v, pos, cu, lengths_out, arrived, st, s);
    case 128: return launch_append<128, FP8>(c, T, k, v, pos, cu, lengths_out, arrived, st, s);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Eviction: which slots stay.  One block per (head, sequence) finds the
// budget-th largest key by four passes over its digits (radix selection),
// then ranks ties, freed and moving slots in slot order.  A key orders first
// by "protected", then by weight.
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;

__device__ __forceinline__ uint32_t evict_key(float w, int pos, int64_t protect_above) {
  if (pos > protect_above) return 0xffffffffu;
  if (isnan(w)) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // -inf -> 0x007fffff, +inf -> 0xff800000
}

// Exclusive sum over the block's warps of one value per warp (valid on every
// thread); *total receives the sum.  red: kSelectWarps ints.
__device__ __forceinline__ int warp_offsets(int mine, int* red, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) red[warp] = mine;
  __syncthreads();
  int v = red[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  *total = __shfl_sync(0xffffffffu, v, 31);
  const int incl = __shfl_sync(0xffffffffu, v, warp);
  return incl - mine;
}

__global__ void __launch_bounds__(kSelectThreads)
    evict_select_kernel(CacheArgs c, int budget, int recent, int32_t* __restrict__ slots, int32_t* __restrict__ holes,
                        DevStatus st) {
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = checked_length(c, b, st, KID_EVICT_SELECT);
  const int64_t out = (static_cast<int64_t>(b) * c.H + h) * budget;
  slots += out;
  holes += out;
  if (n <= budget) {
    for (int j = threadIdx.x; j < budget; j += kSelectThreads) slots[j] = j < n ? j : -1;
    return;
  }
  __shared__ unsigned int hist[256];
  __shared__ int red[kSelectWarps];
  __shared__ unsigned int s_prefix, s_need;

  // the newest position
  int newest = INT_MIN;
  for (int i = threadIdx.x; i < n; i += kSelectThreads) {
    const int row = cache_row(c, b, h, i, st, KID_EVICT_SELECT);
    if (row >= 0) newest = max(newest, c.pos[row]);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) red[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, red[lane]);
  const int64_t above = static_cast<int64_t>(newest) - recent;
  // slots in a page outside the pool have the lowest key
  const auto key_of = [&](int i) {
    const int row = cache_row(c, b, h, i, st, KID_EVICT_SELECT);
    return row < 0 ? 0u : evict_key(c.weight[row], c.pos[row], above);
  };

  unsigned int prefix = 0, need = budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    const unsigned int mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = threadIdx.x; i < n; i += kSelectThreads) {
      const uint32_t key = key_of(i);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 255;
      while (d > 0 && hist[d] < need) need -= hist[d--];
      s_prefix = prefix | (static_cast<unsigned int>(d) << shift);
      s_need = need;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // kept: keys above `prefix`, and the first `need` slots whose key equals it

  const int seg = (n + kSelectThreads - 1) / kSelectThreads * 32;   // a warp's consecutive slots
  const int i0 = min(n, warp * seg), i1 = min(n, i0 + seg);
  int ties = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32)
    ties += __popc(__ballot_sync(0xffffffffu, i < i1 && key_of(i) == prefix));
  int total;
  const int ties0 = warp_offsets(ties, red, &total);
  // A walk over the warp's slots in order: calls f(slot, kept, freed before
  // it, moving before it) and returns both counts.
  const auto walk = [&](int freed, int moving, auto f) {
    int t = ties0;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
      const bool in = i < i1;
      const uint32_t key = in ? key_of(i) : 0u;
      const unsigned int below = (1u << lane) - 1u;
      const unsigned int tie = __ballot_sync(0xffffffffu, in && key == prefix);
      const bool kept = in && (key > prefix || (key == prefix && t + __popc(tie & below) < static_cast<int>(need)));
      const unsigned int fr = __ballot_sync(0xffffffffu, in && !kept && i < budget);
      const unsigned int mv = __ballot_sync(0xffffffffu, kept && i >= budget);
      if (in) f(i, kept, freed + __popc(fr & below), moving + __popc(mv & below));
      t += __popc(tie);
      freed += __popc(fr);
      moving += __popc(mv);
    }
    return make_int2(freed, moving);
  };
  const int2 counts = walk(0, 0, [](int, bool, int, int) {});
  const int freed0 = warp_offsets(counts.x, red, &total);
  const int moving0 = warp_offsets(counts.y, red, &total);
  walk(freed0, moving0, [&](int i, bool kept, int freed, int) {
    if (i >= budget) return;
    if (kept)
      slots[i] = i;
    else
      holes[freed] = i;
  });
  __syncthreads();   // holes[] is complete
  walk(freed0, moving0, [&](int i, bool kept, int, int moving) {
    if (kept && i >= budget) slots[holes[moving]] = i;
  });
}

// ---------------------------------------------------------------------------
// Eviction: the moves, and the lengths.  A warp takes 32 new slots and copies
// the rows that change, one after the other, 16 bytes a lane.  Sources lie at
// or above the budget and destinations below it, so no copy disturbs another.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    evict_move_kernel(CacheArgs c, int budget, const int32_t* __restrict__ slots, int32_t* lengths_out, int kchunks,
                      int vchunks, DevStatus st) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
  const int j = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 32 + lane;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int n = c.lengths[b], cap = c.capacity();
    lengths_out[b] = min(budget, max(0, min(n, cap)));
  }
  int64_t src = -1, dst = -1;
  if (j < budget) {
    const int from = __ldg(slots + (static_cast<int64_t>(b) * c.H + h) * budget + j);
    if (from != j && from >= 0) {
      src = cache_row(c, b, h, from, st, KID_EVICT_MOVE);
      dst = cache_row(c, b, h, j, st, KID_EVICT_MOVE);
    }
  }
  const bool moves = src >= 0 && dst >= 0;
  unsigned int todo = __ballot_sync(0xffffffffu, moves);
  if (moves) {
    c.weight[dst] = c.weight[src];
    c.pos[dst] = c.pos[src];
    if (c.k_scale) {
      c.k_scale[dst] = c.k_scale[src];
      c.v_scale[dst] = c.v_scale[src];
    }
  }
  while (todo) {
    const int who = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t s = __shfl_sync(0xffffffffu, src, who), d = __shfl_sync(0xffffffffu, dst, who);
    if (lane < kchunks)
      reinterpret_cast<uint4*>(c.k)[d * kchunks + lane] = reinterpret_cast<const uint4*>(c.k)[s * kchunks + lane];
    else if (lane < kchunks + vchunks)
      reinterpret_cast<uint4*>(c.v)[d * vchunks + lane - kchunks] =
          reinterpret_cast<const uint4*>(c.v)[s * vchunks + lane - kchunks];
  }
}

}  // namespace
}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_cache_append_workspace_bytes(const qkvp_cache* cache) {
  CacheArgs a;
  return check_cache(cache, &a) == QKVP_OK ? kCacheStatusBytes : 0;
}

int qkvp_cache_append(const qkvp_cache* cache, int T, const uint16_t* k, const uint16_t* v, const int32_t* pos,
                      const int32_t* cu, int32_t* lengths_out, void* ws, size_t ws_bytes, void* stream) {
  CacheArgs a;
  const int rc = check_cache(cache, &a);
  if (rc != QKVP_OK) return rc;
  if (T < 0 || !ws || (T > 0 && (!k || !v || !pos))) return QKVP_ERR_INVALID_ARGUMENT;
  if (!cu && T != a.B) return QKVP_ERR_INVALID_ARGUMENT;
  if (T > (1 << 24)) return QKVP_ERR_UNSUPPORTED;
  if (!lengths_out) lengths_out = cache->lengths;
  const void* ptrs[] = {k, v, pos, cu, lengths_out, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return QKVP_ERR_MISALIGNED;
  if (ws_bytes < kCacheStatusBytes) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int* arrived = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + 192);
  const DevStatus st{static_cast<int*>(ws), 0};
  mark(s);
  const cudaError_t e = cache->fp8 ? launch_append_d<true>(a, T, k, v, pos, cu, lengths_out, arrived, st, s)
                                   : launch_append_d<false>(a, T, k, v, pos, cu, lengths_out, arrived, st, s);
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

size_t qkvp_cache_evict_workspace_bytes(const qkvp_cache* cache, int budget) {
  CacheArgs a;
  if (check_cache(cache, &a) != QKVP_OK || budget < 1 || budget > a.capacity()) return 0;
  return kCacheStatusBytes + static_cast<size_t>(a.B) * a.H * budget * sizeof(int32_t);
}

int qkvp_cache_evict(const qkvp_cache* cache, int budget, int recent, int32_t* slots, int32_t* lengths_out, void* ws,
                     size_t ws_bytes, void* stream) {
  CacheArgs a;
  const int rc = check_cache(cache, &a);
  if (rc != QKVP_OK) return rc;
  if (!a.weight || !a.pos || !slots || !ws) return QKVP_ERR_INVALID_ARGUMENT;
  if (budget < 1 || budget > a.capacity() || recent < 0 || recent > budget) return QKVP_ERR_INVALID_ARGUMENT;
  if (!lengths_out) lengths_out = cache->lengths;
  const void* ptrs[] = {slots, lengths_out, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return QKVP_ERR_MISALIGNED;
  if (ws_bytes < qkvp_cache_evict_workspace_bytes(cache, budget)) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const DevStatus st{static_cast<int*>(ws), 0};
  int32_t* holes = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kCacheStatusBytes);
  mark(s);
  evict_select_kernel<<<dim3(a.H, a.B), kSelectThreads, 0, s>>>(a, budget, recent, slots, holes, st);
  if (cudaGetLastError() != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  const int esize = cache->fp8 ? 1 : 2;
  evict_move_kernel<<<dim3((budget + 255) / 256, a.H, a.B), 256, 0, s>>>(a, budget, slots, lengths_out,
                                                                         a.d * esize / 16, kDv * esize / 16, st);
  if (cudaGetLastError() != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

}  // extern "C"
