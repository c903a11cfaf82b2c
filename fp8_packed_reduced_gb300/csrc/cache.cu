// The paged key-value cache: argument checks, append and eviction.
#include <algorithm>
#include <atomic>
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

int device_sms() {
  static std::atomic<int> cache[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = cache[dev].load(std::memory_order_relaxed))) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

// ---------------------------------------------------------------------------
// Append.  Reads every new row once and writes it once, so it is bound by
// memory (by latency for one token per sequence).  Four lanes hold a row of k
// (D / 32 chunks of 16 bytes each) and of v (four), so a warp takes eight
// consecutive tokens of one head with 3.5 KB of loads in flight, and the work
// per row of the E4M3 form (maximum, scale, its reciprocal) is done for eight
// rows at once.  Every access is 64 bytes (32 of codes) of a row, whole
// sectors.  49152 tokens x 6 heads to E4M3, 203 MB: 35.2 us, 5.77 TB/s (with
// sixteen lanes a row 75 us; in blocks of 256 threads 37.1); 23843 tokens x 8
// heads of d_qk = 128 as bf16, 197 MB: 31.0 us, 6.35 TB/s.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;

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

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Largest magnitudes, by halves of a word, of m and a chunk (NaN is passed over).
__device__ __forceinline__ __nv_bfloat162 absmax8(__nv_bfloat162 m, const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = u[i] & 0x7FFF7FFFu;
    m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
  }
  return m;
}
__device__ __forceinline__ float larger_half(__nv_bfloat162 m) { return fmaxf(__low2float(m), __high2float(m)); }

// The codes E(x / s) of N chunks of eight bf16 values, to out[4 i].  With one
// scale per row the bracketing products of quant8 straddle a rounding boundary
// in every few instructions of a warp (a row whose largest mantissa is 128 or
// 224 has ties throughout), so the float32 quotient itself is formed, correctly
// rounded, by Markstein's iteration (IBM J. Res. Dev. 34, 1990): from y =
// RN(1/s) and q = RN(x y), r = x - q s is exact and RN(q + r y) the quotient.
// For s = RN(amax / 448) with amax and x bf16 there are 128 x 128 pairs of
// mantissas, on which it gave the rounded quotient every time (without the
// step a quarter of them are off).  r is exact and no power leaves the normal
// numbers for s in [2^-80, inf) wherever the quotient reaches 2^-11 (below that
// every code is zero); other scales, of rows that no projection gives, are
// left to the division.  A zero loses its sign in q + r y, so signs come from x.
template <int N>
__device__ __forceinline__ void store_codes(uint2* out, const uint4 (&w)[N], float s) {
  const bool usual = s >= 8.271806125530277e-25f && s < INFINITY;
  const float y1 = __frcp_rn(s);
  const f2 y = f2_make(y1, y1), ns = f2_make(-s, -s);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    if (!usual) {
      out[4 * i] = quant8_exact(f2_from_bf16x2(u[0]), f2_from_bf16x2(u[1]), f2_from_bf16x2(u[2]), f2_from_bf16x2(u[3]), s);
      continue;
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f2 x = f2_from_bf16x2(u[j]);
      const f2 q = f2_mul(x, y);
      c[j] = cvt_e4m3x2(f2_fma(f2_fma(q, ns, x), y, q));
    }
    out[4 * i] = make_uint2(__byte_perm(c[0], c[1], 0x5410) | (__byte_perm(u[0], u[1], 0x7531) & 0x80808080u),
                            __byte_perm(c[2], c[3], 0x5410) | (__byte_perm(u[2], u[3], 0x7531) & 0x80808080u));
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(CacheArgs c, int T, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                  const int32_t* __restrict__ pos, const int32_t* __restrict__ cu, int32_t* lengths_out, int in_place,
                  unsigned int* arrived, DevStatus st) {
  constexpr int KN = D / 32, VN = kDv / 32;   // chunks of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 3;
  const int h = blockIdx.y;
  const int t0 = (blockIdx.x * (kAppendThreads / 32) + warp) * 8, t = t0 + (lane >> 2);
  wait_for_previous();

  // Offsets that fall anywhere give rows to no sequence or to two: every block
  // then stores nothing, and no length grows.  (Asked for ahead of k and v: with
  // the offsets behind them the calls above took 36.1 and 31.5 us.  4096
  // sequences of one token each x 8 heads: 12.4 us, without the test 10.9.)
  bool fall = false;
  if (cu != nullptr)
    for (int b = threadIdx.x; b < c.B; b += kAppendThreads) fall |= __ldg(cu + b + 1) < __ldg(cu + b);

  uint4 kx[KN], vx[VN];
  if (t < T) {
    const int64_t in = static_cast<int64_t>(h) * T + t;
    const uint4* kp = reinterpret_cast<const uint4*>(k) + in * (4 * KN) + l;
    const uint4* vp = reinterpret_cast<const uint4*>(v) + in * (4 * VN) + l;
#pragma unroll
    for (int i = 0; i < KN; ++i) kx[i] = __ldg(kp + 4 * i);
#pragma unroll
    for (int i = 0; i < VN; ++i) vx[i] = __ldg(vp + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < KN; ++i) kx[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < VN; ++i) vx[i] = make_uint4(0, 0, 0, 0);
  }

  // the place of the lane's token
  fall = __syncthreads_or(fall);
  int64_t row = -1;
  if (t0 < T && !fall) {
    int b = t, start = t;
    if (cu != nullptr) {
      b = warp_upper_bound(cu, c.B + 1, t0) - 1;
      while (b < c.B && t < T && __ldg(cu + b + 1) <= t) ++b;   // the warp's later tokens, past empty sequences
      start = b >= 0 && b < c.B ? max(0, __ldg(cu + b)) : 0;
    }
    if (t < T) {
      if (b < 0 || b >= c.B) {
        record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
      } else {
        const int64_t slot = static_cast<int64_t>(checked_length(c, b, st, KID_CACHE_APPEND)) + (t - start);
        if (slot < 0 || slot >= c.capacity())
          record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
        else
          row = cache_row(c, b, h, static_cast<int>(slot), st, KID_CACHE_APPEND);
      }
      if (row >= 0 && l == 0) {
        if (c.weight) c.weight[row] = 0.f;
        if (c.pos) c.pos[row] = __ldg(pos + t);
      }
    }
  }

  if (FP8) {
    __nv_bfloat162 ak = __float2bfloat162_rn(0.f), av = ak;
#pragma unroll
    for (int i = 0; i < KN; ++i) ak = absmax8(ak, kx[i]);
#pragma unroll
    for (int i = 0; i < VN; ++i) av = absmax8(av, vx[i]);
    const float sk = scale_from_amax(quad_max(larger_half(ak))), sv = scale_from_amax(quad_max(larger_half(av)));
    if (row >= 0) {
      store_codes(reinterpret_cast<uint2*>(c.k) + row * (4 * KN) + l, kx, sk);
      store_codes(reinterpret_cast<uint2*>(c.v) + row * (4 * VN) + l, vx, sv);
      if (l == 0) {
        c.k_scale[row] = sk;
        c.v_scale[row] = sv;
      }
    }
  } else if (row >= 0) {
#pragma unroll
    for (int i = 0; i < KN; ++i) reinterpret_cast<uint4*>(c.k)[row * (4 * KN) + l + 4 * i] = kx[i];
#pragma unroll
    for (int i = 0; i < VN; ++i) reinterpret_cast<uint4*>(c.v)[row * (4 * VN) + l + 4 * i] = vx[i];
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
    int add = 1;   // rows that there are for the sequence
    if (cu != nullptr) {
      const int first = __ldg(cu + b), end = __ldg(cu + b + 1);
      if (fall || (b == 0 && first != 0) || (b == c.B - 1 && end != T)) record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
      add = fall ? 0 : min(T, max(0, end)) - min(T, max(0, first));
    }
    const int64_t m = static_cast<int64_t>(n < 0 ? 0 : n) + add;
    if (n < 0 || m > cap) record_error(st, QKVP_ERR_DEVICE_INPUT, KID_CACHE_APPEND);
    lengths_out[b] = static_cast<int32_t>(m > cap ? cap : m);
  }
}

template <int D, bool FP8>
cudaError_t launch_append(const CacheArgs& c, int T, const uint16_t* k, const uint16_t* v, const int32_t* pos,
                          const int32_t* cu, int32_t* lengths_out, unsigned int* arrived, DevStatus st,
                          cudaStream_t s) {
  const dim3 grid(std::max(1, (T + kAppendThreads / 4 - 1) / (kAppendThreads / 4)), c.H);
  return launch_dependent(append_kernel<D, FP8>, grid, kAppendThreads, 0, s, c, T, k, v, pos, cu, lengths_out,
                          static_cast<int>(lengths_out == c.lengths), arrived, st);
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
// Eviction: which slots stay.  A cluster of blocks per (head, sequence) reads
// weights and positions once, into keys that order first by "protected", then
// by weight, kept in shared memory; finds the budget-th largest key by three
// passes over its digits (radix selection, the blocks' histograms added
// through distributed shared memory), then ranks freed and moving slots in
// slot order: the j-th of both make a pair for the moves.  Every step costs
// little beside its latency, so the slots of one head are spread over as many
// blocks as a cluster and the GPU hold.
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSelectAlone = 4 * kSelectThreads;  // slots that one block selects from, whatever the cluster
constexpr int kListed = 2048, kGathered = 4096;   // keys that share the first digit, of a block and of all
constexpr int kSelectKeys = 176 * 1024 / 4;       // keys in shared memory, at most

__device__ __forceinline__ uint32_t evict_key(float w, int pos, int64_t protect_above) {
  if (pos > protect_above) return 0xffffffffu;
  if (isnan(w)) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // -inf -> 0x007fffff, +inf -> 0xff800000
}

// The value of this block's shared variable `p` in block `rank` of the cluster.
__device__ __forceinline__ int ld_rank(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_rank(p, rank)) : "memory");
  return v;
}

// A barrier of the blocks of one piece.
template <int BLOCKS>
__device__ __forceinline__ void sync_blocks() {
  if (BLOCKS > 1)
    cluster_sync_all();
  else
    __syncthreads();
}
// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int4 ld_rank4(const int* p, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(mapa_rank(p, rank))
               : "memory");
  return v;
}

// Sums over the block of one value per thread, in thread order: the
// inclusive prefix up to this thread, and *total.  red: kSelectWarps ints.
__device__ __forceinline__ int block_prefix(int v, int* red, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();   // red is free
  if (lane == 31) red[warp] = incl;
  __syncthreads();
  const int w = lane < kSelectWarps ? red[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, w);
  return incl + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

struct __align__(16) SelectShared {
  int hist[3][kBins];
  // the block's slots with a larger, an equal key, below and above the budget (read as one int4)
  int above_lo, above_hi, ties_lo, ties_hi;
  int4 warps[kSelectWarps];   // the same of its warps
  int red[kSelectWarps];
  int newest, slice, listed, digit, need, ties;
};

// Where, counted from the highest bin, does the sum of counts reach `need`
// (which it does)?  `v`: the counts of bins top - 4 t - 0 .. 3 on thread t (0
// past the bins).  Leaves the bin, what is still needed of it and what it
// holds in x.digit, x.need and x.ties, for every thread after the barrier
// inside.
__device__ __forceinline__ void find_digit(const int4& v, int top, int need, SelectShared& x) {
  const int n[4] = {v.x, v.y, v.z, v.w};
  const int sum = n[0] + n[1] + n[2] + n[3];
  int total, before = block_prefix(sum, x.red, &total) - sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (before < need && need <= before + n[i]) {
      x.digit = top - 4 * static_cast<int>(threadIdx.x) - i;
      x.need = need - before;
      x.ties = n[i];
    }
    before += n[i];
  }
  __syncthreads();
}
__device__ __forceinline__ int4 reversed(const int4& v) { return make_int4(v.w, v.z, v.y, v.x); }

// Workspace of an eviction: pairs of (freed, moving) slots and their number.
struct EvictPairs {
  int* count;     // [B, H]
  int* freed;     // [B, H, budget]
  int* moving;    // [B, H, budget]
};

// The selection of one piece by BLOCKS blocks of the cluster.
template <int BLOCKS>
__device__ __forceinline__ void select_slots(const CacheArgs& c, int b, int h, int n, int budget, int recent, int rank,
                                             uint32_t* keys, int key_slots, SelectShared& x,
                                             int32_t* __restrict__ slots, const EvictPairs& pairs, const DevStatus& st) {
  constexpr int blocks = BLOCKS;   // their remote loads are issued together
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t piece = static_cast<int64_t>(b) * c.H + h;
  // this block's consecutive slots, a multiple of 32 for every warp
  const int seg = ((n + blocks - 1) / blocks + kSelectThreads - 1) / kSelectThreads * kSelectThreads;
  const int s0 = min(n, rank * seg), cnt = min(n, s0 + seg) - s0;
  for (int i = threadIdx.x; i < 3 * kBins; i += kSelectThreads) (&x.hist[0][0])[i] = 0;
  if (threadIdx.x == 0) x.listed = 0;
  const bool cached = seg <= key_slots;

  // The newest position; the weights go into keys[] meanwhile.
  int newest = INT_MIN;
#pragma unroll 4
  for (int i = threadIdx.x * 4; i < cnt; i += kSelectThreads * 4) {   // four slots lie in one page
    const int row = cache_row(c, b, h, s0 + i, st, KID_EVICT_SELECT);
    if (row < 0) continue;
    const int4 p = *reinterpret_cast<const int4*>(c.pos + row);
    if (cached) *reinterpret_cast<float4*>(keys + i) = *reinterpret_cast<const float4*>(c.weight + row);
    newest = max(newest, p.x);
    if (i + 1 < cnt) newest = max(newest, p.y);
    if (i + 2 < cnt) newest = max(newest, p.z);
    if (i + 3 < cnt) newest = max(newest, p.w);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) x.red[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, x.red[lane % kSelectWarps]);
  if (threadIdx.x == 0) x.newest = newest;
  sync_blocks<BLOCKS>();
#pragma unroll
  for (int r = 0; r < blocks; ++r) newest = max(newest, ld_rank(&x.newest, r));
  const int64_t above = static_cast<int64_t>(newest) - recent;

  // slots in a page outside the pool have the lowest key
  const auto key_of = [&](int i) {
    if (cached) return keys[i];
    const int row = cache_row(c, b, h, s0 + i, st, KID_EVICT_SELECT);
    return row < 0 ? 0u : evict_key(c.weight[row], c.pos[row], above);
  };

  // First digit: the highest 11 bits (sign, exponent and two of the mantissa).
  if (cached) {   // (each thread finds the weights that it has put there; the positions come from L1 or L2)
#pragma unroll 4
    for (int i = threadIdx.x * 4; i < cnt; i += kSelectThreads * 4) {
      const int row = cache_row(c, b, h, s0 + i, st, KID_EVICT_SELECT);
      uint4 k = make_uint4(0, 0, 0, 0);
      if (row >= 0) {
        const int4 p = *reinterpret_cast<const int4*>(c.pos + row);
        const float4 w = *reinterpret_cast<const float4*>(keys + i);
        k = make_uint4(evict_key(w.x, p.x, above), evict_key(w.y, p.y, above), evict_key(w.z, p.z, above),
                       evict_key(w.w, p.w, above));
      }
      *reinterpret_cast<uint4*>(keys + i) = k;
      atomicAdd(&x.hist[0][k.x >> 21], 1);
      if (i + 1 < cnt) atomicAdd(&x.hist[0][k.y >> 21], 1);
      if (i + 2 < cnt) atomicAdd(&x.hist[0][k.z >> 21], 1);
      if (i + 3 < cnt) atomicAdd(&x.hist[0][k.w >> 21], 1);
    }
  } else {
    for (int i = threadIdx.x; i < cnt; i += kSelectThreads) atomicAdd(&x.hist[0][key_of(i) >> 21], 1);
  }
  sync_blocks<BLOCKS>();
  int need = budget;
  if constexpr (blocks == 1) {
    find_digit(reversed(*reinterpret_cast<const int4*>(&x.hist[0][kBins - 4 - 4 * threadIdx.x])), kBins - 1, need, x);
  } else {
    // Each block adds up its part of the bins; all then read the sums of the
    // parts, and of the part that the digit lies in its bins.  (Every block
    // reading every bin of every block took 3 us a digit.)
    constexpr int PART = kBins / blocks;
    int4 v = make_int4(0, 0, 0, 0);
    if (4 * threadIdx.x < PART) {
      int4 q[blocks];
#pragma unroll
      for (int r = 0; r < blocks; ++r) q[r] = ld_rank4(&x.hist[0][rank * PART + 4 * threadIdx.x], r);
#pragma unroll
      for (int r = 0; r < blocks; ++r) {
        v.x += q[r].x;
        v.y += q[r].y;
        v.z += q[r].z;
        v.w += q[r].w;
      }
      *reinterpret_cast<int4*>(&x.hist[1][4 * threadIdx.x]) = v;
    }
    int total;
    block_prefix(v.x + v.y + v.z + v.w, x.red, &total);
    if (threadIdx.x == 0) x.slice = total;
    sync_blocks<BLOCKS>();
    int sums[blocks], part = blocks - 1;
#pragma unroll
    for (int r = 0; r < blocks; ++r) sums[r] = ld_rank(&x.slice, r);
#pragma unroll
    for (int r = blocks - 1; r > 0; --r)
      if (part == r && sums[r] < need) {
        need -= sums[r];
        part = r - 1;
      }
    v = make_int4(0, 0, 0, 0);
    if (4 * threadIdx.x < PART) v = reversed(ld_rank4(&x.hist[1][PART - 4 - 4 * threadIdx.x], part));
    find_digit(v, part * PART + PART - 1, need, x);
  }
  uint32_t prefix = x.digit;
  need = x.need;

  // The keys with that digit, gathered from the whole cluster, are few unless
  // weights repeat: then every block finds the other digits by itself.
  uint32_t* listed = keys + key_slots;   // [kListed] of this block, then [kGathered] of all
  uint32_t* gathered = listed + kListed;
  // (One place in the list per warp: a shared counter asked for every 32 keys
  // would be waited for every time.)
  const auto each_mine = [&](const auto& f) {
    if (cached) {
#pragma unroll 4
      for (int i = threadIdx.x * 4; i < cnt; i += kSelectThreads * 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        if (k.x >> 21 == prefix) f(k.x);
        if (i + 1 < cnt && k.y >> 21 == prefix) f(k.y);
        if (i + 2 < cnt && k.z >> 21 == prefix) f(k.z);
        if (i + 3 < cnt && k.w >> 21 == prefix) f(k.w);
      }
    } else {
      for (int i = threadIdx.x; i < cnt; i += kSelectThreads) {
        const uint32_t k = key_of(i);
        if (k >> 21 == prefix) f(k);
      }
    }
  };
  int own = 0;
  each_mine([&](uint32_t) { ++own; });
  int at = own;   // inclusive prefix over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += u;
  }
  int base = 0;
  if (lane == 31) base = atomicAdd(&x.listed, at);
  at += __shfl_sync(0xffffffffu, base, 31) - own;
  each_mine([&](uint32_t key) {
    if (at < kListed) listed[at] = key;
    ++at;
  });
  sync_blocks<BLOCKS>();   // (also: the part sums in hist[1] have been read)
  int counts[blocks], all = 0;
  bool few = true;
#pragma unroll
  for (int r = 0; r < blocks; ++r) {
    counts[r] = ld_rank(&x.listed, r);
    few = few && counts[r] <= kListed;
    all += counts[r];
  }
  few = few && all <= kGathered;
  if (blocks > 1)   // clear what the part sums have used
    for (int i = threadIdx.x; i < kBins; i += kSelectThreads) x.hist[1][i] = 0;
  if (few) {
#pragma unroll 4
    for (int i = threadIdx.x; i < all; i += kSelectThreads) {
      int r = 0, at = i;   // the block that has listed it, and where
#pragma unroll
      for (int k = 0; k < blocks; ++k)
        if (r == k && k + 1 < blocks && at >= counts[k]) {
          at -= counts[k];
          r = k + 1;
        }
      gathered[i] = ld_rank(reinterpret_cast<const int*>(listed + at), r);
    }
  } else if (blocks > 1) {
    sync_blocks<BLOCKS>();   // every block's hist[1] is clear
  }
  __syncthreads();
  for (int pass = 1; pass < 3; ++pass) {
    const auto count = [&](uint32_t key) {
      if (pass == 1 ? key >> 21 == prefix : key >> 10 == prefix)
        atomicAdd(&x.hist[pass][pass == 1 ? (key >> 10) & 2047 : key & 1023], 1);
    };
    int4 v = make_int4(0, 0, 0, 0);
    const int first = kBins - 4 - 4 * threadIdx.x;
    if (few) {
      for (int i = threadIdx.x; i < all; i += kSelectThreads) count(gathered[i]);
      __syncthreads();
      v = *reinterpret_cast<const int4*>(&x.hist[pass][first]);
    } else {
      for (int i = threadIdx.x; i < cnt; i += kSelectThreads) count(key_of(i));
      sync_blocks<BLOCKS>();
#pragma unroll
      for (int r = 0; r < blocks; ++r) {
        const int4 q = ld_rank4(&x.hist[pass][first], r);
        v.x += q.x;
        v.y += q.y;
        v.z += q.z;
        v.w += q.w;
      }
    }
    find_digit(reversed(v), kBins - 1, need, x);
    prefix = pass == 1 ? prefix << 11 | x.digit : prefix << 10 | x.digit;
    need = x.need;
    __syncthreads();   // x.digit is read
  }
  // kept: keys above `prefix`, and the first `need` slots whose key equals it

  // Ties matter only where not all of them are kept.
  const bool all_ties = x.ties == need;
  if (all_ties) --prefix;   // then: keys above `prefix` (a kept key is not 0: `need` of a 0 are all only if n = budget)

  // The warp's slots with a larger and with an equal key, below and above the
  // budget, and those of the slots before: in lower blocks, in lower warps.
  const int wseg = seg / kSelectWarps, i0 = min(cnt, warp * wseg), i1 = min(cnt, i0 + wseg);
  int a_lo = 0, a_hi = 0, t_lo = 0, t_hi = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t key = key_of(i);
    const bool lo = s0 + i < budget;
    if (key > prefix) {
      a_lo += lo;
      a_hi += !lo;
    }
    if (!all_ties && key == prefix) {
      t_lo += lo;
      t_hi += !lo;
    }
  }
  a_lo = __reduce_add_sync(0xffffffffu, a_lo);
  a_hi = __reduce_add_sync(0xffffffffu, a_hi);
  t_lo = __reduce_add_sync(0xffffffffu, t_lo);
  t_hi = __reduce_add_sync(0xffffffffu, t_hi);
  if (lane == 0) x.warps[warp] = make_int4(a_lo, a_hi, t_lo, t_hi);
  __syncthreads();
  const int4 wv = lane < kSelectWarps ? x.warps[lane] : make_int4(0, 0, 0, 0);
  if (warp == 0) {
    const int ta = __reduce_add_sync(0xffffffffu, wv.x), tb = __reduce_add_sync(0xffffffffu, wv.y);
    const int tc = __reduce_add_sync(0xffffffffu, wv.z), td = __reduce_add_sync(0xffffffffu, wv.w);
    if (lane == 0) *reinterpret_cast<int4*>(&x.above_lo) = make_int4(ta, tb, tc, td);
  }
  a_lo = __reduce_add_sync(0xffffffffu, lane < warp ? wv.x : 0);
  a_hi = __reduce_add_sync(0xffffffffu, lane < warp ? wv.y : 0);
  t_lo = __reduce_add_sync(0xffffffffu, lane < warp ? wv.z : 0);
  t_hi = __reduce_add_sync(0xffffffffu, lane < warp ? wv.w : 0);
  sync_blocks<BLOCKS>();
  int all_t_lo = 0, all_a_lo = 0;
  int4 others[blocks];
#pragma unroll
  for (int r = 0; r < blocks; ++r) others[r] = ld_rank4(&x.above_lo, r);
#pragma unroll
  for (int r = 0; r < blocks; ++r) {
    all_a_lo += others[r].x;
    all_t_lo += others[r].z;
    if (r < rank) {
      a_lo += others[r].x;
      a_hi += others[r].y;
      t_lo += others[r].z;
      t_hi += others[r].w;
    }
  }
  if (blocks > 1) cluster_arrive();   // this block reads no other's shared memory any more
  allow_dependents();
  if (all_ties) need = 0;
  const int kept_lo = all_a_lo + min(need, all_t_lo);   // of all slots below the budget
  int* freed_at = pairs.freed + piece * budget;
  int* moving_at = pairs.moving + piece * budget;
  int ties = t_lo + t_hi, kept = a_lo + a_hi + min(need, ties);   // before the warp's next slot
  const unsigned int before = (1u << lane) - 1u;
#pragma unroll 2
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const bool in = i < i1;
    const int slot = s0 + i;
    const uint32_t key = in ? key_of(i) : 0u;
    bool keep = in && key > prefix;
    if (!all_ties) {
      const unsigned int t = __ballot_sync(0xffffffffu, in && key == prefix);
      keep = keep || (in && key == prefix && ties + __popc(t & before) < need);
      ties += __popc(t);
    }
    const unsigned int k = __ballot_sync(0xffffffffu, keep);
    const int rank_kept = kept + __popc(k & before);   // kept slots before this one
    if (in && slot < budget) {
      if (keep)
        slots[slot] = slot;
      else
        freed_at[slot - rank_kept] = slot;
    } else if (keep) {
      moving_at[rank_kept - kept_lo] = slot;
    }
    kept += __popc(k);
  }
  if (rank == 0 && threadIdx.x == 0) pairs.count[piece] = budget - kept_lo;
  if (blocks > 1) cluster_wait();   // no block leaves while another reads its shared memory
}

template <int BLOCKS>
__global__ void __launch_bounds__(kSelectThreads, 2)
    evict_select_kernel(CacheArgs c, int budget, int recent, int key_slots, int32_t* __restrict__ slots, EvictPairs pairs,
                        DevStatus st) {
  extern __shared__ __align__(16) uint32_t keys[];   // [key_slots], then the lists
  __shared__ SelectShared x;
  const int rank = BLOCKS > 1 ? cluster_rank() : 0;
  const int h = blockIdx.x / BLOCKS, b = blockIdx.y;
  wait_for_previous();
  const int n = checked_length(c, b, st, KID_EVICT_SELECT);
  const int64_t piece = static_cast<int64_t>(b) * c.H + h;
  slots += piece * budget;
  if (n <= budget) {   // (the same for the whole cluster)
    for (int j = rank * kSelectThreads + threadIdx.x; j < budget; j += BLOCKS * kSelectThreads) slots[j] = j < n ? j : -1;
    if (rank == 0 && threadIdx.x == 0) pairs.count[piece] = 0;
    return;
  }
  if constexpr (BLOCKS > 1)
    if (n <= min(kSelectAlone, key_slots)) {
      if (rank == 0) select_slots<1>(c, b, h, n, budget, recent, 0, keys, key_slots, x, slots, pairs, st);
      return;   // nobody reads these blocks' shared memory
    }
  select_slots<BLOCKS>(c, b, h, n, budget, recent, rank, keys, key_slots, x, slots, pairs, st);
}

// ---------------------------------------------------------------------------
// Eviction: the moves, and the lengths.  Reads and writes the rows that move,
// 16 bytes a lane: a warp takes 32 pairs and copies one row (E4M3: two) a step,
// the next four steps' loads on their way before the last four are stored.
// Sources lie at or above the budget and destinations below it, so no copy
// disturbs another.  Blocks of one warp, since they end one by one (eviction of
// 24 x 8192 slots: 74 us, 87 with two warps, 103 with eight).
// ---------------------------------------------------------------------------
template <bool FP8>
__global__ void __launch_bounds__(32)
    evict_move_kernel(CacheArgs c, int budget, int32_t* __restrict__ slots, EvictPairs pairs, int32_t* lengths_out,
                      DevStatus st) {
  constexpr int ES = FP8 ? 1 : 2, VC = kDv * ES / 16, ROWS = FP8 ? 2 : 1, STEPS = 4, BATCH = STEPS * ROWS;
  const int kc = c.d * ES / 16;
  const int lane = threadIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t piece = static_cast<int64_t>(b) * c.H + h;
  wait_for_previous();
  if (blockIdx.x == 0 && h == 0 && lane == 0) {   // (in place: the selection has read it)
    const int n = c.lengths[b], cap = c.capacity();
    lengths_out[b] = min(budget, max(0, min(n, cap)));
  }
  const int part = FP8 ? lane >> 4 : 0, l = FP8 ? lane & 15 : lane;   // which of a step's rows, and the lane in it
  const bool is_k = l < kc;
  const uint4* from = reinterpret_cast<const uint4*>(is_k ? c.k : c.v);
  uint4* to = reinterpret_cast<uint4*>(is_k ? c.k : c.v);
  const int chunks = is_k ? kc : VC, ch = is_k ? l : l - kc;
  const int count = __ldcg(pairs.count + piece);
  for (int j0 = blockIdx.x * 32; j0 < count; j0 += gridDim.x * 32) {
    const int n = min(32, count - j0);
    int src = -1, dst = -1, to_slot = 0, from_slot = 0;
    float w = 0.f, ks = 0.f, vs = 0.f;
    int p = 0;
    if (lane < n) {
      to_slot = __ldcg(pairs.freed + piece * budget + j0 + lane);
      from_slot = __ldcg(pairs.moving + piece * budget + j0 + lane);
      src = cache_row(c, b, h, from_slot, st, KID_EVICT_MOVE);
      dst = cache_row(c, b, h, to_slot, st, KID_EVICT_MOVE);
      if (src < 0) dst = -1;
      if (dst >= 0) {
        w = c.weight[src];
        p = c.pos[src];
        if (FP8) {
          ks = c.k_scale[src];
          vs = c.v_scale[src];
        }
      }
    }
    const auto load = [&](int i0, uint4 (&r)[STEPS], int (&d)[STEPS]) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int pair = i0 + i * ROWS + part;
        const int s = __shfl_sync(0xffffffffu, src, pair & 31);
        d[i] = __shfl_sync(0xffffffffu, dst, pair & 31);
        if (l >= kc + VC || pair >= n) d[i] = -1;
        if (d[i] >= 0) r[i] = __ldcg(from + static_cast<int64_t>(s) * chunks + ch);
      }
    };
    const auto store = [&](const uint4 (&r)[STEPS], const int (&d)[STEPS]) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        if (d[i] >= 0) to[static_cast<int64_t>(d[i]) * chunks + ch] = r[i];
    };
    uint4 r0[STEPS], r1[STEPS];
    int d0[STEPS], d1[STEPS];
    load(0, r0, d0);
    for (int i0 = 0; i0 < n; i0 += 2 * BATCH) {
      load(i0 + BATCH, r1, d1);
      store(r0, d0);
      load(i0 + 2 * BATCH, r0, d0);
      store(r1, d1);
    }
    if (lane < n) slots[piece * budget + to_slot] = from_slot;
    if (dst >= 0) {
      c.weight[dst] = w;
      c.pos[dst] = p;
      if (FP8) {
        c.k_scale[dst] = ks;
        c.v_scale[dst] = vs;
      }
    }
  }
}

template <int BLOCKS>
cudaError_t launch_evict_select_n(const CacheArgs& c, int budget, int recent, int key_slots, int32_t* slots,
                                  const EvictPairs& pairs, DevStatus st, cudaStream_t s) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(evict_select_kernel<BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kSelectKeys + kListed + kGathered) * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(c.H * BLOCKS, c.B);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(key_slots + kListed + kGathered) * 4;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = BLOCKS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<BLOCKS>, c, budget, recent, key_slots, slots, pairs, st);
}

// Blocks per (head, sequence): more while a block would still have over 2048
// slots (four a thread) and the GPU holds them all at once, two to an SM, or
// while the keys do not fit into shared memory.
cudaError_t launch_evict_select(const CacheArgs& c, int budget, int recent, int sms, int32_t* slots,
                                const EvictPairs& pairs, DevStatus st, cudaStream_t s) {
  const int64_t pieces = static_cast<int64_t>(c.B) * c.H;
  const auto per_block = [&](int n) {
    return ((c.capacity() + n - 1) / n + kSelectThreads - 1) / kSelectThreads * kSelectThreads;
  };
  int blocks = 1;
  while (blocks < kMaxCluster && ((per_block(blocks) > kSelectAlone && 2 * blocks * pieces <= 2 * sms) ||
                                  per_block(blocks) > kSelectKeys))
    blocks *= 2;
  const int key_slots = std::min(per_block(blocks), kSelectKeys);
  switch (blocks) {
    case 1: return launch_evict_select_n<1>(c, budget, recent, key_slots, slots, pairs, st, s);
    case 2: return launch_evict_select_n<2>(c, budget, recent, key_slots, slots, pairs, st, s);
    case 4: return launch_evict_select_n<4>(c, budget, recent, key_slots, slots, pairs, st, s);
    default: return launch_evict_select_n<8>(c, budget, recent, key_slots, slots, pairs, st, s);
  }
}
}  // namespace
}  // namespace qkvp

using namespace qkvp;

extern "C" {

size_t qkvp_cache_append_workspace_bytes(const qkvp_cache* cache) {
  CacheArgs a;
  return check_cache(cache, &a) == QKVP_OK ? kCacheHeaderBytes : 0;
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
  if (ws_bytes < kCacheHeaderBytes) return QKVP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int* arrived = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + kAppendCounter);
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
  return kCacheHeaderBytes + static_cast<size_t>(a.B) * a.H * (2 * static_cast<size_t>(budget) + 1) * sizeof(int32_t);
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
  const int sms = device_sms();
  if (sms <= 0) return QKVP_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const DevStatus st{static_cast<int*>(ws), 0};
  EvictPairs pairs;
  pairs.count = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kCacheHeaderBytes);
  pairs.freed = pairs.count + static_cast<int64_t>(a.B) * a.H;
  pairs.moving = pairs.freed + static_cast<int64_t>(a.B) * a.H * budget;
  mark(s);
  if (launch_evict_select(a, budget, recent, sms, slots, pairs, st, s) != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  // Blocks for as many pairs as there may be, up to three times the 32 that an
  // SM holds: there may be far fewer pairs, and blocks without any cost too
  // (256 x 8 heads of 300 slots, a budget of 16384: 31 us for the call, 549 with
  // blocks for them all).
  const int64_t pieces = static_cast<int64_t>(a.B) * a.H, full = (96 * sms + pieces - 1) / pieces;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((budget + 31) / 32, full)), a.H, a.B);
  if (launch_dependent(cache->fp8 ? evict_move_kernel<true> : evict_move_kernel<false>, grid, 32, 0, s, a, budget, slots,
                       pairs, lengths_out, st) != cudaSuccess)
    return QKVP_ERR_CUDA;
  mark(s);
  return QKVP_OK;
}

}  // extern "C"
