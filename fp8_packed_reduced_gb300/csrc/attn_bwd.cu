// Gradient of the causal attention over packed sequences on the 5th-generation
// tensor cores (attn.cuh has the formulas), in two passes that both form the
// scores and da . v again: one over the keys of 128 queries for dq, one over the
// queries of 128 keys for dk and dv.  A single pass would have to add dq up in
// memory, in an order that changes from run to run.
#include <atomic>

#include "attn.cuh"

namespace qkvp {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 352;                // eight computing warps, a loading and two issuing ones
constexpr int kBox = kTile * 128;            // bytes of 128 rows x 64 bf16
using VTile = AttnTile<kDv, kTile>;                 // of v and da
// Rings of tiles: in dq of k and v, in dk and dv of q and da.  As many stages as
// fit; in dk and dv a tile of q is back in use sooner than one of da.
__host__ __device__ constexpr int dq_stages(int d) { return d == 128 ? 3 : 4; }
__host__ __device__ constexpr int q_stages(int d) { return d == 128 ? 2 : 4; }
__host__ __device__ constexpr int da_stages(int d) { return d == 64 ? 3 : 2; }
template <int D>
constexpr int dq_smem() {
  return 1024 + dq_stages(D) * (AttnTile<D, kTile>::kBytes + VTile::kBytes);
}
template <int D>
constexpr int dkv_smem() {
  return 1024 + (1 + q_stages(D)) * AttnTile<D, kTile>::kBytes + (1 + da_stages(D)) * VTile::kBytes;
}
// Columns of TMEM
constexpr int kScores = 0, kDp = 128, kAcc0 = 256, kAcc1 = 384, kOpQ = 384, kOpDa = 448;

constexpr int kMaxStages = 4;
struct Shared {
  uint64_t fixed_full, a_full[kMaxStages], a_empty[kMaxStages], b_full[kMaxStages], b_empty[kMaxStages];
  uint64_t s_full, dp_full, s_free, p_full[2], ds_full[2], acc_full;   // (p and ds in two parts)
  uint32_t tmem;
  int abort;
  int lo[4], hi[4], start[4];
  uint32_t again[4];            // rows to be computed again
  Range range;
};

// b_users: issuing warps that release a stage of b.
__device__ __forceinline__ void init_barriers(Shared& g, int b_users) {
  g.abort = 0;
  mbar_init(&g.fixed_full, 1);
  for (int s = 0; s < kMaxStages; ++s) {
    mbar_init(&g.a_full[s], 1);
    mbar_init(&g.a_empty[s], 1);
    mbar_init(&g.b_full[s], 1);
    mbar_init(&g.b_empty[s], b_users);
  }
  mbar_init(&g.s_full, 1);
  mbar_init(&g.dp_full, 1);
  mbar_init(&g.s_free, 8);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&g.p_full[i], 8);
    mbar_init(&g.ds_full[i], 8);
  }
  mbar_init(&g.acc_full, 2);
  fence_mbar_init();
}
// Two pairs of floats of shared memory.
__device__ __forceinline__ void lds_f2x2(uint32_t at, f2 (&z)[2]) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(z[0]), "=l"(z[1]) : "r"(at));
}
// 8 warps of a group have done something to TMEM: arrive once per warp.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// delta = da . a of every row and head, and beside it the row's lse in base 2
// (+inf where the row has no weight at all, so that its probabilities are 0), both
// negative.  A half warp a row, 16 rows a warp.  Its first blocks put the tiles of the two
// passes in order.
constexpr int kPrepThreads = 256, kPrepRows = kPrepThreads / 32 * 16;
static_assert(kPrepRows == kTile, "the statistics cover whole tiles");
__global__ void __launch_bounds__(kPrepThreads) delta_kernel(const __grid_constant__ AttnArgs p, int tiles, DevStatus st) {
  wait_for_previous();
  if (blockIdx.x == 0) check_offsets(p, st, KID_ATTN_DELTA);
  const int sorts = p.order[0] ? 2 : 0;
  if (static_cast<int>(blockIdx.x) < sorts) {
    sort_tiles<kPrepThreads>(p, tiles, kTile, blockIdx.x == 1, p.order[blockIdx.x]);
    return;
  }
  const int block = blockIdx.x - sorts, hq = block / tiles;
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  const int r0 = (block - hq * tiles) * kTile + (threadIdx.x >> 5) * 16;
  float mine = 0.f;   // lane c < 8 of a half keeps row r0 + 2 c + half
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + 2 * i + half;
    float s = 0.f;
    if (row < p.T) {
      const int64_t at = (static_cast<int64_t>(row) * p.Hq + hq) * kDv;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.da + at) + c), y = __ldg(reinterpret_cast<const uint4*>(p.a + at) + c);
      s = bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x) + bf16_lo(x.y) * bf16_lo(y.y) + bf16_hi(x.y) * bf16_hi(y.y) +
          bf16_lo(x.z) * bf16_lo(y.z) + bf16_hi(x.z) * bf16_hi(y.z) + bf16_lo(x.w) * bf16_lo(y.w) + bf16_hi(x.w) * bf16_hi(y.w);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == i) mine = s;
  }
  const int row = r0 + 2 * c + half;
  if (c < 8) {
    const float z = row < p.T ? __ldg(p.lse + static_cast<int64_t>(hq) * p.T + row) : -INFINITY;
    float* to = p.stat + static_cast<int64_t>(hq) * 2 * p.Tp + row;
    to[0] = z == -INFINITY ? -INFINITY : z * -1.4426950408889634f;
    to[p.Tp] = -mine;
  }
}

// ---------------------------------------------------------------------------
// dq: 128 queries of a head.  q and da are operands in TMEM for the whole of
// it, dq adds up there; per tile of 128 keys
//   S = q k^T, dP = da v^T, ds = e^(S - lse) (dP - delta), dq += ds k
// The products are issued dP(j), S(j + 1), dq(j): S(j + 1) covers the forming of ds(j).
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ AttnArgs p, DevStatus st) {
  using KTile = AttnTile<D, kTile>;
  constexpr int kKBytes = KTile::kBytes, kVBytes = VTile::kBytes, kStages = dq_stages(D), KB = (D + 63) / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared g;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = sk + kStages * kKBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) init_barriers(g, 1);
  if (threadIdx.x < 4) g.again[threadIdx.x] = 0;
  if (warp == 9) {
    tmem_alloc(&g.tmem, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  const Place at = place_of(p.order[0], p.Hq);
  const int hq = at.head, h = hq / p.G, r0 = at.tile * kTile;
  const int half = warp >> 2, row = r0 + (threadIdx.x & 127);
  Span sp{-1, -1};
  int seen0 = 0;
  if (warp < 8) {
    if (row < p.T) sp = span_of(p, row);
    if (sp.start >= 0 && alone(p, row, sp.start)) sp.start = -1;   // it passes nothing on
    seen0 = sp.start < 0 ? INT_MAX : window_start(p, row, sp.start);
    const int lo = __reduce_min_sync(0xffffffffu, seen0), hi = __reduce_max_sync(0xffffffffu, sp.start < 0 ? -1 : row);
    const int s0 = __reduce_min_sync(0xffffffffu, sp.start < 0 ? INT_MAX : sp.start);
    if (lane == 0 && half == 0) g.lo[warp] = lo, g.hi[warp] = hi, g.start[warp] = s0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) g.range = range_of<kTile>(p, g.lo, g.hi, g.start);
  const uint32_t tmem = g.tmem, quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
  if (warp < 8) {   // one half of the warps loads q, the other da
    const uint4* from = reinterpret_cast<const uint4*>(half == 0 ? p.q + (static_cast<int64_t>(hq) * p.T + row) * D
                                                                 : p.da + (static_cast<int64_t>(row) * p.Hq + hq) * kDv);
    const uint32_t to = tmem + (half == 0 ? kOpQ : kOpDa) + quarter;
    const int parts = half == 0 ? D / 32 : kDv / 32;
    for (int c = 0; c < parts; ++c) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = row < p.T ? __ldg(from + 4 * c + i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
      tmem_st16(to + 16 * c, w);
    }
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Range r = g.range;
  const int kt0 = r.sink0 < r.sink1 ? r.sink0 : r.first;
  const auto next_of = [&](int kt) { return kt + 1 == r.sink1 ? r.first : kt + 1; };

  if (warp == 8) {
    if (lane == 0) {
      int n = 0;
      for (int kt = kt0; kt < r.last; kt = next_of(kt), ++n) {
        const int s = n % kStages, par = (n / kStages) & 1;
        if (!mbar_wait(&g.a_empty[s], par ^ 1, &g.abort, st, KID_ATTN_DQ)) break;
        mbar_arrive_expect_tx(&g.a_full[s], kKBytes);
        KTile::load(sk + s * kKBytes, &tm_k, &g.a_full[s], kt * kTile, h);
        if (!mbar_wait(&g.b_empty[s], par ^ 1, &g.abort, st, KID_ATTN_DQ)) {
          mbar_wait(&g.a_full[s], par, nullptr, st, KID_ATTN_DQ);
          break;
        }
        mbar_arrive_expect_tx(&g.b_full[s], kVBytes);
        VTile::load(sv + s * kVBytes, &tm_v, &g.b_full[s], kt * kTile, h);
      }
      for (int i = max(0, n - kStages); i < n; ++i) {   // every copy has landed before the block may leave
        mbar_wait(&g.a_full[i % kStages], (i / kStages) & 1, nullptr, st, KID_ATTN_DQ);
        mbar_wait(&g.b_full[i % kStages], (i / kStages) & 1, nullptr, st, KID_ATTN_DQ);
      }
    }
  } else if (warp >= 9) {
    // One warp issues the scores, the other the rest: while one finds out what
    // is ready, the products of the other run.  A whole warp goes the same way
    // (umma_bf16_ss says why).
    constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile, false), id_q = idesc_bf16_f32(kTile, D, true);
    const uint32_t elected = elect_one();
    const auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, &g.abort, st, KID_ATTN_DQ));
    };
    int n = 0;
    if (warp == 9) {
      const uint64_t k0 = KTile::desc(sk);
      for (int kt = kt0; kt < r.last; kt = next_of(kt), ++n) {
        const int s = n % kStages;
        if (!wait(&g.a_full[s], (n / kStages) & 1) || (n > 0 && !wait(&g.s_free, (n - 1) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16_ts(tmem + kScores, tmem + kOpQ + kk * 8, k0 + ((s * kKBytes) >> 4) + KTile::cols16(kk), id_s, kk > 0, elected);
        umma_commit_elected(&g.s_full, elected);
      }
    } else {
      const uint64_t v0 = VTile::desc(sv), k0 = KTile::desc(sk);
      const auto dps = [&](int s) {
#pragma unroll
        for (int kk = 0; kk < kDv / 16; ++kk)
          umma_bf16_ts(tmem + kDp, tmem + kOpDa + kk * 8, v0 + ((s * kVBytes) >> 4) + VTile::cols16(kk), id_s, kk > 0, elected);
        umma_commit_elected(&g.dp_full, elected);
        umma_commit_elected(&g.b_empty[s], elected);
      };
      bool ok = kt0 < r.last && wait(&g.b_full[0], 0);
      if (ok) {
        tc_fence_after();
        dps(0);
      }
      for (int kt = kt0; ok && kt < r.last; ++n) {
        const int s = n % kStages, s1 = (n + 1) % kStages, next = next_of(kt);
        ok = wait(&g.a_full[s], (n / kStages) & 1) && (next >= r.last || wait(&g.b_full[s1], ((n + 1) / kStages) & 1)) &&
             wait(&g.ds_full[0], n & 1);
        if (!ok) break;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1) ok = wait(&g.ds_full[1], n & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 32 keys of each half
            const int kk = (i >> 1) * 4 + 2 * part + (i & 1);
            umma_bf16_ts(tmem + kAcc0, tmem + kDp + (kk / 4) * 64 + (kk % 4) * 8, k0 + ((s * kKBytes) >> 4) + KTile::rows16(kk), id_q,
                         n > 0 || part > 0 || i > 0, elected);
          }
        }
        if (!ok) break;
        umma_commit_elected(&g.a_empty[s], elected);
        if (next < r.last) dps(s1);
        kt = next;
      }
    }
    umma_commit_elected(&g.acc_full, elected);
    mbar_wait(&g.acc_full, 0, nullptr, st, KID_ATTN_DQ);   // all products are done
  } else {
    // this thread's row, and the half of the keys that its warpgroup takes
    const uint32_t ts = tmem + kScores + 64 * half + quarter, td = tmem + kDp + 64 * half + quarter;
    const float* stat = p.stat + static_cast<int64_t>(hq) * 2 * p.Tp + row;   // (row < Tp)
    const float z0 = __ldcg(stat), delta = __ldcg(stat + p.Tp);
    const int sink_end = sp.start < 0 ? 0 : sp.start + min(p.sinks, p.T);
    const f2 sc = f2_make(p.scale_log2, p.scale_log2), mz = f2_make(z0, z0), md = f2_make(delta, delta);
    bool ok = true;
    int n = 0;
    for (int kt = kt0; kt < r.last; kt = next_of(kt), ++n) {
      ok = mbar_wait(&g.s_full, n & 1, &g.abort, st, KID_ATTN_DQ);
      if (!ok) break;
      tc_fence_after();
      uint32_t x[64];
      tmem_ld32(ts, x);
      tmem_ld32(ts + 32, x + 32);
      tmem_ld_wait();
      arrive_warp(&g.s_free);
      f2 w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 z = f2_split(f2_fma(f2_make(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc, mz));
        w[i] = f2_make(ex2(z.x), ex2(z.y));
      }
      const int j0 = kt * kTile + 64 * half;
      const bool whole = __all_sync(0xffffffffu, sp.start >= 0 && j0 >= seen0 && j0 + 64 <= row + 1);
      ok = mbar_wait(&g.dp_full, n & 1, &g.abort, st, KID_ATTN_DQ);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_ld32(td + 32 * c, x);
        tmem_ld_wait();
        uint32_t out[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          out[i] = f2_to_bf16x2(f2_mul(f2_add(f2_make(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), md), w[16 * c + i]));
        if (!whole) {
          uint32_t see = 0;
          if (sp.start >= 0) see = bits(seen0, row + 1, j0 + 32 * c) | bits(sp.start, min(sink_end, row + 1), j0 + 32 * c);
#pragma unroll
          for (int i = 0; i < 16; ++i) out[i] &= (see >> (2 * i) & 1 ? 0xFFFFu : 0u) | (see >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
        }
        tmem_st16(td + 16 * c, out);   // over what this warp has read
        tmem_st_wait();
        arrive_warp(&g.ds_full[c]);
      }
    }
    if (ok) ok = mbar_wait(&g.acc_full, 0, &g.abort, st, KID_ATTN_DQ);
    if (ok) {
      tc_fence_after();
      // each warpgroup writes one box of 64 columns (with d = 64 the first alone)
      bool bad = false;
      const bool some = kt0 < r.last;
      uint8_t* stage = smem + half * kBox + (warp & 3) * 4096;
      if (half < KB) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld32(tmem + kAcc0 + quarter + 64 * half + 32 * c, o);
          tmem_ld_wait();
          const bool in = 64 * half + 32 * c < D;
          float big = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = __uint_as_float(o[i + 2 * k]) * p.scale, b = __uint_as_float(o[i + 2 * k + 1]) * p.scale;
              big += fabsf(a) + fabsf(b);
              w[k] = some ? pack_bf16x2(a, b) : 0u;
            }
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + i / 8) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          bad |= in && !(big < INFINITY);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && row < p.T) {
          tma_store_3d(&tm_dq, stage, 64 * half, row, hq);
          bulk_commit();
          bulk_wait_all<0>();
        }
      }
      __syncwarp();
      const uint32_t again = __ballot_sync(0xffffffffu, bad && some && row < p.T);
      if (lane == 0 && again) atomicOr(&g.again[warp & 3], again);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  // Rows that are not finite may owe that to what they do not see (0 * NaN):
  // they are computed again from what they see.
  if (warp < 4)
    for (uint32_t again = g.again[warp]; again; again &= again - 1) dq_row<D>(p, r0 + warp * 32 + __ffs(again) - 1, hq);
}

// ---------------------------------------------------------------------------
// dk and dv: 128 keys of a head, and the query tiles that see them, of all
// query heads in turn, the keys along the rows:
//   S^T = k q^T, P^T = e^(S^T - lse), dv += P^T da
//   dP^T = v da^T, ds^T = P^T (dP^T - delta), dk += ds^T q
// issued dv(i), S(i + 1), dk(i), dP(i + 1): each step's forming of P^T and ds^T is
// covered by two products.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_da,
               const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
               const __grid_constant__ AttnArgs p, DevStatus st) {
  using KTile = AttnTile<D, kTile>;
  constexpr int kKBytes = KTile::kBytes, kVBytes = VTile::kBytes, SQ = q_stages(D), SD = da_stages(D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared g;
  __shared__ alignas(128) float stats[SQ][2][kTile];   // -lse (base 2) and -delta of a tile of queries
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sk = smem, *sv = sk + kKBytes, *sq = sv + kVBytes, *sd = sq + SQ * kKBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) init_barriers(g, 2);
  if (threadIdx.x < 4) g.again[threadIdx.x] = 0;
  if (warp == 9) {
    tmem_alloc(&g.tmem, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  const Place at = place_of(p.order[1], p.H);
  const int h = at.head, r0 = at.tile * kTile;
  // queries [row, end) see this thread's key; those from ds0 on pass something on
  const int half = warp >> 2, row = r0 + (threadIdx.x & 127);
  int begin = row, end = row, ds0 = row;
  if (warp < 8) {
    const Span sp = row < p.T ? span_of(p, row) : Span{-1, -1};
    if (sp.start >= 0) {
      end = last_seer(p, row, sp);
      ds0 = row + (alone(p, row, sp.start) ? 1 : 0);
    }
    const int hi = __reduce_max_sync(0xffffffffu, end > row ? end : -1), lo = __reduce_min_sync(0xffffffffu, end > row ? row : INT_MAX);
    if (lane == 0 && half == 0) g.hi[warp] = hi, g.lo[warp] = lo;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = g.tmem, quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int hi = max(max(g.hi[0], g.hi[1]), max(g.hi[2], g.hi[3]));
  const int tiles = hi < 0 ? 0 : (hi + kTile - 1) / kTile - at.tile;   // query tiles of a head, from this one on
  const int count = tiles * p.G;

  if (warp == 8) {
    if (lane == 0 && count > 0) {
      mbar_arrive_expect_tx(&g.fixed_full, kKBytes + kVBytes);
      KTile::load(sk, &tm_k, &g.fixed_full, r0, h);
      VTile::load(sv, &tm_v, &g.fixed_full, r0, h);
      int na = 0, nb = 0;
      for (; nb < count; ++nb) {
        // da of this step behind q of it and of as many as there is room for
        const int s = nb % SD, hq = h * p.G + nb / tiles, i0 = r0 + (nb % tiles) * kTile;
        bool ok = true;
        for (; na < count && na <= nb + (SQ - SD); ++na) {
          const int sa = na % SQ, ha = h * p.G + na / tiles, ia = r0 + (na % tiles) * kTile;
          ok = mbar_wait(&g.a_empty[sa], (na / SQ & 1) ^ 1, &g.abort, st, KID_ATTN_DKV);
          if (!ok) break;
          mbar_arrive_expect_tx(&g.a_full[sa], kKBytes + sizeof(stats[0]));
          KTile::load(sq + sa * kKBytes, &tm_q, &g.a_full[sa], ia, ha);
          for (int b = 0; b < 2; ++b)
            bulk_load(stats[sa][b], p.stat + (static_cast<int64_t>(ha) * 2 + b) * p.Tp + ia, sizeof(stats[sa][b]), &g.a_full[sa]);
        }
        if (!ok || !mbar_wait(&g.b_empty[s], (nb / SD & 1) ^ 1, &g.abort, st, KID_ATTN_DKV)) break;
        mbar_arrive_expect_tx(&g.b_full[s], kVBytes);
        for (int b = 0; b < 2; ++b) tma_load_2d(sd + s * kVBytes + b * kBox, &tm_da, &g.b_full[s], hq * kDv + b * 64, i0);
      }
      mbar_wait(&g.fixed_full, 0, nullptr, st, KID_ATTN_DKV);
      // every copy has landed before the block may leave
      for (int i = max(0, na - SQ); i < na; ++i) mbar_wait(&g.a_full[i % SQ], (i / SQ) & 1, nullptr, st, KID_ATTN_DKV);
      for (int i = max(0, nb - SD); i < nb; ++i) mbar_wait(&g.b_full[i % SD], (i / SD) & 1, nullptr, st, KID_ATTN_DKV);
    }
  } else if (warp >= 9) {
    // As for dq: one warp issues dv and the scores, the other dk and dP.
    constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile, false), id_k = idesc_bf16_f32(kTile, D, true),
                       id_v = idesc_bf16_f32(kTile, kDv, true);
    const uint32_t elected = elect_one();
    const auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, &g.abort, st, KID_ATTN_DKV));
    };
    bool ok = count > 0 && wait(&g.fixed_full, 0);
    if (warp == 9) {
      const uint64_t k0 = KTile::desc(sk), q0 = KTile::desc(sq), d0 = VTile::desc(sd);
      const auto scores = [&](int s) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16_ss(tmem + kScores, k0 + KTile::cols16(kk), q0 + ((s * kKBytes) >> 4) + KTile::cols16(kk), id_s, kk > 0, elected);
        umma_commit_elected(&g.s_full, elected);
      };
      ok = ok && wait(&g.a_full[0], 0);
      if (ok) {
        tc_fence_after();
        scores(0);
      }
      for (int n = 0; ok && n < count; ++n) {
        const int s = n % SD, s1 = (n + 1) % SQ;
        ok = wait(&g.b_full[s], (n / SD) & 1) && (n + 1 == count || wait(&g.a_full[s1], ((n + 1) / SQ) & 1)) &&
             wait(&g.p_full[0], n & 1);
        if (!ok) break;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1) ok = wait(&g.p_full[1], n & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 32 queries of each half
            const int kk = (i >> 1) * 4 + 2 * part + (i & 1);
            umma_bf16_ts(tmem + kAcc0, tmem + kScores + (kk / 4) * 64 + (kk % 4) * 8, d0 + ((s * kVBytes) >> 4) + VTile::rows16(kk), id_v,
                         n > 0 || part > 0 || i > 0, elected);
          }
        }
        if (!ok) break;
        umma_commit_elected(&g.b_empty[s], elected);
        if (n + 1 < count) scores(s1);
      }
    } else {
      const uint64_t v0 = VTile::desc(sv), d0 = VTile::desc(sd), q0 = KTile::desc(sq);
      const auto dps = [&](int s) {
#pragma unroll
        for (int kk = 0; kk < kDv / 16; ++kk)
          umma_bf16_ss(tmem + kDp, v0 + VTile::cols16(kk), d0 + ((s * kVBytes) >> 4) + VTile::cols16(kk), id_s, kk > 0, elected);
        umma_commit_elected(&g.dp_full, elected);
        umma_commit_elected(&g.b_empty[s], elected);
      };
      ok = ok && wait(&g.b_full[0], 0);
      if (ok) {
        tc_fence_after();
        dps(0);
      }
      for (int n = 0; ok && n < count; ++n) {
        const int s = n % SQ, s1 = (n + 1) % SD;
        ok = wait(&g.a_full[s], (n / SQ) & 1) && (n + 1 == count || wait(&g.b_full[s1], ((n + 1) / SD) & 1)) &&
             wait(&g.ds_full[0], n & 1);
        if (!ok) break;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1) ok = wait(&g.ds_full[1], n & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 32 queries of each half
            const int kk = (i >> 1) * 4 + 2 * part + (i & 1);
            umma_bf16_ts(tmem + kAcc1, tmem + kDp + (kk / 4) * 64 + (kk % 4) * 8, q0 + ((s * kKBytes) >> 4) + KTile::rows16(kk), id_k,
                         n > 0 || part > 0 || i > 0, elected);
          }
        }
        if (!ok) break;
        umma_commit_elected(&g.a_empty[s], elected);
        if (n + 1 < count) dps(s1);
      }
    }
    umma_commit_elected(&g.acc_full, elected);
    mbar_wait(&g.acc_full, 0, nullptr, st, KID_ATTN_DKV);   // all products are done
  } else {
    // this thread's key, and the half of the queries that its warpgroup takes
    const uint32_t ts = tmem + kScores + 64 * half + quarter, td = tmem + kDp + 64 * half + quarter;
    const f2 sc = f2_make(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int n = 0; n < count; ++n) {
      const int s = n % SQ, i0 = r0 + (n % tiles) * kTile + 64 * half;
      ok = mbar_wait(&g.a_full[s], (n / SQ) & 1, &g.abort, st, KID_ATTN_DKV) && mbar_wait(&g.s_full, n & 1, &g.abort, st, KID_ATTN_DKV);
      if (!ok) break;
      tc_fence_after();
      const uint32_t stat = smem_u32(stats[s][0]) + 4 * 64 * half;
      const bool whole = __all_sync(0xffffffffu, i0 >= ds0 && i0 + 64 <= end);
      uint32_t x[64];
      tmem_ld32(ts, x);
      tmem_ld32(ts + 32, x + 32);
      tmem_ld_wait();
      f2 w[32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t out[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          f2 z[2];
          lds_f2x2(stat + 128 * c + 8 * i, z);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = 16 * c + i + k;
            const float2 y = f2_split(f2_fma(f2_make(__uint_as_float(x[2 * at]), __uint_as_float(x[2 * at + 1])), sc, z[k]));
            w[at] = f2_make(ex2(y.x), ex2(y.y));
            out[i + k] = f2_to_bf16x2(w[at]);
          }
        }
        if (!whole) {
          const uint32_t see = bits(begin, end, i0 + 32 * c);
#pragma unroll
          for (int i = 0; i < 16; ++i) out[i] &= (see >> (2 * i) & 1 ? 0xFFFFu : 0u) | (see >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
        }
        tmem_st16(ts + 16 * c, out);   // over what this warp has read
        tmem_st_wait();
        arrive_warp(&g.p_full[c]);
      }
      ok = mbar_wait(&g.dp_full, n & 1, &g.abort, st, KID_ATTN_DKV);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_ld32(td + 32 * c, x);
        tmem_ld_wait();
        uint32_t out[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          f2 z[2];
          lds_f2x2(stat + 4 * kTile + 128 * c + 8 * i, z);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            out[i + k] = f2_to_bf16x2(f2_mul(f2_add(f2_make(__uint_as_float(x[2 * (i + k)]), __uint_as_float(x[2 * (i + k) + 1])), z[k]),
                                             w[16 * c + i + k]));
        }
        if (!whole) {
          const uint32_t see = bits(ds0, end, i0 + 32 * c);
#pragma unroll
          for (int i = 0; i < 16; ++i) out[i] &= (see >> (2 * i) & 1 ? 0xFFFFu : 0u) | (see >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
        }
        tmem_st16(td + 16 * c, out);
        tmem_st_wait();
        arrive_warp(&g.ds_full[c]);
      }
    }
    if (ok) ok = mbar_wait(&g.acc_full, 0, &g.abort, st, KID_ATTN_DKV);
    if (ok) {
      tc_fence_after();
      // one warpgroup writes dv, the other dk
      const int width = half == 0 ? kDv : D, nb = (width + 63) / 64;
      const float f = half == 0 ? 1.f : p.scale;
      uint8_t* stage = (half == 0 ? sv : sq) + (warp & 3) * nb * 4096;
      bool bad = false;
      for (int c = 0; c < 2 * nb; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + (half == 0 ? kAcc0 : kAcc1) + quarter + 32 * c, o);
        tmem_ld_wait();
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = __uint_as_float(o[i + 2 * k]) * f, b = __uint_as_float(o[i + 2 * k + 1]) * f;
            big += fabsf(a) + fabsf(b);
            w[k] = count > 0 ? pack_bf16x2(a, b) : 0u;
          }
          *reinterpret_cast<uint4*>(stage + (c >> 1) * 4096 + lane * 128 + (((4 * (c & 1) + i / 8) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        bad |= 32 * c < width && !(big < INFINITY);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0 && row < p.T) {
        for (int b = 0; b < nb; ++b) tma_store_3d(half == 0 ? &tm_dv : &tm_dk, stage + b * 4096, 64 * b, row, h);
        bulk_commit();
        bulk_wait_all<0>();
      }
      __syncwarp();
      const uint32_t again = __ballot_sync(0xffffffffu, bad && count > 0 && row < p.T);
      if (lane == 0 && again) atomicOr(&g.again[warp & 3], again);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (warp < 4)   // as for dq
    for (uint32_t again = g.again[warp]; again; again &= again - 1) dkv_row<D>(p, r0 + warp * 32 + __ffs(again) - 1, h);
}

template <class... Args>
cudaError_t allow_smem(void (*kernel)(Args...), int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <int D>
cudaError_t launch(AttnArgs a, DevStatus st, cudaStream_t s) {
  static std::atomic<bool> ready[2][64];
  cudaError_t e = allow_smem(dq_kernel<D>, dq_smem<D>(), ready[0]);
  if (e == cudaSuccess) e = allow_smem(dkv_kernel<D>, dkv_smem<D>(), ready[1]);
  if (e != cudaSuccess) return e;
  constexpr auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  using KTile = AttnTile<D, kTile>;
  CUtensorMap q, k, v, da, dq, dk, dv;
  if (!map3d(&q, bf16, 2, a.q, D, a.T, a.Hq, KTile::kCols, kTile, 1, KTile::kSwizzle) ||
      !map3d(&k, bf16, 2, a.k, D, a.T, a.H, KTile::kCols, kTile, 1, KTile::kSwizzle) ||
      !map3d(&v, bf16, 2, a.v, kDv, a.T, a.H, VTile::kCols, kTile, 1, VTile::kSwizzle) ||
      !map2d_bf16(&da, a.da, static_cast<uint64_t>(a.Hq) * kDv, a.T, 64, kTile) ||
      !map3d(&dq, bf16, 2, a.dq, D, a.T, a.Hq, 64, 32, 1, sw) || !map3d(&dk, bf16, 2, a.dk, D, a.T, a.H, 64, 32, 1, sw) ||
      !map3d(&dv, bf16, 2, a.dv, kDv, a.T, a.H, 64, 32, 1, sw))
    return cudaErrorInvalidValue;
  const int tiles = a.Tp / kTile;
  if (static_cast<int64_t>(tiles) * a.Hq <= device_sms()) a.order[0] = a.order[1] = nullptr;   // all blocks start at once
  const unsigned prep = (a.order[0] ? 2 : 0) + static_cast<unsigned>(tiles) * a.Hq;
  e = launch_dependent(delta_kernel, dim3(prep), kPrepThreads, 0, s, a, tiles, st);
  if (e != cudaSuccess) return e;
  e = launch_dependent(dkv_kernel<D>, dim3(static_cast<unsigned>(tiles) * a.H), kThreads, dkv_smem<D>(), s, q, da, k, v, dk, dv, a, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(dq_kernel<D>, dim3(static_cast<unsigned>(tiles) * a.Hq), kThreads, dq_smem<D>(), s, k, v, dq, a, st);
}

}  // namespace

cudaError_t launch_attention_backward(const AttnArgs& a, DevStatus st, cudaStream_t s) {
  return a.d == 64 ? launch<64>(a, st, s) : a.d == 96 ? launch<96>(a, st, s) : launch<128>(a, st, s);
}

}  // namespace qkvp
