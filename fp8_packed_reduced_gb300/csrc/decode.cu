// Attention of one new token per sequence over the paged cache.
//   s_i = scale * q . k_i,  a = sum_i e^(s_i) v_i / sum_i e^(s_i)
//
// Every live row is read once: 2 (d + 128) bytes (bf16) or d + 128 + 8 (E4M3)
// per slot and head for 4 (d + 128) operations per query head, so the kernel
// is bound by memory, and its parts are chosen to keep loads in flight:
//   - The live slots of all (sequence, head) pairs, in units of KS slots, form
//     one list that is cut into equal contiguous parts, one for each warp of
//     the grid (one block of eight warps per SM), whatever the lengths are.
//     Warps never meet inside their parts.
//   - Each warp has its own ring of stages in shared memory, filled by
//     cp.async.  A unit lies inside one page (E4M3: its two halves do), so
//     its k and v are contiguous; chunks are swizzled so that the reads below
//     meet no bank twice.
//   - S^T = K Q^T and O^T = V^T P^T on mma.m16n8k16, slots (or value columns)
//     along M and up to eight query heads of a K/V head along N: they share
//     its one read.  k's dims may be permuted freely if q's are too, so a
//     lane's operands are whole 16-byte (8-byte) chunks of a row.
//   - Running maximum and sum per head in float32, exponentials of base 2.
//   - E4M3: codes become f16 exactly.  q is scaled per head by a power of two
//     into f16's range (a bf16 loses nothing above 2^-14 of its row's largest,
//     2^-25 of it below), row scales multiply scores and probabilities in
//     float32.  The probabilities times v's row scales are held relative to
//     their own running maximum, since rows of very different scale may meet.
//   - Probabilities enter the second product as bf16 (E4M3: f16): half a step
//     of 2^-8 (2^-11) relative, no more than the rounding of the output; the
//     sum of the probabilities, lse and the weights use them unrounded.
// A part that holds only a piece of a (sequence, head) leaves a record (m, l,
// O); pieces inside one block are joined by a warp of it, pieces across blocks
// by the block that arrives last, in the order of the slots: the result does
// not depend on the order of arrival.
#include <atomic>
#include <cmath>

#include "cache.cuh"
#include "kernels.cuh"

namespace qkvp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 160;            // one per SM, and the workspace's bound
constexpr int kSmemMax = 232448 - 1024;
constexpr int kMaxHeadTile = 16;           // query heads of one K/V head that share a read
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeParams {
  CacheArgs c;
  int G;                 // query heads per K/V head
  int chunks, nh;        // the G heads are taken in `chunks` parts of at most nh
  float scale_log2;      // scale * log2(e)
  const uint16_t* q;     // [H * G, B, d]
  uint16_t* a;           // [B, H * G, 128]
  float* lse;            // [B, H * G] natural logarithm, or null
  float* lse2;           // [B, H * G] base 2
  float* scores;         // [B, H * G, capacity] base 2, or null
  float* records;        // [2 * warps] of record_floats(nh)
  unsigned int* arrived; // [B * H * chunks] blocks that have left their records, zero between calls
};

__host__ __device__ constexpr int record_floats(int nh) { return nh * (kDv + 4); }

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t lo16) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(lo16 & 0xFFFFu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// exp2(x - m) with the weight of a score of -inf zero, also where m is -inf
__device__ __forceinline__ float exp2_below(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

// ---------------------------------------------------------------------------
// Shapes of a unit and of a stage
// ---------------------------------------------------------------------------
template <int D, bool FP8>
struct Tile {
  static constexpr int SUB = FP8 ? 2 : 1;              // halves of 16 slots
  static constexpr int KS = 16 * SUB;                  // slots of a unit
  static constexpr int ES = FP8 ? 1 : 2;               // bytes per value
  static constexpr int KC = D * ES / 16;               // 16-byte chunks of a k row
  static constexpr int VC = kDv * ES / 16;             // and of a v row
  static constexpr int K_BYTES = KS * D * ES;
  static constexpr int V_BYTES = KS * kDv * ES;
  static constexpr int SCALE_BYTES = FP8 ? 2 * KS * 4 : 0;
  static constexpr int META_BYTES = 32;
  __host__ __device__ static constexpr int stage_bytes(int nh) {
    return K_BYTES + V_BYTES + SCALE_BYTES + META_BYTES + nh * D * 2;
  }
  // Places of 16-byte chunk `ch` of row r, conflict-free for the reads below:
  // k is read by 8 lanes at a time as two rows x 64 bytes (bf16) or by 16 as
  // four rows x 32 bytes (E4M3), v by ldmatrix as eight rows x 16 bytes.
  __device__ static int k_at(int r, int ch) {
    int s = ch;
    if (!FP8 && D != 96) s ^= (r & 1) << 2;
    if (FP8 && D == 64) s ^= (r & 2);
    if (FP8 && D == 128) s ^= (r & 3) << 1;
    return (r * KC + s) * 16;
  }
  __device__ static int v_at(int r, int ch) { return (r * VC + (ch ^ (r & 7))) * 16; }
};

struct Unit {
  int64_t row[2];   // pool row of each half's first slot, -1: none
  int b, hv, u;     // sequence, head x chunk, unit of the sequence
  int valid;        // live slots
};

// The list of units: sequence b holds units[b] per (head, chunk), prefix[b]
// of them come before it.
struct Plan {
  const int* prefix;   // [B + 1]
  const int* length;   // [B]
  int B, Hv;
  int64_t total, part; // units, units per warp
};

// Exclusive prefix over the block of one value per thread.
__device__ __forceinline__ int block_exclusive(int v, int* red, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += red[w];
    sum += red[w];
  }
  *total = sum;
  __syncthreads();
  return before + x - v;
}

template <class TL>
__device__ __forceinline__ Unit locate(const Plan& pl, const DecodeParams& p, int64_t f, const DevStatus& st) {
  int lo = 0, hi = pl.B;   // prefix[lo] * Hv <= f < prefix[hi] * Hv
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(pl.prefix[mid]) * pl.Hv <= f)
      lo = mid;
    else
      hi = mid;
  }
  Unit r;
  r.b = lo;
  const int per = pl.prefix[lo + 1] - pl.prefix[lo];
  const int64_t rest = f - static_cast<int64_t>(pl.prefix[lo]) * pl.Hv;
  r.hv = static_cast<int>(rest / per);
  r.u = static_cast<int>(rest - static_cast<int64_t>(r.hv) * per);
  r.valid = min(TL::KS, pl.length[lo] - r.u * TL::KS);
  const int h = r.hv / p.chunks;
#pragma unroll
  for (int s = 0; s < 2; ++s)
    r.row[s] = s < TL::SUB && 16 * s < r.valid ? cache_row(p.c, lo, h, r.u * TL::KS + 16 * s, st, KID_DECODE) : -1;
  return r;
}

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
// Writes a and lse of query head hq from l, m (base 2) and four columns of O
// relative to 2^mo per lane.
__device__ __forceinline__ void write_head(const DecodeParams& p, int b, int hq, float m, float l, float mo, float4 o) {
  const int lane = threadIdx.x & 31, Hq = p.c.H * p.G;
  const bool none = l == 0.f;
  const float f = none ? 0.f : exp2_below(mo, m) / l;
  const int64_t at = static_cast<int64_t>(b) * Hq + hq;
  uint2 w = make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
  if (none) w = make_uint2(0, 0);
  reinterpret_cast<uint2*>(p.a + at * kDv)[lane] = w;
  if (lane == 0) {
    const float x = none ? -INFINITY : m + log2f(l);
    p.lse2[at] = x;
    if (p.lse) p.lse[at] = none ? -INFINITY : x * 0.6931471805599453f;
  }
}

// Joins, for head n, the records of warps w0, w0 + step, .. <= w1 of one
// (sequence, head): the first warp of the whole piece, `first`, holds it in
// its second record, the others in their first.
__device__ __forceinline__ void join_records(const DecodeParams& p, int n, int first, int w0, int w1, int step, float& m,
                                             float& l, float& mo, float4& o) {
  const int lane = threadIdx.x & 31, rs = record_floats(p.nh);
  const auto rec = [&](int w) { return p.records + static_cast<int64_t>(2 * w + (w == first)) * rs; };
  m = mo = -INFINITY;
  for (int w = w0 + step * lane; w <= w1; w += 32 * step) {
    m = fmaxf(m, __ldcg(rec(w) + p.nh * kDv + n));
    mo = fmaxf(mo, __ldcg(rec(w) + p.nh * (kDv + 2) + n));
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, s));
  }
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int w = w0; w <= w1; w += step) {
    const float* r = rec(w);
    l += exp2_below(__ldcg(r + p.nh * kDv + n), m) * __ldcg(r + p.nh * (kDv + 1) + n);
    const float f = exp2_below(__ldcg(r + p.nh * (kDv + 2) + n), mo);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(r + n * kDv) + lane);
    o.x += f * x.x;
    o.y += f * x.y;
    o.z += f * x.z;
    o.w += f * x.w;
  }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, bool FP8, int NT, int S>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ DecodeParams p, DevStatus st) {
  using TL = Tile<D, FP8>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int red[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int B = p.c.B, Hq = p.c.H * p.G;

  // --- the list of units -------------------------------------------------
  int* prefix = reinterpret_cast<int*>(smem);
  int* length = prefix + B + 1;
  int run = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int n = b < B ? checked_length(p.c, b, st, KID_DECODE) : 0;
    int sum;
    const int before = block_exclusive((n + TL::KS - 1) / TL::KS, red, &sum);
    if (b < B) {
      prefix[b] = run + before;
      length[b] = n;
    }
    run += sum;
  }
  if (threadIdx.x == 0) prefix[B] = run;
  __syncthreads();
  Plan pl{prefix, length, B, p.c.H * p.chunks, 0, 0};
  pl.total = static_cast<int64_t>(run) * pl.Hv;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  pl.part = (pl.total + nwarps - 1) / nwarps;

  // sequences without a live slot
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (length[b] == 0) {
      for (int i = threadIdx.x; i < Hq * (kDv / 8); i += kThreads)
        reinterpret_cast<uint4*>(p.a)[static_cast<int64_t>(b) * Hq * (kDv / 8) + i] = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; p.lse && i < Hq; i += kThreads) p.lse[static_cast<int64_t>(b) * Hq + i] = -INFINITY;
    }

  // --- the warp's part ----------------------------------------------------
  const int wid = blockIdx.x * kWarps + warp;
  const int64_t f0 = min(pl.total, wid * pl.part), f1 = min(pl.total, f0 + pl.part);
  const int stage_bytes = TL::stage_bytes(p.nh);
  uint8_t* ring = smem + ((2 * B + 1) * 4 + 127) / 128 * 128 + warp * S * stage_bytes;
  const uint32_t ring_u32 = smem_u32(ring);

  Unit mine;             // lane i: unit batch + i
  int64_t batch = f0 - 32;
  int prev_hv = -1, prev_b = -1;   // of the unit issued last
  const auto issue = [&](int64_t f) {
    if (f < f1) {
      if (f - batch >= 32) {
        batch = f;
        if (batch + lane < f1) mine = locate<TL>(pl, p, batch + lane, st);
      }
      const int who = static_cast<int>(f - batch);
      const int stage = static_cast<int>((f - f0) % S);
      const uint32_t s0 = ring_u32 + stage * stage_bytes;
      const int b = __shfl_sync(0xffffffffu, mine.b, who), hv = __shfl_sync(0xffffffffu, mine.hv, who);
      const int valid = __shfl_sync(0xffffffffu, mine.valid, who);
#pragma unroll
      for (int s = 0; s < TL::SUB; ++s) {
        const int64_t row = __shfl_sync(0xffffffffu, mine.row[s], who);
        const uint8_t* ks = p.c.k + (row < 0 ? 0 : row) * (D * TL::ES);
        const uint8_t* vs = p.c.v + (row < 0 ? 0 : row) * (kDv * TL::ES);
        const int live = row < 0 ? 0 : valid - 16 * s;   // live rows of this half
#pragma unroll
        for (int i = 0; i < TL::KC / 2; ++i) {
          const int id = i * 32 + lane, r = id / TL::KC, ch = id % TL::KC;
          cp16(s0 + TL::k_at(16 * s + r, ch), ks + id * 16, r < live);
        }
#pragma unroll
        for (int i = 0; i < TL::VC / 2; ++i) {
          const int id = i * 32 + lane, r = id / TL::VC, ch = id % TL::VC;
          cp16(s0 + TL::K_BYTES + TL::v_at(16 * s + r, ch), vs + id * 16, r < live);
        }
        if (FP8 && lane < 8) {   // 16 scales of k, then of v
          const float* sc = (lane < 4 ? p.c.k_scale : p.c.v_scale) + (row < 0 ? 0 : row) + (lane & 3) * 4;
          cp16(s0 + TL::K_BYTES + TL::V_BYTES + (lane < 4 ? 0 : TL::KS * 4) + 64 * s + (lane & 3) * 16, sc, live > 0);
        }
      }
      if (hv != prev_hv || b != prev_b) {   // q comes with the first unit of a (sequence, head)
        prev_hv = hv;
        prev_b = b;
        const int h = hv / p.chunks, ch0 = (hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
        constexpr int QC = D / 8;
        for (int i = lane; i < nh * QC; i += 32)
          cp16(s0 + TL::K_BYTES + TL::V_BYTES + TL::SCALE_BYTES + TL::META_BYTES + i * 16,
               p.q + (static_cast<int64_t>(h * p.G + ch0 + i / QC) * B + b) * D + (i % QC) * 8, true);
      }
      if (lane == who) {
        int* meta = reinterpret_cast<int*>(ring + stage * stage_bytes + TL::K_BYTES + TL::V_BYTES + TL::SCALE_BYTES);
        *reinterpret_cast<int4*>(meta) = make_int4(mine.b, mine.hv, mine.u, mine.valid);
        *reinterpret_cast<int2*>(meta + 4) = make_int2(mine.row[0] >= 0, mine.row[1] >= 0);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(f0 + i);

  uint4 qf[NT][D / 32];           // q of head 8 t + g: chunk c of every 32 dims
  float qmul[NT][2];              // score multiplier of heads 8 t + 2 c, + 1
  float m[NT][2], l[NT][2], mo[NT][2], o[NT][8][4];
  int cur_b = -1, cur_hv = -1;
  bool from_start = false;        // the piece being read begins with unit 0

  // Leaves the finished piece: the whole (sequence, head) as the result, part
  // of one as a record.
  const auto flush = [&](bool to_end) {
    const int h = cur_hv / p.chunks, ch0 = (cur_hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
    float* rec = p.records + static_cast<int64_t>(2 * wid + (from_start ? 1 : 0)) * record_floats(p.nh);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        const int n = 8 * t + 2 * c + e;
        if (n >= nh) continue;
        if (from_start && to_end) {
          const int64_t at = static_cast<int64_t>(cur_b) * Hq + h * p.G + ch0 + n;
          const bool none = x == 0.f;
          const float f = none ? 0.f : exp2_below(mo[t][e], m[t][e]) / x;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
            if (FP8) {
              const uint32_t w = pack_bf16x2(o[t][mt][e] * f, o[t][mt][2 + e] * f);
              reinterpret_cast<uint32_t*>(p.a + at * kDv)[8 * mt + g] = none ? 0u : w;
            } else {
              const uint32_t w = pack_bf16x2(o[t][mt][e] * f, o[t][mt][2 + e] * f);
              p.a[at * kDv + 16 * mt + g] = none ? 0 : static_cast<uint16_t>(w);
              p.a[at * kDv + 16 * mt + g + 8] = none ? 0 : static_cast<uint16_t>(w >> 16);
            }
          if (g == 0) {
            const float y = none ? -INFINITY : m[t][e] + log2f(x);
            p.lse2[at] = y;
            if (p.lse) p.lse[at] = none ? -INFINITY : y * 0.6931471805599453f;
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
            if (FP8) {
              *reinterpret_cast<float2*>(rec + n * kDv + 16 * mt + 2 * g) = make_float2(o[t][mt][e], o[t][mt][2 + e]);
            } else {
              rec[n * kDv + 16 * mt + g] = o[t][mt][e];
              rec[n * kDv + 16 * mt + g + 8] = o[t][mt][2 + e];
            }
          if (g == 0) {
            rec[p.nh * kDv + n] = m[t][e];
            rec[p.nh * (kDv + 1) + n] = x;
            rec[p.nh * (kDv + 2) + n] = mo[t][e];
          }
        }
      }
  };

  for (int64_t f = f0; f < f1; ++f) {
    cp_wait<S - 2>();
    __syncwarp();
    issue(f + S - 1);   // into the stage read in the last round
    const int stage = static_cast<int>((f - f0) % S);
    const uint32_t s0 = ring_u32 + stage * stage_bytes;
    const uint32_t sv = s0 + TL::K_BYTES, ss = sv + TL::V_BYTES, sm = ss + TL::SCALE_BYTES, sq = sm + TL::META_BYTES;
    const uint4 meta = lds128(sm);
    const uint2 good = lds64(sm + 16);
    const int b = meta.x, hv = meta.y, u = meta.z, valid = meta.w;
    if (b != cur_b || hv != cur_hv) {
      if (cur_b >= 0) flush(true);
      cur_b = b;
      cur_hv = hv;
      from_start = u == 0;
      const int nh = min(p.nh, p.G - (hv % p.chunks) * p.nh);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bool head = 8 * t + g < nh;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          qf[t][j] = head ? lds128(sq + (8 * t + g) * D * 2 + j * 64 + c * 16) : make_uint4(0, 0, 0, 0);
        float back = 1.f;   // what the scaled q is multiplied with again
        if (FP8) {
          float am = 0.f;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint32_t w[4] = {qf[t][j].x, qf[t][j].y, qf[t][j].z, qf[t][j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) am = fmaxf(am, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
          }
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
          // 2^-e and 2^e for am in [2^e, 2^(e+1)), from am's exponent bits, kept to normal numbers
          const int eb = min(253, max(1, static_cast<int>(__float_as_uint(am) >> 23)));
          const float down = __uint_as_float(static_cast<uint32_t>(254 - eb) << 23);
          back = __uint_as_float(static_cast<uint32_t>(eb) << 23);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t w[4] = {qf[t][j].x, qf[t][j].y, qf[t][j].z, qf[t][j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
            qf[t][j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qmul[t][e] = p.scale_log2 * (FP8 ? __shfl_sync(0xffffffffu, back, 8 * c + 4 * e) : 1.f);
          m[t][e] = mo[t][e] = -INFINITY;
          l[t][e] = 0.f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) o[t][mt][e] = o[t][mt][2 + e] = 0.f;
        }
      }
    }

    // scores of slots 16 s + g and + 8, heads 8 t + 2 c and + 1
    float x[NT][TL::SUB][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = 0; s < TL::SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][s][i] = 0.f;
#pragma unroll
    for (int s = 0; s < TL::SUB; ++s)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t ka[4], kb[4];   // rows g and g + 8: dims 32 j + 8 c .. + 7
        if (FP8) {
          const uint2 ra = lds64(s0 + TL::k_at(16 * s + g, 2 * j + (c >> 1)) + (c & 1) * 8);
          const uint2 rb = lds64(s0 + TL::k_at(16 * s + g + 8, 2 * j + (c >> 1)) + (c & 1) * 8);
          ka[0] = e4m3x2_to_f16x2(ra.x);
          ka[1] = e4m3x2_to_f16x2(ra.x >> 16);
          ka[2] = e4m3x2_to_f16x2(ra.y);
          ka[3] = e4m3x2_to_f16x2(ra.y >> 16);
          kb[0] = e4m3x2_to_f16x2(rb.x);
          kb[1] = e4m3x2_to_f16x2(rb.x >> 16);
          kb[2] = e4m3x2_to_f16x2(rb.y);
          kb[3] = e4m3x2_to_f16x2(rb.y >> 16);
        } else {
          const uint4 ra = lds128(s0 + TL::k_at(g, 4 * j + c)), rb = lds128(s0 + TL::k_at(g + 8, 4 * j + c));
          ka[0] = ra.x, ka[1] = ra.y, ka[2] = ra.z, ka[3] = ra.w;
          kb[0] = rb.x, kb[1] = rb.y, kb[2] = rb.z, kb[3] = rb.w;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<FP8>(x[t][s], ka[0], kb[0], ka[1], kb[1], qf[t][j].x, qf[t][j].y);
          mma16816<FP8>(x[t][s], ka[2], kb[2], ka[3], kb[3], qf[t][j].z, qf[t][j].w);
        }
      }

    uint32_t pb[NT][TL::SUB][2];   // the probabilities as the second product's operand
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[TL::SUB][4];   // E4M3: the score plus log2 of v's row scale
      float top[2] = {-INFINITY, -INFINITY}, otop[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int s = 0; s < TL::SUB; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * s + 8 * r + g;
          const bool live = i < valid && (s == 0 ? good.x : good.y) != 0;
          float ks = 1.f, vs = 0.f;
          if (FP8) {
            ks = lds32(ss + i * 4);
            vs = __log2f(lds32(ss + TL::KS * 4 + i * 4));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = x[t][s][2 * r + e];
            v = live ? v * qmul[t][e] * ks : -INFINITY;
            top[e] = fmaxf(top[e], v);
            if (FP8) {
              y[s][2 * r + e] = live ? v + vs : -INFINITY;
              otop[e] = fmaxf(otop[e], y[s][2 * r + e]);
            }
          }
          if (p.scores != nullptr && i < valid) {
            const int h = hv / p.chunks, ch0 = (hv % p.chunks) * p.nh;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = 8 * t + 2 * c + e;
              if (n < p.nh && ch0 + n < p.G)
                p.scores[(static_cast<int64_t>(b) * Hq + h * p.G + ch0 + n) * p.c.capacity() + u * TL::KS + i] =
                    x[t][s][2 * r + e];
            }
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], s));
          if (FP8) otop[e] = fmaxf(otop[e], __shfl_xor_sync(0xffffffffu, otop[e], s));
        }
        top[e] = fmaxf(top[e], m[t][e]);
        otop[e] = FP8 ? fmaxf(otop[e], mo[t][e]) : top[e];
      }
      const bool grows = top[0] > m[t][0] || top[1] > m[t][1] || otop[0] > mo[t][0] || otop[1] > mo[t][1];
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[t][e] *= exp2_below(m[t][e], top[e]);
          const float fo = exp2_below(mo[t][e], otop[e]);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[t][mt][e] *= fo;
            o[t][mt][2 + e] *= fo;
          }
          m[t][e] = top[e];
          mo[t][e] = otop[e];
        }
      }
#pragma unroll
      for (int s = 0; s < TL::SUB; ++s) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float pr = exp2_below(x[t][s][i], m[t][i & 1]);
          l[t][i & 1] += pr;
          w[i] = FP8 ? exp2_below(y[s][i], mo[t][i & 1]) : pr;
        }
        pb[t][s][0] = movmatrix_trans(FP8 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]));
        pb[t][s][1] = movmatrix_trans(FP8 ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]));
      }
    }

#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint32_t r[4];
      if (FP8) {
        // eight slots x 16 columns each: column pairs 2 g, 2 g + 1 of slots 2 c and 2 c + 1
        ldmatrix4_trans(r, sv + TL::v_at(lane, mt));
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = __byte_perm(r[i], 0, 0x3120);
          lo[i] = e4m3x2_to_f16x2(w);
          hi[i] = e4m3x2_to_f16x2(w >> 16);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int s = 0; s < TL::SUB; ++s)
            mma16816<true>(o[t][mt], lo[2 * s], hi[2 * s], lo[2 * s + 1], hi[2 * s + 1], pb[t][s][0], pb[t][s][1]);
      } else {
        // slots 0-7 and 8-15, columns 16 mt .. + 7 and + 8 .. + 15
        ldmatrix4_trans(r, sv + TL::v_at((lane & 7) + (lane >> 4) * 8, 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816<false>(o[t][mt], r[0], r[1], r[2], r[3], pb[t][0][0], pb[t][0][1]);
      }
    }
  }
  cp_wait<0>();
  // The last piece of the part: to its end?
  const auto piece_of = [&](int64_t f, int64_t& start, int64_t& end, int& b, int& hv) {   // the (sequence, head) of unit f
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<int64_t>(prefix[mid]) * pl.Hv <= f)
        lo = mid;
      else
        hi = mid;
    }
    const int per = prefix[lo + 1] - prefix[lo];
    const int64_t base = static_cast<int64_t>(prefix[lo]) * pl.Hv;
    b = lo;
    hv = static_cast<int>((f - base) / per);
    start = base + static_cast<int64_t>(hv) * per;
    end = start + per;
  };
  if (cur_b >= 0) {
    int64_t s, e;
    int b, hv;
    piece_of(f1 - 1, s, e, b, hv);
    flush(e == f1);
  }
  __threadfence();
  __syncthreads();

  // --- joining ---------------------------------------------------------------
  const int64_t c0 = min(pl.total, blockIdx.x * kWarps * pl.part), c1 = min(pl.total, c0 + kWarps * pl.part);
  if (c0 >= c1) return;
  // pieces that begin in this warp's part, end in another warp's of this block
  if (f0 < f1) {
    int64_t s, e;
    int b, hv;
    piece_of(f1 - 1, s, e, b, hv);
    if (s >= f0 && e > f1 && e <= c1) {
      const int h = hv / p.chunks, ch0 = (hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
      const int last = static_cast<int>((e - 1) / pl.part);
      for (int n = 0; n < nh; ++n) {
        float jm, jl, jo;
        float4 x;
        join_records(p, n, wid, wid, last, 1, jm, jl, jo, x);
        write_head(p, b, h * p.G + ch0 + n, jm, jl, jo, x);
      }
    }
  }
  // pieces that reach over the block's ends: the first and the last of it
  __shared__ bool is_last;
  float* part = reinterpret_cast<float*>(smem + ((2 * B + 1) * 4 + 127) / 128 * 128);
  for (int side = 0; side < 2; ++side) {
    int64_t s, e;
    int b, hv;
    piece_of(side == 0 ? c0 : c1 - 1, s, e, b, hv);
    const bool reaches = side == 0 ? s < c0 : s >= c0 && e > c1;   // one that covers the whole block counts once
    if (!reaches) continue;
    const int first = static_cast<int>(s / pl.part), last = static_cast<int>((e - 1) / pl.part);
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned int* cnt = p.arrived + static_cast<int64_t>(b) * pl.Hv + hv;
      const unsigned int blocks = last / kWarps - first / kWarps + 1;
      is_last = atomicAdd(cnt, 1u) == blocks - 1;
      if (is_last) *cnt = 0;
      __threadfence();
    }
    __syncthreads();
    if (!is_last) continue;
    const int h = hv / p.chunks, ch0 = (hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
    const int rs = record_floats(p.nh);
    for (int n = 0; n < nh; ++n) {   // every warp joins some of the records, in the order of the slots
      const int count = last - first + 1, each = (count + kWarps - 1) / kWarps;
      float jm, jl, jo;
      float4 x;
      join_records(p, n, first, first + warp * each, min(last, first + (warp + 1) * each - 1), 1, jm, jl, jo, x);
      float* r = part + warp * rs;
      reinterpret_cast<float4*>(r + n * kDv)[lane] = x;
      if (lane == 0) {
        r[p.nh * kDv + n] = jm;
        r[p.nh * (kDv + 1) + n] = jl;
        r[p.nh * (kDv + 2) + n] = jo;
      }
    }
    __syncthreads();
    for (int n = warp; n < nh; n += kWarps) {
      float jm = -INFINITY, jl = 0.f, jo = -INFINITY;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        jm = fmaxf(jm, part[w * rs + p.nh * kDv + n]);
        jo = fmaxf(jo, part[w * rs + p.nh * (kDv + 2) + n]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* r = part + w * rs;
        jl += exp2_below(r[p.nh * kDv + n], jm) * r[p.nh * (kDv + 1) + n];
        const float fo = exp2_below(r[p.nh * (kDv + 2) + n], jo);
        const float4 y = reinterpret_cast<const float4*>(r + n * kDv)[lane];
        x.x += fo * y.x;
        x.y += fo * y.y;
        x.z += fo * y.z;
        x.w += fo * y.w;
      }
      write_head(p, b, h * p.G + ch0 + n, jm, jl, jo, x);
    }
  }
}

// weight += the probabilities of the head's query heads
__global__ void __launch_bounds__(kThreads) decode_weight_kernel(const __grid_constant__ DecodeParams p, DevStatus st) {
  const int h = blockIdx.y, b = blockIdx.z, Hq = p.c.H * p.G, i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= checked_length(p.c, b, st, KID_DECODE_WEIGHT)) return;
  const int64_t row = cache_row(p.c, b, h, i, st, KID_DECODE_WEIGHT);
  if (row < 0) return;
  float w = 0.f;
  for (int g = 0; g < p.G; ++g) {
    const int64_t at = static_cast<int64_t>(b) * Hq + h * p.G + g;
    w += exp2_below(p.scores[at * p.c.capacity() + i], p.lse2[at]);
  }
  p.c.weight[row] += w;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_heads(const CacheArgs& a, int Hq) {
  if (Hq < 1) return QKVP_ERR_INVALID_ARGUMENT;
  return Hq % a.H || Hq > 1024 ? QKVP_ERR_UNSUPPORTED : QKVP_OK;
}

// Parts of the workspace: status, arrival counters, lse2, records, scores.
struct DecodeLayout {
  size_t arrived, lse2, records, scores, bytes;
};
int head_chunks(const CacheArgs& a, int Hq) { return (Hq / a.H + kMaxHeadTile - 1) / kMaxHeadTile; }
int heads_per_chunk(const CacheArgs& a, int Hq) {
  const int G = Hq / a.H, n = head_chunks(a, Hq);
  return (G + n - 1) / n;
}
int64_t most_units(const CacheArgs& a, int Hq) {
  return static_cast<int64_t>(a.B) * a.H * head_chunks(a, Hq) * (a.capacity() / 16);
}
DecodeLayout decode_layout(const CacheArgs& a, int Hq, int accumulate) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const int64_t warps = most_units(a, Hq) < kMaxBlocks * kWarps ? most_units(a, Hq) : kMaxBlocks * kWarps;
  DecodeLayout w;
  w.arrived = kCacheStatusBytes;
  w.lse2 = w.arrived + up(static_cast<size_t>(a.B) * a.H * head_chunks(a, Hq) * sizeof(unsigned int));
  w.records = w.lse2 + up(static_cast<size_t>(a.B) * Hq * sizeof(float));
  w.scores = w.records + up(static_cast<size_t>(2 * (warps + kWarps)) * record_floats(heads_per_chunk(a, Hq)) * sizeof(float));
  w.bytes = w.scores + (accumulate ? static_cast<size_t>(a.B) * Hq * a.capacity() * sizeof(float) : 0);
  return w;
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

template <int D, bool FP8, int NT, int S>
cudaError_t launch_decode_s(const DecodeParams& p, int grid, int smem, DevStatus st, cudaStream_t s) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(decode_kernel<D, FP8, NT, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev].store(true, std::memory_order_relaxed);
  }
  decode_kernel<D, FP8, NT, S><<<grid, kThreads, smem, s>>>(p, st);
  return cudaGetLastError();
}

// As many stages as fit: three, or two beside the q rows of many heads.
template <int D, bool FP8, int NT>
cudaError_t launch_decode_nt(const DecodeParams& p, int grid, DevStatus st, cudaStream_t s) {
  const int head = ((2 * p.c.B + 1) * 4 + 127) / 128 * 128;
  const int stage = kWarps * Tile<D, FP8>::stage_bytes(p.nh);
  if (head + 3 * stage <= kSmemMax) return launch_decode_s<D, FP8, NT, 3>(p, grid, head + 3 * stage, st, s);
  return launch_decode_s<D, FP8, NT, 2>(p, grid, head + 2 * stage, st, s);
}

template <int D, bool FP8>
cudaError_t launch_decode(const DecodeParams& p, int grid, DevStatus st, cudaStream_t s) {
  return p.nh <= 8 ? launch_decode_nt<D, FP8, 1>(p, grid, st, s) : launch_decode_nt<D, FP8, 2>(p, grid, st, s);
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
  p.arrived = reinterpret_cast<unsigned int*>(wsb + w.arrived);
  p.lse2 = reinterpret_cast<float*>(wsb + w.lse2);
  p.lse = lse;
  p.records = reinterpret_cast<float*>(wsb + w.records);
  p.scores = accumulate ? reinterpret_cast<float*>(wsb + w.scores) : nullptr;
  const int64_t blocks = (most_units(p.c, Hq) + kWarps - 1) / kWarps;
  const int most = sms < kMaxBlocks ? sms : kMaxBlocks;
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  mark(s);
  cudaError_t e;
  switch (p.c.d) {
    case 64: e = cache->fp8 ? launch_decode<64, true>(p, grid, st, s) : launch_decode<64, false>(p, grid, st, s); break;
    case 96: e = cache->fp8 ? launch_decode<96, true>(p, grid, st, s) : launch_decode<96, false>(p, grid, st, s); break;
    default: e = cache->fp8 ? launch_decode<128, true>(p, grid, st, s) : launch_decode<128, false>(p, grid, st, s);
  }
  if (e != cudaSuccess) return QKVP_ERR_CUDA;
  mark(s);
  if (accumulate) {
    decode_weight_kernel<<<dim3((p.c.capacity() + kThreads - 1) / kThreads, p.c.H, p.c.B), kThreads, 0, s>>>(p, st);
    if (cudaGetLastError() != cudaSuccess) return QKVP_ERR_CUDA;
    mark(s);
  }
  return QKVP_OK;
}

}  // extern "C"
