// Attention of one new token per sequence over the paged cache.
//   s_i = scale * q . k_i,  a = sum_i e^(s_i) v_i / sum_i e^(s_i)
//
// Every live row is read once: 2 (d + 128) bytes (bf16) or d + 128 + 8 (E4M3)
// per slot and head for 4 (d + 128) operations per query head, so the kernel
// is bound by memory, and its parts are chosen to keep loads in flight:
//   - The live slots of all (sequence, head) pairs, in units of KS slots, form
//     one list that is cut into equal contiguous parts, one for each warp of
//     the grid (a block per SM, of 12 warps or, where registers or shared memory
//     do not hold them, 8), whatever the lengths are.  Warps never meet inside their parts.
//   - Each warp has its own ring of stages in shared memory, filled by
//     cp.async.  A unit lies inside one page (E4M3: its two halves do), so
//     its k and v are contiguous; chunks are swizzled so that the reads below
//     meet no bank twice.
//   - S^T = K Q^T and O^T = V^T P^T on mma.m16n8k16, slots (or value columns)
//     along M and up to eight query heads of a K/V head along N: they share
//     its one read.  k's dims may be permuted freely if q's are too, so a
//     lane's operands are whole 16-byte (8-byte) chunks of a row.
//   - Running maximum and sum per head in float32, exponentials of base 2.
//   - E4M3: codes become f16 exactly.  q is scaled per head by a power of two to
//     the top of f16's range (a bf16 is exact down to 2^-31 of its row's
//     largest), row scales multiply scores and probabilities in float32.  The
//     probabilities times v's row scales are held relative to 2^-15 of their own
//     running maximum (rows of very different scale may meet), again at the top
//     of the range, so that rounding is relative down to 2^-29 of it.  Both are
//     taken relative to the scores' maximum first: the logarithm of a scale
//     added to a score of 2^16 would keep 2^-8 of itself.
//   - Probabilities enter the second product as two bf16, which hold 2^-15 of
//     them relatively (one holds 2^-8, as much again as the rounding of the
//     output): the second takes the tile's odd columns, which up to four heads
//     leave empty, or with more heads a product of its own (32 sequences of up to
//     6001 slots, 4 x 8 heads of 96 50.4 us, with one bf16 50.3; 4 x 16 of 64
//     49.6 / 48.4).
//     E4M3: as one f16, 2^-11, an eighth of the output's rounding.  The sum of
//     the probabilities, lse and the weights use them unrounded.
// A part that holds only a piece of a (sequence, head) leaves a record (m, l,
// O); pieces inside one block are joined by a warp of it, pieces across blocks
// by the block that arrives last, in the order of the slots: the result does
// not depend on the order of arrival.
//
// Measured (GB300, bytes of the live rows over the whole call): 64 sequences
// of up to 8191 slots x 6 heads, 606 MB, 103.6 us, 5.85 TB/s (86 % of a copy's
// rate); one of 131072 slots 64.5 us, 5.46 TB/s; 256 of up to 333 slots x 8
// heads of 128 with weights 34.4 us, 4.30 TB/s; 32 of up to 6001 slots, 4 x 4
// heads of 64 with weights 37 us, 3.44 TB/s; 48 of up to 8192 slots of E4M3
// with weights 55.6 us, 4.22 TB/s.  While a block reads it does so at the
// copy's rate; the rest is 2.5 us until the first loads are issued, up to 4 us
// between the first and the last SM to end (those of some GPCs are slower in
// every run), 4 - 7 us of joins and 3 us of the weights' kernel.
//
// Under a window (kWindow) a sequence's units are those that hold a slot below
// `sinks` or one of its last `window`, and what the other slots of such a unit
// hold is not used: their rows read as zero, their scores as -inf.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "cache.cuh"
#include "kernels.cuh"

namespace qkvp {

struct DecodeParams {
  CacheArgs c;
  int G;                 // query heads per K/V head
  int chunks, nh;        // the G heads are taken in `chunks` parts of at most nh
  int smem_records;      // the warps' records fit into shared memory
  int window, sinks;     // slots that are seen under a window
  float scale_log2;      // scale * log2(e)
  const uint16_t* q;     // [H * G, B, d]
  uint16_t* a;           // [B, H * G, 128]
  float* lse;            // [B, H * G] natural logarithm, or null
  float* lse2;           // [B, H * G] base 2
  float* scores;         // [B, H * G, capacity] base 2, or null
  float* records;        // [2 * blocks] records of blocks, then [warps] of warps (unless smem_records)
  unsigned int* arrived; // [blocks] for the piece that a block ends with, the blocks that have left their records of
                         // it; zero between calls
};
// The attention under a window (its kernels are a translation unit of their own).
cudaError_t launch_decode_window(DecodeParams& p, bool fp8, int grid, DevStatus st, cudaStream_t s);

namespace {

constexpr int kMaxWarps = 12;
constexpr int kWeightThreads = 256;        // at most
constexpr int kMaxBlocks = 160;            // one per SM, and the workspace's bound
static_assert(kMaxBlocks <= kMaxDecodeBlocks, "too few counters");
constexpr int kSmemMax = 232448 - 1024;
constexpr float kLog2e = 1.4426950408889634f;

// A record: O [nh][128] relative to 2^(m + mo), then m [nh], l [nh] (relative to 2^m), mo [nh].
__host__ __device__ constexpr int record_floats(int nh) { return nh * (kDv + 4); }

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
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
// The four E4M3 codes of a word as f16, exactly: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x to 2^-22 relative; results below the normal numbers are zero.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The bf16 next to x >= 0 towards zero, and what it leaves of x: never zero
// beside an x that is not, so that infinities of v times it are those of v
// times x.
__device__ __forceinline__ float bf16_below(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_rest(float x) {
  return x > 0.f ? fmaxf(x - bf16_below(x), 1.1754943508222875e-38f) : 0.f;
}
// What scores are taken relative to: their maximum m, or 0 where all are -inf
// (so that each of them has the weight 2^-inf = 0).
__device__ __forceinline__ float below(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float exp2_below(float x, float m) { return ex2(x - below(m)); }

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
  static constexpr int META_BYTES = 16;
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
  int row[2];       // pool row of each half's first slot, -1: none
  int b, hv, u;     // sequence, head x chunk, unit of the sequence
  int valid;        // live slots
  int first;        // the sequence's first unit
  int hole;         // under a window: slots hole & 63 .. (hole >> 8) - 1 are not seen
};

// The units of a sequence of n live slots that hold what is seen: all, or the
// first `sinks` and those behind the next `skip`.
struct Seen {
  int sinks, skip, count;
};
template <bool kWindow, int KS>
__device__ __forceinline__ Seen seen_units(const DecodeParams& p, int n) {
  const int all = (n + KS - 1) / KS;
  if (!kWindow) return Seen{all, 0, all};
  const int w0 = max(0, n - p.window), first = w0 / KS;   // the window's first slot and unit
  const int s = min(first, (min(p.sinks, w0) + KS - 1) / KS);
  return Seen{s, first - s, all - (first - s)};
}

// The list of units: sequence b holds as many per (head, chunk) as lie
// between prefix[b] and prefix[b + 1].
struct Plan {
  const int* prefix;   // [B + 1]
  const int* length;   // [B]
  int B, Hv;
};

// Quotients of numbers that are below 2^31 but for caches of the largest size:
// a 64-bit division is several times as long.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? static_cast<int64_t>(static_cast<unsigned int>(a) / static_cast<unsigned int>(b)) : a / b;
}
__device__ __forceinline__ int64_t divide_up(int64_t a, int64_t b) { return divide(a + b - 1, b); }

// A (sequence, head, chunk) as a piece of the list.
struct Piece {
  int64_t start, end;
  int b, hv;
};
__device__ __forceinline__ Piece piece_of(const Plan& pl, int64_t f) {
  int lo = 0, hi = pl.B;   // prefix[lo] * Hv <= f < prefix[hi] * Hv
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(pl.prefix[mid]) * pl.Hv <= f)
      lo = mid;
    else
      hi = mid;
  }
  const int per = pl.prefix[lo + 1] - pl.prefix[lo];
  const int64_t base = static_cast<int64_t>(pl.prefix[lo]) * pl.Hv, rest = f - base;
  Piece r;
  r.b = lo;
  r.hv = static_cast<int>(divide(rest, per));
  r.start = base + static_cast<int64_t>(r.hv) * per;
  r.end = r.start + per;
  return r;
}

// Exclusive prefix over the block of one value per thread.
template <int kWarps>
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

template <bool kWindow, class TL>
__device__ __forceinline__ Unit locate(const Plan& pl, const DecodeParams& p, int64_t f, const DevStatus& st) {
  const Piece pc = piece_of(pl, f);
  Unit r;
  r.b = pc.b;
  r.hv = pc.hv;
  r.u = static_cast<int>(f - pc.start);
  r.first = r.u == 0;
  r.hole = 0;
  if (kWindow) {
    const int n = pl.length[r.b];
    const Seen se = seen_units<true, TL::KS>(p, n);
    if (r.u >= se.sinks) r.u += se.skip;
    const int from = min(max(p.sinks - r.u * TL::KS, 0), TL::KS), to = min(max(n - p.window - r.u * TL::KS, 0), TL::KS);
    if (from < to) r.hole = from | to << 8;
  }
  r.valid = min(TL::KS, pl.length[r.b] - r.u * TL::KS);
  const int h = r.hv / p.chunks;
#pragma unroll
  for (int s = 0; s < 2; ++s)
    r.row[s] = s < TL::SUB && 16 * s < r.valid ? cache_row(p.c, r.b, h, r.u * TL::KS + 16 * s, st, KID_DECODE) : -1;
  return r;
}

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
// Writes a and lse of query head hq from l, m (base 2) and four columns of O
// relative to 2^(m + mo) per lane.
__device__ __forceinline__ void write_head(const DecodeParams& p, int b, int hq, float m, float l, float mo, float4 o) {
  const int lane = threadIdx.x & 31, Hq = p.c.H * p.G;
  const bool none = l == 0.f;
  const float f = none ? 0.f : ex2(mo) / l;
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

// Records joined, for one head: m, l and four columns of O per lane.
struct Joined {
  float m, l, mo;
  float4 o;
  __device__ void store(float* r, int n, int nh) const {
    const int lane = threadIdx.x & 31;
    reinterpret_cast<float4*>(r + n * kDv)[lane] = o;
    if (lane == 0) {
      r[nh * kDv + n] = m;
      r[nh * (kDv + 1) + n] = l;
      r[nh * (kDv + 2) + n] = mo;
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Records of this block (in shared memory, or not), and of other blocks.
struct AnyLoad {
  template <class T>
  __device__ T operator()(const T* p) const { return *p; }
};
struct L2Load {
  template <class T>
  __device__ T operator()(const T* p) const { return __ldcg(p); }
};

// Counts an arrival; everything the block has written (before a barrier) is
// visible to whoever counts after it.  Returns the arrivals before.
__device__ __forceinline__ unsigned int count_arrival(unsigned int* p) {
  unsigned int old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// The join of head n of `count` records, record i at rec(i).  32 at a time: a
// lane takes the maximum and the sum of one of them, so that every record's
// factor is known at once and the loads of O do not wait for each other.
template <class Load, class Rec>
__device__ __forceinline__ Joined join_records(const Load& load, const Rec& rec, int count, int n, int nh) {
  const int lane = threadIdx.x & 31;
  Joined j{-INFINITY, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int k = min(32, count - i0);
    float rm = -INFINITY, rl = 0.f, rmo = 0.f;
    if (lane < k) {
      const float* r = rec(i0 + lane);
      rm = load(r + nh * kDv + n);
      rl = load(r + nh * (kDv + 1) + n);
      rmo = load(r + nh * (kDv + 2) + n);
    }
    const float m = fmaxf(j.m, warp_max(rm)), up = below(m);
    const float z = rm - up + rmo, zj = j.m - up + j.mo;   // where the records' O stand, relative to 2^m
    const float mo = below(fmaxf(zj, warp_max(z)));
    const float f = ex2(z - mo), back = ex2(zj - mo);
    j.l = j.l * ex2(j.m - up) + warp_sum(rl * ex2(rm - up));
    j.o = make_float4(j.o.x * back, j.o.y * back, j.o.z * back, j.o.w * back);
    j.m = m;
    j.mo = mo;
#pragma unroll 4
    for (int i = 0; i < k; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      const float4 x = load(reinterpret_cast<const float4*>(rec(i0 + i) + n * kDv) + lane);
      j.o.x += fi * x.x;
      j.o.y += fi * x.y;
      j.o.z += fi * x.z;
      j.o.w += fi * x.w;
    }
  }
  return j;
}

// ---------------------------------------------------------------------------
// The kernel.  E query heads per lane and tile of eight columns: two, or with
// at most four heads one, on the even columns (half the work between the two
// products).
// ---------------------------------------------------------------------------
template <int D, bool FP8, bool kWindow, int NT, int E, int kWarps, int S>
__global__ void __launch_bounds__(32 * kWarps, 1) decode_kernel(const __grid_constant__ DecodeParams p, DevStatus st) {
  using TL = Tile<D, FP8>;
  constexpr int SUB = TL::SUB, KS = TL::KS, kThreads = 32 * kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int red[kWarps], red_max[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int B = p.c.B, Hq = p.c.H * p.G, nrec = record_floats(p.nh);
  constexpr float kTop = FP8 ? 15.f : 0.f;   // O is relative to 2^(m + mo - kTop); bf16: mo is 0
  const auto head_of = [&](int t, int e) { return E == 1 ? c : 8 * t + 2 * c + e; };   // of this lane's scores

  wait_for_previous();
  // The page table is first needed after the lengths: it comes into L2 meanwhile.
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 32; i < static_cast<int64_t>(B) * p.c.max_pages;
       i += static_cast<int64_t>(gridDim.x) * kThreads * 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + i));

  // --- the list of units -------------------------------------------------
  int* prefix = reinterpret_cast<int*>(smem);
  int* length = prefix + B + 1;
  int run = 0, longest = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int n = b < B ? checked_length(p.c, b, st, KID_DECODE) : 0;
    int sum;
    const int units = seen_units<kWindow, KS>(p, n).count;
    const int before = block_exclusive<kWarps>(units, red, &sum);
    if (b < B) {
      prefix[b] = run + before;
      length[b] = n;
    }
    run += sum;
    longest = max(longest, __reduce_max_sync(0xffffffffu, kWindow ? units * KS : n));
  }
  if (threadIdx.x == 0) prefix[B] = run;
  if (lane == 0) red_max[warp] = longest;
  __syncthreads();
  const Plan pl{prefix, length, B, p.c.H * p.chunks};
  const int64_t total = static_cast<int64_t>(run) * pl.Hv;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  // Even parts, [c0, c1) for the block.  An end of it that lies within one
  // warp's part of a piece's end moves there: a piece cut between blocks costs
  // about 5 us (two rounds through L2 after the last load).
  const int64_t even = divide_up(total, nwarps);
  int64_t part = even;
  const auto block_start = [&](int64_t blk) {
    const int64_t f = blk * kWarps * even;
    if (f >= total) return total;
    const Piece pc = piece_of(pl, f);
    return f - pc.start <= even && f - pc.start <= pc.end - f ? pc.start : pc.end - f <= even ? pc.end : f;
  };
  const int64_t start = block_start(blockIdx.x + (lane & 1));   // both ends at once
  int64_t c0 = __shfl_sync(0xffffffffu, start, 0), c1 = __shfl_sync(0xffffffffu, start, 1);
  if (c1 - c0 > 0) part = (c1 - c0 + kWarps - 1) / kWarps;
  // But where a block for every piece makes no warp's part longer by more than
  // a few units (0.7 us each), it has one.
  if (static_cast<int64_t>(B) * pl.Hv <= gridDim.x) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) longest = max(longest, red_max[w]);
    if ((longest + kWarps * KS - 1) / (kWarps * KS) <= even + 4) {
      const int b = blockIdx.x / pl.Hv, hv = blockIdx.x % pl.Hv;
      c0 = c1 = 0;
      if (b < B) {
        const int per = prefix[b + 1] - prefix[b];
        c0 = static_cast<int64_t>(prefix[b]) * pl.Hv + static_cast<int64_t>(hv) * per;
        c1 = c0 + per;
        part = max(1, (per + kWarps - 1) / kWarps);
      }
    }
  }
  // sequences without a live slot
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (length[b] == 0) {
      for (int i = threadIdx.x; i < Hq * (kDv / 8); i += kThreads)
        reinterpret_cast<uint4*>(p.a)[static_cast<int64_t>(b) * Hq * (kDv / 8) + i] = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; p.lse && i < Hq; i += kThreads) p.lse[static_cast<int64_t>(b) * Hq + i] = -INFINITY;
    }
  if (c0 >= c1) return;

  // --- the warp's part ----------------------------------------------------
  const int64_t f0 = min(c1, c0 + warp * part), f1 = min(c1, f0 + part);
  const int count = static_cast<int>(f1 - f0);
  const int stage_bytes = TL::stage_bytes(p.nh);
  uint8_t* rings = smem + ((2 * B + 1) * 4 + 127) / 128 * 128;
  uint8_t* ring = rings + warp * S * stage_bytes;
  const uint32_t ring_u32 = smem_u32(ring);
  // Records of the warps: of a piece begun in an earlier part, here; of one
  // begun in its own and not ended there, in the warp's ring once it is empty.
  float* begun_before = p.smem_records ? reinterpret_cast<float*>(rings + kWarps * S * stage_bytes)
                                       : p.records + (2 * gridDim.x + static_cast<int64_t>(blockIdx.x) * kWarps) * nrec;
  const auto begun_here = [&](int w) { return reinterpret_cast<float*>(rings + w * S * stage_bytes); };

  // places of the lane's chunks of 16 slots
  int koff[TL::KC / 2], voff[TL::VC / 2];
#pragma unroll
  for (int i = 0; i < TL::KC / 2; ++i) koff[i] = TL::k_at((i * 32 + lane) / TL::KC, (i * 32 + lane) % TL::KC);
#pragma unroll
  for (int i = 0; i < TL::VC / 2; ++i)
    voff[i] = TL::K_BYTES + TL::v_at((i * 32 + lane) / TL::VC, (i * 32 + lane) % TL::VC);

  Unit mine{};           // lane i: unit batch + i of the part
  int batch = -32, to = 0;   // the stage to fill
  const auto issue = [&](int f) {
    if (f < count) {
      if (f - batch >= 32) {
        batch = f;
        if (batch + lane < count) mine = locate<kWindow, TL>(pl, p, f0 + batch + lane, st);
      }
      const int who = f - batch;
      const uint32_t s0 = ring_u32 + to * stage_bytes;
      const int valid = __shfl_sync(0xffffffffu, mine.valid, who);
      const bool first = f == 0 || __shfl_sync(0xffffffffu, kWindow ? mine.first : mine.u == 0, who);
      const int hole = kWindow ? __shfl_sync(0xffffffffu, mine.hole, who) : 0;
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int row = __shfl_sync(0xffffffffu, mine.row[s], who);
        const int live = row < 0 ? 0 : valid - 16 * s;   // live rows of this half
        const int64_t at = row < 0 ? 0 : row;
        const uint8_t* ks = p.c.k + at * (D * TL::ES) + lane * 16;
        const uint8_t* vs = p.c.v + at * (kDv * TL::ES) + lane * 16;
        const uint32_t dk = s0 + s * (16 * D * TL::ES), dv = s0 + s * (16 * kDv * TL::ES);
        if (kWindow && hole != 0 && row >= 0) {
          const auto seen = [&](int r) { return r < live && (r + 16 * s < (hole & 63) || r + 16 * s >= hole >> 8); };
#pragma unroll
          for (int i = 0; i < TL::KC / 2; ++i) cp16_or_zero(dk + koff[i], ks + i * 512, seen((i * 32 + lane) / TL::KC));
#pragma unroll
          for (int i = 0; i < TL::VC / 2; ++i) cp16_or_zero(dv + voff[i], vs + i * 512, seen((i * 32 + lane) / TL::VC));
        } else if (live >= 16) {
#pragma unroll
          for (int i = 0; i < TL::KC / 2; ++i) cp16(dk + koff[i], ks + i * 512);
#pragma unroll
          for (int i = 0; i < TL::VC / 2; ++i) cp16(dv + voff[i], vs + i * 512);
        } else {   // what is not live reads as zero: 0 * NaN would be NaN
#pragma unroll
          for (int i = 0; i < TL::KC / 2; ++i) cp16_or_zero(dk + koff[i], ks + i * 512, (i * 32 + lane) / TL::KC < live);
#pragma unroll
          for (int i = 0; i < TL::VC / 2; ++i) cp16_or_zero(dv + voff[i], vs + i * 512, (i * 32 + lane) / TL::VC < live);
        }
        if (FP8 && lane < 8) {   // 16 scales of k, then of v
          const float* sc = (lane < 4 ? p.c.k_scale : p.c.v_scale) + at + (lane & 3) * 4;
          cp16_or_zero(s0 + TL::K_BYTES + TL::V_BYTES + (lane < 4 ? 0 : KS * 4) + 64 * s + (lane & 3) * 16, sc, live > 0);
        }
      }
      if (first) {   // q comes with a piece's first unit
        const int b = __shfl_sync(0xffffffffu, mine.b, who), hv = __shfl_sync(0xffffffffu, mine.hv, who);
        const int h = hv / p.chunks, ch0 = (hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
        constexpr int QC = D / 8;
        for (int i = lane; i < nh * QC; i += 32)
          cp16(s0 + TL::K_BYTES + TL::V_BYTES + TL::SCALE_BYTES + TL::META_BYTES + i * 16,
               p.q + (static_cast<int64_t>(h * p.G + ch0 + i / QC) * B + b) * D + (i % QC) * 8);
      }
      if (lane == who) {
        const int flags = mine.valid | (first ? 64 : 0) | (mine.row[0] >= 0 ? 128 : 0) | (mine.row[1] >= 0 ? 256 : 0) |
                          (kWindow ? (mine.first ? 512 : 0) | mine.hole << 16 : 0);
        *reinterpret_cast<int4*>(ring + to * stage_bytes + TL::K_BYTES + TL::V_BYTES + TL::SCALE_BYTES) =
            make_int4(flags, mine.u, mine.b, mine.hv);
      }
    }
    to = to + 1 == S ? 0 : to + 1;
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  // The pieces at the block's ends and at the end of the warp's part, while the
  // first loads are on their way.
  struct End {
    Piece piece;
    int first, last;   // the blocks that hold it
  };
  __shared__ End ends[2];
  if (lane == 0 && warp < 2) {
    // the block that holds unit f, from where it would be with even parts
    const auto block_of = [&](int64_t f) {
      int64_t blk = divide(f, kWarps * even);
      while (f < block_start(blk)) --blk;
      while (f >= block_start(blk + 1)) ++blk;
      return static_cast<int>(blk);
    };
    End e;
    e.piece = piece_of(pl, warp == 0 ? c0 : c1 - 1);
    e.first = e.last = blockIdx.x;
    if (e.piece.start < c0) e.first = block_of(e.piece.start);
    if (e.piece.end > c1) e.last = block_of(e.piece.end - 1);
    ends[warp] = e;
  }
  const Piece last_piece = piece_of(pl, count > 0 ? f1 - 1 : c1 - 1);

  uint4 qf[NT][D / 32];           // q of column 8 t + g: chunk c of every 32 dims
  float qmul[NT][E];              // score multipliers
  float m[NT][E], l[NT][E], mo[NT][E], o[NT][8][4];
  float* score_at[NT][E];         // where the scores of this lane's heads go, or null
  int cur_b = -1, cur_hv = -1;
  bool from_start = false;        // the piece being read begins with unit 0

  // Leaves the finished piece: the whole of it as the result, part of it as a
  // record.
  const auto flush = [&](bool to_end) {
    if (E == 1 && !FP8)   // what bf16 has left of the probabilities joins them
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        o[0][mt][0] += o[0][mt][1];
        o[0][mt][2] += o[0][mt][3];
      }
    const int h = cur_hv / p.chunks, ch0 = (cur_hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
    float* rec = from_start ? begun_here(warp) : begun_before + warp * nrec;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        const int n = head_of(t, e);
        if (n >= nh) continue;
        if (from_start && to_end) {
          const int64_t at = static_cast<int64_t>(cur_b) * Hq + h * p.G + ch0 + n;
          const bool none = x == 0.f;
          const float f = none ? 0.f : ex2(below(mo[t][e]) - kTop) / x;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            const uint32_t w = none ? 0u : pack_bf16x2(o[t][mt][e] * f, o[t][mt][2 + e] * f);
            if (FP8) {
              reinterpret_cast<uint32_t*>(p.a + at * kDv)[8 * mt + g] = w;
            } else {
              p.a[at * kDv + 16 * mt + g] = static_cast<uint16_t>(w);
              p.a[at * kDv + 16 * mt + g + 8] = static_cast<uint16_t>(w >> 16);
            }
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
            rec[p.nh * (kDv + 2) + n] = below(mo[t][e]) - kTop;
          }
        }
      }
  };

  int from = 0;   // the stage to read
  for (int f = 0; f < count; ++f) {
    cp_wait<S - 2>();
    __syncwarp();
    issue(f + S - 1);   // into the stage read in the last round
    const uint32_t s0 = ring_u32 + from * stage_bytes;
    from = from + 1 == S ? 0 : from + 1;
    const uint32_t sv = s0 + TL::K_BYTES, ss = sv + TL::V_BYTES, sm = ss + TL::SCALE_BYTES, sq = sm + TL::META_BYTES;
    const uint4 meta = lds128(sm);
    const int valid = meta.x & 63, u = meta.y;
    if (meta.x & 64) {
      if (f > 0) flush(true);
      cur_b = meta.z;
      cur_hv = meta.w;
      from_start = kWindow ? (meta.x & 512) != 0 : u == 0;
      const int h = cur_hv / p.chunks, ch0 = (cur_hv % p.chunks) * p.nh, nh = min(p.nh, p.G - ch0);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n = E == 1 ? g >> 1 : 8 * t + g;
        const bool head = n < nh && (E == 2 || (g & 1) == 0);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          qf[t][j] = head ? lds128(sq + n * D * 2 + j * 64 + c * 16) : make_uint4(0, 0, 0, 0);
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
          // 2^(14-e) and 2^(e-14) for am in [2^e, 2^(e+1)), from am's exponent bits, kept to normal numbers
          const int eb = min(253, max(15, static_cast<int>(__float_as_uint(am) >> 23)));
          const float down = __uint_as_float(static_cast<uint32_t>(268 - eb) << 23);
          back = __uint_as_float(static_cast<uint32_t>(eb - 14) << 23);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t w[4] = {qf[t][j].x, qf[t][j].y, qf[t][j].z, qf[t][j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
            qf[t][j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][mt][i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          qmul[t][e] = p.scale_log2 * (FP8 ? __shfl_sync(0xffffffffu, back, 8 * c + 4 * e) : 1.f);
          m[t][e] = -INFINITY;
          mo[t][e] = FP8 ? -INFINITY : 0.f;
          l[t][e] = 0.f;
          const int hn = head_of(t, e);
          score_at[t][e] = p.scores != nullptr && hn < nh
                               ? p.scores + (static_cast<int64_t>(cur_b) * Hq + h * p.G + ch0 + hn) * p.c.capacity() + g
                               : nullptr;
        }
      }
    }

    // scores of slots 16 s + g and + 8 (x[..][0, 1] and [2, 3])
    float x[NT][SUB][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][s][i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        uint32_t ka[4], kb[4];   // rows g and g + 8: dims 32 j + 8 c .. + 7
        if (FP8) {
          const uint2 ra = lds64(s0 + TL::k_at(16 * s + g, 2 * j + (c >> 1)) + (c & 1) * 8);
          const uint2 rb = lds64(s0 + TL::k_at(16 * s + g + 8, 2 * j + (c >> 1)) + (c & 1) * 8);
          const uint2 a0 = e4m3x4_to_f16x4(ra.x), a1 = e4m3x4_to_f16x4(ra.y);
          const uint2 b0 = e4m3x4_to_f16x4(rb.x), b1 = e4m3x4_to_f16x4(rb.y);
          ka[0] = a0.x, ka[1] = a0.y, ka[2] = a1.x, ka[3] = a1.y;
          kb[0] = b0.x, kb[1] = b0.y, kb[2] = b1.x, kb[3] = b1.y;
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

    // The row scales: of k into the multiplier, of v as a logarithm (E4M3);
    // what is not live gets the score -inf.
    float ks[SUB][2], lv[SUB][2];
    bool live[SUB][2];
#pragma unroll
    for (int s = 0; s < SUB; ++s)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = 16 * s + 8 * r + g;
        live[s][r] = i < valid && (meta.x & (s == 0 ? 128 : 256));
        if (kWindow) live[s][r] = live[s][r] && (i < static_cast<int>(meta.x >> 16 & 63) || i >= static_cast<int>(meta.x >> 24));
        if (FP8) {
          ks[s][r] = lds32(ss + i * 4);
          lv[s][r] = __log2f(lds32(ss + KS * 4 + i * 4));
        }
      }

    uint32_t pb[NT][SUB][2];   // the probabilities as the second product's operand
    uint32_t rest[NT][2];      // and what bf16 leaves of them, where they fill the tile
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[SUB][4];   // E4M3: the score relative to the maximum, plus log2 of v's row scale
      float next[E];     // the maximum with this unit
      bool grows = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float top = m[t][e];
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float& v = x[t][s][2 * r + e];
            v = live[s][r] ? v * (FP8 ? qmul[t][e] * ks[s][r] : qmul[t][e]) : -INFINITY;
            top = fmaxf(top, v);
            if (score_at[t][e] && 16 * s + 8 * r + g < valid) score_at[t][e][u * KS + 16 * s + 8 * r] = v;
          }
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        next[e] = top;
        grows |= top > m[t][e];
      }
      float otop[E];
      if (FP8) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          otop[e] = mo[t][e] + (m[t][e] - below(next[e]));
#pragma unroll
          for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& v = y[s][2 * r + e];
              v = live[s][r] ? x[t][s][2 * r + e] - below(next[e]) + lv[s][r] : -INFINITY;
              otop[e] = fmaxf(otop[e], v);
            }
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) otop[e] = fmaxf(otop[e], __shfl_xor_sync(0xffffffffu, otop[e], s));
          grows |= otop[e] > mo[t][e];
        }
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float fall = m[t][e] - below(next[e]), fl = ex2(fall);
          const float fo = FP8 ? ex2(fall + (mo[t][e] - below(otop[e]))) : fl;
          l[t][e] *= fl;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[t][mt][e] *= fo;
            o[t][mt][2 + e] *= fo;
            if (E == 1 && !FP8) {
              o[t][mt][1] *= fo;
              o[t][mt][3] *= fo;
            }
          }
          m[t][e] = next[e];
          if (FP8) mo[t][e] = otop[e];
        }
      }
      float w[SUB][4];
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = i & 1;
          if (e >= E) {
            w[s][i] = FP8 ? 0.f : bf16_rest(w[s][i - 1]);
            continue;
          }
          const float pr = ex2(x[t][s][i] - below(m[t][e]));
          l[t][e] += pr;
          w[s][i] = FP8 ? ex2(y[s][i] - (below(mo[t][e]) - kTop)) : pr;
        }
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w0 = w[s][2 * r], w1 = w[s][2 * r + 1];
          pb[t][s][r] = movmatrix_trans(FP8 ? pack_f16x2(w0, w1) : pack_bf16x2(bf16_below(w0), E == 1 ? w1 : bf16_below(w1)));
          if (!FP8 && E == 2) rest[t][r] = movmatrix_trans(pack_bf16x2(bf16_rest(w0), bf16_rest(w1)));
        }
    }

#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint32_t r[4];
      if (FP8) {
        // eight slots x 16 columns each: columns 2 g and 2 g + 1 of slots 2 c and 2 c + 1
        ldmatrix4_trans(r, sv + TL::v_at(lane, mt));
        uint2 w[4];   // .x column 2 g, .y column 2 g + 1
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e4m3x4_to_f16x4(__byte_perm(r[i], 0, 0x3120));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int s = 0; s < SUB; ++s)
            mma16816<true>(o[t][mt], w[2 * s].x, w[2 * s].y, w[2 * s + 1].x, w[2 * s + 1].y, pb[t][s][0], pb[t][s][1]);
      } else {
        // slots 0-7 and 8-15, columns 16 mt .. + 7 and + 8 .. + 15
        ldmatrix4_trans(r, sv + TL::v_at((lane & 7) + (lane >> 4) * 8, 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<false>(o[t][mt], r[0], r[1], r[2], r[3], pb[t][0][0], pb[t][0][1]);
          if (E == 2)
            mma16816<false>(o[t][mt], r[0], r[1], r[2], r[3], rest[t][0], rest[t][1]);
        }
      }
    }
  }
  cp_wait<0>();
  __syncwarp();   // the ring is read: a record may take its place

  // --- joining ------------------------------------------------------------
  if (count > 0) flush(last_piece.end == f1);
  __syncthreads();
  allow_dependents();
  const Piece &head = ends[0].piece, &tail = ends[1].piece;
  const int part32 = static_cast<int>(part);   // (a block's parts together are below 2^31 units)
  const auto warp_of = [&](int64_t f) { return static_cast<int>(static_cast<unsigned int>(f - c0) / part32); };
  const auto join_warps = [&](const Piece& pc, int n) {   // the records of one piece in this block
    const int wa = pc.start <= c0 ? 0 : warp_of(pc.start), wb = warp_of(min(pc.end, c1) - 1);
    const bool begins = pc.start >= c0;
    return join_records(AnyLoad{}, [&](int i) { return i == 0 && begins ? begun_here(wa) : begun_before + (wa + i) * nrec; },
                        wb - wa + 1, n, p.nh);
  };
  const auto heads_in = [&](const Piece& pc) { return min(p.nh, p.G - (pc.hv % p.chunks) * p.nh); };
  const auto head_at = [&](const Piece& pc, int n) { return pc.hv / p.chunks * p.G + (pc.hv % p.chunks) * p.nh + n; };

  // Pieces that reach over the block's ends (one that covers it counts as the
  // first): one record of the block for each, then the count of arrivals.
  const bool over0 = head.start < c0, over1 = tail.start >= c0 && tail.end > c1;
  __shared__ int is_last[2];
  if (over0 || over1) {
    const int n0 = over0 ? heads_in(head) : 0, n1 = over1 ? heads_in(tail) : 0;
    for (int i = warp; i < n0 + n1; i += kWarps) {
      const bool second = i >= n0;
      const int n = second ? i - n0 : i;
      join_warps(second ? tail : head, n).store(p.records + (2 * blockIdx.x + second) * static_cast<int64_t>(nrec), n, p.nh);
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      is_last[threadIdx.x] = 0;
      if (threadIdx.x == 0 ? over0 : over1) {
        const unsigned int blocks = ends[threadIdx.x].last - ends[threadIdx.x].first + 1;
        unsigned int* cnt = p.arrived + ends[threadIdx.x].first;
        if (count_arrival(cnt) == blocks - 1) {   // releases the block's record, acquires the others'
          is_last[threadIdx.x] = 1;
          *cnt = 0;
        }
      }
    }
  }
  // meanwhile, pieces begun in this warp's part and ended in another's of the block
  if (count > 0 && last_piece.start >= f0 && last_piece.end > f1 && last_piece.end <= c1)
    for (int n = 0; n < heads_in(last_piece); ++n) {
      const Joined j = join_warps(last_piece, n);
      write_head(p, last_piece.b, head_at(last_piece, n), j.m, j.l, j.mo, j.o);
    }
  if (!over0 && !over1) return;
  __syncthreads();
  float* parts = reinterpret_cast<float*>(rings);   // the warps' records are joined
  for (int side = 0; side < 2; ++side) {
    if (!is_last[side]) continue;
    const Piece& pc = side == 0 ? head : tail;
    const int b0 = ends[side].first, nb = ends[side].last - b0 + 1, nh = heads_in(pc);
    // a warp per head, or with many records and few heads, several
    const int split = nb > 8 ? max(1, kWarps / nh) : 1, each = (nb + split - 1) / split;
    for (int i = warp; i < nh * split; i += kWarps) {
      const int n = i / split, r0 = (i % split) * each, r1 = min(nb, r0 + each);
      const Joined j = join_records(
          L2Load{}, [&](int r) { return p.records + (2 * (b0 + r0 + r) + (r0 + r == 0)) * static_cast<int64_t>(nrec); }, r1 - r0, n, p.nh);
      if (split == 1)
        write_head(p, pc.b, head_at(pc, n), j.m, j.l, j.mo, j.o);
      else
        j.store(parts + i * record_floats(1), 0, 1);
    }
    if (split > 1) {
      __syncthreads();
      for (int n = warp; n < nh; n += kWarps) {
        const Joined j = join_records(AnyLoad{}, [&](int i) { return parts + (n * split + i) * record_floats(1); }, split, 0, 1);
        write_head(p, pc.b, head_at(pc, n), j.m, j.l, j.mo, j.o);
      }
      __syncthreads();   // before the other side's
    }
  }
}

// weight += the probabilities of the head's query heads.  Four slots a thread:
// a page and the row of scores both begin on 16 of them.
template <bool kWindow>
__global__ void __launch_bounds__(kWeightThreads) decode_weight_kernel(const __grid_constant__ DecodeParams p, DevStatus st) {
  const int h = blockIdx.y, b = blockIdx.z, Hq = p.c.H * p.G, i0 = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
  // What the attention does not write is read ahead of its end, from L2 (which
  // the kernels before it have left up to date; it has waited for them).
  const int n = checked_length<true>(p.c, b, st, KID_DECODE_WEIGHT);
  // Under a window only the units that the attention has read count (a slot in
  // them that is not seen has the score -inf).
  const int shift = p.c.k_scale ? 5 : 4;
  const Seen se = !kWindow ? Seen{} : p.c.k_scale ? seen_units<true, 32>(p, n) : seen_units<true, 16>(p, n);
  const int end = kWindow ? min(n, se.count << shift) : n;   // of the slots as they are counted here
  const auto slot_of = [&](int i) { return kWindow && i >> shift >= se.sinks ? i + (se.skip << shift) : i; };
  const auto row_of = [&](int i) { return i < end && slot_of(i) < n ? cache_row<true>(p.c, b, h, slot_of(i), st, KID_DECODE_WEIGHT) : -1; };
  const auto weights_at = [&](int row) {
    return row >= 0 ? __ldcg(reinterpret_cast<const float4*>(p.c.weight + row)) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  int row = row_of(i0);
  float4 old = weights_at(row);
  wait_for_previous();
  const int64_t head = static_cast<int64_t>(b) * Hq + h * p.G;
  for (int i = i0; i < end; i += gridDim.x * blockDim.x * 4) {
    if (i > i0) {
      row = row_of(i);
      old = weights_at(row);
    }
    if (row < 0) continue;
    const int slot = slot_of(i);
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < p.G; ++g) {
      const float z = __ldcg(p.lse2 + head + g);
      const float4 s = __ldcg(reinterpret_cast<const float4*>(p.scores + (head + g) * p.c.capacity() + slot));
      w.x += exp2_below(s.x, z);
      w.y += exp2_below(s.y, z);
      w.z += exp2_below(s.z, z);
      w.w += exp2_below(s.w, z);
    }
    float* at = p.c.weight + row;
    if (slot + 3 < n) {
      *reinterpret_cast<float4*>(at) = make_float4(old.x + w.x, old.y + w.y, old.z + w.z, old.w + w.w);
    } else {   // what lies past the length stays as it is
      at[0] = old.x + w.x;
      if (slot + 1 < n) at[1] = old.y + w.y;
      if (slot + 2 < n) at[2] = old.z + w.z;
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
template <int D, bool FP8, bool kWindow, int NT, int E, int W, int S>
cudaError_t launch_decode_s(const DecodeParams& p, int grid, int smem, DevStatus st, cudaStream_t s) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(decode_kernel<D, FP8, kWindow, NT, E, W, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev].store(true, std::memory_order_relaxed);
  }
  return launch_dependent(decode_kernel<D, FP8, kWindow, NT, E, W, S>, dim3(grid), 32 * W, smem, s, p, st);
}

// Shared memory of W warps with S stages; with the warps' records where they
// fit.
template <int D, bool FP8, int NT, int E, int W, int S>
bool fits(DecodeParams& p, int* smem) {
  *smem = ((2 * p.c.B + 1) * 4 + 127) / 128 * 128 + W * S * Tile<D, FP8>::stage_bytes(p.nh);
  if (*smem > kSmemMax) return false;
  const int recs = W * record_floats(p.nh) * 4;
  p.smem_records = *smem + recs <= kSmemMax;
  if (p.smem_records) *smem += recs;
  return true;
}

template <int D, bool FP8, bool kWindow>
cudaError_t launch_decode(DecodeParams& p, int grid, DevStatus st, cudaStream_t s) {
  int smem;
  if (p.nh <= 4) {
    // Twelve warps with two stages against eight with three: 104.0 / 106.8 us
    // (64 sequences up to 8191 tokens), 58.1 / 60.6 us (48 of E4M3): each warp's
    // chain of dependent steps is what the others have to cover.
    if (fits<D, FP8, 1, 1, 12, 2>(p, &smem)) return launch_decode_s<D, FP8, kWindow, 1, 1, 12, 2>(p, grid, smem, st, s);
    fits<D, FP8, 1, 1, 8, 2>(p, &smem);   // beside the list of very many sequences
    return launch_decode_s<D, FP8, kWindow, 1, 1, 8, 2>(p, grid, smem, st, s);
  }
  if (p.nh <= 8) {
    // Likewise for bf16 (32 sequences of 6001 slots, 4 x 8 heads: d_qk = 64 57.2 /
    // 61.7 us, 96 69.4 / 77.2); E4M3 would spill at twelve warps (57.4 / 49.6).
    if constexpr (!FP8)
      if (fits<D, FP8, 1, 2, 12, 2>(p, &smem)) return launch_decode_s<D, FP8, kWindow, 1, 2, 12, 2>(p, grid, smem, st, s);
    if (fits<D, FP8, 1, 2, 8, 3>(p, &smem)) return launch_decode_s<D, FP8, kWindow, 1, 2, 8, 3>(p, grid, smem, st, s);
    fits<D, FP8, 1, 2, 8, 2>(p, &smem);
    return launch_decode_s<D, FP8, kWindow, 1, 2, 8, 2>(p, grid, smem, st, s);
  }
  fits<D, FP8, 2, 2, 8, 2>(p, &smem);
  return launch_decode_s<D, FP8, kWindow, 2, 2, 8, 2>(p, grid, smem, st, s);
}

}  // namespace
}  // namespace qkvp
