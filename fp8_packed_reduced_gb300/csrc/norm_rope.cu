// Rows of a packed projection, y [T, N] = q heads, k heads, v heads side by
// side, into head-major q, k and v, and back:
//   forward   r = (mean x^2 + eps)^-1/2,  q, k = R(x r gain),  v = x
//   backward  g = R^T(dq),  dgain = sum g x r,
//             dx = r (g gain - x r mean(g gain x r)),  dv as it is
// with R the rotation of the pairs (i, i + d / 2) by their angles.  Sums, r and
// the gains' gradients are float; rounded to bf16 (2^-8) are the results only.
//
// Each value is read once and written once, so memory is the bound, and what it
// takes is enough bytes under way: a thread's rows come into shared memory by its
// own asynchronous copies, a few rows ahead, with no registers held and nothing to
// wait for but these.  Measured with 49152 tokens of 6 + 6 + 6 heads, d = 96
// (warm; bytes at the rate of a copy: 56 / 73 us), forward / gradient with gains:
//   rows loaded as they are needed, two at a time        109 / 187 us
//   three (two) rows at a time, 5 (4) blocks of 128       74 / 105
//   rows ahead in shared memory, pairs of floats          62 / 104
//   rstd among them                                            93
//   even turns instead of a range of tokens for a block        88
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
  int chunk_rows;           // (backward) the most rows of a chunk
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

constexpr int kThreads = 128;
// Blocks a multiprocessor and rows held for a thread.  (Forward: 5 to 8 blocks, 3
// to 8 rows are within 3 %.  Backward: 4 blocks 97 us instead of 93; 6 leave too few
// registers, 117.  More rows change nothing.)
constexpr int kForwardBlocks = 7, kForwardSlots = 4, kBackwardBlocks = 5, kBackwardSlots = 3;
constexpr int kNormHeader = 1024;   // of the workspace: the status word
constexpr int kMaxNormBlocks = 2048;

// A token takes GROUP lanes; lane c < d / 16 has columns 8 c .. 8 c + 7 and the
// same of the second half, that is, eight pairs.
template <int D>
struct Lanes {
  static constexpr int GROUP = D == 64 ? 4 : 8, USED = D / 16;
  static constexpr int TOKENS = kThreads / GROUP;   // of a block
};

// A value that nothing reads again.
__device__ __forceinline__ uint4 load_once(const uint4* p) { return __ldcs(p); }
template <int GROUP>
__device__ __forceinline__ float group_add(float v) {
#pragma unroll
  for (int o = 1; o < GROUP; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void unpack_f2(f2 (&x)[4], uint4 w) {
  x[0] = f2_from_bf16x2(w.x), x[1] = f2_from_bf16x2(w.y), x[2] = f2_from_bf16x2(w.z), x[3] = f2_from_bf16x2(w.w);
}
__device__ __forceinline__ uint4 pack_f2(const f2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}

// Cosines and sines of the lane's eight pairs.
__device__ __forceinline__ void load_turn(const NormArgs& p, int t, int c, f2 (&cs)[4], f2 (&sn)[4], const DevStatus& st, int kid) {
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
    cs[i] = f2_make(e.x, e.y);
    sn[i] = f2_make(e.z, e.w);
  }
}

__device__ __forceinline__ void load_gain(const float* gain, int D, int c, f2 (&lo)[4], f2 (&hi)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2* at = reinterpret_cast<const float2*>(gain + 8 * c) + i;
    const float2 one = make_float2(1.f, 1.f), a = gain ? __ldg(at) : one, b = gain ? __ldg(at + D / 4) : one;
    lo[i] = f2_make(a.x, a.y);
    hi[i] = f2_make(b.x, b.y);
  }
}

// Rows first .. last - 1 of v, copied between y's form and the head-major one.
template <int D, bool BACK>
__device__ __forceinline__ void copy_v(const NormArgs& p, int t, int c, int64_t N, int first, int last) {
  constexpr int GROUP = Lanes<D>::GROUP, EACH = 16 / GROUP, BATCH = 8 / EACH;
  const int64_t col = static_cast<int64_t>(p.Hq + p.H) * D, row = static_cast<int64_t>(p.T) * kDv;
  const uint16_t* from = BACK ? p.dv + static_cast<int64_t>(t) * kDv : p.y + t * p.ldy + col;
  uint16_t* to = BACK ? p.dy + t * N + col : p.v + static_cast<int64_t>(t) * kDv;
  const int64_t from_step = BACK ? row : kDv, to_step = BACK ? kDv : row;
#pragma unroll 1
  for (int h = first; h < last; h += BATCH) {
    uint4 w[BATCH][EACH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (h + b < last) w[b][i] = load_once(reinterpret_cast<const uint4*>(from + (h + b) * from_step) + i * GROUP + c);
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (h + b < last) reinterpret_cast<uint4*>(to + (h + b) * to_step)[i * GROUP + c] = w[b][i];
  }
}

// Heads are cut into gridDim.y parts where the tokens alone do not fill the GPU.
__device__ __forceinline__ void head_part(const NormArgs& p, int& first, int& last) {
  const int rows = p.Hq + 2 * p.H, each = (rows + gridDim.y - 1) / gridDim.y;
  first = min(rows, static_cast<int>(blockIdx.y) * each);
  last = min(rows, first + each);
}

// Rows on their way to a thread: SLOTS places of PARTS words of 16 bytes that are
// its own, so that nothing but its own copies has to be waited for.
template <int PARTS, int SLOTS>
struct Ring {
  uint4 words[SLOTS][PARTS][kThreads];
  __device__ __forceinline__ void bring(int at, int part, const uint4* from) {
    cp16(smem_u32(&words[at % SLOTS][part][threadIdx.x]), from);
  }
  __device__ __forceinline__ uint4 get(int at, int part) const { return words[at % SLOTS][part][threadIdx.x]; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, kForwardBlocks) norm_rope_kernel(const __grid_constant__ NormArgs p, DevStatus st) {
  using L = Lanes<D>;
  constexpr int SLOTS = kForwardSlots;
  __shared__ Ring<2, SLOTS> ring;
  wait_for_previous();
  const int c = threadIdx.x % L::GROUP;
  const int t = blockIdx.x * L::TOKENS + threadIdx.x / L::GROUP;
  const bool real = t < p.T, used = real && c < L::USED;
  const int64_t N = static_cast<int64_t>(p.Hq + p.H) * D + static_cast<int64_t>(p.H) * kDv;
  int first, last;
  head_part(p, first, last);
  const int end = min(last, p.Hq + p.H);   // of the rows of q and k
  const uint16_t* y = p.y + t * p.ldy + 8 * c;
  const auto bring = [&](int h) {
    if (used && h < end) {
      const uint4* x = reinterpret_cast<const uint4*>(y + static_cast<int64_t>(h) * D);
      ring.bring(h, 0, x);
      ring.bring(h, 1, x + D / 16);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < SLOTS - 1; ++i) bring(first + i);
  f2 cs[4], sn[4];
  if (used && first < end) load_turn(p, t, c, cs, sn, st, KID_NORM_FWD);
  const auto heads = [&](int h0, int h1, const float* gain, uint16_t* out) {
    if (h0 >= h1) return;
    f2 glo[4], ghi[4];
    load_gain(gain, D, min(c, L::USED - 1), glo, ghi);
    out += static_cast<int64_t>(t) * D + 8 * c;
#pragma unroll 1
    for (int h = h0; h < h1; ++h, out += static_cast<int64_t>(p.T) * D) {
      cp_wait<SLOTS - 2>();
      f2 lo[4], hi[4], sum = f2_make(0.f, 0.f);
      if (used) {
        unpack_f2(lo, ring.get(h, 0));
        unpack_f2(hi, ring.get(h, 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = f2_fma(hi[i], hi[i], f2_fma(lo[i], lo[i], sum));
      }
      bring(h + SLOTS - 1);
      const float2 s2 = f2_split(sum);
      const float r = 1.f / sqrtf(group_add<L::GROUP>(s2.x + s2.y) * (1.f / D) + p.eps);
      if (!used) continue;
      const f2 rr = f2_make(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 u = f2_mul(f2_mul(lo[i], rr), glo[i]), v = f2_mul(f2_mul(hi[i], rr), ghi[i]);
        lo[i] = f2_sub(f2_mul(u, cs[i]), f2_mul(v, sn[i]));
        hi[i] = f2_fma(u, sn[i], f2_mul(v, cs[i]));
      }
      *reinterpret_cast<uint4*>(out) = pack_f2(lo);
      *reinterpret_cast<uint4*>(out + D / 2) = pack_f2(hi);
      if (c == 0) p.rstd[static_cast<int64_t>(h) * p.T + t] = r;
    }
  };
  heads(first, min(end, p.Hq), p.q_gain, p.q + static_cast<int64_t>(first) * p.T * D);
  heads(max(first, p.Hq), end, p.k_gain, p.k + static_cast<int64_t>(max(first, p.Hq) - p.Hq) * p.T * D);
  if (real) copy_v<D, false>(p, t, c, N, max(first, p.Hq + p.H) - p.Hq - p.H, last - p.Hq - p.H);
}

// Chunks [begin, end) of a kind of rows, `parts` of them a tile.  A token's cosines
// and sines are read once a chunk, but its blocks end together only if chunks are
// short: of at most 2 / 4 / 6 / 8 / 16 rows, six heads of 96 take 109 / 96 / 88 / 88 /
// 88 us, 32 + 8 heads of 128 and 32768 tokens 232 / 188 / 183 / 190 / 199.
constexpr int kChunkRows = 6;
struct Chunks {
  int count, parts, rows, begin, end;
  __device__ Chunks(int tiles, int count, int most, int begin) : count(count), begin(begin) {
    parts = (count + most - 1) / most;
    rows = (count + parts - 1) / parts;
    end = begin + tiles * parts;
  }
};
// The rows of a block's chunks: every gridDim.x-th.
struct Walk {
  const Chunks& of;
  int chunk, tile, h, last;
  __device__ explicit Walk(const Chunks& c) : of(c) {
    const int grid = static_cast<int>(gridDim.x), ahead = (static_cast<int>(blockIdx.x) - c.begin % grid + grid) % grid;
    chunk = ahead < c.end - c.begin ? c.begin + ahead : c.end;
    settle();
  }
  __device__ __forceinline__ void settle() {
    const int at = chunk - of.begin;
    tile = at / of.parts;
    h = (at - tile * of.parts) * of.rows;
    last = min(of.count, h + of.rows);
  }
  __device__ __forceinline__ bool more() const { return chunk < of.end; }
  __device__ __forceinline__ void next_chunk() {
    chunk = of.end - chunk > static_cast<int>(gridDim.x) ? chunk + static_cast<int>(gridDim.x) : of.end;
    settle();
  }
  __device__ __forceinline__ bool next() {   // whether that is another chunk's
    if (++h < last) return false;
    next_chunk();
    return true;
  }
};

template <int D, bool GAIN>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks) norm_rope_back_kernel(const __grid_constant__ NormArgs p, DevStatus st) {
  using L = Lanes<D>;
  constexpr int SLOTS = kBackwardSlots;
  __shared__ Ring<4, SLOTS> ring;
  __shared__ float rstd[SLOTS][kThreads];
  __shared__ float part[GAIN ? kThreads / 32 : 1][2][D];
  __shared__ float4 gain_of[2][D / 4];
  wait_for_previous();
  for (int i = threadIdx.x; i < D / 2; i += kThreads) {
    const float* gain = i < D / 4 ? p.q_gain : p.k_gain;
    (&gain_of[0][0])[i] = gain ? __ldg(reinterpret_cast<const float4*>(gain) + i % (D / 4)) : make_float4(1.f, 1.f, 1.f, 1.f);
  }
  __syncthreads();
  const int c = threadIdx.x % L::GROUP;
  const int64_t N = static_cast<int64_t>(p.Hq + p.H) * D + static_cast<int64_t>(p.H) * kDv;
  // The blocks take chunks (a tile of TOKENS tokens times a few rows of one kind) in
  // turn: all those of q heads, then of k heads, then of v heads.
  const int tiles = (p.T + L::TOKENS - 1) / L::TOKENS, mine = threadIdx.x / L::GROUP;
  const Chunks q_chunks(tiles, p.Hq, p.chunk_rows, 0), k_chunks(tiles, p.H, p.chunk_rows, q_chunks.end),
      v_chunks(tiles, p.H, p.chunk_rows, k_chunks.end);
  // one kind of heads after the other, so that only one gain's sums are held
  const auto heads = [&](const Chunks& chunks, int base, const uint16_t* grad, int kind) {
    f2 sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = f2_make(0.f, 0.f);
    Walk it(chunks), on(chunks);   // the row in hand, the one that is brought next
    if (it.more()) {
      const float4* gains = gain_of[kind] + 2 * c;
      int at_on = 0;
      const auto bring = [&] {
        if (on.more()) {
          const int t_on = on.tile * L::TOKENS + mine;
          if (t_on < p.T && c < L::USED) {
            const uint4* xs = reinterpret_cast<const uint4*>(p.y + t_on * p.ldy + static_cast<int64_t>(base + on.h) * D + 8 * c);
            const uint4* gs = reinterpret_cast<const uint4*>(grad + (static_cast<int64_t>(on.h) * p.T + t_on) * D + 8 * c);
            ring.bring(at_on, 0, xs);
            ring.bring(at_on, 1, xs + D / 16);
            ring.bring(at_on, 2, gs);
            ring.bring(at_on, 3, gs + D / 16);
            cp4(smem_u32(&rstd[at_on % SLOTS][threadIdx.x]), p.rstd + static_cast<int64_t>(base + on.h) * p.T + t_on);
          }
          on.next();
        }
        ++at_on;
        cp_commit();
      };
#pragma unroll 1
      for (int i = 0; i < SLOTS - 1; ++i) bring();
      f2 cs[4], sn[4];
      bool turned = false;
#pragma unroll 1
      for (int at = 0; it.more(); ++at) {
        const int t = it.tile * L::TOKENS + mine, h = it.h;
        const bool used = t < p.T && c < L::USED;
        if (used && !turned) load_turn(p, t, c, cs, sn, st, KID_NORM_BWD);
        turned = true;
        cp_wait<SLOTS - 2>();
        const float r = rstd[at % SLOTS][threadIdx.x];
        f2 lo[4], hi[4], u[4], w[4], dots = f2_make(0.f, 0.f);
        const f2 rr = f2_make(r, r);
        if (used) {
          unpack_f2(lo, ring.get(at, 0));
          unpack_f2(hi, ring.get(at, 1));
          unpack_f2(u, ring.get(at, 2));
          unpack_f2(w, ring.get(at, 3));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 m = f2_fma(w[i], sn[i], f2_mul(u[i], cs[i])), n = f2_sub(f2_mul(w[i], cs[i]), f2_mul(u[i], sn[i]));
            lo[i] = f2_mul(lo[i], rr);
            hi[i] = f2_mul(hi[i], rr);
            if (GAIN) {
              sum[i] = f2_fma(m, lo[i], sum[i]);
              sum[4 + i] = f2_fma(n, hi[i], sum[4 + i]);
            }
            u[i] = m;
            w[i] = n;
          }
#pragma unroll
          for (int i = 0; i < 4; i += 2) {   // (read for every row: held, they took 16 registers)
            const float4 a = gains[i / 2], b = gains[D / 8 + i / 2];
            u[i] = f2_mul(u[i], f2_make(a.x, a.y)), u[i + 1] = f2_mul(u[i + 1], f2_make(a.z, a.w));
            w[i] = f2_mul(w[i], f2_make(b.x, b.y)), w[i + 1] = f2_mul(w[i + 1], f2_make(b.z, b.w));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) dots = f2_fma(w[i], hi[i], f2_fma(u[i], lo[i], dots));
        }
        bring();
        const float2 d2 = f2_split(dots);
        const float dot = group_add<L::GROUP>(d2.x + d2.y) * (-1.f / D);
        if (used) {
          const f2 dd = f2_make(dot, dot);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = f2_mul(f2_fma(lo[i], dd, u[i]), rr);
            w[i] = f2_mul(f2_fma(hi[i], dd, w[i]), rr);
          }
          uint4* to = reinterpret_cast<uint4*>(p.dy + t * N + static_cast<int64_t>(base + h) * D);
          to[c] = pack_f2(u);
          to[D / 16 + c] = pack_f2(w);
        }
        turned = !it.next();
      }
    }
    if (GAIN) {   // lanes with the same columns
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = i % 2 ? f2_split(sum[i / 2]).y : f2_split(sum[i / 2]).x;
#pragma unroll
        for (int o = L::GROUP; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane < L::USED) part[threadIdx.x >> 5][kind][(i >> 3) * (D / 2) + 8 * lane + (i & 7)] = x;
      }
    }
  };
  heads(q_chunks, 0, p.dq, 0);
  heads(k_chunks, p.Hq, p.dk, 1);
  for (Walk it(v_chunks); it.more(); it.next_chunk())
    if (it.tile * L::TOKENS + mine < p.T) copy_v<D, true>(p, it.tile * L::TOKENS + mine, c, N, it.h, it.last);
  if (GAIN) {   // warps, and then (by another kernel) blocks, in a fixed order
    __syncthreads();
    float* to = p.partial + static_cast<int64_t>(blockIdx.x) * (2 * D);
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) x += part[w][i / D][i % D];
      to[i] = x;
    }
  }
}

// Sums `blocks` partials of each of 2 d columns: eight columns (a sector) a block,
// whose threads take the partials in turn.
constexpr int kSumCols = 8, kSumRows = 128;
__global__ void __launch_bounds__(kSumCols * kSumRows) gain_sum_kernel(const __grid_constant__ NormArgs p, int d, int blocks) {
  __shared__ float part[kSumRows / 4][kSumCols];
  wait_for_previous();
  const int row = threadIdx.x / kSumCols, col = threadIdx.x % kSumCols, at = blockIdx.x * kSumCols + col;
  float x = 0.f;
#pragma unroll 4
  for (int b = row; b < blocks; b += kSumRows) x += __ldcg(p.partial + static_cast<int64_t>(b) * 2 * d + at);
#pragma unroll
  for (int o = kSumCols; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);   // a warp's four rows
  if ((threadIdx.x & 31) < kSumCols) part[threadIdx.x >> 5][col] = x;
  __syncthreads();
  if (threadIdx.x >= kSumCols) return;
  x = 0.f;
#pragma unroll
  for (int w = 0; w < kSumRows / 4; ++w) x += part[w][col];
  (at < d ? p.dq_gain : p.dk_gain)[at < d ? at : at - d] = x;
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

// Parts of the heads: as many as bring the blocks to four a multiprocessor.
int head_parts(int64_t token_blocks, int rows, int sms) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, 4 * sms / std::max<int64_t>(1, token_blocks))));
}

template <int D>
cudaError_t forward(const NormArgs& a, int sms, DevStatus st, cudaStream_t s) {
  const int blocks = (a.T + Lanes<D>::TOKENS - 1) / Lanes<D>::TOKENS;
  return launch_dependent(norm_rope_kernel<D>, dim3(blocks, head_parts(blocks, a.Hq + 2 * a.H, sms)), kThreads, 0, s, a, st);
}

template <int D>
cudaError_t backward(NormArgs a, int sms, DevStatus st, cudaStream_t s) {
  // Blocks that are all on the GPU at once; shorter chunks where they would not all have one.
  const int64_t units = static_cast<int64_t>((a.T + Lanes<D>::TOKENS - 1) / Lanes<D>::TOKENS) * (a.Hq + 2 * a.H);
  const int blocks = static_cast<int>(std::min<int64_t>(units, std::min(kBackwardBlocks * sms, kMaxNormBlocks)));
  a.chunk_rows = static_cast<int>(std::min<int64_t>(kChunkRows, units / blocks));
  if (!a.partial) return launch_dependent(norm_rope_back_kernel<D, false>, dim3(blocks), kThreads, 0, s, a, st);
  const cudaError_t e = launch_dependent(norm_rope_back_kernel<D, true>, dim3(blocks), kThreads, 0, s, a, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(gain_sum_kernel, dim3(2 * D / kSumCols), kSumCols * kSumRows, 0, s, a, D, blocks);
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
