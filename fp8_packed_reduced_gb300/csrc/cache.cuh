// The paged key-value cache as the kernels see it: pools of pages, the page
// table and the lengths, with the checks that keep every access in bounds.
#pragma once

#include <utility>

#include "common.cuh"

namespace qkvp {

// Kernel ids recorded beside an error in the status word (they continue the
// ids of KernelId).
enum CacheKernelId : int { KID_CACHE_APPEND = 13, KID_DECODE = 14, KID_DECODE_WEIGHT = 15, KID_EVICT_SELECT = 16,
                           KID_EVICT_MOVE = 17 };

constexpr int kMaxSeqs = 4096;
constexpr int kMaxPage = 256;
constexpr int kDv = 128;
// The start of every workspace: the status word, then counters that every call
// leaves at zero.  They lie at the same place whatever the call and its shape
// are, so that nothing else is ever written there.
constexpr size_t kAppendCounter = 128;      // blocks of an append that have arrived
constexpr size_t kDecodeCounters = 256;     // of an attention, for every block the piece that it ends with
constexpr int kMaxDecodeBlocks = 192;
constexpr size_t kCacheHeaderBytes = 1024;
static_assert(kDecodeCounters + kMaxDecodeBlocks * sizeof(unsigned int) <= kCacheHeaderBytes, "header too small");

struct CacheArgs {
  uint8_t* k;        // [P, H, page, d] bf16 or E4M3 codes
  uint8_t* v;        // [P, H, page, 128]
  float* k_scale;    // [P, H, page] (E4M3)
  float* v_scale;
  float* weight;     // [P, H, page], or null
  int32_t* pos;      // [P, H, page], or null
  const int32_t* table;    // [B, max_pages]
  const int32_t* lengths;  // [B]
  int P, H, B, max_pages, page_shift;
  int d;             // d_qk
  __host__ __device__ int page() const { return 1 << page_shift; }
  __host__ __device__ int capacity() const { return max_pages << page_shift; }
};

// The length of sequence b, clamped to what its pages can hold; a length
// outside [0, capacity] is recorded.  L2: past L1; else a plain load, not one
// of read-only data, since the append in place writes the lengths at its end
// (past L1 it takes 32.0 us instead of 30.9 for 23843 ragged rows x 8 heads).
template <bool L2 = false>
__device__ __forceinline__ int checked_length(const CacheArgs& c, int b, const DevStatus& st, int kid) {
  const int n = L2 ? __ldcg(c.lengths + b) : c.lengths[b], cap = c.capacity();
  if (n < 0 || n > cap) {
    record_error(st, QKVP_ERR_DEVICE_INPUT, kid);
    return n < 0 ? 0 : cap;
  }
  return n;
}

// Row (of the pools seen as [P * H * page, ...]) of slot `slot` of sequence
// b, head h; -1, recorded, when its page lies outside the pool.  The caller
// has checked 0 <= slot < capacity.
template <bool L2 = false>
__device__ __forceinline__ int cache_row(const CacheArgs& c, int b, int h, int slot, const DevStatus& st, int kid) {
  const int* at = c.table + static_cast<int64_t>(b) * c.max_pages + (slot >> c.page_shift);
  const int pid = L2 ? __ldcg(at) : __ldg(at);
  if (pid < 0 || pid >= c.P) {
    record_error(st, QKVP_ERR_DEVICE_INPUT, kid);
    return -1;
  }
  return ((pid * c.H + h) << c.page_shift) + (slot & (c.page() - 1));   // below 2^31: checked on the host
}

// A kernel launched by launch_dependent may start before the one ahead of it
// in its stream is done: when every block of that one has left or has called
// allow_dependents (a kernel of another library does not, so nothing of ours
// runs beside it).  Every thread calls wait_for_previous before it touches
// what the kernels ahead write, and before it returns.
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... KArgs, class... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Host: QKVP_OK or the status an entry point returns for `c`; fills `a`.
int check_cache(const qkvp_cache* c, CacheArgs* a);
// Multiprocessors of the current device, 0 on error.
int device_sms();

}  // namespace qkvp
