// Paged key-value cache: what its kernels share (ft_kv_append.cu,
// ft_kv_attention.cu, ft_kv_evict.cu) and the host calls of ft_kv.cu.
#pragma once

#include <atomic>

#include "ft_common.cuh"

namespace ft {

constexpr int kKvMaxSms = 160;       // SMs a launch is spread over at most; sizes the split workspace
constexpr int kKvMaxSeqs = 65536;    // rows of a block table

// A cache as the kernels take it.  Rows (one entry of one KV head) are
// numbered (page * n_kv + head) * page_size + slot: below 2^31, checked on
// the host, so a row number is an int and only byte offsets are 64-bit.
struct KvView {
  int D, Hq, Hkv, G;          // G query heads a KV head
  int page_shift, page_mask;  // page_size = 1 << page_shift
  int n_seqs, max_pages;
  int n_pages;
  int cap;                    // max_pages * page_size, the longest sequence
  float k_scale, v_scale;
  uint8_t* k;
  uint8_t* v;
  float* mass;
  int32_t* pos;
  const int32_t* table;
  int32_t* lengths;
  int* status;
};

// Length of sequence b; one out of range counts as 0 (and sets the status
// where `tell` is).
__device__ __forceinline__ int kv_length(const KvView& kv, int b, bool tell = false) {
  const int n = kv.lengths[b];
  if ((unsigned)n <= (unsigned)kv.cap) return n;
  if (tell) set_status(kv.status, kStBadId);
  return 0;
}

// Row of entry `slot` of sequence b and KV head h, or -1 (and the status)
// where the table names no page of the pool.
__device__ __forceinline__ int kv_row(const KvView& kv, int b, int h, int slot) {
  const int page = kv.table[(int64_t)b * kv.max_pages + (slot >> kv.page_shift)];
  if ((unsigned)page >= (unsigned)kv.n_pages) {
    set_status(kv.status, kStBadId);
    return -1;
  }
  return ((page * kv.Hkv + h) << kv.page_shift) + (slot & kv.page_mask);
}

__device__ __forceinline__ void kv_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void kv_pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct KvAppendArgs {
  KvView kv;
  int64_t T;
  const uint16_t *q, *k, *v;  // bf16
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu_new;
  const int32_t* positions;
  int n_axes;
  const double* inv_freq;
  const int32_t* axis;
  int rot;
  uint16_t* q_out;
};

struct KvAttnArgs {
  KvView kv;
  const uint16_t* q;  // bf16
  int64_t q_stride;
  float scale;
  uint16_t* out;
  float* lse;
  uint8_t* work;
  bool mass;
};

struct KvEvictArgs {
  KvView kv;
  const int32_t* budgets;
  int recent;
  uint8_t* work;
};

// Workspace bytes of the two calls that take one.
int64_t kv_attn_workspace(const ft_kv_cache& c);
int64_t kv_evict_workspace(const ft_kv_cache& c);

// The attention's split of `total` tiles over `sms` SMs: entries of a tile, tiles of a chunk, chunks used, chunks there are.
void kv_geometry(const ft_kv_cache& c, int total, int sms, int64_t out[4]);

cudaError_t launch_kv_append(const KvAppendArgs& a, bool e4m3, bool adjacent, int sms, cudaStream_t s);
cudaError_t launch_kv_attention(const KvAttnArgs& a, bool e4m3, int device, int sms, cudaStream_t s);
cudaError_t launch_kv_wait(int blocks, uint64_t limit_ns, int64_t arrive_ns, int32_t* lanes, cudaStream_t s);
cudaError_t launch_kv_evict(const KvEvictArgs& a, int row_bytes, int device, int sms, cudaStream_t s);

// Sets a kernel attribute once on each device (`done` has a bit for each; a second thread
// that sets it too does no harm).
template <typename F>
inline cudaError_t kv_attribute_once(std::atomic<uint64_t>& done, int device, F* kern, cudaFuncAttribute what, int value) {
  const uint64_t bit = (uint64_t)1 << (device & 63);
  if (device < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, what, value);
  if (e == cudaSuccess && device < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch with programmatic stream serialisation: the kernel may start while
// its predecessor on the stream still runs.  Every thread of every kernel here executes
// griddepcontrol.wait before it touches memory that another kernel may have
// written or still reads, so a grid ends only after all those before it.  Loads are plain
// ones for the same reason: one that is marked read-only for the whole kernel may be moved
// to before the wait.
template <typename A>
inline cudaError_t kv_launch_after(void (*kern)(const A), dim3 grid, int threads, size_t smem, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace ft
