// What the session-cache operators share: the batch of sessions as the device
// sees it, the lookup of a row's session, and the rule of visibility.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "pa.h"
#include "ptx.cuh"

namespace pa {

constexpr int kPage = 16;  // tokens of a page

// A pa_sessions by value, with the pools' head layout.  Every index read from
// the device arrays is clamped or range-checked where it is read, so that no
// content of theirs leads out of a buffer.
struct Sessions {
  int S, rows, Hq, Hkv, max_pages, num_pages;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu_rows;

  __device__ __forceinline__ int kv_len(int s) const { return min(max(kv_lens[s], 0), max_pages * kPage); }
  __device__ __forceinline__ int row_begin(int s) const { return min(max(cu_rows[s], 0), rows); }
  // The page of logical page j of session s; -1: a hole (an id outside the pool)
  __device__ __forceinline__ int page(int s, int j) const {
    const int p = table[(size_t)s * max_pages + j];
    return (unsigned)p < (unsigned)num_pages ? p : -1;
  }
};

// A row at cached position p sees token t of its session.
struct Window {
  int window, sinks;  // window 0: no limit
  __device__ __forceinline__ bool sees(int p, int t) const {
    return t <= p && (window == 0 || t > p - window || t < sinks);
  }
  // first token past the sinks that a row at position p sees (0 without a window)
  __device__ __forceinline__ int first(int p) const { return window == 0 ? 0 : max(0, p - window + 1); }
};

// The session whose rows contain row r (a whole warp asks; every lane gets the
// answer): the last s with cu_rows[s] <= r.  A 32-way search, so one round
// trip for up to 32 sessions and two for up to 1024.
__device__ __forceinline__ int warp_find_session(const Sessions& b, int r, int lane) {
  int lo = 0, n = b.S;  // cu_rows[lo] <= r, the answer in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int j = lo + lane * step;
    const bool le = lane == 0 || (j < lo + n && b.cu_rows[j] <= r);
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = 31 - __clz(m);
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// A cluster of CTAs and its shared memory.
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// A word of this CTA's shared memory as CTA `rank` of the cluster has it.
template <typename T>
__device__ __forceinline__ T cluster_read(const T* p, unsigned rank) {
  static_assert(sizeof(T) == 4);
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return *reinterpret_cast<T*>(&v);
}

}  // namespace pa

// Host side: the rule of visibility.  Positions are below 2^30, so wider windows
// and more sinks mean the same, and sums with them stay inside 32 bits.
inline pa::Window pa_window(int32_t window, int32_t sinks) {
  constexpr int32_t most = 1 << 30;
  return pa::Window{window < most ? window : most, sinks < most ? sinks : most};
}

// A softmax scale whose product with log2 e, which the kernels scale by, is finite too
// (0 times an infinity would be NaN).
inline bool pa_scale_ok(float scale) { return scale >= 0.f && scale <= 2.3e38f; }

// Checks of a pa_sessions that every operator makes.  `rows`: the
// operator uses the rows of the batch (cu_rows).
inline pa_status pa_check_sessions(const pa_sessions* b, bool rows) {
  if (!b || b->n_sessions < 1 || b->max_pages < 1 || b->num_pages_in_pool < 1 || b->num_q_heads < 1 ||
      b->num_kv_heads < 1 || !b->d_block_table || !b->d_kv_lens)
    return PA_ERR_INVALID;
  if (b->num_q_heads % b->num_kv_heads || b->n_sessions > 65535 || b->num_kv_heads > 65535) return PA_ERR_INVALID;
  if ((int64_t)b->n_sessions * b->num_kv_heads > INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
  if (rows && (b->num_rows < 0 || !b->d_cu_rows)) return PA_ERR_INVALID;
  if (b->page_size != pa::kPage || !(b->head_dim == 64 || b->head_dim == 128)) return PA_ERR_UNSUPPORTED;
  const int G = b->num_q_heads / b->num_kv_heads;
  if (!(G == 1 || G == 2 || G == 4 || G == 8)) return PA_ERR_UNSUPPORTED;
  // token indices and pool rows are 32-bit
  if ((int64_t)b->max_pages * pa::kPage > INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
  if ((int64_t)b->num_pages_in_pool * b->num_kv_heads * pa::kPage > INT32_MAX) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

inline pa::Sessions pa_device_sessions(const pa_sessions& b) {
  return pa::Sessions{b.n_sessions, b.num_rows,      b.num_q_heads, b.num_kv_heads, b.max_pages, b.num_pages_in_pool,
                      b.d_block_table, b.d_kv_lens, b.d_cu_rows};
}

inline bool pa_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Dynamic shared memory of a kernel, allowed once per device (`done`: a bit per device).
template <typename K>
bool pa_allow_smem(K* kernel, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// The current device and its SMs (148 without a device).
struct pa_device {
  int index = -1, sms = 148;
};
inline pa_device pa_current_device() {
  static std::atomic<int> known[64];
  pa_device d;
  if (cudaGetDevice(&d.index) != cudaSuccess) {
    cudaGetLastError();
    return d;
  }
  const bool slot = d.index >= 0 && d.index < 64;
  const int n = slot ? known[d.index].load(std::memory_order_relaxed) : 0;
  if (n > 0) {
    d.sms = n;
  } else if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.index) == cudaSuccess && slot) {
    known[d.index].store(d.sms, std::memory_order_relaxed);
  }
  return d;
}

// The wait that the thread's next call gives up (pa_session_fault), taken once.
inline thread_local int32_t pa_fault = 0;
inline int32_t pa_take_fault() {
  const int32_t wait = pa_fault;
  pa_fault = 0;
  return wait;
}

// Reads the first-failure word of the current device (a __device__ array of four)
// and clears it when it tells of one; synchronises the stream.
template <typename W>
pa_status pa_take_status(const W& words, cudaStream_t cs, pa_status* out) {
  void* word = nullptr;
  int32_t v = 0;
  if (cudaGetSymbolAddress(&word, words) != cudaSuccess ||
      cudaMemcpyAsync(&v, word, 4, cudaMemcpyDeviceToHost, cs) != cudaSuccess || cudaStreamSynchronize(cs) != cudaSuccess)
    return PA_ERR_CUDA;
  if (v != 0 && cudaMemsetAsync(word, 0, sizeof(W), cs) != cudaSuccess) return PA_ERR_CUDA;
  *out = static_cast<pa_status>(v);
  return PA_OK;
}

// Launch of a kernel that begins with griddep_wait (before it touches memory): it
// may be brought up while the kernel before it on the stream still runs.
template <typename... P, typename... A>
bool pa_launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                     const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}
