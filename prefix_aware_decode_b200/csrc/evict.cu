// Eviction of cached tokens by accumulated attention weight (pa_evict_tokens).
//
// Of the n cached tokens of a session, each kv head keeps the first `sinks`,
// the last `recent` and, of the rest, the `quota` = budget - sinks - recent with
// the highest scores, ties to the lowest index; all n when n <= budget.
//
//   select  one CTA per (session, kv head): the quota-th highest score by a
//           radix selection (8 bits a pass over a histogram in shared memory),
//           then one ordered pass that writes the kept indices and scores
//   gather  copies the kept K and V rows, in order, to the destination pages
//
// The selection is bound by its passes over the scores (L2 after the first),
// the gather by memory.
#include "ptx.cuh"
#include "sessions.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kGatherThreads = 256;

struct EvictArgs {
  Sessions b;
  const float* scores;
  int64_t max_tokens;
  const uint16_t *k_pool, *v_pool;  // read and written (other pages)
  const int32_t* dst_table;
  int dst_max_pages, budget, sinks, recent;
  float* scores_out;
  int32_t *kept, *new_lens;
};

// Order-preserving map of a score to an unsigned key: NaN above every number,
// -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int s_pick, s_rank;
  __shared__ uint32_t wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / a.b.Hkv, g = blockIdx.x % a.b.Hkv;
  const int64_t row = (int64_t)s * a.b.Hkv + g;
  const float* x = a.scores + row * a.max_tokens;
  float* out = a.scores_out + row * a.max_tokens;
  int32_t* kept = a.kept + row * a.budget;
  const int n = (int)min((int64_t)a.b.kv_len(s), a.max_tokens);
  const int n_new = min(n, a.budget);
  if (tid == 0 && g == 0) a.new_lens[s] = n_new;
  // tokens past the kept ones
  for (int64_t t = n_new + tid; t < a.max_tokens; t += kSelThreads) out[t] = 0.f;
  for (int t = n_new + tid; t < a.budget; t += kSelThreads) kept[t] = -1;
  if (n <= a.budget) {
    for (int t = tid; t < n; t += kSelThreads) {
      out[t] = x[t];
      kept[t] = t;
    }
    return;
  }
  const int lo = a.sinks, hi = n - a.recent, quota = a.budget - a.sinks - a.recent;
  uint32_t prefix = 0, mask = 0;
  int rank = quota;  // the rank-th highest key among those that match the prefix
  if (quota > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = score_key(x[t]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // bins from the highest down: lane l holds bins 255 - 8l .. 248 - 8l
        int c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;  // keys in higher bins than this lane's
        if (above < rank && above + sum >= rank) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above < rank && above + c[j] >= rank) {
              s_pick = 255 - 8 * lane - j;
              s_rank = rank - above;
            }
            above += c[j];
          }
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_pick << shift;
      mask |= 255u << shift;
      rank = s_rank;
      __syncthreads();
    }
  }
  // one ordered pass: a token stays if held, above the threshold, or among the
  // first `rank` equal to it.  Counts of both kinds in the halves of one word.
  int base = 0, ties = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads) {
    const int t = t0 + tid;
    const float f = t < n ? x[t] : 0.f;
    const bool held = t < n && (t < lo || t >= hi);
    const uint32_t key = score_key(f);
    const bool mid = t < n && !held && quota > 0;
    const bool take = held || (mid && key > prefix), tie = mid && key == prefix;
    uint32_t v = (take ? 1u : 0u) | (tie ? 0x10000u : 0u), inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      uint32_t w = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      wsum[lane] = w;
    }
    __syncthreads();
    const uint32_t exc = inc - v + (warp ? wsum[warp - 1] : 0u);
    const int tie_before = ties + (int)(exc >> 16);
    if (take || (tie && tie_before < rank)) {
      const int j = base + (int)(exc & 0xffffu) + min(tie_before, rank) - min(ties, rank);
      kept[j] = t;
      out[j] = f;
    }
    const uint32_t tot = wsum[31];
    base += (int)(tot & 0xffffu) + min(ties + (int)(tot >> 16), rank) - min(ties, rank);
    ties += (int)(tot >> 16);
    __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  constexpr int V = D / 8;  // 16-byte vectors of a row
  const int s = blockIdx.z, g = blockIdx.y;
  const int n_new = a.new_lens[s];
  const int j = blockIdx.x * (kGatherThreads / V) + threadIdx.x / V, c = threadIdx.x % V;
  if (j >= n_new || j / kPage >= a.dst_max_pages) return;
  const int t = a.kept[((int64_t)s * a.b.Hkv + g) * a.budget + j];
  const int sp = a.b.page(s, t / kPage), dp = a.dst_table[(size_t)s * a.dst_max_pages + j / kPage];
  if (sp < 0 || (unsigned)dp >= (unsigned)a.b.num_pages) return;
  const size_t from = (((size_t)sp * a.b.Hkv + g) * kPage + t % kPage) * D + 8 * c;
  const size_t to = (((size_t)dp * a.b.Hkv + g) * kPage + j % kPage) * D + 8 * c;
  const uint4 x = *reinterpret_cast<const uint4*>(a.k_pool + from);
  const uint4 y = *reinterpret_cast<const uint4*>(a.v_pool + from);
  *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.k_pool) + to) = x;
  *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.v_pool) + to) = y;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_evict_tokens(const pa_sessions* b, const float* scores, int64_t max_tokens, void* k_pool,
                                     void* v_pool, const int32_t* d_dst_table, int32_t dst_max_pages, int32_t budget,
                                     int32_t sinks, int32_t recent, float* scores_out, int32_t* kept,
                                     int32_t* new_lens, void* stream) {
  const pa_status st = pa_check_sessions(b, false);
  if (st != PA_OK) return st;
  if (!scores || !k_pool || !v_pool || !d_dst_table || !scores_out || !kept || !new_lens || scores == scores_out)
    return PA_ERR_INVALID;
  if (max_tokens < 1 || budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget ||
      dst_max_pages < 1 || (int64_t)dst_max_pages * pa::kPage < budget)
    return PA_ERR_INVALID;
  if (!pa_aligned16(k_pool) || !pa_aligned16(v_pool)) return PA_ERR_INVALID;
  pa::EvictArgs a{};
  a.b = pa_device_sessions(*b);
  a.scores = scores;
  a.max_tokens = max_tokens;
  a.k_pool = static_cast<const uint16_t*>(k_pool);
  a.v_pool = static_cast<const uint16_t*>(v_pool);
  a.dst_table = d_dst_table;
  a.dst_max_pages = dst_max_pages;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.scores_out = scores_out;
  a.kept = kept;
  a.new_lens = new_lens;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  pa::evict_select_kernel<<<b->n_sessions * b->num_kv_heads, pa::kSelThreads, 0, cs>>>(a);
  const int rows = pa::kGatherThreads / (b->head_dim / 8);
  const int64_t span = (int64_t)b->max_pages * pa::kPage;
  const int most = (int)(span < budget ? span : budget);
  const dim3 grid((most + rows - 1) / rows, b->num_kv_heads, b->n_sessions);
  if (b->head_dim == 64) pa::evict_gather_kernel<64><<<grid, pa::kGatherThreads, 0, cs>>>(a);
  else pa::evict_gather_kernel<128><<<grid, pa::kGatherThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
