// Eviction of cached tokens by accumulated attention weight (pa_evict_tokens).
//
// Of the n cached tokens of a session, each kv head keeps the first `sinks`,
// the last `recent` and, of the rest, the `quota` = budget - sinks - recent with
// the highest scores, ties to the lowest index; all n when n <= budget.
//
//   select  a cluster of CTAs per (session, kv head), each with a run of the
//           tokens whose order-preserving keys it holds in shared memory (re-read
//           from memory when they do not fit): the quota-th highest key by a radix
//           selection, 11 + 11 + 10 bits, over histograms that the cluster adds up
//           through distributed shared memory (the scores' exponents are few, so
//           8-bit digits made lanes collide; and one copy per four warps); then
//           every warp counts what it keeps of its run, and with the counts before
//           it writes the kept indices and scores in order.  Up to 512 tokens,
//           one a thread, are ranked by comparing each with all
//   gather  copies the kept K and V rows, in order, to the destination pages (zeros for
//           a kept token whose page is a hole)
//
// The selection reads the scores once; the gather, which moves the bytes, is
// bound by memory.  Measured, 16 sessions of 20000-32768 tokens, 8 heads of 128, to
// 4096: selection 34 us, bound by the ALU and shared memory work of its passes;
// gather 92 us for 0.5 GB (5.5 TB/s); the call 127 us.
#include <type_traits>

#include "ptx.cuh"
#include "sessions.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kRankMax = 512;  // most tokens of a row that are ranked by comparison
constexpr int kGatherThreads = 256;
constexpr int kKeysMax = 32768;  // keys that a CTA holds in shared memory (128 KB)
constexpr int kBins = 2048, kCopies = 8;

struct EvictArgs {
  Sessions b;
  const float* scores;
  int64_t max_tokens;
  const uint16_t *k_pool, *v_pool;  // read and written (other pages)
  const int32_t* dst_table;
  int dst_max_pages, budget, sinks, recent;
  float* scores_out;
  int32_t *kept, *new_lens;
  int held_keys;  // keys that the launch's shared memory holds per CTA (0: none)
  int small;      // no row has more than kRankMax tokens
};

// Order-preserving map of a score to an unsigned key: NaN above every number,
// -0 equal to +0.
__device__ __forceinline__ uint32_t score_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return f != f ? 0xffffffffu : k;
}

// The score of a key; not that of an unranked token (0), of a zero (which of the two) or of NaN.
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct SelShared {
  int cta_count[2];  // kept outright, equal to the threshold; read by the cluster
  int pick, rank;
  int warp_count[2][kSelWarps];
  int warp_sum[kSelWarps];
};
struct SelHist {
  int hist[kCopies][kBins];
  int cta_hist[2][kBins];  // by parity of the pass; read by the cluster
};

// Sum of the first n <= 32 of v, by a whole warp.
__device__ __forceinline__ int sum_before(const int* v, int n, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < n ? v[lane] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  __shared__ SelShared sh;
  uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem);
  SelHist& hi_ = *reinterpret_cast<SelHist*>(sel_smem + 4 * a.held_keys);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank_c = (int)cluster_rank();
  griddep_wait();
  const int64_t row = blockIdx.x / C;
  const int s = (int)(row / a.b.Hkv), g = (int)(row % a.b.Hkv);
  const float* x = a.scores + row * a.max_tokens;
  float* out = a.scores_out + row * a.max_tokens;
  int32_t* kept = a.kept + row * a.budget;
  const int n = (int)min((int64_t)a.b.kv_len(s), a.max_tokens);
  const int n_new = min(n, a.budget);
  const int all = C * kSelThreads, me = rank_c * kSelThreads + tid;
  if (me == 0 && g == 0) a.new_lens[s] = n_new;
  if (n <= a.budget) {  // uniform over the cluster
    for (int t = me; t < n; t += all) {
      out[t] = x[t];
      kept[t] = t;
    }
    return;
  }
  const int lo = a.sinks, hi = n - a.recent, quota = a.budget - a.sinks - a.recent;
  if (a.small) {  // one CTA, n <= kRankMax: thread t has token t
    const bool there = tid < n, mid = there && tid >= lo && tid < hi;
    const float f = there ? x[tid] : 0.f;
    // a token's place in the order (key, then the lower index); keys outside the
    // middle are 0, which is no score's key
    const uint32_t key = score_key(f);
    keys[tid] = mid ? key : 0u;
    __syncthreads();
    int before = 0;
    if (quota > 0 && __any_sync(0xffffffffu, mid)) {
      const uint4* k4 = reinterpret_cast<const uint4*>(keys);
      const int end = (n + 3) >> 2, own = warp * 8;
      int b0 = 0, b1 = 0, b2 = 0, b3 = 0;
#pragma unroll 4
      for (int t = 0; t < own; ++t) {  // lower indices: ties count
        const uint4 k = k4[t];
        b0 += k.x >= key, b1 += k.y >= key, b2 += k.z >= key, b3 += k.w >= key;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint32_t k = __shfl_sync(0xffffffffu, mid ? key : 0u, i);
        b0 += i < lane ? k >= key : k > key;
      }
#pragma unroll 4
      for (int t = own + 8; t < end; ++t) {
        const uint4 k = k4[t];
        b0 += k.x > key, b1 += k.y > key, b2 += k.z > key, b3 += k.w > key;
      }
      before = b0 + b1 + b2 + b3;
    }
    const bool keep = there && (!mid || before < quota);
    const unsigned m = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) sh.warp_sum[warp] = __popc(m);
    __syncthreads();
    int j = __popc(m & ((1u << lane) - 1));
    j += sum_before(sh.warp_sum, warp, lane);
    if (keep) {
      kept[j] = tid;
      out[j] = f;
    }
    return;
  }
  // this CTA's tokens [c0, c1), this warp's [w0, w1): multiples of 128, four a lane
  const int seg = ((n + C - 1) / C + 127) & ~127;
  const int c0 = min(n, rank_c * seg), c1 = min(n, c0 + seg);
  const int wseg = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int w0 = min(c1, c0 + warp * wseg), w1 = min(c1, w0 + wseg);
  const bool held = a.held_keys > 0;
  // Four keys of tokens t .. t + 3, 0 for those that the selection does not rank
  // (held or past the run): below every score's key, so no rank counts them.
  const bool vec = (a.max_tokens & 3) == 0 && (reinterpret_cast<uintptr_t>(a.scores) & 15) == 0;
  const int m0 = max(lo, w0), m1 = min(hi, w1);  // the warp's ranked tokens
  auto load_keys = [&](int t) -> uint4 {
    float f[4];
    if (vec) {
      const float4 v = *reinterpret_cast<const float4*>(x + t);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = t + i < w1 ? x[t + i] : 0.f;
    }
    uint32_t k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = t + i >= m0 && t + i < m1 ? score_key(f[i]) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  if (held) {
#pragma unroll 8
    for (int t = w0 + 4 * lane; t < w1; t += 128) *reinterpret_cast<uint4*>(keys + (t - c0)) = load_keys(t);
  }
  __syncwarp();
  auto keys_at = [&](int t) { return held ? *reinterpret_cast<const uint4*>(keys + (t - c0)) : load_keys(t); };
  uint32_t prefix = 0;
  int rank = quota;  // the rank-th highest key among those that match the prefix
  auto pass = [&](auto shift_tag, auto bits_tag, int parity) {
    constexpr int shift = decltype(shift_tag)::value, bits = decltype(bits_tag)::value;
    constexpr uint32_t digit = (1u << bits) - 1, mask = shift + bits == 32 ? 0u : ~0u << (shift + bits);
    int* hist = hi_.hist[warp / (kSelWarps / kCopies)];
    for (int i = tid; i < kCopies * kBins / 4; i += kSelThreads)
      reinterpret_cast<int4*>(hi_.hist[0])[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int t = w0 + 4 * lane; t < w1; t += 128) {
      const uint4 k = keys_at(t);
      const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (mask == 0 || ((kk[i] ^ prefix) & mask) == 0) atomicAdd(&hist[(kk[i] >> shift) & digit], 1);
    }
    __syncthreads();
    // bins from the highest down, two a thread
    const int b = kBins - 2 - 2 * tid;
    int2 c = make_int2(0, 0);  // x: bin b + 1, y: bin b
#pragma unroll
    for (int w = 0; w < kCopies; ++w) {
      const int2 v = *reinterpret_cast<const int2*>(&hi_.hist[w][b]);
      c.x += v.y;
      c.y += v.x;
    }
    if (C > 1) {
      hi_.cta_hist[parity][b + 1] = c.x;
      hi_.cta_hist[parity][b] = c.y;
      cluster_sync();
      c = make_int2(0, 0);
      for (int r = 0; r < C; ++r) {
        c.x += cluster_read(&hi_.cta_hist[parity][b + 1], r);
        c.y += cluster_read(&hi_.cta_hist[parity][b], r);
      }
    }
    int above = c.x + c.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, above, o);
      if (lane >= o) above += y;
    }
    if (lane == 31) sh.warp_sum[warp] = above;
    __syncthreads();
    above += sum_before(sh.warp_sum, warp, lane) - c.x - c.y;  // keys in higher bins than this thread's
    if (above < rank && above + c.x >= rank) {
      sh.pick = b + 1;
      sh.rank = rank - above;
    } else if (above + c.x < rank && above + c.x + c.y >= rank) {
      sh.pick = b;
      sh.rank = rank - above - c.x;
    }
    __syncthreads();
    prefix |= (uint32_t)sh.pick << shift;
    rank = sh.rank;
  };
  if (quota > 0) {
    using std::integral_constant;
    pass(integral_constant<int, 21>{}, integral_constant<int, 11>{}, 0);
    pass(integral_constant<int, 10>{}, integral_constant<int, 11>{}, 1);
    pass(integral_constant<int, 0>{}, integral_constant<int, 10>{}, 0);
  } else {
    prefix = 0xffffffffu;  // nothing is above it, and `rank` = 0 takes no tie
  }
  // A token stays if held outright (sinks, recent), above the threshold, or among
  // the first `rank` equal to it: every warp counts both kinds of its run ...
  int takes = 0, ties = 0;
  for (int t = w0 + 4 * lane; t < w1; t += 128) {
    const uint4 k = keys_at(t);
    takes += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
    ties += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
  }
  takes = __reduce_add_sync(0xffffffffu, takes) + max(0, min(w1, lo) - w0) + max(0, w1 - max(w0, hi));
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    sh.warp_count[0][warp] = takes;
    sh.warp_count[1][warp] = ties;
  }
  __syncthreads();
  if (warp < 2) {
    const int sum = sum_before(sh.warp_count[warp], kSelWarps, lane);
    if (lane == 0) sh.cta_count[warp] = sum;
  }
  if (C > 1) cluster_sync();
  // ... and adds up what lies before them
  takes = ties = 0;
  for (int c = 0; c < rank_c; ++c) {
    takes += cluster_read(&sh.cta_count[0], c);
    ties += cluster_read(&sh.cta_count[1], c);
  }
  takes += sum_before(sh.warp_count[0], warp, lane);
  ties += sum_before(sh.warp_count[1], warp, lane);
  const unsigned below = (1u << lane) - 1;
  // 128 tokens at a time, four a lane; 32 at a time, where a ballot gives a token's
  // place, for those with held tokens, ties, NaN, or a zero or negative threshold
  for (int t1 = w0; t1 < w1; t1 += 128) {
    const int t4 = t1 + 4 * lane;
    const uint4 k4 = t4 < w1 ? keys_at(t4) : make_uint4(0, 0, 0, 0);
    const uint32_t kk[4] = {k4.x, k4.y, k4.z, k4.w};
    bool odd = prefix <= 0x80000000u;
    int c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      odd |= kk[i] == prefix || kk[i] == 0xffffffffu;
      c += kk[i] > prefix;
    }
    if (t1 >= lo && min(t1 + 128, w1) <= hi && !__any_sync(0xffffffffu, odd)) {
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      int j = takes + min(ties, rank) + inc - c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (kk[i] > prefix) {
          kept[j] = t4 + i;
          out[j] = score_of(kk[i]);
          ++j;
        }
      takes += __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    for (int t0 = t1; t0 < min(t1 + 128, w1); t0 += 32) {
      const int t = t0 + lane;
      uint32_t key = 0;
      if (t < w1) key = held ? keys[t - c0] : t >= m0 && t < m1 ? score_key(x[t]) : 0u;
      const unsigned out_of = __ballot_sync(0xffffffffu, t < w1 && (t < lo || t >= hi));
      const unsigned above = __ballot_sync(0xffffffffu, key > prefix) | out_of;
      const unsigned tied = __ballot_sync(0xffffffffu, key == prefix);
      const int tie_before = ties + __popc(tied & below);
      if ((above >> lane & 1) || ((tied >> lane & 1) && tie_before < rank)) {
        const int j = takes + __popc(above & below) + min(tie_before, rank);
        kept[j] = t;
        out[j] = x[t];
      }
      takes += __popc(above);
      ties += __popc(tied);
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another reads its counts
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  constexpr int V = D / 8;  // 16-byte vectors of a row
  griddep_wait();  // the selection's results
  const int s = blockIdx.z, g = blockIdx.y;
  const int n_new = a.new_lens[s];
  const int j = blockIdx.x * (kGatherThreads / V) + threadIdx.x / V, c = threadIdx.x % V;
  // what lies past the kept tokens, in equal parts
  const int64_t row = (int64_t)s * a.b.Hkv + g;
  const int64_t me = (int64_t)blockIdx.x * kGatherThreads + threadIdx.x, all = (int64_t)gridDim.x * kGatherThreads;
  for (int64_t i = n_new + me; i < a.max_tokens; i += all) a.scores_out[row * a.max_tokens + i] = 0.f;
  for (int64_t i = n_new + me; i < a.budget; i += all) a.kept[row * a.budget + i] = -1;
  if (j >= n_new || j / kPage >= a.dst_max_pages) return;
  const int t = a.kept[row * a.budget + j];
  const int sp = a.b.page(s, t / kPage), dp = a.dst_table[(size_t)s * a.dst_max_pages + j / kPage];
  if ((unsigned)dp >= (unsigned)a.b.num_pages) return;
  const size_t to = (((size_t)dp * a.b.Hkv + g) * kPage + j % kPage) * D + 8 * c;
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (sp >= 0) {  // of a hole's token zeros: the slot will be seen, and may hold another session's rows
    const size_t from = (((size_t)sp * a.b.Hkv + g) * kPage + t % kPage) * D + 8 * c;
    x = *reinterpret_cast<const uint4*>(a.k_pool + from);
    y = *reinterpret_cast<const uint4*>(a.v_pool + from);
  }
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
  const int64_t span = (int64_t)b->max_pages * pa::kPage;
  // CTAs per (session, kv head): more while SMs would be idle and a CTA would
  // still have 8192 tokens, or until the keys fit shared memory.  8 rows of 32768
  // tokens: 1 CTA each 24 us, 2 20.9 us, 4 21.5 us, 8 33.9 us (a cluster of 8 such
  // CTAs starts late); 8 rows of 16384: 1 18.4 us, 2 18.7 us, 4 21.0 us
  const int64_t longest = span < max_tokens ? span : max_tokens;
  const int64_t pairs = (int64_t)b->n_sessions * b->num_kv_heads;
  const pa_device dev = pa_current_device();
  int C = 1;
  while (C < 8 && (longest / C > pa::kKeysMax || (C < 4 && pairs * C * 2 <= dev.sms && longest / (2 * C) >= 8192))) C *= 2;
  // ranked by comparison against the radix selection, 4 sessions of 2 heads: 320
  // tokens 6.1 and 8.9 us, 512 tokens 8.7 and 9.3 us, 640 tokens 10.9 and 9.1 us
  a.small = longest <= pa::kRankMax;
  // (a warp's run is padded to 128 tokens)
  const int64_t per_cta = ((longest + C - 1) / C + 127) / 128 * 128 + 128 * pa::kSelWarps;
  constexpr int64_t most_held = pa::kKeysMax + 128 * pa::kSelWarps;
  a.held_keys = a.small ? pa::kSelThreads : (int)(per_cta <= most_held ? per_cta : 0);
  const int smem = 4 * a.held_keys + (a.small ? 0 : (int)sizeof(pa::SelHist));
  static std::atomic<uint64_t> allowed{0};
  if (!pa_allow_smem(pa::evict_select_kernel, 4 * (int)most_held + (int)sizeof(pa::SelHist), dev.index, allowed))
    return PA_ERR_CUDA;
  if (!pa_launch_early(pa::evict_select_kernel, dim3((unsigned)(pairs * C)), dim3(pa::kSelThreads), smem, cs, C, a))
    return PA_ERR_CUDA;
  const int rows = pa::kGatherThreads / (b->head_dim / 8);
  const int most = (int)(span < budget ? span : budget);
  const dim3 grid((most + rows - 1) / rows, b->num_kv_heads, b->n_sessions);
  auto* gather = b->head_dim == 64 ? pa::evict_gather_kernel<64> : pa::evict_gather_kernel<128>;
  return pa_launch_early(gather, grid, dim3(pa::kGatherThreads), 0, cs, 1, a) ? PA_OK : PA_ERR_CUDA;
}
