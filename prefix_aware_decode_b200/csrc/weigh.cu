// Accumulated attention weight of cached tokens (pa_weigh_tokens):
//     scores[s][g][t] += sum over the rows r of session s that see t and the
//                        query heads h of kv head g of e^{scale q_rh . k_t - lse_rh}
// with the lse of pa_window_attend, so a row's weights sum to one.
#include "ptx.cuh"
#include "sessions.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct WeighArgs {
  Sessions b;
  Window w;
  const uint16_t *q, *k_pool;
  const float* lse;
  float* scores;
  int64_t max_tokens;
  float scale_log2;
};

// One warp per (session, kv head, token); lane l holds dims [l D/32, (l + 1) D/32).
template <int D>
__global__ void __launch_bounds__(256) weigh_kernel(const WeighArgs a) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.z, g = blockIdx.y, t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int kv = a.b.kv_len(s);
  if (t >= kv || t >= a.max_tokens) return;
  const int page = a.b.page(s, t / kPage);
  const int r0 = a.b.row_begin(s), n = a.b.row_begin(s + 1) - r0, p0 = kv - n;
  if (page < 0 || n <= 0) return;
  const int G = a.b.Hq / a.b.Hkv;
  const uint32_t* k =
      reinterpret_cast<const uint32_t*>(a.k_pool + (((size_t)page * a.b.Hkv + g) * kPage + t % kPage) * D) + lane * W;
  float2 kf[W];
#pragma unroll
  for (int i = 0; i < W; ++i) kf[i] = bf16x2_to_f2(k[i]);
  float sum = 0.f;
  for (int i = max(0, t - p0); i < n; ++i) {
    if (!a.w.sees(p0 + i, t)) break;  // later rows see it no more
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const size_t at = (size_t)(r0 + i) * a.b.Hq + h;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + at * D) + lane * W;
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float2 qf = bf16x2_to_f2(q[j]);
        x += qf.x * kf[j].x + qf.y * kf[j].y;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      const float l = a.lse[at];
      if (l > -INFINITY) sum += ex2(x * a.scale_log2 - l * kLog2e);
    }
  }
  if (lane == 0) a.scores[((size_t)s * a.b.Hkv + g) * a.max_tokens + t] += sum;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_weigh_tokens(const pa_sessions* b, int32_t window, int32_t sinks, float softmax_scale,
                                     const void* q, const void* k_pool, const float* lse, float* scores,
                                     int64_t max_tokens, void* stream) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (window < 0 || sinks < 0 || max_tokens < 1 || !scores || !(softmax_scale >= 0.f) || softmax_scale > 3.4e38f)
    return PA_ERR_INVALID;
  if (b->num_rows == 0) return PA_OK;
  if (!q || !k_pool || !lse || !pa_aligned16(q) || !pa_aligned16(k_pool)) return PA_ERR_INVALID;
  pa::WeighArgs a{};
  a.b = pa_device_sessions(*b);
  a.w = pa::Window{window, sinks};
  a.q = static_cast<const uint16_t*>(q);
  a.k_pool = static_cast<const uint16_t*>(k_pool);
  a.lse = lse;
  a.scores = scores;
  a.max_tokens = max_tokens;
  a.scale_log2 = (softmax_scale != 0.f ? softmax_scale : 1.f / sqrtf((float)b->head_dim)) * pa::kLog2e;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t span = (int64_t)b->max_pages * pa::kPage;
  const int64_t most = span < max_tokens ? span : max_tokens;
  const dim3 grid((unsigned)((most + 7) / 8), b->num_kv_heads, b->n_sessions);
  if (b->head_dim == 64) pa::weigh_kernel<64><<<grid, 256, 0, cs>>>(a);
  else pa::weigh_kernel<128><<<grid, 256, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
