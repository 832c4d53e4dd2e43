// Attention of the last rows of every session over its paged cache: causal,
// with a sliding window and sinks (pa_window_attend).
//
// A row at cached position p sees token t when t <= p and (t > p - window or
// t < sinks); out = sum_t e^{s_t - m} v_t / l, lse = m + ln l in one pass over
// the visible tokens with a running maximum.
#include "ptx.cuh"
#include "sessions.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendArgs {
  Sessions b;
  Window w;
  const uint16_t *q, *k_pool, *v_pool;
  uint16_t* out;
  float* lse;
  float scale_log2;
};

// One warp per (row, query head); lane l holds dims [l D/32, (l + 1) D/32).
template <int D>
__global__ void __launch_bounds__(256) window_attend_kernel(const AttendArgs a) {
  constexpr int W = D / 64;  // bf16x2 words per lane
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = (int)(unit / a.b.Hq), h = (int)(unit % a.b.Hq);
  if (r >= a.b.rows) return;
  const int s = warp_find_session(a.b, r, lane);
  const int r0 = a.b.row_begin(s), n = a.b.row_begin(s + 1) - r0;
  if (r < r0 || r >= r0 + n) return;
  const int p = a.b.kv_len(s) - n + (r - r0), g = h / (a.b.Hq / a.b.Hkv);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((size_t)r * a.b.Hq + h) * D) + lane * W;
  float2 qf[W], acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) qf[i] = bf16x2_to_f2(q[i]), acc[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const int first = a.w.first(p);
  for (int t = min(a.w.sinks, first) > 0 ? 0 : first; t <= p; ++t) {
    if (t >= a.w.sinks && t < first) t = first;
    const int page = a.b.page(s, t / kPage);
    if (page < 0) continue;
    const size_t at = (((size_t)page * a.b.Hkv + g) * kPage + t % kPage) * D;
    const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k_pool + at) + lane * W;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v_pool + at) + lane * W;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 kf = bf16x2_to_f2(k[i]);
      x += qf[i].x * kf.x + qf[i].y * kf.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x);
    const float c = mn == -INFINITY ? 1.f : ex2(m - mn), e = mn == -INFINITY ? 0.f : ex2(x - mn);
    m = mn;
    l = l * c + e;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 vf = bf16x2_to_f2(v[i]);
      acc[i] = make_float2(acc[i].x * c + e * vf.x, acc[i].y * c + e * vf.y);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* o = reinterpret_cast<uint32_t*>(a.out + ((size_t)r * a.b.Hq + h) * D) + lane * W;
#pragma unroll
  for (int i = 0; i < W; ++i) o[i] = pack_bf16x2(acc[i].x * inv, acc[i].y * inv);
  if (a.lse && lane == 0) a.lse[(size_t)r * a.b.Hq + h] = l > 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_window_workspace_size(const pa_sessions* b, int32_t window, int32_t sinks, size_t* bytes) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (!bytes || window < 0 || sinks < 0) return PA_ERR_INVALID;
  *bytes = 256;
  return PA_OK;
}

extern "C" pa_status pa_window_attend(const pa_sessions* b, int32_t window, int32_t sinks, float softmax_scale,
                                      const void* q, const void* k_pool, const void* v_pool, void* d_workspace,
                                      size_t workspace_bytes, void* out, float* lse, void* stream) {
  size_t need = 0;
  const pa_status st = pa_window_workspace_size(b, window, sinks, &need);
  if (st != PA_OK) return st;
  if (b->num_rows == 0) return PA_OK;
  if (!q || !k_pool || !v_pool || !out || !d_workspace) return PA_ERR_INVALID;
  if (!pa_aligned16(q) || !pa_aligned16(k_pool) || !pa_aligned16(v_pool) || !pa_aligned16(out) ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 255))
    return PA_ERR_INVALID;
  if (workspace_bytes < need) return PA_ERR_NOMEM;
  pa::AttendArgs a{};
  a.b = pa_device_sessions(*b);
  a.w = pa::Window{window, sinks};
  a.q = static_cast<const uint16_t*>(q);
  a.k_pool = static_cast<const uint16_t*>(k_pool);
  a.v_pool = static_cast<const uint16_t*>(v_pool);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.scale_log2 = (softmax_scale != 0.f ? softmax_scale : 1.f / sqrtf((float)b->head_dim)) * pa::kLog2e;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t units = (int64_t)b->num_rows * b->num_q_heads;
  const unsigned grid = (unsigned)((units + 7) / 8);
  if (b->head_dim == 64) pa::window_attend_kernel<64><<<grid, 256, 0, cs>>>(a);
  else pa::window_attend_kernel<128><<<grid, 256, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
