// Rotary positions with several axes, fused with the write of new K and V rows
// into their pages (pa_rope_append).
//
// Pair i of a head turns by angle(r, i) = positions[axis(i)][r] * inv_freq[i]:
// (x, y) -> (x cos - y sin, x sin + y cos).  The angle is formed and reduced to
// half turns in fp64: at position 2^20 an fp32 product would be off by 2^-4
// radian, the fp64 one by 2^-33.  One sincospif per (row, pair), shared by all
// heads of the row through shared memory; the rotation itself is fp32, rounded
// to bf16 once.
//
// Bound by memory: each q, k, v element is read and written once.  10306 rows of
// 32/8 heads of 128: 0.25 GB in 48 us (5.3 TB/s); 64 rows 4.0 us.
#include "ptx.cuh"
#include "sessions.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  Sessions b;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from row to row
  const int32_t* positions;              // [n_axes][rows]
  const double* inv_freq;                // [R / 2]
  uint16_t *k_pool, *v_pool, *q_out;
  int R, interleaved;
  uint32_t axes[4];  // 2 bits per pair: its axis
};

// Turns the 8 pairs of a unit: with `split` element i of the vectors is pair i,
// else the elements 2i, 2i + 1 are.
__device__ __forceinline__ void turn_unit(uint4& x0, uint4& x1, const float2* cs, bool split) {
  uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float2 p = bf16x2_to_f2(w0[m]), y = bf16x2_to_f2(w1[m]);
    if (split) {
      const float2 t0 = cs[2 * m], t1 = cs[2 * m + 1];
      w0[m] = pack_bf16x2(p.x * t0.x - y.x * t0.y, p.y * t1.x - y.y * t1.y);
      w1[m] = pack_bf16x2(p.x * t0.y + y.x * t0.x, p.y * t1.y + y.y * t1.x);
    } else {
      const float2 t0 = cs[m], t1 = cs[4 + m];
      w0[m] = pack_bf16x2(p.x * t0.x - p.y * t0.y, p.x * t0.y + p.y * t0.x);
      w1[m] = pack_bf16x2(y.x * t1.x - y.y * t1.y, y.x * t1.y + y.y * t1.x);
    }
  }
  x0 = make_uint4(w0[0], w0[1], w0[2], w0[3]);
  x1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
}

// ROWS consecutive rows per CTA: one while all CTAs are resident at once (the fewest
// dependent steps), four when there are enough (each thread then has six
// vectors in flight).
template <int D, int ROWS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
  __shared__ float2 turn[ROWS][D / 2];  // (cos, sin)
  __shared__ long long slot[ROWS];      // pool offset of the row's kv head 0 slot; -1: none
  __shared__ int live[ROWS];            // the row belongs to a session
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * ROWS;
  const int pairs = a.R >> 1;
  griddep_wait();
  for (int i = tid; i < ROWS * pairs; i += kRopeThreads) {
    const int j = i / pairs, p = i - j * pairs, r = r0 + j;
    if (r < a.b.rows) {
      const int axis = (a.axes[p >> 4] >> (2 * (p & 15))) & 3;
      const double half_turns =
          (double)a.positions[(size_t)axis * a.b.rows + r] * a.inv_freq[p] * 0.31830988618379067154;
      float s, c;
      sincospif((float)(half_turns - 2.0 * rint(0.5 * half_turns)), &s, &c);
      turn[j][p] = make_float2(c, s);
    }
  }
  for (int j = warp; j < ROWS; j += kRopeThreads / 32) {
    const int r = r0 + j;
    long long at = -1;
    int in = 0;
    if (r < a.b.rows) {
      const int s = warp_find_session(a.b, r, lane);
      const int b0 = a.b.row_begin(s), n = a.b.row_begin(s + 1) - b0;
      in = r >= b0 && r < b0 + n;
      const int t = a.b.kv_len(s) - n + (r - b0);
      if (in && t >= 0) {
        const int page = a.b.page(s, t / kPage);
        if (page >= 0) at = ((long long)page * a.b.Hkv * kPage + t % kPage) * D;
      }
    }
    if (lane == 0) {
      slot[j] = at;
      live[j] = in;
    }
  }
  __syncthreads();
  // Units of 16 elements (two 16-byte vectors) of a head: a thread keeps its unit
  // u of the heads and walks the (row, head) pairs, kBatch of them with their
  // loads in flight together.
  constexpr int U = D / 16, STEP = kRopeThreads / U;
  constexpr int kBatch = 2;
  const int Hq = a.b.Hq, Hkv = a.b.Hkv, H = Hq + 2 * Hkv;
  const int u = tid % U;
  const bool rot = u < a.R / 16, split = rot && !a.interleaved;
  const int e0 = split ? 8 * u : 16 * u, e1 = split ? e0 + a.R / 2 : e0 + 8;  // the unit's two vectors
  int j = 0, h = tid / U;
  while (h >= H) h -= H, ++j;
  while (j < ROWS) {
    uint4 x0[kBatch], x1[kBatch];
    uint16_t* dst[kBatch];
    int row[kBatch];  // the turns to apply; -1: copy
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      dst[k] = nullptr;
      if (j < ROWS && r0 + j < a.b.rows && live[j]) {
        const int64_t r = r0 + j;
        const uint16_t* src = nullptr;
        row[k] = rot && h < Hq + Hkv ? j : -1;
        if (h < Hq) {
          src = a.q + r * a.q_stride + h * D;
          dst[k] = a.q_out + (r * Hq + h) * D;
        } else if (slot[j] >= 0) {
          const bool is_v = h >= Hq + Hkv;
          const int g = is_v ? h - Hq - Hkv : h - Hq;
          src = (is_v ? a.v + r * a.v_stride : a.k + r * a.k_stride) + g * D;
          dst[k] = (is_v ? a.v_pool : a.k_pool) + slot[j] + (int64_t)g * kPage * D;
        }
        if (src) {
          x0[k] = *reinterpret_cast<const uint4*>(src + e0);
          x1[k] = *reinterpret_cast<const uint4*>(src + e1);
        }
      }
      h += STEP;
      while (h >= H) h -= H, ++j;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!dst[k]) continue;
      if (row[k] >= 0) turn_unit(x0[k], x1[k], &turn[row[k]][8 * u], split);
      *reinterpret_cast<uint4*>(dst[k] + e0) = x0[k];
      *reinterpret_cast<uint4*>(dst[k] + e1) = x1[k];
    }
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_rope_append(const pa_sessions* b, const pa_rope* rope, const void* q, int64_t q_row_stride,
                                    const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                    void* k_pool, void* v_pool, void* q_out, void* stream) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (!rope || rope->n_axes < 1 || rope->n_axes > 4 || rope->rotary_dim < 16 || rope->rotary_dim > b->head_dim ||
      rope->rotary_dim % 16)
    return PA_ERR_INVALID;
  if (rope->axes)
    for (int i = 0; i < rope->rotary_dim / 2; ++i)
      if (rope->axes[i] >= rope->n_axes) return PA_ERR_INVALID;
  if (b->num_rows == 0) return PA_OK;
  if (!q || !k || !v || !k_pool || !v_pool || !q_out || !rope->d_positions || !rope->d_inv_freq) return PA_ERR_INVALID;
  const void* ptrs[] = {q, k, v, k_pool, v_pool, q_out};
  for (const void* p : ptrs)
    if (!pa_aligned16(p)) return PA_ERR_INVALID;
  const int64_t hq = (int64_t)b->num_q_heads * b->head_dim, hk = (int64_t)b->num_kv_heads * b->head_dim;
  if (q_row_stride < hq || k_row_stride < hk || v_row_stride < hk || (q_row_stride | k_row_stride | v_row_stride) % 8)
    return PA_ERR_INVALID;
  pa::RopeArgs a{};
  a.b = pa_device_sessions(*b);
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.positions = rope->d_positions;
  a.inv_freq = rope->d_inv_freq;
  a.k_pool = static_cast<uint16_t*>(k_pool);
  a.v_pool = static_cast<uint16_t*>(v_pool);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.R = rope->rotary_dim;
  a.interleaved = rope->interleaved;
  if (rope->axes)
    for (int i = 0; i < rope->rotary_dim / 2; ++i) a.axes[i >> 4] |= (uint32_t)rope->axes[i] << (2 * (i & 15));
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // a CTA a row while they are all resident at once: 700 rows of 32/8 heads of 128 5.1
  // us, four rows a CTA 7.0 us; 800 rows 7.3 and 7.1 us, 4736 rows 28.5 and 24.9 us;
  // 900 rows of 8/1 heads of 64 4.8 and 3.2 us
  const bool many = b->num_rows > 5 * pa_current_device().sms;
  const unsigned grid = many ? (b->num_rows + 3) / 4 : b->num_rows;
  auto* kernel = b->head_dim == 64 ? (many ? pa::rope_append_kernel<64, 4> : pa::rope_append_kernel<64, 1>)
                                   : (many ? pa::rope_append_kernel<128, 4> : pa::rope_append_kernel<128, 1>);
  return pa_launch_early(kernel, dim3(grid), dim3(pa::kRopeThreads), 0, cs, 1, a) ? PA_OK : PA_ERR_CUDA;
}
