// Device helpers of the session-cache tensor-core kernels.
#pragma once

#include "ptx.cuh"

namespace pa {

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The larger, the smaller one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// y minus the two bf16 numbers of a word (lower half first), in one mixed-precision step
// each, which is exact where they are y rounded or cut to bf16.
__device__ __forceinline__ float2 minus_bf16x2(float2 y, uint32_t w) {
  float2 d;
  asm("{\n .reg .b16 a, b, m;\n mov.b32 {a, b}, %2;\n mov.b16 m, 0xbf80;\n"
      " fma.rn.f32.bf16 %0, a, m, %3;\n fma.rn.f32.bf16 %1, b, m, %4;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(w), "f"(y.x), "f"(y.y));
  return d;
}

// After a wait gave up the barriers no longer tell what is in flight: 5 ms are
// far more than any copy or product of this CTA can take to land.
__device__ __forceinline__ void settle() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 5000000ull) __nanosleep(1000);
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// A block of `np` <= 8 pages (lane from + i of the warp holds the pool row of the
// i-th) into 128-row x 64-dim swizzled tiles, by a converged warp whose elected
// lane issues: the rows come by shuffles, so that each copy's operands are
// uniform (copies issued by eight lanes each took 78 cycles apiece).
template <int HALVES>
__device__ __forceinline__ void load_pages(uint32_t dst, const void* tmap, int row, int from, int np, uint32_t bar,
                                           bool lead) {
  int r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __shfl_sync(0xffffffffu, row, from + i);
  if (lead) {
    mbar_arrive_expect_tx(bar, (uint32_t)np * (HALVES * 2048));
    if (np == 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) tma_load_2d(dst + h * 16384 + i * 2048, tmap, 64 * h, r[i], bar);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < np)
#pragma unroll
          for (int h = 0; h < HALVES; ++h) tma_load_2d(dst + h * 16384 + i * 2048, tmap, 64 * h, r[i], bar);
    }
  }
  __syncwarp();
}

// umma_sdesc_sw128 from an address already in 16-byte units.
__device__ __forceinline__ uint64_t sdesc_sw128_lo(uint32_t addr16, uint32_t lbo16, uint32_t sbo16) {
  return (uint64_t)(addr16 | (lbo16 << 16)) | ((uint64_t)(sbo16 | (1u << 14) | (2u << 29)) << 32);
}

// Whole warp: 8 fp32 columns of its 32 TMEM lanes times each lane's f.
__device__ __forceinline__ void tmem_scale8(uint32_t taddr, float f) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 2^x of two x on the FMA pipe: x = n + f, f in [-1/2, 1/2]; 2^f by the degree-5
// polynomial of least relative error with a constant of 1 (by Lawson's reweighted least
// squares: 9.2e-8; with these fp32 coefficients and fp32 steps 1.6e-7, bias -1.9e-8, over
// 2 million f) times 2^n, made of its bits.  As ex2 at the ends: 0 below -126.5 (-inf
// among it), inf from 127.5 on, NaN of NaN (which the clamps keep and the product then
// carries).
__device__ __forceinline__ float2 exp2_fma(float2 x) {
  x.x = min_nan(max_nan(x.x, -127.f), 128.f);
  x.y = min_nan(max_nan(x.y, -127.f), 128.f);
  // adding 1.5 * 2^23 rounds to an integer, which its low bits then hold
  const float2 t = fadd2(x, make_float2(12582912.f, 12582912.f));
  const float2 n = fadd2(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = ffma2(n, make_float2(-1.f, -1.f), x);
  float2 p = make_float2(1.3264702865853906e-3f, 1.3264702865853906e-3f);
  p = ffma2(p, f, make_float2(9.671504609286785e-3f, 9.671504609286785e-3f));
  p = ffma2(p, f, make_float2(5.550734326243401e-2f, 5.550734326243401e-2f));
  p = ffma2(p, f, make_float2(0.24022239446640015f, 0.24022239446640015f));
  p = ffma2(p, f, make_float2(0.6931469440460205f, 0.6931469440460205f));
  p = ffma2(p, f, make_float2(1.f, 1.f));
  return fmul2(p, make_float2(__uint_as_float(0x3f800000u + (__float_as_uint(t.x) << 23)),
                              __uint_as_float(0x3f800000u + (__float_as_uint(t.y) << 23))));
}

}  // namespace pa
