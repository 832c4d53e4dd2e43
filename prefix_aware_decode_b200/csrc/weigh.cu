// Accumulated attention weight of cached tokens (pa_weigh_tokens):
//     scores[s][g][t] += sum over the rows r of session s that see t and the
//                        query heads h of kv head g of e^{scale q_rh . k_t - lse_rh}
// with the lse of pa_window_attend, so a row's weights sum to one.
//
// S^T = K Q^T on the 5th-generation tensor cores with the keys as the rows of
// the product: a key is a lane of tensor memory and a thread, and its sum over
// the (row, head) columns stays in that thread's registers.  Nothing is
// exchanged but one number per key, and no two CTAs add to one score: the
// result is the same on every run.
//
// An item is (session, kv head, up to 256 keys as two blocks of 8 pages); the
// tiles of 128 columns that see any of them stream past the resident K blocks
// (Q tiles by TMA, their lse beside them).  When the batch has few rows (one
// tile of columns per session) the K blocks stream instead: a CTA takes a
// contiguous run of items and keeps the Q tile while session and head stay.
//
// Bounds: with few rows the K bytes.  With many rows the exponentials: one per
// (row, head, visible key), 16 a cycle and SM on the MUFU pipe against 128 x 128
// scores in 512 tensor cycles; so a part of them is computed on the FMA pipe
// (kFmaPairs), which leaves both pipes about equally busy.  Measured, 32/8 heads of
// 128: a decode step of 64 sessions of 2000-20000 tokens, 1.41 GB in 231-241 us (6.0
// TB/s); chunks of 1500 and 2048 rows over 9000 and 16384 tokens, 361 GFLOP in 405
// us (0.89 PFLOP/s; the exponential pipe about 72% busy, 80% on the fullest SM).
//
// Roles (640 threads): warps 0-15 four groups of one thread per key, each with
// its own score buffer in tensor memory; warp 16 issues the products; warp 17
// walks the items and loads the Q tiles, warps 18 and 19 an item's first and
// second K block (one warp took 3300 cycles an item to issue the copies of both).
#include <type_traits>

#include "ptx.cuh"
#include "sessions.cuh"
#include "tmap.h"
#include "umma.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 640;
constexpr int kGroups = 1024;  // entries of the table of item prefixes
constexpr int kQueue = 4;      // entries of the CTA's item queue
// Of 16 pairs of scores: exponentials on the FMA pipe.  Prompt chunks (above) with
// 0, 3, 4, 6: 450, 405, 413, 431 us.
constexpr int kFmaPairs = 3;
constexpr uint64_t kTimeoutNs = 2000000000ull;

// First failure of a device-side wait since pa_weigh_status last read it.
__device__ int32_t g_weigh_status[4];

struct WeighArgs {
  Sessions b;
  Window w;
  int lg;                 // log2 G
  int per_group;          // sessions per entry of the prefix table
  int nk, nq;             // ring slots of first (and of second) K blocks, and of Q tiles
  int run;                // 1: contiguous runs of items, 0: every gridDim.x-th item
  int pair;               // key blocks of an item: 2, or 1
  int give_up;            // the wait (its code) that gives up at once; 0: none
  const float* lse;
  float* scores;
  int64_t max_tokens;
  float scale_log2;
};

// The cached pages of a session that its rows see: virtual pages 0 .. ns - 1
// (sinks), then from page ns + off on, np in all.
struct Span {
  int r0, n, p0;  // rows [r0, r0 + n), the first at position p0
  int kv, np, ns, off;
  __device__ __forceinline__ int page_index(int v) const { return v < ns ? v : v + off; }
};

__device__ __forceinline__ Span make_span(const WeighArgs& a, int s) {
  Span x{};
  x.r0 = a.b.row_begin(s);
  x.n = a.b.row_begin(s + 1) - x.r0;
  x.kv = a.b.kv_len(s);
  x.p0 = x.kv - x.n;
  if (x.n <= 0 || x.kv <= 0) return x;
  const int last = (x.kv - 1) / kPage, first = a.w.first(max(x.p0, 0)) / kPage;
  const int sink = (min(a.w.sinks, x.kv) + kPage - 1) / kPage;
  if (sink < first) {
    x.ns = sink;
    x.off = first - sink;
  }
  x.np = last + 1 - x.off;
  return x;
}

struct Item {
  Span x;
  int s, g, v0;      // v0: first virtual page; -1 ends the line
  int rt0, rt1;      // column tiles
  int q_new, q_last; // the item loads its Q tile / releases it (one-tile items)
};

template <int D>
struct Shape {
  static constexpr int HALVES = D / 64;
  static constexpr int BLK = 128 * 128;      // 128 rows x 64 dims
  static constexpr int TILE = HALVES * BLK;  // a K block, a Q tile
  static constexpr int SLOTS = D == 128 ? 6 : 10;  // nk <= 8, nq <= 8
  static constexpr int OFF_MISC = SLOTS * TILE;
};

struct Misc {
  uint64_t kfull[2][8], kempty[2][8], qfull[8], qempty[8], sfull[4], sempty[4], done;
  uint64_t it_full[kQueue], it_empty[kQueue], comb[kQueue];
  uint32_t tmem;
  int fail;
  Item items[kQueue];
  long long warp_sum[kThreads / 32];
  long long prefix[kGroups + 1];  // items before group i
  float ex[kQueue][4][128];       // by queue entry and group of warps: sums of a key
  alignas(16) float nlse[8][128];  // per Q slot and column: -lse log2 e
};

template <int D>
constexpr int weigh_smem() {
  return Shape<D>::OFF_MISC + (int)sizeof(Misc);
}
static_assert(weigh_smem<128>() <= 232448 && weigh_smem<64>() <= 232448, "shared memory");

// Slot and phase of a ring, stepped through in order.
struct Ring {
  int slot = 0, phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, ++phase;
  }
  __device__ __forceinline__ void skip(int k, int n) {
    slot += k;
    phase += slot / n;
    slot %= n;
  }
};

// FAULT: the kernel of a call whose waits of one number give up (pa_session_fault); a
// comparison in every wait would cost all calls 3-8 %
template <int D, bool FAULT>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_kernel(const WeighArgs a, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the swizzle needs it; the kernel has no other shared memory before it
    griddep_wait();  // a launch ends no earlier than those before it on the stream
    if (threadIdx.x == 0) record_status(g_weigh_status, PA_ERR_DEVICE, blockIdx.x, 0);
    return;
  }
  Misc& mi = *reinterpret_cast<Misc*>(smem + S::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lt = 7 - a.lg;  // log2 of the tokens of a column tile
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const int step = 8 * a.pair;  // pages of an item

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar(mi.kfull[b][i]), 1);
        mbar_init(bar(mi.kempty[b][i]), 1);
      }
      mbar_init(bar(mi.qfull[i]), 2);               // the tile's bytes; the lse
      mbar_init(bar(mi.qempty[i]), a.run ? 17 : 1 + 4 * a.pair);  // products; the warps that read the lse
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(mi.sfull[i]), 1);
      mbar_init(bar(mi.sempty[i]), 4);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(bar(mi.it_full[i]), 1);
      mbar_init(bar(mi.it_empty[i]), 19);
      mbar_init(bar(mi.comb[i]), 16);
    }
    mbar_init(bar(mi.done), 1);
    mi.fail = 0;
    fence_mbar_init();
  }
  if (warp == 16) tmem_alloc(smem_u32(&mi.tmem), 512);
  griddep_wait();

  // ---------------- items before each group of sessions
  auto items_of = [&](int s) -> long long {
    if (s >= a.b.S) return 0;
    const Span x = make_span(a, s);
    return (long long)((x.np + step - 1) / step) * a.b.Hkv;
  };
  const int groups = (a.b.S + a.per_group - 1) / a.per_group;
  long long run = 0;
  for (int base = 0; base < groups; base += kThreads) {
    const int i = base + tid;
    long long x = 0;
    if (i < groups)
      for (int k = 0; k < a.per_group; ++k) x += items_of(i * a.per_group + k);
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) mi.warp_sum[warp] = inc;
    __syncthreads();
    long long exc = run + inc - x;
    for (int w = 0; w < warp; ++w) exc += mi.warp_sum[w];
    if (i < groups) mi.prefix[i] = exc;
    for (int w = 0; w < kThreads / 32; ++w) run += mi.warp_sum[w];
    __syncthreads();
  }
  if (tid == 0) mi.prefix[groups] = run;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mi.tmem;
  const long long total = run;
  volatile int* fail = &mi.fail;
  auto wwait = [&](uint64_t& b, int phase, int code) -> bool {
    const uint32_t ad = bar(b), par = (uint32_t)phase & 1u;
    const bool quit = FAULT && code == a.give_up;
    if (!quit && __all_sync(0xffffffffu, mbar_try_wait(ad, par))) return true;
    const uint64_t t0 = global_timer_ns();
    while (quit || !__all_sync(0xffffffffu, mbar_try_wait(ad, par))) {
      if (__any_sync(0xffffffffu, *fail != 0)) return false;
      if (quit || __any_sync(0xffffffffu, global_timer_ns() - t0 > kTimeoutNs)) {
        if (lane == 0) {
          *fail = 1;
          record_status(g_weigh_status, PA_ERR_TIMEOUT, blockIdx.x, code);
        }
        return false;
      }
    }
    return true;
  };
  // K slots first (a ring for each block of an item, so that each is filled by one
  // warp that sees all of its phases), then Q slots
  auto k_at = [&](int b, int slot) { return b * a.nk + slot; };
  auto q_at = [&](int slot) { return a.pair * a.nk + slot; };
  auto tile_at = [&](int at) { return smem + at * S::TILE; };

  if (warp == 17) {
    // ---------------- items and loads
    const bool lead = elect_one();
    if (lead) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
    }
    const long long span = a.run ? (total + gridDim.x - 1) / gridDim.x : 1;
    long long k = a.run ? blockIdx.x * span : blockIdx.x;
    const long long k_end = a.run ? min(total, k + span) : total, k_step = a.run ? 1 : gridDim.x;
    int it = 0, n_q = 0;
    Ring qr;
    bool ok = true;
    int s = -1, g = 0, blk = 0, nblk = 0;
    Span x{};
    bool q_held = false;
    for (; k < k_end && ok; k += k_step) {
      // ---- item k: the next one of the run, or looked up
      bool same = false;
      if (a.run && s >= 0) {
        same = ++blk < nblk;
        if (!same) blk = 0, ++g;
      }
      if (!a.run || s < 0 || g == a.b.Hkv) {
        int lo = 0, hi = groups;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (mi.prefix[mid] <= k) lo = mid;
          else hi = mid;
        }
        long long rest = k - mi.prefix[lo];
        s = lo * a.per_group;
        for (;;) {  // at most per_group sessions
          x = make_span(a, s);
          nblk = (x.np + step - 1) / step;
          const long long c = (long long)nblk * a.b.Hkv;
          if (rest < c || s + 1 >= a.b.S) break;
          rest -= c;
          ++s;
        }
        if (nblk == 0) break;
        g = (int)(rest / nblk);
        blk = (int)(rest % nblk);
      }
      const int v0 = blk * step, v1 = min(v0 + step, x.np);
      const int t_first = x.page_index(v0) * kPage, t_last = x.page_index(v1 - 1) * kPage + kPage - 1;
      // rows that see any of the item's tokens
      const int i0 = max(0, t_first - x.p0);
      const int i1 = a.w.window == 0 || v0 < x.ns || t_first < a.w.sinks
                         ? x.n
                         : (int)min((long long)x.n, (long long)t_last + a.w.window - x.p0);
      const int rt0 = i0 >> lt, rt1 = (i1 + (1 << lt) - 1) >> lt;
      const bool one = x.n <= 1 << lt;  // one tile of columns: the Q tile stays
      const bool q_new = !one || !same || !q_held;
      const bool q_last = !one || !a.run || k + 1 >= k_end || blk + 1 >= nblk;
      const int e = it % kQueue;
      if (it >= kQueue && !wwait(mi.it_empty[e], it / kQueue - 1, 1)) break;
      if (lane == 0) {
        Item& im = mi.items[e];
        im.x = x;
        im.s = s;
        im.g = g;
        im.v0 = v0;
        im.rt0 = one ? 0 : rt0;
        im.rt1 = one ? 1 : max(rt1, rt0);
        im.q_new = q_new;
        im.q_last = q_last;
        mbar_arrive(bar(mi.it_full[e]));
      }
      ++it;
      // ---- Q tiles and their lse
      if (q_new) {
        for (int rt = one ? 0 : rt0; rt < (one ? 1 : rt1); ++rt) {
          const int tok = rt << lt;
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 32 * i + lane, t = tok + (c >> a.lg);
            const float l = t < x.n ? a.lse[(size_t)(x.r0 + t) * a.b.Hq + (g << a.lg) + (c & ((1 << a.lg) - 1))] : 0.f;
            v[i] = l == -INFINITY ? -INFINITY : -l * kLog2e;  // a row that sees nothing weighs nothing
          }
          if (qr.phase > 0 && !(ok = wwait(mi.qempty[qr.slot], qr.phase - 1, 3))) break;
          const uint32_t fb = bar(mi.qfull[qr.slot]);
          if (lead) {
            mbar_arrive_expect_tx(fb, S::TILE);
#pragma unroll
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(smem_u32(tile_at(q_at(qr.slot)) + h * S::BLK), &tq, 64 * h, g << a.lg, x.r0 + tok, fb);
          }
          ++n_q;
#pragma unroll
          for (int i = 0; i < 4; ++i) mi.nlse[qr.slot][32 * i + lane] = v[i];
          __syncwarp();
          if (lane == 0) mbar_arrive(fb);
          qr.next(a.nq);
        }
        q_held = one;
      }
    }
    const int e = it % kQueue;
    if (it < kQueue || wwait(mi.it_empty[e], it / kQueue - 1, 4)) {
      if (lane == 0) {
        mi.items[e].v0 = -1;
        mbar_arrive(bar(mi.it_full[e]));
      }
    }
    // loads in flight land before the CTA ends (all have, unless a wait gave up)
    for (int i = max(0, n_q - a.nq); i < n_q; ++i) mbar_wait_bounded(bar(mi.qfull[i % a.nq]), (i / a.nq) & 1, kTimeoutNs);
  } else if (warp >= 18) {
    // ---------------- the items' first (warp 18) and second K blocks
    const int b = warp - 18;
    const bool lead = elect_one();
    const int oob = a.b.num_pages * a.b.Hkv * kPage;
    Ring kr;
    int n_k = 0;
    for (int it = 0;; ++it) {
      const int e = it % kQueue;
      if (!wwait(mi.it_full[e], it / kQueue, 13)) break;
      const Item& im = mi.items[e];
      const Span x = im.x;
      const int s = im.s, g = im.g, v0 = im.v0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.it_empty[e]));
      if (v0 < 0) break;
      if (b == 1 && (a.pair < 2 || v0 + 8 >= x.np)) continue;
      const int v = v0 + 8 * b + lane;
      const int pg = lane < 8 && v < x.np ? a.b.page(s, x.page_index(v)) : -1;
      const int row = pg < 0 ? oob : (pg * a.b.Hkv + g) * kPage;
      if (kr.phase > 0 && !wwait(mi.kempty[b][kr.slot], kr.phase - 1, 14)) break;
      load_pages<S::HALVES>(smem_u32(tile_at(k_at(b, kr.slot))), &tk, row, 0, min(8, x.np - v0 - 8 * b),
                            bar(mi.kfull[b][kr.slot]), lead);
      kr.next(a.nk);
      ++n_k;
    }
    for (int i = max(0, n_k - a.nk); i < n_k; ++i) mbar_wait_bounded(bar(mi.kfull[b][i % a.nk]), (i / a.nk) & 1, kTimeoutNs);
  } else if (warp == 16) {
    // ---------------- products (the whole warp walks, one elected lane issues)
    auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tm = (uint32_t)uni((int)tmem), lo = (uint32_t)uni((int)(smem_u32(smem) >> 4));
    const bool lead = elect_one();
    int it = 0, seq = 0, uses[4] = {0, 0, 0, 0};  // uses: products into each score buffer
    Ring kr[2], qr, qcur;
    bool ok = true;
    auto commit = [&](uint64_t& b) {
      if (lead) umma_commit(bar(b));
      __syncwarp();
    };
    while (ok) {
      const int e = it % kQueue;
      if (!wwait(mi.it_full[e], it / kQueue, 5)) break;
      const Item& im = mi.items[e];
      const int v0 = uni(im.v0), np = uni(im.x.np), n = uni(im.x.n), rt0 = uni(im.rt0), rt1 = uni(im.rt1);
      const int q_new = uni(im.q_new), q_last = uni(im.q_last);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.it_empty[e]));
      if (v0 < 0) break;
      const int nb = a.pair == 2 && v0 + 8 < np ? 2 : 1;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (b < nb && ok) ok = wwait(mi.kfull[b][kr[b].slot], kr[b].phase, 6);
      for (int rt = rt0; rt < rt1 && ok; ++rt, ++seq) {
        if (q_new) {
          qcur = qr;
          qr.next(a.nq);
          if (!(ok = wwait(mi.qfull[qcur.slot], qcur.phase, 7))) break;
        }
        const int cols = min(128, (n - (rt << lt)) << a.lg), N = (cols + 15) & ~15;
        const uint32_t idesc = umma_idesc_bf16(128, N, false, false);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b >= nb || !ok) continue;
          const int buf = a.pair == 2 ? (seq & 1) * 2 + b : seq & 3;
          int u = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) u = i == buf ? uses[i]++ : u;
          if (u > 0 && !(ok = wwait(mi.sempty[buf], u - 1, 8))) continue;
          tc_fence_after();
          const uint32_t ka = lo + k_at(b, kr[b].slot) * (S::TILE >> 4), qa = lo + q_at(qcur.slot) * (S::TILE >> 4);
          if (lead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t o = (k >> 2) * (S::BLK >> 4) + (k & 3) * 2;
              umma_bf16(tm + buf * 128, sdesc_sw128_lo(ka + o, 1, 64), sdesc_sw128_lo(qa + o, 1, 64), idesc,
                        k > 0 ? 1u : 0u);
            }
            umma_commit(bar(mi.sfull[buf]));
          }
          __syncwarp();
        }
        if (ok && q_last) commit(mi.qempty[qcur.slot]);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (b < nb && ok) {
          commit(mi.kempty[b][kr[b].slot]);
          kr[b].next(a.nk);
        }
      ++it;
    }
    commit(mi.done);  // every product has completed before the tensor memory is released
    mbar_wait_bounded(bar(mi.done), 0, kTimeoutNs);
    __syncwarp();
  } else {
    // ---------------- sums: group of warps `buf` reads score buffer `buf`, key (= TMEM lane) `key`
    const int buf = warp >> 2, key = (warp & 3) * 32 + lane;
    const uint32_t t_s = tmem + buf * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const int blk = a.pair == 2 ? buf & 1 : 0;               // its key block of an item
    const int mine = a.pair == 2 ? buf >> 1 : buf, of = a.pair == 2 ? 2 : 4;  // its turn among the column tiles
    int it = 0, seq = 0, uses = 0;
    Ring qr, qcur;
    bool ok = true;
    while (ok) {
      const int e = it % kQueue;
      if (!wwait(mi.it_full[e], it / kQueue, 9)) break;
      const Item& im = mi.items[e];
      if (im.v0 < 0) break;
      const Span& x = im.x;
      const int v0 = im.v0 + 8 * blk, rt0 = im.rt0, rt1 = im.rt1, p0 = x.p0, n = x.n;
      const bool there = v0 < x.np, q_new = im.q_new, q_last = im.q_last;
      // who adds the item's sums to the scores: the group whose turn the only column
      // tile is, else the block's first group; it asks for what it needs now
      const bool single = rt1 - rt0 == 1, owner = single ? seq % of == mine : mine == 0;
      // Nothing to add up: the barriers only (see below).  64 sessions of 2000-8000,
      // 8/8 heads, dims 64: 99 -> 88 us, bound by these warps' steps per item; with
      // dims 128, bound by memory, the shorter way made it slower (231 -> 247 us for
      // 64 sessions of 2000-20000): the warps then poll beside the loaders.
      if (D == 64 && a.run && single && !owner) {
        if (q_new) {
          qcur = qr;
          qr.next(a.nq);
        }
        if (!(ok = wwait(mi.qfull[qcur.slot], qcur.phase, 11))) break;
        ++seq;
        __syncwarp();
        if (lane == 0) {
          if (q_last) mbar_arrive(bar(mi.qempty[qcur.slot]));
          mbar_arrive(bar(mi.comb[e]));
          mbar_arrive(bar(mi.it_empty[e]));
        }
        ++it;
        continue;
      }
      const int v1 = min(v0 + 8, x.np);
      const int t = x.page_index(v0 + (key >> 4)) * kPage + (key & 15);  // this thread's token
      const int t_first = x.page_index(v0) * kPage, t_last = x.page_index(max(v1 - 1, 0)) * kPage + kPage - 1;
      // rows that see token t: indices [i0, i1)
      const bool always = a.w.window == 0 || t < a.w.sinks;
      const int i0 = max(0, t - p0), i1 = always ? n : (int)min((long long)n, (long long)t + a.w.window - p0);
      const bool writes = owner && v0 + (key >> 4) < x.np && t < x.kv && t < a.max_tokens;
      float* score = a.scores + ((size_t)im.s * a.b.Hkv + im.g) * a.max_tokens + t;
      float old = 0.f;
      bool hole = false;
      if (writes) {
        old = *score;
        hole = a.b.page(im.s, t / kPage) < 0;
      }
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // one column tile, in Q slot q
      auto tile = [&](int rt, const Ring& q) -> bool {
        const int tok = rt << lt, cols = min(128, (n - tok) << a.lg);
        // every key of the block sees every column
        const bool all = cols == 128 && v1 - v0 == 8 && p0 + tok >= t_last &&
                         (a.w.window == 0 || (v0 >= x.ns && p0 + tok + (128 >> a.lg) - 1 < (long long)t_first + a.w.window) ||
                          t_last < a.w.sinks);
        if (!wwait(mi.sfull[buf], uses++, 10)) return false;
        tc_fence_after();
        // the columns [cl, cr) of the tile see the key
        const int cl = min(max(i0 - tok, 0), 1 << lt) << a.lg, cr = min(max(i1 - tok, 0), 1 << lt) << a.lg;
        const float* nl = mi.nlse[q.slot];
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        auto chunk = [&](auto all_tag, float(&y)[32], int c) {
          constexpr bool ALL = decltype(all_tag)::value;
          uint32_t see = 0xffffffffu;  // bit i: column 32 c + i sees the key
          if (!ALL) {
            const int l0 = min(max(cl - 32 * c, 0), 32);
            const int l1 = min(max(cr - 32 * c, 0), 32);
            see = l1 > l0 ? (0xffffffffu >> (32 - (l1 - l0))) << l0 : 0u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(nl + 32 * c + i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float2 z = ffma2(make_float2(y[i + 2 * k], y[i + 2 * k + 1]), sc,
                               k == 0 ? make_float2(l4.x, l4.y) : make_float2(l4.z, l4.w));
              if (!ALL) {
                z.x = see >> (i + 2 * k) & 1 ? z.x : -INFINITY;
                z.y = see >> (i + 2 * k + 1) & 1 ? z.y : -INFINITY;
              }
              const int pr = (i >> 1) + k;
              const bool fma = ALL && (pr * kFmaPairs) / 16 != ((pr + 1) * kFmaPairs) / 16;
              sum[k] = fadd2(sum[k], fma ? exp2_fma(z) : make_float2(ex2(z.x), ex2(z.y)));
            }
          }
        };
        auto sweep = [&](auto all_tag) {
          const int nc = (cols + 31) >> 5;
#pragma unroll 1
          for (int c = 0; c < nc; ++c) {
            float y[32];
            tmem_ld32(t_s + 32 * c, y);
            tmem_wait_ld_into(y);
            chunk(all_tag, y, c);
          }
        };
        if (all) sweep(std::true_type{});
        else sweep(std::false_type{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(mi.sempty[buf]));
        return true;
      };
      // In a run every warp waits for every tile, its turn or not, and arrives when
      // the slot is given back, so that its arrival belongs to this use of the slot.
      // Else every tile is loaded anew, and a group takes the slots of its turn,
      // always the same ones (the ring's size is a multiple of the turns).
      const int skip = a.run ? 0 : (mine - seq) & (of - 1);
      if (!a.run) {
        qcur = qr;
        qcur.skip(skip, a.nq);
      }
      for (int rt = rt0 + skip; rt < rt1; rt += a.run ? 1 : of) {
        if (a.run && q_new) {
          qcur = qr;
          qr.next(a.nq);
        }
        if (!(ok = wwait(mi.qfull[qcur.slot], qcur.phase, 11))) break;
        if (there && (!a.run || seq % of == mine) && !(ok = tile(rt, qcur))) break;
        __syncwarp();
        if (lane == 0 && (!a.run || q_last)) mbar_arrive(bar(mi.qempty[qcur.slot]));
        if (a.run) ++seq;
        else qcur.skip(of, a.nq);
      }
      if (!a.run) {
        qr.skip(rt1 - rt0, a.nq);
        seq += rt1 - rt0;
      }
      if (!ok) break;
      // ---------------- the item's end: the groups of a block join their sums
      float w = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (!single) mi.ex[e][buf][key] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.comb[e]));
      if (!single && owner) {
        if (!(ok = wwait(mi.comb[e], it / kQueue, 12))) break;
        w = 0.f;
        for (int j = 0; j < of; ++j) w += mi.ex[e][a.pair == 2 ? 2 * j + blk : j][key];
      }
      if (writes && !hole) *score = old + w;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.it_empty[e]));
      ++it;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*fail) settle();
  if (warp == 16) tmem_free(tmem, 512);
}

template <int D>
pa_status launch(WeighArgs& a, const pa_sessions& b, const void* q, const void* k_pool, cudaStream_t cs) {
  CUtensorMap tq, tk;
  const int G = 1 << a.lg;
  if (!tmap_q(&tq, q, b.num_rows, b.num_q_heads, D, G, 128 / G) ||
      !tmap_pool(&tk, k_pool, b.num_pages_in_pool, b.num_kv_heads, D))
    return PA_ERR_CUDA;
  const pa_device dev = pa_current_device();
  const int sms = dev.sms;
  // The longest possible line: every session at the table's width (or its window).
  int64_t pages = b.max_pages;
  if (a.w.window) {
    const int64_t seen = ((int64_t)a.w.window + b.num_rows + 14) / kPage + 1 + ((int64_t)a.w.sinks + 15) / kPage + 1;
    if (seen < pages) pages = seen;
  }
  // K blocks in pairs halve the Q traffic; single ones when each of them can have
  // an SM of its own: a chunk of 2000 rows, 8/8 heads of 64, over 2000 tokens (64
  // pairs) 25 us in pairs, 16 us single; 512 rows, 32/8 heads of 128, over 4096
  // tokens (128 pairs) 28.5 and 30.7 us, over 8192 tokens x 4 sessions 156 and
  // 176 us; the decode step of 20000 tokens 13.6 and 17.3 us
  const int64_t pairs = (pages + 15) / 16 * b.num_kv_heads * b.n_sessions;
  a.pair = 2 * pairs > sms ? 2 : 1;
  const int64_t line = (pages + 8 * a.pair - 1) / (8 * a.pair) * b.num_kv_heads * b.n_sessions;
  const int grid = (int)(line < sms ? line : sms);
  // few rows (one tile of columns a session): K streams (runs of items, the Q tile
  // stays); many: Q streams.  8 sessions of 4000-8000, 32/8 heads of 128: 20 rows
  // each 30.8 us with K streaming, 37.9 us with Q; 64 rows 53.6 and 54.0 us; 128
  // rows 93.7 and 90.4 us; one session with 512 rows over 8192 tokens 74.5 and 55.9 us
  a.run = (int64_t)b.num_rows * G <= (int64_t)128 * b.n_sessions;
  a.nq = a.run ? 2 : Shape<D>::SLOTS - 2;  // 4 or 8 when not a.run: a multiple of the groups' turns
  a.nk = (Shape<D>::SLOTS - a.nq) / a.pair;
  a.per_group = (b.n_sessions + kGroups - 1) / kGroups;
  constexpr int smem = weigh_smem<D>();
  auto* kernel = a.give_up ? weigh_kernel<D, true> : weigh_kernel<D, false>;
  static std::atomic<uint64_t> allowed[2];
  if (!pa_allow_smem(kernel, smem, dev.index, allowed[a.give_up ? 1 : 0])) return PA_ERR_CUDA;
  return pa_launch_early(kernel, dim3(grid), dim3(kThreads), smem, cs, 1, a, tq, tk) ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_weigh_tokens(const pa_sessions* b, int32_t window, int32_t sinks, float softmax_scale,
                                     const void* q, const void* k_pool, const float* lse, float* scores,
                                     int64_t max_tokens, void* stream) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (window < 0 || sinks < 0 || max_tokens < 1 || !scores || !pa_scale_ok(softmax_scale))
    return PA_ERR_INVALID;
  if (b->num_rows == 0) return PA_OK;
  if (!q || !k_pool || !lse || !pa_aligned16(q) || !pa_aligned16(k_pool)) return PA_ERR_INVALID;
  pa::WeighArgs a{};
  a.b = pa_device_sessions(*b);
  a.w = pa_window(window, sinks);
  const int G = b->num_q_heads / b->num_kv_heads;
  a.lg = G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
  a.give_up = pa_take_fault();
  a.lse = lse;
  a.scores = scores;
  a.max_tokens = max_tokens;
  a.scale_log2 = (softmax_scale != 0.f ? softmax_scale : 1.f / sqrtf((float)b->head_dim)) * pa::kLog2e;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return b->head_dim == 64 ? pa::launch<64>(a, *b, q, k_pool, cs) : pa::launch<128>(a, *b, q, k_pool, cs);
}

extern "C" pa_status pa_weigh_status(void* stream, pa_status* out) {
  if (!out) return PA_ERR_INVALID;
  return pa_take_status(pa::g_weigh_status, static_cast<cudaStream_t>(stream), out);
}
