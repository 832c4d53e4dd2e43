// Attention of the last rows of every session over its paged cache: causal,
// with a sliding window and sinks (pa_window_attend), on the 5th-generation
// tensor cores.
//
// A row at cached position p sees token t when t <= p and (t > p - window or
// t < sinks); out = sum_t e^{s_t - m} v_t / l, lse = m + ln l in one pass over
// the visible tokens with a running maximum m and sum l.
//
// Tiles.  The rows of one kv head are (token, head of the group) pairs, 128 to
// a tensor-core tile.  A work item is (session, up to 256 / G tokens, kv head)
// over the pages that any of its rows sees, 8 pages (128 keys) a block:
//   pair   more than 128 rows: two tiles share every K, V block
//   alone  at most 128 rows: one tile; even blocks go to one accumulator and
//          softmax group, odd blocks to the other, joined at the item's end
// so in both forms two softmax groups alternate and the tensor cores always
// have a product to run while a group works on its scores.
//
// Schedule.  The kv heads are dealt to `lanes` (up to 4); a lane's items' blocks
// form a line, cut into equal spans, one per CTA (one CTA per SM): every SM gets
// the same work whatever the lengths, and the CTAs of the lanes walk the same
// pages side by side (a page holds its heads one behind the other).  Lengths live
// on the device, so every CTA sums the items' blocks itself to find its span.  An
// item cut by a span's end leaves normalised partial rows (o, lse) in the
// workspace, at most two a CTA, joined by a short second launch.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax groups, one thread per row;
// warp 8 issues the products; warp 9 walks the items and loads (TMA).  Per
// block and tile: S = Q K^T (TMEM), P = exp2(S c - m c) written over S as P_hi + P_lo,
// O += P V (TMEM).  P_hi is P rounded or cut to bf16, so that P - P_hi is exact in fp32,
// P_lo that rest rounded to bf16: together within 2^-16 of P, as the planned decode's
// weights (one bf16 alone is off by up to 2^-8 of a weight, up to 0.9 % of an output); l
// sums P.
//   items of at most 64 rows   each row has two lanes of the tile (Q is loaded to both),
//     16 rows to a warp's 32 lanes: one lane writes P_hi, the other P_lo, one product
//     serves both and the epilogue adds the two
//   more rows                  two products, P_hi V and P_lo V
// The running maximum is raised, and O rescaled, only when it grows by more than 2^8:
// numerator and denominator use the same maximum, so the result is unchanged.
//
// Measured: with one bf16 64 windowed decodes 178 us, windowed chunks 43 us, a prompt
// chunk 1.92 ms; as it is 181 us, 47 us, 2.5 ms; with two products for few rows too 192
// us, 64 decodes of 3000-4000 tokens 164 and not 155 us.  The rests by masks and packed
// fp32 steps in place of mixed-precision ones: 199 us, 50 us, 2.6 ms.  Before that step,
// weights handed over at once 2.75 ms and 51 us, P_hi first (in 1, 2 or 4 parts) and P_lo
// while its product runs 2.8, 2.85, 3.4 ms and 54, 56, 65 us: with two tiles the product
// warp then waits where it could serve the other one.
//
// Bounds and measured device times, 32/8 heads of 128: decode rows by the bytes of
// the visible cache and by how long a block's slots are held through its softmax (64
// sessions, window 4096: 1.08 GB in 181 us, 6.0 TB/s; two of 100001-131072: 0.98 GB in
// 160 us, 6.1 TB/s); a prompt chunk of 4096 rows over 32768 tokens by the chain scores -
// softmax - product of a tile, two tiles being all that tensor memory holds at 128 dims,
// and by power (2.25 ms alone, 2.5-2.6 ms in a loop, 0.79-0.92 PFLOP/s of the definition's
// operations, 1.5 times as many done; tensor pipe 76%, exponential pipe 51% busy); a call
// of one short item by its steps, about 12 us.
#include <type_traits>

#include "ptx.cuh"
#include "sessions.cuh"
#include "tmap.h"
#include "umma.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 384;
constexpr int kMaxChunks = 256;      // chunks of kThreads tile slots that a CTA sums
constexpr int kQueue = 2;            // entries of the CTA's item queue
// items of at most so many blocks are not cut: 8 windowed chunks of 1-700 rows 47 us,
// all items cut 55 us; whole up to 32 blocks: 4 sessions of 4096, 3 rows, 46 and 28 us
constexpr int kWholeBlocks = 8;
// most kv heads walked side by side (148 SMs = 37 spans of 4); 1: 64 windowed decodes
// 204 and 180 us, 64 of 300-1000 with 5 rows 67 and 60 us
constexpr int kLanes = 4;
constexpr int kTwinRows = 64;        // most rows of an item that has each in two lanes
constexpr float kRaise = 8.f;        // log2 growth of a maximum that raises it
constexpr uint64_t kTimeoutNs = 2000000000ull;

// First failure of a device-side wait since pa_window_status(NULL, ...) last read it.
__device__ int32_t g_window_status[4];

struct Desc {  // a partial item at the head of a CTA's span
  int first, last;  // spans that share the item
  int slot0;        // partial slot of the first
  int row0, n_tok, g, pad0, pad1;
};

struct AttendArgs {
  Sessions b;
  Window w;
  int lg;              // log2 G
  int slots, min_span, lanes;
  int whole;           // items are not cut: a CTA takes those that start in its span
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* status;
  Desc* desc;
  float *part_lse, *part_o;  // [2 grid][256], [2 grid][256][D]
};

// What an item's tile slot covers: tokens [i0, i0 + n_tok) of session s, and
// the virtual pages that its rows see: pages 0 .. ns - 1 (sinks), then from
// page ns + off on, np in all.
struct Tile {
  int s, r0, i0, n_tok, p0;  // r0: first row of the tile; p0: its position
  int np, ns, off;
  __device__ __forceinline__ int blocks() const { return (np + 7) >> 3; }
  __device__ __forceinline__ int page_index(int v) const { return v < ns ? v : v + off; }
};

// Sessions' first rows and lengths, from the device arrays or a shared copy.
struct FromGlobal {
  const Sessions& b;
  __device__ __forceinline__ int begin(int s) const { return b.row_begin(s); }
  __device__ __forceinline__ int kv(int s) const { return b.kv_len(s); }
};
struct FromShared {
  const int *cu, *len;
  __device__ __forceinline__ int begin(int s) const { return cu[s]; }
  __device__ __forceinline__ int kv(int s) const { return len[s]; }
};

// Tile slots: session s owns [begin(s) / T + s, begin(s + 1) / T + s + 1), at
// least as many as it has tiles of T = 2^lt tokens; the rest are empty.
template <typename From>
__device__ __forceinline__ Tile make_tile(const AttendArgs& a, const From& f, int slot, int s) {
  const int lt = 8 - a.lg;
  Tile t;
  t.s = s;
  const int b0 = f.begin(s), n = f.begin(s + 1) - b0, kv = f.kv(s);
  t.i0 = (slot - ((b0 >> lt) + s)) << lt;
  t.n_tok = min(1 << lt, n - t.i0);
  t.r0 = b0 + t.i0;
  t.p0 = kv - n + t.i0;
  t.np = t.ns = t.off = 0;
  if (t.n_tok <= 0 || t.i0 < 0) {
    t.n_tok = 0;
    return t;
  }
  const int p1 = max(t.p0 + t.n_tok - 1, 0);  // last position; rows that all see nothing get page 0, masked
  const int last = p1 / kPage, first = a.w.first(max(t.p0, 0)) / kPage;
  const int sink = (min(a.w.sinks, p1 + 1) + kPage - 1) / kPage;
  if (sink < first) {
    t.ns = sink;
    t.off = first - sink;
  }
  t.np = last + 1 - t.off;
  return t;
}

// Session of a slot by bisection (one thread).
template <typename From>
__device__ __forceinline__ int find_slot_session(const From& f, int S, int slot, int lt) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((f.begin(mid) >> lt) + mid <= slot) lo = mid;
    else hi = mid;
  }
  return lo;
}

// An entry of the item queue: a segment [b0, b1) of an item's blocks.
struct Item {
  Tile t;
  int g, b0, b1;
  int part;  // partial slot, -1: the whole item
};

struct Misc {
  uint64_t full[8], empty[8];          // ring
  uint64_t q_full, q_empty, o_free, joined, done;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t it_full[kQueue], it_empty[kQueue];
  uint32_t tmem;
  int fail;
  Item items[kQueue];
  float2 exch[2][128];                 // (m, l) of the two groups
};

template <int D>
struct Shape {
  static constexpr int HALVES = D / 64;
  static constexpr int BLK = 128 * 128;               // 128 rows x 64 dims
  static constexpr int TILE = HALVES * BLK;           // a Q tile, a K block, a V block
  static constexpr int NS = D == 128 ? 5 : 8;         // ring slots
  static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE, OFF_MISC = OFF_RING + NS * TILE;
  static constexpr int SMEM = OFF_MISC + (int)sizeof(Misc);
  static constexpr uint32_t T_S = 0, T_O = 256;       // TMEM columns: S0, S1, O0, O1
};
static_assert(Shape<128>::SMEM <= 232448 && Shape<64>::SMEM <= 232448, "shared memory");

// What a CTA finds its span with (aliases the ring before any load): sums of
// kThreads slots' blocks, per chunk, and a copy of the sessions' rows and
// lengths when there are at most kCopied (bisecting the device arrays costs a
// memory round trip a step).
constexpr int kCopied = 4096;
struct Sums {
  long long chunk[kMaxChunks];
  long long warp[kThreads / 32];
  long long lo_rest;
  int lo_slot, pad;
  int cu[kCopied + 1], len[kCopied];
};
static_assert(sizeof(Sums) <= 5 * Shape<64>::TILE, "ring");

// FAULT: the kernel of a call whose waits number give_up give up (pa_session_fault); a
// comparison in every wait would cost all calls 3 %
template <int D, bool FAULT>
__global__ void __launch_bounds__(kThreads, 1)
    window_attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tq16, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const int give_up) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the swizzle needs it; the kernel has no other shared memory before it
    griddep_wait();
    if (threadIdx.x == 0) {
      a.desc[blockIdx.x].first = -1;
      record_status(a.status, PA_ERR_DEVICE, blockIdx.x, 0);
      record_status(g_window_status, PA_ERR_DEVICE, blockIdx.x, 0);
    }
    return;
  }
  Misc& mi = *reinterpret_cast<Misc*>(smem + S::OFF_MISC);
  Sums& su = *reinterpret_cast<Sums*>(smem + S::OFF_RING);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lt = 8 - a.lg;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (tid == 0) {
    for (int i = 0; i < S::NS; ++i) {
      mbar_init(bar(mi.full[i]), 1);
      mbar_init(bar(mi.empty[i]), 1);
    }
    mbar_init(bar(mi.q_full), 1);
    mbar_init(bar(mi.q_empty), 1);
    mbar_init(bar(mi.o_free), 8);
    mbar_init(bar(mi.joined), 8);
    mbar_init(bar(mi.done), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(mi.s_full[i]), 1);
      mbar_init(bar(mi.p_full[i]), 4);
      mbar_init(bar(mi.o_full[i]), 1);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(bar(mi.it_full[i]), 1);
      mbar_init(bar(mi.it_empty[i]), 9);  // product warp, 8 softmax warps
    }
    mi.fail = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tq16);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }

  griddep_wait();
  if (tid == 0 && blockIdx.x == 0) *a.status = 0;

  // ---------------- the line of blocks and this CTA's span
  const int heads = a.b.Hkv / a.lanes, in_lane = blockIdx.x % a.lanes;  // head k of the lane is k lanes + in_lane
  const bool copied = a.b.S <= kCopied;
  if (copied) {
    for (int s = tid; s <= a.b.S; s += kThreads) {
      su.cu[s] = a.b.row_begin(s);
      if (s < a.b.S) su.len[s] = a.b.kv_len(s);
    }
    __syncthreads();
  }
  auto slot_blocks = [&](int slot) -> long long {
    if (slot >= a.slots) return 0;
    auto blocks = [&](auto f) { return make_tile(a, f, slot, find_slot_session(f, a.b.S, slot, lt)).blocks(); };
    return (long long)(copied ? blocks(FromShared{su.cu, su.len}) : blocks(FromGlobal{a.b})) * heads;
  };
  // exclusive prefix of x over the CTA's threads, and its sum
  auto scan = [&](long long x, long long& sum) -> long long {
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) su.warp[warp] = inc;
    __syncthreads();
    long long before = 0;
    sum = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) before = sum;
      sum += su.warp[w];
    }
    return before + inc - x;
  };
  const int n_chunks = (a.slots + kThreads - 1) / kThreads;
  long long total = 0, x = 0, exc = 0, sum = 0;
  for (int c = 0; c < n_chunks; ++c) {
    x = slot_blocks(c * kThreads + tid);
    exc = scan(x, sum);
    if (tid == 0) su.chunk[c] = sum;
    total += sum;
  }
  const int spans = gridDim.x / a.lanes, mine = blockIdx.x / a.lanes;
  const long long span = max((long long)a.min_span, (total + spans - 1) / spans);
  const long long lo = mine * span, hi = min(total, lo + span);
  if (lo >= total) {
    if (tid == 0) a.desc[blockIdx.x].first = -1;
    return;  // uniform over the CTA
  }
  if (warp == 8) tmem_alloc(smem_u32(&mi.tmem), 512);
  {
    int c = 0;
    if (n_chunks > 1) {
      __syncthreads();
      long long before = 0;
      while (before + su.chunk[c] <= lo) before += su.chunk[c++];
      x = slot_blocks(c * kThreads + tid);
      exc = before + scan(x, sum);
    }
    if (x > 0 && exc <= lo && lo < exc + x) {
      su.lo_slot = c * kThreads + tid;
      su.lo_rest = lo - exc;
    }
    __syncthreads();
  }
  const int lo_slot = su.lo_slot;
  const long long lo_rest = su.lo_rest;
  fence_proxy_async_smem();  // the ring held the sums
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = mi.tmem;
  volatile int* fail = &mi.fail;

  // A whole warp waits for a phase; false when that took kTimeoutNs, or when
  // another role has given up.  A phase that is over costs one vote: the branch
  // is uniform (a loop that lanes leave one by one took 100 cycles).
  auto wwait = [&](uint64_t& b, int phase, int code) -> bool {
    const uint32_t ad = bar(b), par = (uint32_t)phase & 1u;
    const bool quit = FAULT && code == give_up;
    if (!quit && __all_sync(0xffffffffu, mbar_try_wait(ad, par))) return true;
    const uint64_t t0 = global_timer_ns();
    while (quit || !__all_sync(0xffffffffu, mbar_try_wait(ad, par))) {
      if (__any_sync(0xffffffffu, *fail != 0)) return false;
      if (quit || __any_sync(0xffffffffu, global_timer_ns() - t0 > kTimeoutNs)) {
        if (lane == 0) {
          *fail = 1;
          record_status(a.status, PA_ERR_TIMEOUT, blockIdx.x, code);
        }
        return false;
      }
    }
    return true;
  };
  // Ring position of the loads of a segment of n blocks whose first load is
  // number `base`: K0 K1 V0 K2 V1 ... V(n-1), the order in which they are used.
  auto pos_k = [](int base, int j) { return j == 0 ? base : base + 2 * j - 1; };
  auto pos_v = [](int base, int j, int n) { return j < n - 1 ? base + 2 * j + 2 : base + 2 * n - 1; };
  uint8_t* ring = smem + S::OFF_RING;

  // Registers: 384 threads x 168 at launch; a softmax thread holds a row of
  // scores: 2 x 128 x 216 + 128 x 72 = 64512
  if (warp == 9) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------- items and loads
    const bool lead = elect_one();
    const FromGlobal from{a.b};
    int slot = lo_slot;
    Tile t = make_tile(a, from, slot, find_slot_session(from, a.b.S, slot, lt));
    int b0 = (int)(lo_rest % t.blocks()), head = (int)(lo_rest / t.blocks()), g = head * a.lanes + in_lane;
    long long left = hi - lo;
    int base = 0, it = 0, issued = 0, n_q = 0;
    bool ok = true;
    auto next_item = [&]() {  // when there is more to do
      b0 = 0;
      if (++head == heads) {
        head = 0;
        while (left > 0 && ++slot < a.slots) {
          t = make_tile(a, from, slot, find_slot_session(from, a.b.S, slot, lt));
          if (t.np > 0) break;
        }
      }
      g = head * a.lanes + in_lane;
    };
    if (a.whole && b0 > 0) {  // that item is the CTA's before
      left -= t.blocks() - b0;
      next_item();
    }
    const int oob = a.b.num_pages * a.b.Hkv * kPage;  // a row past the pool: zeros
    if (lane == 0) {
      Desc d{};
      d.first = -1;
      if (b0 > 0 && !a.whole) {
        const long long start = lo - b0, end = start + t.blocks();
        d.first = (int)(start / span);
        d.last = (int)((end - 1) / span);
        d.slot0 = 2 * (d.first * a.lanes + in_lane) + (start == d.first * span ? 0 : 1);
        d.row0 = t.r0;
        d.n_tok = t.n_tok;
        d.g = g;
      }
      a.desc[blockIdx.x] = d;
    }
    while (left > 0 && ok) {
      const int nb = t.blocks();
      const int b1 = a.whole ? nb : (int)min((long long)nb, b0 + left);
      const int n = b1 - b0, e = it % kQueue;
      if (it >= kQueue && !wwait(mi.it_empty[e], it / kQueue - 1, 1)) break;
      if (lane == 0) {
        Item& x = mi.items[e];
        x.t = t;
        x.g = g;
        x.b0 = b0;
        x.b1 = b1;
        x.part = b0 == 0 && b1 == nb ? -1 : left == hi - lo ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1;
        mbar_arrive(bar(mi.it_full[e]));
      }
      if (it > 0 && !wwait(mi.q_empty, it - 1, 2)) break;
      const int rows = t.n_tok << a.lg;
      const bool pair = rows > 128;
      ++n_q;
      if (lead && rows <= kTwinRows) {  // 16 rows to lanes 32 i .. 32 i + 15 of the tile, and again to the 16 after them
        const int n16 = (rows + 15) >> 4;
        mbar_arrive_expect_tx(bar(mi.q_full), n16 * 2 * S::HALVES * 2048);
        for (int i = 0; i < n16; ++i)
#pragma unroll
          for (int h = 0; h < 2 * S::HALVES; ++h)
            tma_load_3d(smem_u32(smem + S::OFF_Q + (h >> 1) * S::BLK + (2 * i + (h & 1)) * 2048), &tq16, 64 * (h >> 1),
                        g << a.lg, t.r0 + i * (16 >> a.lg), bar(mi.q_full));
      } else if (lead) {
        mbar_arrive_expect_tx(bar(mi.q_full), (pair ? 2 : 1) * S::TILE);
        for (int i = 0; i < (pair ? 2 : 1); ++i)
#pragma unroll
          for (int h = 0; h < S::HALVES; ++h)
            tma_load_3d(smem_u32(smem + S::OFF_Q + i * S::TILE + h * S::BLK), &tq, 64 * h, g << a.lg,
                        t.r0 + i * (128 >> a.lg), bar(mi.q_full));
      }
      __syncwarp();
      // rows of the pool of the block's pages, lane l < 8: page 8 j + l
      auto rows_of = [&](int j) -> int {
        const int v = 8 * j + lane;
        if (lane >= 8 || v >= t.np) return -1;
        const int pg = a.b.page(t.s, t.page_index(v));
        return pg < 0 ? oob : (pg * a.b.Hkv + g) * kPage;
      };
      auto load = [&](int pos, const CUtensorMap* tm, int j, int row) -> bool {
        const int sl = pos % S::NS;
        if (pos >= S::NS && !wwait(mi.empty[sl], pos / S::NS - 1, 3)) return false;
        issued = pos + 1;
        load_pages<S::HALVES>(smem_u32(ring + sl * S::TILE), tm, row, 0, min(8, t.np - 8 * j), bar(mi.full[sl]), lead);
        return true;
      };
      int row = rows_of(b0), prev = row;
      for (int j = 0; j < n && ok; ++j) {
        const int next = j + 1 < n ? rows_of(b0 + j + 1) : -1;
        ok = load(pos_k(base, j), &tk, b0 + j, row);
        if (ok && j > 0) ok = load(pos_v(base, j - 1, n), &tv, b0 + j - 1, prev);
        prev = row;
        row = next;
      }
      if (ok) ok = load(pos_v(base, n - 1, n), &tv, b1 - 1, prev);
      base += 2 * n;
      left -= n;
      ++it;
      next_item();
    }
    // end of the line for the other roles
    const int e = it % kQueue;
    if (it < kQueue || wwait(mi.it_empty[e], it / kQueue - 1, 4)) {
      if (lane == 0) {
        mi.items[e].b1 = -1;
        mbar_arrive(bar(mi.it_full[e]));
      }
    }
    // loads in flight land before the CTA ends (all of them have, unless a wait gave up)
    for (int p = max(0, issued - S::NS); p < issued; ++p)
      mbar_wait_bounded(bar(mi.full[p % S::NS]), (p / S::NS) & 1, kTimeoutNs);
    if (n_q > 0) mbar_wait_bounded(bar(mi.q_full), (n_q - 1) & 1, kTimeoutNs);
  } else if (warp == 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------- products.  The whole warp walks the blocks, one elected lane
    // issues: what the products take (descriptors, addresses) then stays in uniform
    // registers (a single-lane branch took 80-150 cycles to issue a 64-cycle product)
    constexpr uint32_t idesc_s = umma_idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_o = umma_idesc_bf16(128, D, false, true);
    auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tm = (uint32_t)uni((int)tmem);
    const uint32_t q_lo = (uint32_t)uni((int)(smem_u32(smem + S::OFF_Q) >> 4));
    const uint32_t ring_lo = (uint32_t)uni((int)(smem_u32(ring) >> 4));
    const bool lead = elect_one();
    int base = 0, it = 0, c0 = 0, c1 = 0;  // c0, c1: P phases used of each tile
    bool ok = true;
    // S = Q K^T of Q tile q into score buffer `tile`, K in ring slot sl
    auto issue_s = [&](int tile, int q, int sl) {
      tc_fence_after();
      const uint32_t qa = q_lo + q * (S::TILE >> 4), ka = ring_lo + sl * (S::TILE >> 4), d = tm + S::T_S + tile * 128;
      if (lead) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t o = (k >> 2) * (S::BLK >> 4) + (k & 3) * 2;
          umma_bf16(d, sdesc_sw128_lo(qa + o, 1, 64), sdesc_sw128_lo(ka + o, 1, 64), idesc_s, k > 0 ? 1u : 0u);
        }
        umma_commit(bar(mi.s_full[tile]));
      }
      __syncwarp();
    };
    // O += P V, V in ring slot sl
    auto issue_o = [&](int tile, int sl, int pages, bool first, bool twin) {
      tc_fence_after();
      const uint32_t va = ring_lo + sl * (S::TILE >> 4), d = tm + S::T_O + tile * D, p = tm + S::T_S + tile * 128;
      auto pv = [&](int c) {
        const uint64_t v = sdesc_sw128_lo(va + c * 128, S::BLK >> 4, 64);
        if (twin) {
          umma_bf16_ts(d, p + 8 * c, v, idesc_o, first && c == 0 ? 0u : 1u);
        } else {
          umma_bf16_ts(d, p + 16 * c, v, idesc_o, first && c == 0 ? 0u : 1u);
          umma_bf16_ts(d, p + 16 * c + 8, v, idesc_o, 1u);
        }
      };
      if (lead) {
        if (pages == 8) {
#pragma unroll
          for (int c = 0; c < 8; ++c) pv(c);
        } else {
          for (int c = 0; c < pages; ++c) pv(c);
        }
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t& b) {
      if (lead) umma_commit(bar(b));
      __syncwarp();
    };
    auto wait_load = [&](int pos) -> bool { return wwait(mi.full[pos % S::NS], pos / S::NS, 6); };
    while (ok) {
      const int e = it % kQueue;
      if (!wwait(mi.it_full[e], it / kQueue, 5)) break;
      const Item& x = mi.items[e];
      const int b1 = uni(x.b1), jb = uni(x.b0), n = b1 - jb, np = uni(x.t.np);
      const int rows = uni(x.t.n_tok) << a.lg;
      const bool pair = rows > 128, twin = rows <= kTwinRows;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.it_empty[e]));
      if (b1 < 0) break;
      if (!wwait(mi.q_full, it, 7)) break;
      if (pair) {
        const int p0 = pos_k(base, 0);
        if (!(ok = wait_load(p0))) break;
        issue_s(0, 0, p0 % S::NS);
        issue_s(1, 1, p0 % S::NS);
        commit(mi.empty[p0 % S::NS]);
        if (n == 1) commit(mi.q_empty);
        for (int j = 0; j < n; ++j) {
          const int pv = pos_v(base, j, n), pk = pos_k(base, j + 1), pages = min(8, np - 8 * (jb + j));
          const bool more = j + 1 < n;
          // tile 0
          // (what does not depend on the weights is waited for first: the way from a
          // tile's last weights to its next scores is what a block costs)
          ok = wait_load(pv) && (!more || wait_load(pk)) && (j || it == 0 || wwait(mi.o_free, it - 1, 9)) &&
               wwait(mi.p_full[0], c0, 8);
          if (!ok) break;
          ++c0;
          issue_o(0, pv % S::NS, pages, j == 0, false);
          if (more) {
            issue_s(0, 0, pk % S::NS);
          } else {
            commit(mi.o_full[0]);
          }
          // tile 1, which frees the slots
          if (!(ok = wwait(mi.p_full[1], c1, 8))) break;
          ++c1;
          issue_o(1, pv % S::NS, pages, j == 0, false);
          commit(mi.empty[pv % S::NS]);
          if (more) {
            issue_s(1, 1, pk % S::NS);
            commit(mi.empty[pk % S::NS]);
            if (j + 2 == n) commit(mi.q_empty);
          } else {
            commit(mi.o_full[1]);
          }
        }
      } else {
        for (int j = 0; j < min(n, 2); ++j) {
          const int pk = pos_k(base, j);
          if (!(ok = wait_load(pk))) break;
          issue_s(j, 0, pk % S::NS);
          commit(mi.empty[pk % S::NS]);
          if (j == n - 1) commit(mi.q_empty);
        }
        for (int j = 0; j < n && ok; ++j) {
          const int tile = j & 1, pv = pos_v(base, j, n), pages = min(8, np - 8 * (jb + j));
          const int phase = tile ? c1++ : c0++;
          const bool more = j + 2 < n;
          const int pk = pos_k(base, j + 2);
          ok = wait_load(pv) && (j || it == 0 || wwait(mi.o_free, it - 1, 11)) && wwait(mi.p_full[tile], phase, 10);
          if (!ok) break;
          issue_o(tile, pv % S::NS, pages, j < 2, twin);
          commit(mi.empty[pv % S::NS]);
          if (more) {
            if (!(ok = wait_load(pk))) break;
            issue_s(tile, 0, pk % S::NS);
            commit(mi.empty[pk % S::NS]);
            if (j + 3 == n) commit(mi.q_empty);
          } else {
            commit(mi.o_full[tile]);
          }
        }
      }
      base += 2 * n;
      ++it;
    }
    // every product issued has completed before the tensor memory is released
    commit(mi.done);
    mbar_wait_bounded(bar(mi.done), 0, kTimeoutNs);
    __syncwarp();
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---------------- softmax: group `grp`, row (= TMEM lane) quad * 32 + lane of its tile
    const int grp = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + S::T_S + grp * 128 + lane_off, t_o = tmem + S::T_O + grp * D + lane_off;
    int it = 0, base = 0, ps = 0, po = 0, pj = 0;  // phases used of s_full, o_full, joined
    bool ok = true;
    while (ok) {
      const int e = it % kQueue;
      if (!wwait(mi.it_full[e], it / kQueue, 12)) break;
      const Tile t = mi.items[e].t;
      const int g = mi.items[e].g, b0 = mi.items[e].b0, b1 = mi.items[e].b1, part = mi.items[e].part;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.it_empty[e]));
      if (b1 < 0) break;
      const int n = b1 - b0;
      const bool pair = (t.n_tok << a.lg) > 128, twin = t.n_tok << a.lg <= kTwinRows;
      const bool low = twin && (lane & 16);              // this thread writes P_lo of its row
      const int trow = twin ? quad * 16 + (lane & 15) : row;  // row of the tile
      const int tok0 = pair ? grp << (7 - a.lg) : 0;     // first token of this group's tile
      const int tok = tok0 + (trow >> a.lg);             // this row's token
      const int p = t.p0 + min(tok, t.n_tok - 1);        // rows past the tile repeat its last
      const int p_min = t.p0 + tok0, p_max = t.p0 + min(tok0 + (128 >> a.lg), t.n_tok) - 1;
      const int kv_end = a.b.kv_len(t.s), seen_from = a.w.first(max(t.p0, 0));
      // a warp without rows keeps the protocol and leaves its rows of P and O as they are
      const bool busy = __any_sync(0xffffffffu, tok < t.n_tok);
      // the page (or hole, -1) of lane's page of block j, asked for a block ahead
      auto page_of = [&](int j) -> int {
        const int v = 8 * (b0 + j) + lane;
        return j < n && lane < 8 && v < t.np ? a.b.page(t.s, t.page_index(v)) : 0;
      };
      int page_next = page_of(pair ? 0 : grp);
      float m = -INFINITY, l = 0.f;
      bool first = true;
      // (two copies; in one the registers of both ways are live: prompt chunk 2.57 -> 2.7 ms)
      auto walk = [&](auto twin_tag) {
        constexpr bool TWIN = decltype(twin_tag)::value;
        for (int j = pair ? 0 : grp; j < n && ok; j += pair ? 1 : 2) {
          const int v0 = 8 * (b0 + j), pages = min(8, t.np - v0);
          const unsigned holes = __ballot_sync(0xffffffffu, page_next < 0);
          page_next = page_of(j + (pair ? 1 : 2));
          const int t_first = t.page_index(v0) * kPage, t_last = t.page_index(v0 + pages - 1) * kPage + kPage - 1;
          const bool all = pages == 8 && holes == 0 && t_last <= p_min &&
                           (a.w.window == 0 || (v0 >= t.ns && t_first > p_max - a.w.window) || t_last < a.w.sinks);
          // tokens that no row of the item sees (past the session's end, between the
          // sinks and the first window) may hold anything: a weight of 0 times NaN is
          // NaN, so their V rows are zeroed; the first tile of a pair does it for both
          bool dead = false;
          if (!all && lane < pages) {
            const int t0 = t.page_index(v0 + lane) * kPage;
            dead = t0 + kPage > kv_end || (t0 + kPage > a.w.sinks && t0 < seen_from);
          }
          if (!(ok = wwait(mi.s_full[grp], ps++, 13))) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, dead) && (grp == 0 || !pair)) {
            const int pv = pos_v(base, j, n);
            // (after the block's scores: the slot's last use is then over, which the
            // parity of a phase alone would not tell)
            if (!(ok = wwait(mi.full[pv % S::NS], pv / S::NS, 14))) break;
            const int key = tid & 127, tk0 = t.page_index(v0 + (key >> 4)) * kPage + (key & 15);
            if ((key >> 4) < pages && (tk0 >= kv_end || (tk0 >= a.w.sinks && tk0 < seen_from))) {
              uint8_t* vt = ring + (pv % S::NS) * S::TILE + key * 128;
#pragma unroll
              for (int i = 0; i < 8 * S::HALVES; ++i)
                *reinterpret_cast<uint4*>(vt + (i >> 3) * S::BLK + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          // none of the tile's rows sees a key of the block: all weights are 0
          const bool none = t_first > p_max || (a.w.window != 0 && v0 >= t.ns && t_last <= p_min - a.w.window &&
                                                t_first >= a.w.sinks);
          if (!busy || none) {
            if (busy) {
              float z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = 0.f;
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_st32(t_s + 32 * c, z);
              tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(mi.p_full[grp]));
            continue;
          }
          float x[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, x[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld_into(x[c]);
          if (!all) {
#pragma unroll
            for (int pg = 0; pg < 8; ++pg) {
              const int t0 = t.page_index(v0 + pg) * kPage;
              const bool gone = pg >= pages || (holes >> pg & 1);
              // bit i: this row sees token t0 + i
              const int top = p - t0, under = a.w.window ? p - a.w.window - t0 : -1, sk = a.w.sinks - t0;
              const uint32_t upto = top < 0 ? 0u : 0xffffu >> (15 - min(top, 15));
              const uint32_t from = under < 0 ? 0xffffu : 0xffffu << min(under + 1, 16);
              const uint32_t sink = sk <= 0 ? 0u : 0xffffu >> (16 - min(sk, 16));
              const uint32_t see = gone ? 0u : upto & (from | sink);
              if (__any_sync(0xffffffffu, see != 0xffffu)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float& y = x[pg >> 1][16 * (pg & 1) + i];
                  y = see & (1u << i) ? y : -INFINITY;
                }
              }
            }
          }
          float mq[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mq[c] = x[c][0];
#pragma unroll
            for (int i = 1; i < 31; i += 2) mq[c] = max3(mq[c], x[c][i], x[c][i + 1]);
          }
          float mx = max3(max3(mq[0], mq[1], x[0][31]), max3(mq[2], mq[3], x[1][31]), fmaxf(x[2][31], x[3][31]));
          if (TWIN) mx = __shfl_sync(0xffffffffu, mx, lane & 15);  // both lanes of a row rescale alike
          mx *= a.scale_log2;
          if (first) {
            m = mx;
          } else if (__any_sync(0xffffffffu, mx > m + kRaise)) {
            const float mn = mx > m + kRaise ? mx : m;
            const float f = mn == -INFINITY ? 1.f : ex2(m - mn);  // O and l are 0 while m is -inf
            l *= f;
            m = mn;
#pragma unroll 1
            for (int c = 0; c < D; c += 8) tmem_scale8(t_o + c, f);
            tmem_wait_st();
          }
          first = false;
          const float mc = m == -INFINITY ? 0.f : -m;
          const float2 sc = make_float2(a.scale_log2, a.scale_log2), mm = make_float2(mc, mc);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // the weights, 32 keys at a time
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float pw[32];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 z = ffma2(make_float2(x[c][i], x[c][i + 1]), sc, mm);
              const float2 y = make_float2(ex2(z.x), ex2(z.y));
              sum[(i >> 1) & 1] = fadd2(sum[(i >> 1) & 1], y);
              if (TWIN) {  // (P_hi rounded; cut: 64 windowed decodes 188 and 182 us)
                const uint32_t hi = pack_bf16x2(y.x, y.y);
                const float2 v = minus_bf16x2(y, hi);
                const uint32_t lo = pack_bf16x2(v.x, v.y);
                pw[i >> 1] = __uint_as_float(low ? lo : hi);
              } else {  // of 16 keys 8 words P_hi, cut, and 8 words P_lo
                const uint32_t hi = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
                const float2 v = minus_bf16x2(y, hi);
                const int w = (i & 16) + ((i & 15) >> 1);
                pw[w] = __uint_as_float(hi);
                pw[w + 8] = __uint_as_float(pack_bf16x2(v.x, v.y));
              }
            }
            if (TWIN) tmem_st16<0>(t_s + 16 * c, pw);
            else tmem_st32(t_s + 32 * c, pw);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(mi.p_full[grp]));
          l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        }
      };
      if (twin) walk(std::true_type{});
      else walk(std::false_type{});
      if (!ok) break;
      // ---------------- the item's end
      const int n_mine = pair ? n : (n - grp + 1) >> 1;  // blocks of this group
      if (n_mine > 0 && !(ok = wwait(mi.o_full[grp], po++, 15))) break;
      tc_fence_after();
      // (a sum of 0: the row saw nothing; one that is NaN makes its out and lse NaN)
      float w0 = l == 0.f ? 0.f : 1.f / l, w1 = 0.f, lse2 = l == 0.f ? -INFINITY : m + lg2(l);
      int d0 = 0, dn = D;  // dims this thread writes
      uint32_t src0 = t_o, src1 = t_o;
      bool two = false;
      if (!pair) {
        mi.exch[grp][row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(mi.joined));
        if (!(ok = wwait(mi.joined, pj++, 16))) break;
        tc_fence_after();
        const float2 ml = mi.exch[grp ^ 1][row];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(mi.joined));  // read by both before the next item's are written
        if (!(ok = wwait(mi.joined, pj++, 17))) break;
        const float mm = fmaxf(m, ml.x);
        const float f0 = l == 0.f ? 0.f : ex2(m - mm), f1 = ml.y == 0.f ? 0.f : ex2(ml.x - mm);
        const float lt2 = l * f0 + ml.y * f1, inv = lt2 == 0.f ? 0.f : 1.f / lt2;
        lse2 = lt2 == 0.f ? -INFINITY : mm + lg2(lt2);
        w0 = f0 * inv;
        w1 = f1 * inv;
        d0 = grp * (D / 2);
        dn = D / 2;
        src1 = tmem + S::T_O + (grp ^ 1) * D + lane_off;
        two = n > 1;
      }
      const bool have = n_mine > 0;  // this group's accumulator was written
      const bool live = tok < t.n_tok && !low;
      const int r = t.r0 + tok, h = (g << a.lg) + (trow & ((1 << a.lg) - 1));
      const int prow = (pair ? grp * 128 : 0) + trow;
#pragma unroll 1
      for (int c = d0; c < d0 + dn; c += 32) {
        float o[32];
        if (have) {
          tmem_ld32(src0 + c, o);
          tmem_wait_ld_into(o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = have ? o[i] * w0 : 0.f;
        if (two || (!pair && !have)) {
          float o1[32];
          tmem_ld32(src1 + c, o1);
          tmem_wait_ld_into(o1);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] += o1[i] * w1;
        }
        if (twin) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], 16);
        }
        if (live) {
          if (part < 0) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((size_t)r * a.b.Hq + h) * D + c);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(dst + i / 2) =
                  make_uint4(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]),
                             pack_bf16x2(o[i + 4], o[i + 5]), pack_bf16x2(o[i + 6], o[i + 7]));
          } else {
            float* dst = a.part_o + ((size_t)part * 256 + prow) * D + c;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              st_global_v8(dst + i, o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
          }
        }
      }
      if (live && (pair || grp == 0)) {
        if (part < 0) {
          if (a.lse) a.lse[(size_t)r * a.b.Hq + h] = lse2 * kLn2;
        } else {
          a.part_lse[(size_t)part * 256 + prow] = lse2;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(mi.o_free));
      base += 2 * n;
      ++it;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*fail) {
    if (tid == 0) record_status(g_window_status, PA_ERR_TIMEOUT, blockIdx.x, 0);
    settle();
  }
  griddep_launch_dependents();
  if (warp == 8) tmem_free(tmem, 512);
}

// Joins the partial rows of the items that the spans cut: blocks (c, y) take the
// item cut at the start of the span after CTA c's, when that is its first cut.
// A warp per row; when there are few rows and many parts the block's eight warps
// per row, each every eighth part (the sum is kept in that order on every run).
// One session of 60000 tokens, 8 heads of 1 kv head, whole call: 1 row 21 us, 4 rows 23
// us, 8 rows 28 us (a warp a row and 8 blocks an item throughout: 47, 47, 66 us).  32 blocks an item (most find nothing
// to do) cost other calls nothing measurable against 8.
constexpr int kJoinY = 32;
template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(const AttendArgs a) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W = D / 32;
  const Desc d = a.desc[blockIdx.x + a.lanes];
  if (d.first != (int)blockIdx.x / a.lanes) return;
  const int in_lane = blockIdx.x % a.lanes;
  const int rows = d.n_tok << a.lg;  // tile 1 of a pair starts at row 128, token 128 / G
  __shared__ float part[8][D], part_sum[8];
  const int team = rows <= 2 * kJoinY && d.last - d.first >= 16 ? 8 : 1, rank = team == 8 ? warp : 0;
  for (int prow = (blockIdx.y * 8 + warp) / team; prow < rows; prow += kJoinY * 8 / team) {
    auto slot_of = [&](int c) { return (size_t)(c == d.first ? d.slot0 : 2 * (c * a.lanes + in_lane)) * 256 + prow; };
    float mx = -INFINITY;
    for (int c = d.first + lane; c <= d.last; c += 32) mx = fmaxf(mx, a.part_lse[slot_of(c)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float sum = 0.f, acc[W] = {};
#pragma unroll 4
    for (int c = d.first + rank; c <= d.last; c += team) {
      const size_t at = slot_of(c);
      const float pl = a.part_lse[at], f = pl == -INFINITY ? 0.f : ex2(pl - mx);
      sum += f;
#pragma unroll
      for (int i = 0; i < W; ++i) acc[i] += f * a.part_o[at * D + lane * W + i];
    }
    if (team == 8) {  // all eight warps are at the same row
#pragma unroll
      for (int i = 0; i < W; ++i) part[warp][lane * W + i] = acc[i];
      if (lane == 0) part_sum[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < 8; ++w) {
          sum += part_sum[w];
#pragma unroll
          for (int i = 0; i < W; ++i) acc[i] += part[w][lane * W + i];
        }
      }
      __syncthreads();
      if (warp) continue;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t ro = (size_t)(d.row0 + (prow >> a.lg)) * a.b.Hq + (d.g << a.lg) + (prow & ((1 << a.lg) - 1));
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ro * D) + lane * (W / 2);
#pragma unroll
    for (int i = 0; i < W; i += 2) dst[i / 2] = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (a.lse && lane == 0) a.lse[ro] = sum == 0.f ? -INFINITY : (mx + lg2(sum)) * kLn2;
  }
}

// ---------------- few rows over short caches
//
// One CTA per (row, kv head), or a cluster of up to 8 when that leaves SMs free,
// each warp a page in turn: such a call is bound by its latency, and this form
// has a fourth of the other's steps between launch and end (no tensor memory, no
// roles, no join launch).  A warp keeps its own running maxima and sums (fp32), so
// K and V of its next page are in flight while it works on one.  S (16 keys x 8
// heads of the group) by warp-level products (mma.sync; K rows straight from
// memory: the contraction may take the dims in any order, so each lane's 16-byte
// piece serves two products); the weights stay in fp32; P V on the CUDA cores; the
// warps' results are joined in shared memory, the CTAs' through the cluster's.
//
// Taken for two rows a session on average and up to 128 pages a CTA (of the table's
// width, or what a window leaves of it), 64 and 32 for groups of 4 and 8, whose P V costs
// more.  Measured, this form against the other (device time of a call; query / kv heads x
// dims):
//   1 x 20 tokens, 8/8x64           2.7   13.8 us    64 x 300-900, 8/1x128        12.6  18.9 us
//   4 x 300, 8/2x64                 4.5   11.8       8 x 500-1000, 32/4x128        9.5  18.0
//   4 x 1500-2000, 32/8x128        10.8   21.8       2 x 900-1000, 64/8x64         6.8  16.7
//   1 x 6000-8000, 32/8x128        18.5   23.2       1 x 12000-16000, 8/8x128     24.4  26.3
//   64 x 500-1000, 32/8x128        44.3   59.6       64 x 1500-2000, 8/8x64       45.0  83.5
//   256 x 400-900, 32/8x128       124.0  173.9       256 x 1200-1900, 8/4x128    130.0 149.8 (6.1 TB/s)
// Past the rule: 64 x 1500-2000, 32/8x128: 89.5 and 91.3 us; 64 x 3000-4000: 169 and 155
// us; 256 x 100-900, 64/8x128: 143 and 157 us; 4 rows a session, each a read of the same
// pages, 16 x 500-900: 39.6 and 26.7 us.  The rows are counted on average, since the host
// does not know them one by one: a chunk of 64 rows over 800 tokens among 63 single rows,
// 32/8x128: 52.0 and 49.4 us; of 256 over 1000 among 255: 209 and 187 us.
constexpr int kShortPages = 128;
constexpr int kShortCluster = 8;
constexpr int kShortThreads = 256, kShortWarps = kShortThreads / 32;

template <int D, int G>
__global__ void __launch_bounds__(kShortThreads, 2) window_short_kernel(const AttendArgs a, const uint16_t* q,
                                                                        const uint16_t* k_pool,
                                                                        const uint16_t* v_pool) {
  constexpr int W = D / 32;  // dims of a lane in P V
  __shared__ __align__(16) float weight[kShortWarps][kPage][G];  // of the warp's page
  __shared__ float scale[kShortWarps][8];                        // of what the warp holds, for a new maximum
  __shared__ float top[kShortWarps][8], sums[kShortWarps][8];
  __shared__ __align__(16) float part[kShortWarps][G][D];
  __shared__ __align__(16) float joined[G][D];  // the CTA's, read by the cluster
  __shared__ float joined_top[G], joined_sum[G];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tq = lane & 3;
  const int C = (int)cluster_size(), rank = (int)cluster_rank(), r = blockIdx.x / C, g = blockIdx.y;
  const int warps = kShortWarps * C, wid = kShortWarps * rank + warp;  // of the cluster
  griddep_wait();
  if (blockIdx.x == 0 && g == 0 && tid == 0) *a.status = 0;
  const int s = warp_find_session(a.b, r, lane);
  const int r0 = a.b.row_begin(s), n = a.b.row_begin(s + 1) - r0;
  if (r < r0 || r >= r0 + n) return;  // a row of no session
  const int p = a.b.kv_len(s) - n + (r - r0);
  // virtual pages 0 .. ns - 1 (sinks), then from page ns + off on, np in all
  int np = 0, ns = 0, off = 0;
  if (p >= 0) {
    const int first = a.w.first(p) / kPage, sink = (min(a.w.sinks, p + 1) + kPage - 1) / kPage;
    if (sink < first) ns = sink, off = first - sink;
    np = p / kPage + 1 - off;
  }
  auto logical = [&](int v) { return v < ns ? v : v + off; };
  // lane j: the page id of the warp's j-th page (-1: a hole)
  const int mine = wid + warps * lane < np ? a.b.page(s, logical(wid + warps * lane)) : -1;
  // the group's query rows as the second operand (heads past G: zeros)
  const size_t row = ((size_t)r * a.b.Hq + g * G) * D;
  uint4 qf[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    qf[i] = gr < G ? *reinterpret_cast<const uint4*>(q + row + gr * D + 32 * i + 8 * tq) : make_uint4(0, 0, 0, 0);
  uint4 k0[D / 32], k1[D / 32];  // rows gr and gr + 8 of the page's keys
  uint32_t raw[kPage][W / 2];    // its V rows; those that the row does not see are not read
  // (plain loads: the kernel before this one may still be filling the pages when it starts)
  auto load_k = [&](int page) {
    if (page < 0) return;
    const uint16_t* k = k_pool + (((size_t)page * a.b.Hkv + g) * kPage + gr) * D + 8 * tq;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      k0[i] = *reinterpret_cast<const uint4*>(k + 32 * i);
      k1[i] = *reinterpret_cast<const uint4*>(k + 8 * D + 32 * i);
    }
  };
  auto load_v = [&](int page, int t0) {
    if (page < 0) return;
    const uint16_t* vp = v_pool + ((size_t)page * a.b.Hkv + g) * kPage * D + lane * W;
#pragma unroll
    for (int key = 0; key < kPage; ++key) {
      const bool see = a.w.sees(p, t0 + key);
      if (W == 2) {
        raw[key][0] = see ? *reinterpret_cast<const uint32_t*>(vp + key * D) : 0u;
      } else {
        const uint2 y = see ? *reinterpret_cast<const uint2*>(vp + key * D) : make_uint2(0u, 0u);
        raw[key][0] = y.x;
        raw[key][W / 2 - 1] = y.y;
      }
    }
  };
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of heads 2 tq, 2 tq + 1; l: of this lane's keys
  float acc[G][W] = {};
  int page = __shfl_sync(0xffffffffu, mine, 0);
  load_k(page);
  load_v(page, logical(wid) * kPage);
  for (int v = wid, j = 0; v < np; v += warps) {
    const int t0 = logical(v) * kPage, next = __shfl_sync(0xffffffffu, mine, ++j & 31);
    const int t1 = logical(v + warps) * kPage;
    if (page < 0) {  // nothing to see: on to the next
      page = next;
      load_k(page);
      load_v(page, t1);
      continue;
    }
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      mma_bf16_16816(x, {k0[i].x, k1[i].x, k0[i].y, k1[i].y}, qf[i].x, qf[i].y);
      mma_bf16_16816(x, {k0[i].z, k1[i].z, k0[i].w, k1[i].w}, qf[i].z, qf[i].w);
    }
    load_k(next);
    const bool see0 = a.w.sees(p, t0 + gr), see1 = a.w.sees(p, t0 + gr + 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float y0 = see0 ? x[i] * a.scale_log2 : -INFINITY, y1 = see1 ? x[2 + i] * a.scale_log2 : -INFINITY;
      float mx = fmaxf(y0, y1);  // (drops NaN: a row of NaN logits has no maximum, but weights and a sum of NaN)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(mx, m[i]);
      const float c = m[i] == mx ? 1.f : ex2(m[i] - mx);  // no key yet: 0, of nothing
      const float w0 = y0 == -INFINITY ? 0.f : ex2(y0 - mx), w1 = y1 == -INFINITY ? 0.f : ex2(y1 - mx);
      m[i] = mx;
      l[i] = l[i] * c + w0 + w1;
      if (2 * tq + i < G) {
        weight[warp][gr][2 * tq + i] = w0;
        weight[warp][gr + 8][2 * tq + i] = w1;
        if (gr == 0) scale[warp][2 * tq + i] = c;
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float c = scale[warp][h];
#pragma unroll
      for (int i = 0; i < W; ++i) acc[h][i] *= c;
    }
#pragma unroll
    for (int key = 0; key < kPage; ++key) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float w = weight[warp][key][h];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          const float2 f = bf16x2_to_f2(raw[key][i]);
          acc[h][2 * i] += w * f.x;
          acc[h][2 * i + 1] += w * f.y;
        }
      }
    }
    page = next;
    load_v(page, t1);
    __syncwarp();  // the weights are read
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    if (gr == 0) top[warp][2 * tq + i] = m[i], sums[warp][2 * tq + i] = l[i];
  }
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int i = 0; i < W; ++i) part[warp][h][lane * W + i] = acc[h][i];
  __syncthreads();
  // the CTA's warps, then the cluster's CTAs: head h's maximum, sum and dims i, i + 1
  for (int i = 2 * tid; i < G * D; i += 2 * kShortThreads) {
    const int h = i / D, d = i % D;
    float mx = -INFINITY, sum = 0.f;
    float2 o = make_float2(0.f, 0.f);
    auto add = [&](float t, float l1, float2 y) {
      const float f = l1 == 0.f ? 0.f : ex2(t - mx);  // a sum of 0: it saw nothing
      sum += f * l1;
      o.x += f * y.x;
      o.y += f * y.y;
    };
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) mx = fmaxf(mx, top[w][h]);
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) add(top[w][h], sums[w][h], *reinterpret_cast<const float2*>(&part[w][h][d]));
    if (C == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint32_t*>(a.out + row + i) = pack_bf16x2(o.x * inv, o.y * inv);
      if (a.lse && d == 0) a.lse[(size_t)r * a.b.Hq + g * G + h] = sum == 0.f ? -INFINITY : (mx + lg2(sum)) * kLn2;
    } else {
      *reinterpret_cast<float2*>(&joined[h][d]) = o;
      if (d == 0) joined_top[h] = mx, joined_sum[h] = sum;
    }
  }
  if (C == 1) return;
  __syncwarp();
  cluster_sync();
  for (int i = 2 * (tid + kShortThreads * rank); i < G * D; i += 2 * kShortThreads * C) {
    const int h = i / D, d = i % D;
    float t[kShortCluster], l1[kShortCluster], mx = -INFINITY, sum = 0.f;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kShortCluster; ++c) {
      t[c] = c < C ? cluster_read(&joined_top[h], c) : -INFINITY;
      l1[c] = c < C ? cluster_read(&joined_sum[h], c) : 0.f;
      mx = fmaxf(mx, t[c]);
    }
#pragma unroll
    for (int c = 0; c < kShortCluster; ++c) {
      if (l1[c] == 0.f) continue;  // it saw nothing
      const float f = ex2(t[c] - mx);
      sum += f * l1[c];
      o.x += f * cluster_read(&joined[h][d], c);
      o.y += f * cluster_read(&joined[h][d + 1], c);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(a.out + row + i) = pack_bf16x2(o.x * inv, o.y * inv);
    if (a.lse && d == 0) a.lse[(size_t)r * a.b.Hq + g * G + h] = sum == 0.f ? -INFINITY : (mx + lg2(sum)) * kLn2;
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another reads its results
}

// log2 of G (1, 2, 4, 8)
int log2_group(const pa_sessions& b) {
  const int G = b.num_q_heads / b.num_kv_heads;
  return G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
}

struct Launch {
  int grid, slots, min_span, lanes, whole, device;
  int cluster;  // > 0: the form for few rows over short caches, so many CTAs for each row and head
  size_t off_desc, off_lse, off_o, bytes;
};

// At most one CTA per SM, and no more than the longest possible line of blocks fills.
bool plan_launch(const pa_sessions& b, const Window& w, Launch* out) {
  const pa_device dev = pa_current_device();
  const int sms = dev.sms;
  out->device = dev.index;
  const int T = 256 >> log2_group(b);
  const int64_t slots = (int64_t)b.num_rows / T + b.n_sessions;
  if (slots > (int64_t)kMaxChunks * kThreads) return false;
  int64_t pages = b.max_pages, row_pages = pages;
  if (w.window) {
    const int64_t row_sees = ((int64_t)w.window + kPage - 2) / kPage + 1 + ((int64_t)w.sinks + kPage - 1) / kPage;
    if (row_sees < row_pages) row_pages = row_sees;
    const int64_t seen = ((int64_t)w.window + T + kPage - 2) / kPage + 1 + ((int64_t)w.sinks + kPage - 1) / kPage + 1;
    if (seen < pages) pages = seen;
  }
  // a cut costs partial rows, a second load of Q and the join: about as much as
  // 8 blocks, so items of no more than that stay whole
  out->whole = (pages + 7) / 8 <= kWholeBlocks;
  out->min_span = 2;
  out->lanes = b.num_kv_heads < kLanes ? b.num_kv_heads : kLanes;
  while (b.num_kv_heads % out->lanes) --out->lanes;
  const int64_t line = slots * (b.num_kv_heads / out->lanes) * ((pages + 7) / 8);
  int64_t spans = (line + out->min_span - 1) / out->min_span;
  const int64_t most = sms / out->lanes > 1 ? sms / out->lanes : 1;
  if (spans > most) spans = most;
  if (spans < 1) spans = 1;
  out->grid = (int)spans * out->lanes;
  // the form for few rows over short caches, above: CTAs for a row until they
  // cover the SMs twice or each warp has a page
  out->cluster = 0;
  if (b.num_rows <= 2 * b.n_sessions) {
    int c = 1;
    while (c < kShortCluster && row_pages > c * kShortWarps && (int64_t)b.num_rows * b.num_kv_heads * c <= sms) c *= 2;
    const int lg = log2_group(b);
    if (row_pages <= c * (lg == 0 ? kShortPages : 2 * kShortPages >> lg)) out->cluster = c;
  }
  out->slots = (int)slots;
  out->off_desc = 256;
  out->off_lse = out->off_desc + ((size_t)out->grid * sizeof(Desc) + 255) / 256 * 256;
  out->off_o = out->off_lse + (size_t)out->grid * 2 * 256 * 4;
  out->bytes = out->off_o + (size_t)out->grid * 2 * 256 * b.head_dim * 4;
  return true;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_window_workspace_size(const pa_sessions* b, int32_t window, int32_t sinks, size_t* bytes) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (!bytes || window < 0 || sinks < 0) return PA_ERR_INVALID;
  pa::Launch l;
  if (!pa::plan_launch(*b, pa_window(window, sinks), &l)) return PA_ERR_UNSUPPORTED;
  *bytes = l.bytes;
  return PA_OK;
}

extern "C" pa_status pa_window_status(const void* d_workspace, void* stream, pa_status* out) {
  if (!out) return PA_ERR_INVALID;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!d_workspace) return pa_take_status(pa::g_window_status, cs, out);
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, d_workspace, 4, cudaMemcpyDeviceToHost, cs) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaStreamSynchronize(cs) != cudaSuccess) return PA_ERR_CUDA;
  *out = static_cast<pa_status>(word);
  return PA_OK;
}

extern "C" pa_status pa_session_fault(int32_t wait) {
  if (wait < 0) return PA_ERR_INVALID;
  pa_fault = wait;
  return PA_OK;
}

namespace {

template <int D, int G>
bool launch_short(const pa::AttendArgs& a, int cluster, const void* q, const void* k_pool, const void* v_pool,
                  cudaStream_t cs) {
  return pa_launch_early(pa::window_short_kernel<D, G>, dim3(a.b.rows * cluster, a.b.Hkv), dim3(pa::kShortThreads), 0, cs,
                         cluster, a,
                         static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k_pool),
                         static_cast<const uint16_t*>(v_pool));
}

template <int D>
bool launch_short(const pa::AttendArgs& a, int cluster, const void* q, const void* k_pool, const void* v_pool,
                  cudaStream_t cs) {
  switch (a.lg) {
    case 0: return launch_short<D, 1>(a, cluster, q, k_pool, v_pool, cs);
    case 1: return launch_short<D, 2>(a, cluster, q, k_pool, v_pool, cs);
    case 2: return launch_short<D, 4>(a, cluster, q, k_pool, v_pool, cs);
    default: return launch_short<D, 8>(a, cluster, q, k_pool, v_pool, cs);
  }
}

template <int D>
bool launch(const pa::AttendArgs& a, const pa::Launch& l, const CUtensorMap& tq, const CUtensorMap& tq16,
            const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t cs) {
  const int give_up = pa_take_fault();
  auto* k = give_up ? pa::window_attend_kernel<D, true> : pa::window_attend_kernel<D, false>;
  constexpr int smem = pa::Shape<D>::SMEM;
  static std::atomic<uint64_t> allowed[2];
  if (!pa_allow_smem(k, smem, l.device, allowed[give_up ? 1 : 0])) return false;
  if (!pa_launch_early(k, dim3(l.grid), dim3(pa::kThreads), smem, cs, 1, a, tq, tq16, tk, tv, give_up)) return false;
  if (l.grid == l.lanes || a.whole) return true;  // no item is cut
  return pa_launch_early(pa::window_join_kernel<D>, dim3(l.grid - l.lanes, pa::kJoinY), dim3(256), 0, cs, 1, a);
}

}  // namespace

extern "C" pa_status pa_window_attend(const pa_sessions* b, int32_t window, int32_t sinks, float softmax_scale,
                                      const void* q, const void* k_pool, const void* v_pool, void* d_workspace,
                                      size_t workspace_bytes, void* out, float* lse, void* stream) {
  const pa_status st = pa_check_sessions(b, true);
  if (st != PA_OK) return st;
  if (window < 0 || sinks < 0 || !pa_scale_ok(softmax_scale)) return PA_ERR_INVALID;
  pa::Launch l;
  if (!pa::plan_launch(*b, pa_window(window, sinks), &l)) return PA_ERR_UNSUPPORTED;
  if (b->num_rows == 0) {  // nothing but the status of a workspace that is given
    if (!d_workspace || (reinterpret_cast<uintptr_t>(d_workspace) & 255) || workspace_bytes < 4) return PA_OK;
    return cudaMemsetAsync(d_workspace, 0, 4, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  if (!q || !k_pool || !v_pool || !out || !d_workspace) return PA_ERR_INVALID;
  if (!pa_aligned16(q) || !pa_aligned16(k_pool) || !pa_aligned16(v_pool) || !pa_aligned16(out) ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 255))
    return PA_ERR_INVALID;
  if (workspace_bytes < l.bytes) return PA_ERR_NOMEM;
  pa::AttendArgs a{};
  a.b = pa_device_sessions(*b);
  a.w = pa_window(window, sinks);
  a.lg = pa::log2_group(*b);
  a.slots = l.slots;
  a.min_span = l.min_span;
  a.whole = l.whole;
  a.lanes = l.lanes;
  a.scale_log2 = (softmax_scale != 0.f ? softmax_scale : 1.f / sqrtf((float)b->head_dim)) * pa::kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  a.status = reinterpret_cast<int32_t*>(ws);
  a.desc = reinterpret_cast<pa::Desc*>(ws + l.off_desc);
  a.part_lse = reinterpret_cast<float*>(ws + l.off_lse);
  a.part_o = reinterpret_cast<float*>(ws + l.off_o);
  const int D = b->head_dim, G = 1 << a.lg;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (l.cluster > 0) {
    const bool ok = D == 64 ? launch_short<64>(a, l.cluster, q, k_pool, v_pool, cs)
                            : launch_short<128>(a, l.cluster, q, k_pool, v_pool, cs);
    return ok ? PA_OK : PA_ERR_CUDA;
  }
  CUtensorMap tq, tq16, tk, tv;
  if (!pa::tmap_q(&tq, q, b->num_rows, b->num_q_heads, D, G, 128 / G) ||
      !pa::tmap_q(&tq16, q, b->num_rows, b->num_q_heads, D, G, 16 / G) ||
      !pa::tmap_pool(&tk, k_pool, b->num_pages_in_pool, b->num_kv_heads, D) ||
      !pa::tmap_pool(&tv, v_pool, b->num_pages_in_pool, b->num_kv_heads, D))
    return PA_ERR_CUDA;
  return (D == 64 ? launch<64>(a, l, tq, tq16, tk, tv, cs) : launch<128>(a, l, tq, tq16, tk, tv, cs)) ? PA_OK : PA_ERR_CUDA;
}
