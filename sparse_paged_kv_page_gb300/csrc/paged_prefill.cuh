// sa_paged_prefill and sa_paged_prefill8: causal softmax attention of new tokens (a
// prompt, a chunk of one, a few drafted tokens) over the paged cache that already holds
// them, in 16 bits or (kQ8) in 8.
//
// Mathematics: o = sum_j p_j v_j, p = softmax(scale q . k_j) over the visible
// positions j, in one pass with a running reference m near the maximum and the sum l;
// O and l are rescaled only where the weights 2^(scale (s - m)) have grown large; the
// quotient o / l at the end makes any m right.
//
// A CTA owns 128 packed rows (token, query head of one KV head's group) at head dim 64,
// two CTAs an SM, and 2 x 128 at 128, one an SM, so a key is read once for all G heads,
// and walks the visible keys 128 at a time. The products run on the 5th-generation
// tensor cores, accumulators in TMEM: S = Q K^T (128 x 128), P over S's columns as the A
// operand from TMEM, O += P V. A warpgroup takes each 128 rows, one a thread (no
// shuffles): while one turns S into P the tensor cores work for the other, so the time
// from S to P counts. One warp issues the products, one the copies: keys and values in a
// ring of 128-row slots, page by page through a tensor map (pages of 8 tokens and more),
// or row by row with cp.async (smaller pages). Where the rows of a CTA of two halves
// fill one only, the halves take every other step of the same rows and meet at the end.
//
// In 8 bits (kQ8) the copy warps turn codes into values, exactly, on the way to the slots:
// 16-byte cp.async into a lane's own chunks a step ahead, no barrier but the slots'. At head
// dim 128 a team of three warps for the keys and one for the values. What the turning costs,
// and when the codes are turned before instead: at worth_pages.
//
// Value rows that no query of the CTA sees are zeroed in shared memory (a weight 0
// times what a freed page holds must be 0), key rows masked.
//
// Times here and below are of the kernel in replayed graphs, where they vary by 2% with
// the machine and its power; calls from Python of the two long prompts take 2 - 3% more.
// Bound by the tensor cores for prompts (16384 tokens, 32 / 8 heads of 128, pages of 16:
// 1315 us, 1.67 PFLOP/s; 2048 tokens behind 64000, 64 / 8 heads, 2540 us, 1.72 PFLOP/s:
// the rate that the power limit leaves a dense product); at head dim 64 by
// the rows' turn from S to P and the number of page copies (an operation costs about 80
// cycles whatever its size: a prompt of 8192 over 4096 in pages of 16 1145 us, of 128
// 920); for a few rows over a long cache by HBM, where each item's keys are cut into
// parts of about the same number of steps, one a CTA, and the last of an item's CTAs
// merges the parts in order.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "kv8.cuh"
#include "paged.cuh"
#include "tc5.cuh"
#include "tma_map.h"

namespace sa {
namespace {

constexpr int kKeys = 128;                // positions per step
constexpr int kTileRing = 8;              // steps whose row masks are kept
// The running maximum m follows the row only when a step's sum of weights 2^(scale (s - m)) passes this: below it
// every weight is inside both 16-bit types, and float32 sums do not mind. So no step but the first looks for its
// maximum (60 instructions of 380 a row), the sum that is made anyway tells.
constexpr float kMostSum = 8192.0f;
constexpr int kRun = 8;                   // words of P stored at a time
// Steps of a part at least, and of an item that is cut at all: a merge costs about six. Measured (us) with items of two
// halves: 30 tokens x 64 heads over 500, 5 steps, whole 15 and in parts 22; over 2000, 16 steps, parts of 4 24, of 6 28.
constexpr int kMinPart = 4, kMinCut = 9;
constexpr int kTailPart = 16, kMostTail = 8;   // steps at least and number at most of the parts of a unit behind the last full round
// Steps of all items (64 KB of keys and values each) up to which they stay near, in L2, for a second reader: items of a
// call in parts are of one half then. Measured (us), two halves / one: 30 tokens x 64 heads over 2000 24.5 / 19, 8000 49 /
// 28, 32000 (2000 steps) 62 / 56, 120000 129 / 153, four requests over 16000 (3776 steps) 66 / 94.
constexpr int kNear = 2048;
constexpr int kLag = 2;                   // row-by-row copies under way behind the newest

struct PagedPrefillArgs {
  const void* k;
  const void* v;
  const uint8_t* scale;   // kQ8
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* new_cu;
  void* out;
  float* lse;
  float4* part_o;       // [CTAs][D / 4][rows]: a warp stores adjacent rows
  float* part_lse;      // [CTAs][rows]
  int32_t* tickets;     // [units that can be cut], no more than CTAs run at once
  int32_t* status;
  int H_kv, H_q, G, ps_shift, num_blocks, bt_stride, batch, T, window, n_sink, items;
  int split;              // rounds of CTAs that the parts of items may fill (0: items are whole)
  int whole, tail_parts;  // without split: CTAs before the last units, and parts of each of those
  float scale_log2;
  const int32_t* turn;    // nullable: the kernel has work only if turn[0] is 1 and turn[1] 0 (or, with `otherwise`, if not)
  int otherwise;
};

// Halves of 128 packed rows of a CTA, a warpgroup each. At head dim 64 one, and two CTAs an SM, of which one works while
// the other begins or ends (us, two halves / one: sliding-window prompts 177 / 166, 6 tokens of 4 requests over 30000 75 / 51).
constexpr int ways(int D) { return D == 128 ? 2 : 1; }

template <int D, bool kTma, bool kQ8>
struct Cfg {
  // copy warps; kQ8 at head dim 128: a team of three for the keys, one for the values, which take turns at head dim 64
  static constexpr int kTeams = kQ8 && D == 128 ? 2 : 1;
  static constexpr int kParts = 2 / kTeams;                        // a warp's parts of a step: keys, values
  static constexpr int kProducers = kTma ? 1 : 3 * kTeams;
  static constexpr int kHalves = D / 64;                           // 64-column halves of a row
  static constexpr int kWays = ways(D);
  static constexpr int kRows = 128 * kWays, kMmaWarp = 4 * kWays;  // the warps before are the softmax
  static constexpr int kSoftmaxThreads = 32 * kMmaWarp, kThreads = kSoftmaxThreads + 128 * kTeams;
  // Registers: the softmax warpgroups take (a row of 128 scores a thread) what the last one gives back:
  // 256 x 208 + 128 x 88 = 384 x 168, 128 x 192 + 128 x 64 = 256 x 128, 256 x 176 + 256 x 80 = 512 x 128.
  static constexpr int kSoftmaxRegs = kWays == 2 && kTeams == 1 ? 208 : kTeams == 2 ? 176 : 192, kOtherRegs = kWays == 2 && kTeams == 1 ? 88 : kTeams == 2 ? 80 : 64;
  static constexpr int kGroupBytes = kHalves * 1024;               // 8 rows of a slot: [half][8 rows of 128 bytes]
  static constexpr int kSlotBytes = kKeys / 8 * kGroupBytes;
  // kQ8: an even number, so that each team waits for slots of its own copies alone (a wait for a phase after the next one
  // of a barrier passes at once)
  static constexpr int kSlots = kQ8 ? 4 : 5;
  // kQ8: codes of a step's keys and values behind the slots, a lane's own chunks of 16 side by side
  static constexpr int kRawBytes = kQ8 ? 2 * kKeys * D : 0;
  static constexpr int kQBytes = kWays * kSlotBytes;
  // TMEM columns: S of the halves, overwritten by P, and O of the halves. At D = 64, where there is room, S and P take turns
  // in three blocks of 64 columns: step j has S in blocks j and j + 1 (mod 3) and P in block j, so that the next step's S,
  // in the block left over and the one of the P before this (whose products come first), is made while P is (a prompt of
  // 8192 over 4096, pages of 128: 945 -> 915 us against P in a place of its own, for which the products before had to end).
  static constexpr bool kAhead = D == 64;
  static constexpr int kOCol = kAhead ? 192 : 128 * kWays, kCols = 256 * kWays;
  static constexpr int kRawAt = kQBytes + kSlots * kSlotBytes, kSharedAt = kRawAt + kRawBytes;
};

// What a CTA does: tokens [t0, t0 + nt) of request b for KV head h, steps [tb, tb + steps) of the visible keys.
struct Work {
  int b, item, h, per, part, parts, unit, slot, c0, n, L;   // per: tokens of an item; unit, slot: of the tickets and of the parts' results
};

struct Shared {
  // of the halves: s made, p made, the last products complete (o); where S is made ahead p is of even and odd steps
  // (the rows may be two P ahead of the products), s is read (r), a step's products complete (v)
  uint64_t full[8], empty[8], q, s[2], p[2], o[2], r, v, edge, drain;
  uint32_t tile[kTileRing][1 + kKeys / 32];   // [0]: rows of the step are masked by the words that follow
  int64_t off[kKeys];                         // pool row of each position of a step copied row by row, -1: none
  float x[2][kKeys];                          // the second half's maxima and sums, where both have the same rows
  Work work;
  uint32_t tmem;
  int abort, last, bad;                       // bad: a page that was to be read has no block
};

// Wait for a phase; false once any wait of the CTA has given up. The clock is read
// only after many tries (each try suspends the thread for a while by itself).
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, Shared& sh, int32_t* status) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if (i & 63) continue;
    if (*reinterpret_cast<volatile int*>(&sh.abort)) return false;
    const uint64_t t = global_ns();
    if (!t0) t0 = t;
    if (t - t0 > kWaitLimitNs) {
      flag(status, SA_DEV_TIMEOUT);
      *reinterpret_cast<volatile int*>(&sh.abort) = 1;
      return false;
    }
  }
}

// Barriers of part of the block: 1 the copy warps, 2 the softmax warps.
template <int kCount>
__device__ __forceinline__ void named_sync(int id) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "n"(kCount) : "memory");
}
template <int kCount>
__device__ __forceinline__ bool named_any(int id, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"(id), "n"(kCount), "r"(uint32_t(x))
               : "memory");
  return r != 0;
}

// Steps of a request's last item of `per` tokens, which has the most, as its items' parts are cut.
__device__ __forceinline__ int request_steps(const PagedPrefillArgs& a, int L, int n, int per, int cap) {
  return Span<kKeys>(L - min(n, per), L - 1, min(max(L, 0), cap), a.window, a.n_sink).tiles;
}

// Parts of about `chunk` steps that an item is cut into.
__device__ __forceinline__ int parts_of(int steps, int chunk) { return steps < kMinCut ? 1 : (steps + chunk - 1) / chunk; }

// The CTA's work, found by one warp. False if there is none.
__device__ __forceinline__ bool find_work(const PagedPrefillArgs& a, int cap, int half_tokens, int ways, Work& w) {
  const int lane = threadIdx.x & 31;
  int per = ways * half_tokens;
  w.per = per;
  // Item and head u. Heads outermost: the CTAs of a wave share one head's keys in L2; long items first.
  auto whole_item = [&](int u, bool there) {
    w.h = u / a.items;
    return there && find_item(a.new_cu, a.seq_lens, a.batch, per, a.items - 1 - u % a.items, w.b, w.item, w.c0, w.n, w.L);
  };
  if (!a.split) {
    const int tail = max(0, int(blockIdx.x) - a.whole);
    w.parts = int(blockIdx.x) < a.whole ? 1 : a.tail_parts;
    w.part = tail % w.parts, w.unit = tail / w.parts, w.slot = tail;
    if (!whole_item(min(int(blockIdx.x), a.whole) + w.unit, true)) return false;
    if (w.parts > 1) {
      const int t0 = w.item * per, first = w.L - w.n + t0;
      const int steps = Span<kKeys>(first, first + min(per, w.n - t0) - 1, min(max(w.L, 0), cap), a.window, a.n_sink).tiles;
      w.parts = max(1, min(w.parts, steps / kTailPart));
      if (w.part >= w.parts) return false;
    }
    return true;
  }
  // Every (item, head) of request b in ceil(steps_b / chunk) parts, chunk the least
  // that gives no more parts than CTAs. At most 96 requests (three a lane).
  int c0[3], n[3], L[3], units[3], steps[3];
  int most = 1;
  int64_t rows = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int b = 32 * i + lane;
    c0[i] = n[i] = L[i] = units[i] = steps[i] = 0;
    if (b < a.batch) {
      c0[i] = a.new_cu[b], n[i] = a.new_cu[b + 1] - c0[i], L[i] = a.seq_lens[b];
      if (c0[i] < 0 || int64_t(c0[i]) + n[i] > a.T) {
        if (blockIdx.x == 0) flag(a.status, SA_DEV_BAD_COUNT);
      } else if (n[i] > 0) {
        rows += n[i];
        units[i] = (n[i] + per - 1) / per * a.H_kv;
        steps[i] = request_steps(a, L[i], n[i], per, cap);
      }
    }
    most = max(most, steps[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) rows += __shfl_xor_sync(kFull, rows, o);
  if (rows > a.T) {                          // not a list of offsets within the rows: some part might have no CTA
    if (blockIdx.x == 0 && lane == 0) flag(a.status, SA_DEV_BAD_COUNT);
    return false;
  }
  most = __reduce_max_sync(kFull, most);
  const int ctas = int(gridDim.x) / a.split; // that run at once
  if (ways == 2) {
    // items of one half, whose CTAs' halves take the steps in turn, where there are CTAs for them
    int all = 0, near = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      all += units[i] ? (n[i] + half_tokens - 1) / half_tokens * a.H_kv : 0;
      near += units[i] * min(steps[i], kNear + 1);
    }
    if (__reduce_add_sync(kFull, all) <= ctas && __reduce_add_sync(kFull, near) <= kNear) {
      w.per = per = half_tokens;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (!units[i]) continue;
        units[i] = (n[i] + per - 1) / per * a.H_kv;
        steps[i] = request_steps(a, L[i], n[i], per, cap);
      }
    }
  }
  int lo = kMinPart, hi = max(kMinPart, most);
  if (a.split > 1) {
    // several rounds of CTAs: parts of a good length, or whole items where the longest do not make much more than the mean
    int all = 0, total = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) all += units[i], total += units[i] * min(steps[i], 1 << 20);
    all = __reduce_add_sync(kFull, all), total = __reduce_add_sync(kFull, total) / ctas;
    lo = min(kTailPart, hi);
    if ((all <= ctas ? most : total + most / 2) <= total + total / 16 + kTailPart) {
      w.parts = 1, w.part = w.unit = w.slot = 0;
      if (per == ways * half_tokens) return whole_item(int(blockIdx.x), int(blockIdx.x) < a.items * a.H_kv);
      lo = hi;
    }
  }
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int parts = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) parts += units[i] * parts_of(steps[i], mid);
    if (__reduce_add_sync(kFull, parts) <= int(gridDim.x)) hi = mid;
    else lo = mid + 1;
  }
  int before = 0, units_before = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int np = parts_of(steps[i], lo), mine = units[i] * np;
    int x = mine, y = units[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, x, o), v = __shfl_up_sync(kFull, y, o);
      if (lane >= o) x += u, y += v;
    }
    const int k = __popc(__ballot_sync(kFull, before + x <= int(blockIdx.x)));
    if (k < 32) {
      const int first = before + __shfl_sync(kFull, x, k) - __shfl_sync(kFull, mine, k);
      const int unit0 = units_before + __shfl_sync(kFull, y, k) - __shfl_sync(kFull, units[i], k);
      w.parts = __shfl_sync(kFull, np, k);
      const int at = int(blockIdx.x) - first, unit = at / w.parts;
      w.part = at % w.parts;
      w.unit = unit0 + unit, w.slot = int(blockIdx.x);
      w.h = unit % a.H_kv, w.item = unit / a.H_kv, w.b = 32 * i + k;
      w.c0 = __shfl_sync(kFull, c0[i], k), w.n = __shfl_sync(kFull, n[i], k), w.L = __shfl_sync(kFull, L[i], k);
      return true;
    }
    before += __shfl_sync(kFull, x, 31);
    units_before += __shfl_sync(kFull, y, 31);
  }
  return false;
}

template <typename T, int D, bool kTma, bool kQ8>
__global__ void __launch_bounds__(Cfg<D, kTma, kQ8>::kThreads, 3 - ways(D))
    paged_prefill_kernel(const __grid_constant__ PagedPrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using E = Elem<T>;
  using C = Cfg<D, kTma, kQ8>;
  static_assert(!(kTma && kQ8), "codes are copied row by row");
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];               // Q, the ring, Shared
  uint8_t* ring = smem + C::kQBytes;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kSharedAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G, pss = a.ps_shift, half_tokens = 128 / G;
  if (a.turn && (a.turn[0] == 1 && a.turn[1] == 0) == (a.otherwise != 0)) return;
  const int cap = int(min(int64_t(a.bt_stride) << pss, int64_t(0x7fffffff)));

  if (warp == 0) {
    Work w;
    const bool any = find_work(a, cap, half_tokens, C::kWays, w);
    if (any && w.item == 0 && w.h == 0 && w.part == 0 && lane == 0) {
      if (w.c0 < 0 || int64_t(w.c0) + w.n > a.T || w.L < w.n) flag(a.status, SA_DEV_BAD_COUNT);
      if (w.L > cap) flag(a.status, SA_DEV_OVERFLOW);
    }
    if (!any || w.c0 < 0 || int64_t(w.c0) + w.n > a.T) w.b = -1;
    if (lane == 0) {
      sh.work = w;
      sh.abort = 0;
      sh.bad = 0;
    }
  } else if (threadIdx.x == 32) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), kQ8 ? 3 : 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.q), 1);
    mbar_init(smem_u32(&sh.edge), 1);
    mbar_init(smem_u32(&sh.drain), 1);
    mbar_init(smem_u32(&sh.r), 4);
    mbar_init(smem_u32(&sh.v), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s[i]), 1);
      mbar_init(smem_u32(&sh.p[i]), 4);
      mbar_init(smem_u32(&sh.o[i]), 1);
    }
    mbar_init_fence();
  } else if (warp == C::kMmaWarp) {
    tc5_alloc(smem_u32(&sh.tmem), C::kCols);
  } else if (threadIdx.x == C::kSoftmaxThreads + 32) {
    prefetch_map(&tmq);
    if (kTma) {
      prefetch_map(&tmk);
      prefetch_map(&tmv);
    }
  }
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = sh.tmem;                                  // columns: S/P of the halves, then O of the halves
  const Work w = sh.work;
  if (w.b < 0) {
    if (warp == C::kMmaWarp) tc5_dealloc(tmem, C::kCols);
    return;
  }
  const int h = w.h, t0 = w.item * w.per, nt = min(w.per, w.n - t0);
  const int first = w.L - w.n + t0, last = first + nt - 1, len = min(max(w.L, 0), cap);
  const Span<kKeys> sp(first, last, len, a.window, a.n_sink);
  const int per = (sp.tiles + w.parts - 1) / w.parts;
  const int tb = min(sp.tiles, w.part * per), steps = min(sp.tiles, tb + per) - tb;
  const bool two = C::kWays == 2 && nt > half_tokens;                              // the second half has rows of its own
  const bool dual = C::kWays == 2 && !two && steps > 1;                            // the halves take every other step of the same rows

  if (warp < C::kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------- softmax: one row a thread
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(warp & 3) << 21;              // TMEM lane 32 * (warp % 4)
    const uint32_t s_col = tmem + lanes + half * 128, o_col = tmem + lanes + C::kOCol + half * D;
    const int t = (dual ? 0 : half * half_tokens) + row / G;
    const bool in = row / G < half_tokens && t < nt;
    const int pos = in ? first + t : -1;
    const int64_t orow = in ? int64_t(w.c0 + t0 + t) * a.H_q + int64_t(h) * G + row % G : -1;
    float m = in ? -INFINITY : 0.f, l = 0.f;                      // m: -inf until the row has seen a key
    const bool act = half == 0 || two || dual;
    const int stride = dual ? 2 : 1;
    uint32_t parity = 0;
    int block = 0;                                                // first one of the step's S
    bool ok = steps > 0;
    // the warp's rows: steps that end behind `low`, or begin before `high`'s window, hide keys from one of them
    const int low = __reduce_min_sync(kFull, in ? min(pos, len - 1) : 0x7fffffff);
    const int high = __reduce_max_sync(kFull, pos);
    for (int j = dual ? half : 0; act && j < steps; j += stride, parity ^= 1) {
      const int j0 = sp.start(tb + j);
      const bool cut = j0 + kKeys - 1 > low || (a.window > 0 && j0 <= high - a.window && j0 + kKeys > a.n_sink);
      ok = wait_on(&sh.s[half], parity, sh, a.status) && ok;       // (a wait that gave up: the rest runs on to its end)
      __syncwarp();
      tc5_fence_after();
      const uint32_t s_at = C::kAhead ? s_col + 64 * block : s_col, s_next = s_col + 64 * (block < 2 ? block + 1 : 0);
      block = block < 2 ? block + 1 : 0;
      float s[kKeys];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tc5_ld32(reinterpret_cast<uint32_t*>(s) + 32 * c, (C::kAhead && c >= 2 ? s_next - 64 : s_at) + 32 * c);
      const int bad = *reinterpret_cast<volatile int*>(&sh.bad);   // looked at with the sum below
      tc5_wait_ld();
      if constexpr (C::kAhead) {
        tc5_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.r));
      }
      auto hide = [&]() {
        // columns seen: up to hi, from lo on or below sk, and those whose rows the step has
        const int hi = min(pos, len - 1) - j0;
        const int lo = a.window > 0 ? pos - a.window + 1 - j0 : 0, sk = a.n_sink - j0;
        const volatile uint32_t* words = sh.tile[j % kTileRing];
        const bool some = words[0];
        auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t see = below(hi + 1 - 32 * x) & (~below(lo - 32 * x) | below(sk - 32 * x));
          if (some) see &= words[1 + x];
#pragma unroll
          for (int c = 0; c < 32; ++c) keep_if(s[32 * x + c], see, 1u << c);
        }
      };
      auto maximum = [&]() {
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kKeys - 4; c += 8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], s[c + x], s[c + 4 + x]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], s[kKeys - 4 + x]);
        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      };
      if (cut || bad) hide();
      float sum = INFINITY;                                        // (of the first step, before it is known)
      bool grow = j < stride;                                      // some row's reference follows its maximum
#pragma unroll 1
      for (int turn = 0;; ++turn) {
        if (grow) {
          // this row's: where its own sum says so, so that a result does not depend on the rows beside it
          const float top = maximum();
          const float m_new = in && (sum > kMostSum || sum != sum || m == -INFINITY) ? fmaxf(m, top) : m;
          if (j >= stride) {
            // O and l follow; the products into O before this step are complete
            if (C::kAhead) ok = wait_on(&sh.v, parity ^ 1, sh, a.status) && ok;
            __syncwarp();
            tc5_fence_after();
            const float f = m_new == m ? 1.f : ex2_approx((m - m_new) * a.scale_log2);
            l *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              tc5_ld16(reinterpret_cast<uint32_t*>(o), o_col + 16 * c);
              tc5_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] *= f;
              tc5_st16(o_col + 16 * c, reinterpret_cast<uint32_t*>(o));
            }
          }
          m = m_new;
        }
        // P = 2^(scale s - scale m) to TMEM, eight words at a time and one run behind; the row's sum
        const float base = m == -INFINITY ? 0.f : -m * a.scale_log2;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pw[2][kRun];
#pragma unroll
        for (int c = 0; c <= 64 / kRun; ++c) {
          if (c < 64 / kRun) {
#pragma unroll
            for (int x = 0; x < kRun; ++x) {
              float p0, p1;
              fma2(p0, p1, s[2 * kRun * c + 2 * x], s[2 * kRun * c + 2 * x + 1], a.scale_log2, base);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              add2(part[2 * (x & 1)], part[2 * (x & 1) + 1], p0, p1);
              pw[c & 1][x] = E::pack(p0, p1);
            }
          }
          if (c > 0) tc5_st8(s_at + kRun * (c - 1), pw[(c - 1) & 1]);
        }
        sum = (part[0] + part[1]) + (part[2] + part[3]);
        if (turn || j < stride) break;
        grow = __any_sync(kFull, in && (!(sum <= kMostSum) || m == -INFINITY));
        if (!grow) break;                                          // else P is made again (it has not been handed over)
      }
      l += sum;
      tc5_wait_st();
      tc5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.p[C::kAhead ? j & 1 : half]));
    }
    // ------------------------------------------------------------- outputs
    if (act) {
      ok = ok && wait_on(&sh.o[half], 0, sh, a.status);
      if (dual) ok = wait_on(&sh.o[half ^ 1], 0, sh, a.status) && ok;   // the ring is free: no product reads it
      ok = __all_sync(kFull, ok);
      tc5_fence_after();
      float* other = reinterpret_cast<float*>(ring);                      // [D columns][128 rows] of the second half
      float f0 = 1.f, f1 = 0.f;
      if (dual) {
        if (half == 1) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            __syncwarp();
            if (ok) tc5_ld32(reinterpret_cast<uint32_t*>(o), o_col + 32 * c);
            tc5_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) other[(32 * c + x) * kKeys + row] = o[x];
          }
          sh.x[0][row] = m;
          sh.x[1][row] = l;
        }
        named_sync<C::kSoftmaxThreads>(2);
        const float m1 = sh.x[0][row], l1 = sh.x[1][row], top = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.f : ex2_approx((m - top) * a.scale_log2);
        f1 = m1 == -INFINITY ? 0.f : ex2_approx((m1 - top) * a.scale_log2);
        l = l * f0 + l1 * f1;
        m = top;
      }
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      const float row_lse = l != 0.f ? (m * a.scale_log2 + lg2_approx(l)) * kLn2 : -INFINITY;
      const int prow = (dual ? 0 : half * 128) + row;
      if (in && !(dual && half == 1)) {
        if (w.parts > 1) a.part_lse[int64_t(w.slot) * C::kRows + prow] = row_lse;
        else if (a.lse) a.lse[orow] = row_lse;
      }
      f0 *= inv;
      f1 *= inv;
      uint8_t* stage = smem + half * C::kSlotBytes + row * (D * 2);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if (dual && half == 1) break;                                     // (whole warps)
        float o[32];
        __syncwarp();
        if (ok) tc5_ld32(reinterpret_cast<uint32_t*>(o), o_col + 32 * c);
        tc5_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          o[x] = l != 0.f ? o[x] * f0 : 0.f;
          if (dual && l != 0.f) o[x] = fmaf(other[(32 * c + x) * kKeys + row], f1, o[x]);
        }
        if (w.parts > 1) {
          if (in) {
            float4* dst = a.part_o + (int64_t(w.slot) * (D / 4) + 8 * c) * C::kRows + prow;
#pragma unroll
            for (int x = 0; x < 8; ++x) dst[x * C::kRows] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        } else {
          // through the half's query rows in shared memory (every product with them is complete), so that a store
          // instruction covers whole rows of out and not 16 bytes of 32 of them
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(stage + ((4 * c + x) ^ (row & 7)) * 16) =
                make_uint4(E::pack(o[8 * x], o[8 * x + 1]), E::pack(o[8 * x + 2], o[8 * x + 3]),
                           E::pack(o[8 * x + 4], o[8 * x + 5]), E::pack(o[8 * x + 6], o[8 * x + 7]));
        }
      }
      if (w.parts == 1 && !(dual && half == 1)) {
        __syncwarp();
        constexpr int kChunks = D / 8, kRows = 32 / kChunks;               // 16-byte chunks of a row, rows at a time
        const int chunk = lane % kChunks;
        uint8_t* rows = stage - lane * (D * 2);
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += kRows) {
          const int r = r0 + lane / kChunks;
          const int64_t to = __shfl_sync(kFull, orow, r);
          const uint4 x = *reinterpret_cast<const uint4*>(rows + r * (D * 2) + (chunk ^ (r & 7)) * 16);
          if (to >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + to * D + chunk * 8) = x;
        }
      }
      tc5_fence_before();
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kOtherRegs));
  if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------- products, issued by one thread
    if (steps > 0 && elect_one()) {
      constexpr uint32_t id_s2 = tc5_idesc(kBf16, 128, kKeys / 2, false), id_s = tc5_idesc(kBf16, 128, kKeys, false), id_o = tc5_idesc(kBf16, 128, D, true);
      const uint64_t q_desc = tc5_desc(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = tc5_desc(smem_u32(ring), 16, C::kGroupBytes);
      const uint64_t v_desc = tc5_desc(smem_u32(ring), 1024, C::kGroupBytes);
      auto scores = [&](int half, int slot, int block) {                       // S = Q K^T
        const uint64_t qd = q_desc + (dual ? 0u : uint32_t(half * C::kSlotBytes / 16));
        const uint64_t kd = k_desc + uint32_t(slot * C::kSlotBytes / 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t q_at = (kk >> 2) * (128 * 128) + (kk & 3) * 32, k_at = (kk >> 2) * 1024 + (kk & 3) * 32;
          if (!C::kAhead) {
            tc5_mma_ss(tmem + half * 128, qd + q_at / 16, kd + k_at / 16, id_s, kk > 0);
          } else if (block < 2) {
            tc5_mma_ss(tmem + 64 * block, qd + q_at / 16, kd + k_at / 16, id_s, kk > 0);
          } else {                                                  // blocks 2 and 0
            tc5_mma_ss(tmem + 128, qd + q_at / 16, kd + k_at / 16, id_s2, kk > 0);
            tc5_mma_ss(tmem, qd + q_at / 16, kd + (k_at + 8 * C::kGroupBytes) / 16, id_s2, kk > 0);
          }
        }
        tc5_commit(smem_u32(&sh.s[half]));
      };
      auto outputs = [&](int half, int slot, bool add, int turn, uint32_t parity, int block) {   // O += P V once P is there
        if (!wait_on(&sh.p[turn], parity, sh, a.status)) return false;
        tc5_fence_after();
        const uint64_t vd = v_desc + uint32_t(slot * C::kSlotBytes / 16);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc5_mma_ts(tmem + C::kOCol + half * D, tmem + (C::kAhead ? 64 * block : half * 128) + kk * 8, vd + uint32_t(kk * 2 * C::kGroupBytes / 16), id_o,
                     add || kk > 0);
        return true;
      };
      auto wait_full = [&](int seq) {
        const bool got = wait_on(&sh.full[seq % C::kSlots], (seq / C::kSlots) & 1, sh, a.status);
        tc5_fence_after();
        return got;
      };
      auto release = [&](int seq) { tc5_commit(smem_u32(&sh.empty[seq % C::kSlots])); };
      // keys of step j are copy 2j of the ring, its values copy 2j + 1
      bool ok = wait_on(&sh.q, 0, sh, a.status) && wait_full(0);
      if (ok) {
        scores(0, 0, 0);
        if (two) scores(1, 0, 0);
        release(0);
      }
      if (ok && dual && (ok = wait_full(2))) {
        scores(1, 2 % C::kSlots, 0);
        release(2);
      }
      if (dual) {
        for (int j = 0; ok && j < steps; ++j) {
          const int half = j & 1, sv = 2 * j + 1, sk = 2 * j + 4;
          if (!(ok = wait_full(sv) && outputs(half, sv % C::kSlots, j > 1, half, (j >> 1) & 1, 0))) break;
          release(sv);
          if (j + 2 >= steps) {
            tc5_commit(smem_u32(&sh.o[half]));
          } else if ((ok = wait_full(sk))) {
            scores(half, sk % C::kSlots, 0);
            release(sk);
          }
        }
      } else if (C::kAhead) {
        int block = 0, next = 1;
        for (int j = 0; ok && j < steps; ++j) {
          const int sv = 2 * j + 1, sk = 2 * j + 2;
          if (j + 1 < steps) {                                      // S of the next step, once this one's is read
            if (!(ok = wait_full(sk) && wait_on(&sh.r, j & 1, sh, a.status))) break;
            tc5_fence_after();
            scores(0, sk % C::kSlots, next);
            release(sk);
          }
          if (!(ok = wait_full(sv) && outputs(0, sv % C::kSlots, j > 0, j & 1, (j >> 1) & 1, block))) break;
          release(sv);
          tc5_commit(smem_u32(&sh.v));
          block = next, next = next < 2 ? next + 1 : 0;
        }
        if (ok) tc5_commit(smem_u32(&sh.o[0]));
      } else {
        for (int j = 0; ok && j < steps; ++j) {
          const int sv = 2 * j + 1, sk = 2 * j + 2;
          const bool more = j + 1 < steps;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half && !two) break;
            if (half == 0 && !(ok = wait_full(sv))) break;
            if (!(ok = outputs(half, sv % C::kSlots, j > 0, half, j & 1, 0))) break;
            if (half == 1 || !two) release(sv);
            if (!more) {
              tc5_commit(smem_u32(&sh.o[half]));
            } else {
              if (half == 0 && !(ok = wait_full(sk))) break;
              scores(half, sk % C::kSlots, 0);
            }
          }
          if (ok && more) release(sk);
        }
      }
      if (!ok) {                                                    // let what was issued finish
        tc5_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, a.status);
      }
    }
    __syncwarp();
  } else if (warp <= C::kMmaWarp + C::kProducers) {
    // ------------------------------------------------------------- copies
    constexpr int kCopyThreads = 32 * C::kProducers;
    const int ct = threadIdx.x - 32 * (C::kMmaWarp + 1);
    auto copy_sync = [&]() {
      if (C::kProducers == 1) __syncwarp();
      else named_sync<kCopyThreads>(1);
    };
    const int w0 = a.window > 0 ? max(0, first - a.window + 1) : 0;
    auto seen = [&](int p) { return p < len && (p >= w0 || p < a.n_sink); };   // by some query of the CTA
    const int32_t* btb = a.bt + int64_t(w.b) * a.bt_stride;
    const int ps = 1 << pss, pages = kKeys >> pss;
    // Block ids of a step through the tensor map, one a lane; -1 where the page holds no row to be read.
    auto page_ids = [&](int j) {
      int id = -1;
      if (kTma && j < steps && lane < pages) {
        const int p = sp.start(tb + j) + (lane << pss);
        if (p < len && (p + ps > w0 || p < a.n_sink)) {
          id = btb[p >> pss];
          if (id < 0 || id >= a.num_blocks) {
            flag(a.status, SA_DEV_BAD_BLOCK);
            *reinterpret_cast<volatile int*>(&sh.bad) = 1;
            id = -1;
          }
        }
      }
      return id;
    };
    if (steps > 0 && ct == 0) {
      const uint32_t bar = smem_u32(&sh.q);
      mbar_arrive_expect_tx(bar, uint32_t((two ? 2 : 1) * C::kHalves * G * half_tokens * 128));
      for (int half = 0; half < (two ? 2 : 1); ++half)
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_u32(smem) + half * C::kSlotBytes + hf * kKeys * 128, &tmq, hf * 64, h * G,
                      w.c0 + t0 + half * half_tokens, bar);
    }
    bool ok = true;
    int seq = 0, done = 0;                                         // copies begun; row-by-row ones handed over
    uint32_t edges = 0;
    auto slot_at = [&](int x) { return smem_u32(ring) + (x % C::kSlots) * C::kSlotBytes; };
    auto claim = [&]() {                                           // the ring slot of copy `seq` is free
      if (seq >= C::kSlots)
        ok = __all_sync(kFull, wait_on(&sh.empty[seq % C::kSlots], (seq / C::kSlots - 1) & 1, sh, a.status));
      if constexpr (!kTma) ok = !named_any<kCopyThreads>(1, !ok);
      return ok;
    };
    auto hand_over = [&](int x) {                                  // generic writes to the slot of copy x are complete
      fence_proxy_async_smem();
      copy_sync();
      if (ct == 0) mbar_arrive(smem_u32(&sh.full[x % C::kSlots]));
    };
    if constexpr (kQ8) {
      // A step is 16 groups of 8 rows; warp x of three has groups x, x + 3, .. from pool to slot by itself. A lane copies the
      // chunks of 16 codes that it will turn into values, chunks lane % 4 (and 4 more) of row lane / 4 of each group, and copies
      // the next step's over them as soon as they are used up, so each copy has the time of a step. Two rows' chunks 0 .. 3 as
      // values lie in different banks.
      constexpr int kGroups = 6, kHv = D / 64, kParts = C::kParts; // groups of a warp at most; chunks of a lane of a row
      constexpr uint32_t kPart = 16 * kHv * 32 * 16;               // bytes of a step's keys, or its values
      constexpr uint32_t kNone = 0xffffffffu;                      // no such row
      constexpr int kHalf = kGroups / 2, kFlight = 2 * kParts;     // a lane's copies under way, by halves of its groups (its own: no barrier)
      const int x = (ct >> 5) % 3, team = ct / 96, r = lane >> 2;
      const bool six = x == 0;                                     // (16 groups: the first warp has six, the others five)
      const uint8_t* pool[2] = {static_cast<const uint8_t*>(team ? a.v : a.k) + (lane & 3) * 16,
                                static_cast<const uint8_t*>(a.v) + (lane & 3) * 16};
      const uint32_t raw = smem_u32(smem + C::kRawAt) + team * kPart + (x * kHv * 32 + lane) * 16;
      // Lane l looks up rows l and 32 + l of the warp's 48. Nothing waits for a load in the step that issues it: block ids are
      // loaded two steps ahead, rows and scale bytes (of this lane's two rows) follow one step ahead. (The loads are without
      // conditions, where there is no such row from a place that there always is: a choice behind a load would wait for it.)
      int id[2];
      uint32_t row[2], byte[2][kParts], valid = 0;                  // valid: bit i, there is row i
      auto place = [&](int j, int i) {                              // of row i in step j, -1 where there is no such row
        const int q = 32 * i + lane, gr = 3 * (q >> 3) + x, p = sp.start(tb + j) + 8 * gr + (q & 7);
        return q < 8 * kGroups && gr < 16 && j < steps && seen(p) ? p : -1;
      };
      auto load_ids = [&](int j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) id[i] = btb[max(place(j, i), 0) >> pss];
      };
      // Rows of step j, whose ids have been loaded, their scale bytes, and which there are, for the masks.
      auto look_up = [&](int j) {
        uint8_t* bits = reinterpret_cast<uint8_t*>(&sh.tile[j % kTileRing][1]);
        valid = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = place(j, i), s = p & (ps - 1);
          const bool block = id[i] >= 0 && id[i] < a.num_blocks, there = p >= 0 && block;
          if (p >= 0 && !block) {
            flag(a.status, SA_DEV_BAD_BLOCK);
            *reinterpret_cast<volatile int*>(&sh.bad) = 1;
          }
          const uint32_t tile = there ? uint32_t(id[i]) * a.H_kv + h : 0u;
          row[i] = there ? (tile << pss) + s : kNone;
          valid |= uint32_t(there) << i;
          const uint8_t* s8 = a.scale + (uint64_t(tile) << (pss + 1)) + (there ? s : 0) + (team ? ps : 0);
#pragma unroll
          for (int c = 0; c < kParts; ++c) byte[i][c] = s8[c * ps];
          const uint32_t have = __ballot_sync(kFull, there);
          const int gr = 3 * (4 * i + lane) + x;
          if (team == 0 && lane < 4 && gr < 16 && 4 * i + lane < kGroups) bits[gr] = uint8_t(have >> (8 * lane));
        }
        if (ct == 0) sh.tile[j % kTileRing][0] = 1;
      };
      // Copies of group n, whose row of this lane is `at`.
      auto copy = [&](int n, int part, uint32_t at) {
        const uint8_t* from = pool[part] + (at == kNone ? 0u : uint64_t(at) * D);
        const int bytes = at == kNone ? 0 : 16;
#pragma unroll
        for (int c = 0; c < kHv; ++c) cp_async_16(raw + part * kPart + (3 * n * kHv + c) * 512, from + 64 * c, bytes);
      };
      uint32_t at[kGroups];                                          // rows of this lane in the groups of the next step
      auto spread = [&]() {
#pragma unroll
        for (int n = 0; n < kGroups; ++n) at[n] = __shfl_sync(kFull, n < 4 ? row[0] : row[1], (8 * n + r) & 31);
      };
      // The keys or the values into the slot at dst, and the next step's copies over them, if there are `more`. sc: scale bytes
      // of this lane's two rows. kWide: some scale is above 2^7.
      auto convert = [&](auto wide, uint32_t dst, int part, uint32_t sc, bool more) {
        constexpr bool kWide = decltype(wide)::value;
        auto read = [&](int n, uint4 (&u)[kHv]) {
#pragma unroll
          for (int c = 0; c < kHv; ++c)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(u[c].x), "=r"(u[c].y), "=r"(u[c].z), "=r"(u[c].w)
                         : "r"(raw + part * kPart + (3 * n * kHv + c) * 512));
        };
        const uint32_t to = dst + x * C::kGroupBytes + r * 128;
        const uint32_t at0 = to + (((2 * (lane & 3)) ^ r) << 4), at1 = to + (((2 * (lane & 3) + 1) ^ r) << 4);
        auto group = [&](int n, const uint4 (&u)[kHv], const Factor<T>& f) {
#pragma unroll
          for (int c = 0; c < kHv; ++c) {
            const uint32_t off = 3 * n * C::kGroupBytes + c * 1024;
            uint32_t w[8];
            values4<T, kWide>(u[c].x, f, w[0], w[1]);
            values4<T, kWide>(u[c].y, f, w[2], w[3]);
            values4<T, kWide>(u[c].z, f, w[4], w[5]);
            values4<T, kWide>(u[c].w, f, w[6], w[7]);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at0 + off), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at1 + off), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          }
        };
        if constexpr (kWide) {
#pragma unroll 1
          for (int n = 0; n < kGroups; ++n) {
            uint4 u[kHv];
            if (n % kHalf == 0) cp_async_wait<kFlight - 1>();
            const uint32_t mine = __shfl_sync(kFull, n < 4 ? row[0] : row[1], (8 * n + r) & 31);
            const Factor<T> f((__shfl_sync(kFull, sc, (8 * n + r) & 31) >> (n < 4 ? 0 : 8)) & 0xffu);
            if (n < kGroups - 1 || six) {
              read(n, u);
              group(n, u, f);
              if (more) copy(n, part, mine);
            }
            if (n % kHalf == kHalf - 1) cp_async_commit();
          }
        } else {
          // factors of this lane's two rows, side by side
          const Factor<T> f0(sc & 0xffu), f1((sc >> 8) & 0xffu);
          const uint32_t two_of = __byte_perm(f0.f, f1.f, 0x5410);
          uint32_t fac[kGroups];
#pragma unroll
          for (int n = 0; n < kGroups; ++n) fac[n] = __shfl_sync(kFull, two_of, (8 * n + r) & 31);
          uint4 u[2][kHv];                                           // a group's chunks are read while those before are turned
          cp_async_wait<kFlight - 1>();
          read(0, u[0]);
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            if (n + 1 == kHalf) cp_async_wait<kFlight - 2>();
            if (n < kGroups - 2 || (n < kGroups - 1 && six)) read(n + 1, u[(n + 1) & 1]);
            if (n < kGroups - 1 || six) {
              Factor<T> f;
              f.f = __byte_perm(fac[n], 0u, n < 4 ? 0x1010 : 0x3232);
              group(n, u[n & 1], f);
              if (more) copy(n, part, at[n]);
            }
            if (n % kHalf == kHalf - 1) cp_async_commit();
          }
        }
      };
      load_ids(0);
      look_up(0);
      spread();
      if (steps > 0) {
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            if (n < kGroups - 1 || six) copy(n, part, at[n]);
            if (n % kHalf == kHalf - 1) cp_async_commit();
          }
        }
      }
      load_ids(1);
      for (int j = 0; ok && j < steps; ++j) {
        const bool more = j + 1 < steps;
        uint32_t sc[kParts];
        bool wide = false;                                          // some scale above 2^7: its factor is two
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const uint32_t b0 = valid & 1u ? byte[0][c] : 0u, b1 = valid & 2u ? byte[1][c] : 0u;
          sc[c] = b0 | b1 << 8;
          wide = wide || Factor<T>(b0).wide() || Factor<T>(b1).wide();
        }
        wide = __any_sync(kFull, wide);
        if (more) look_up(j + 1);
        load_ids(j + 2);
        spread();
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (!ok) break;
          seq = 2 * j + team + part;
          if (seq >= C::kSlots && !wait_on(&sh.empty[seq % C::kSlots], (seq / C::kSlots - 1) & 1, sh, a.status)) ok = false;
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          if (wide) convert(std::true_type(), slot_at(seq), part, sc[part], more);
          else convert(std::false_type(), slot_at(seq), part, sc[part], more);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.full[seq % C::kSlots]));
        }
      }
      cp_async_wait<0>();
      if (!ok && ct == 0) mbar_wait(smem_u32(&sh.q), 0, a.status);
    } else if constexpr (kTma) {
      int ids = page_ids(0);
      int edge_seq = -1;                                           // values whose unseen rows are still to be zeroed
      uint32_t edge_bits[4];
      auto finish_edge = [&]() {
        if (edge_seq < 0) return;
        ok = __all_sync(kFull, wait_on(&sh.edge, edges++ & 1, sh, a.status));
        if (!ok) return;
        constexpr int kChunks = D / 8;
        const int c = lane % kChunks;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (edge_bits[x] == 0xffffffffu) continue;
          for (int r = lane / kChunks; r < 32; r += 32 / kChunks)
            if (!((edge_bits[x] >> r) & 1u))
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(
                               slot_at(edge_seq) + (4 * x + (r >> 3)) * C::kGroupBytes + (c >> 3) * 1024 + (r & 7) * 128 +
                               (c & 7) * 16),
                           "r"(0u)
                           : "memory");
        }
        hand_over(edge_seq);
        edge_seq = -1;
      };
      for (int j = 0; ok && j < steps; ++j) {
        const int j0 = sp.start(tb + j), cur = ids;
        ids = page_ids(j + 1);
        const uint32_t have = __ballot_sync(kFull, cur >= 0);
        const bool clean = __popc(have) == pages && j0 + kKeys <= len && (j0 >= w0 || j0 + kKeys <= a.n_sink);
        uint32_t bits[4];
        if (!clean) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = 32 * x + lane;
            bits[x] = __ballot_sync(kFull, seen(j0 + r) && ((have >> (r >> pss)) & 1u));
            if (lane == 0) sh.tile[j % kTileRing][1 + x] = bits[x];
          }
        }
        if (lane == 0) sh.tile[j % kTileRing][0] = !clean;
        __syncwarp();
        const uint32_t bytes = __popc(have) * (uint32_t(C::kGroupBytes) << pss >> 3);
        const int group = int(((int64_t(max(cur, 0)) * a.H_kv + h) << pss) >> 3);
        auto copy = [&](const CUtensorMap& map, uint32_t bar) {
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (cur >= 0)
            tma_load_4d(slot_at(seq) + (uint32_t(lane * C::kGroupBytes) << pss >> 3), &map, 0, 0, 0, group, bar);
          ++seq;
        };
        if (!claim()) break;
        copy(tmk, smem_u32(&sh.full[seq % C::kSlots]));
        finish_edge();
        if (!ok || !claim()) break;
        if (clean) {
          copy(tmv, smem_u32(&sh.full[seq % C::kSlots]));
        } else {
          edge_seq = seq;
#pragma unroll
          for (int x = 0; x < 4; ++x) edge_bits[x] = bits[x];
          fence_proxy_async_smem();
          copy(tmv, smem_u32(&sh.edge));
        }
      }
      const int left = edge_seq;
      if (ok) finish_edge();
      if (!ok) {                                                   // leave no copy under way (bounded waits)
        mbar_wait(smem_u32(&sh.q), 0, a.status);
        for (int x = max(0, seq - C::kSlots); x < seq; ++x)
          if (x != left) mbar_wait(smem_u32(&sh.full[x % C::kSlots]), (x / C::kSlots) & 1, a.status);
      }
    } else {
      // pool rows of a step's positions, two at most a thread, looked up a step ahead
      auto look_up = [&](int j, int64_t (&off)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i * kCopyThreads + ct, p = sp.start(tb + j) + r;
          off[i] = -1;
          if (j < steps && r < kKeys && seen(p)) {
            const int blk = btb[p >> pss];
            if (blk < 0 || blk >= a.num_blocks) {
              flag(a.status, SA_DEV_BAD_BLOCK);
              *reinterpret_cast<volatile int*>(&sh.bad) = 1;
            } else {
              off[i] = ((int64_t(blk) * a.H_kv + h) << pss) + (p & (ps - 1));
            }
          }
        }
      };
      int64_t next[2];
      look_up(0, next);
      for (int j = 0; ok && j < steps; ++j) {
        copy_sync();                                               // the rows of the step before are used up
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i * kCopyThreads + ct;
          if (r >= kKeys) break;                                   // (whole warps)
          sh.off[r] = next[i];
          const uint32_t bits = __ballot_sync(kFull, next[i] >= 0);
          if (lane == 0) sh.tile[j % kTileRing][1 + r / 32] = bits;
        }
        look_up(j + 1, next);
        copy_sync();
        if (ct == 0) {
          uint32_t all = 0xffffffffu;
          for (int x = 0; x < 4; ++x) all &= sh.tile[j % kTileRing][1 + x];
          sh.tile[j % kTileRing][0] = all != 0xffffffffu;
        }
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          if (!claim()) break;
          const uint8_t* pool = static_cast<const uint8_t*>(part ? a.v : a.k);
          constexpr int kChunks = D / 8;
          const int c = ct % kChunks;
          const uint32_t dst = slot_at(seq);
#pragma unroll 8
          for (int r = ct / kChunks; r < kKeys; r += kCopyThreads / kChunks) {
            const int64_t off = sh.off[r];
            cp_async_16(dst + (r >> 3) * C::kGroupBytes + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4),
                        off >= 0 ? pool + off * (D * 2) + c * 16 : pool, off >= 0 ? 16 : 0);
          }
          cp_async_commit();
          ++seq;
          if (seq - done > kLag) {
            cp_async_wait<kLag>();
            hand_over(done++);
          }
        }
      }
      cp_async_wait<0>();
      while (done < seq) hand_over(done++);
      if (!ok && ct == 0) mbar_wait(smem_u32(&sh.q), 0, a.status);
    }
  }
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc5_fence_after();
    tc5_dealloc(tmem, C::kCols);
  }
  if (w.parts == 1 || warp >= C::kMmaWarp) return;

  // ------------------------------------------------------------- merge the parts of the unit
  if (threadIdx.x == 0) sh.last = ticket(&a.tickets[w.unit]) == w.parts - 1;
  named_sync<C::kSoftmaxThreads>(2);
  if (!sh.last) return;
  // A warp merges 8 rows x 32 columns (eight a lane), two such at once, four parts in flight, in the order of the parts.
  constexpr int kWide = D / 32, kAtOnce = 2;
  const int64_t part0 = w.slot - w.part;
  const int tiles = (two ? 256 : 128) / 8 * kWide;
  for (int g0 = warp; g0 < tiles; g0 += kAtOnce * C::kMmaWarp) {
    float acc[kAtOnce][8], M[kAtOnce], tot[kAtOnce];
    int64_t orow[kAtOnce];
    int r[kAtOnce], c8[kAtOnce];                                   // row, chunk of eight columns
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int g = g0 + u * C::kMmaWarp;
      r[u] = g / kWide * 8 + (lane & 7), c8[u] = g % kWide * 4 + (lane >> 3);
      const int t = (r[u] >> 7) * half_tokens + (r[u] & 127) / G;
      orow[u] = g < tiles && (r[u] & 127) / G < half_tokens && t < nt
                    ? int64_t(w.c0 + t0 + t) * a.H_q + int64_t(h) * G + (r[u] & 127) % G
                    : -1;
      M[u] = -INFINITY, tot[u] = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[u][x] = 0.f;
    }
    if (!__any_sync(kFull, orow[0] >= 0 || orow[kAtOnce - 1] >= 0)) continue;
    for (int p0 = 0; p0 < w.parts; p0 += 4) {
      float4 x[kAtOnce][4][2];
      float z[kAtOnce][4];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[u][k] = -INFINITY;
          x[u][k][0] = x[u][k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (orow[u] >= 0 && p0 + k < w.parts) {
            const float4* src = a.part_o + ((part0 + p0 + k) * (D / 4) + 2 * c8[u]) * C::kRows + r[u];
            z[u][k] = __ldcg(a.part_lse + (part0 + p0 + k) * C::kRows + r[u]);
            x[u][k][0] = __ldcg(src);
            x[u][k][1] = __ldcg(src + C::kRows);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float top = fmaxf(M[u], fmaxf(fmaxf(z[u][0], z[u][1]), fmaxf(z[u][2], z[u][3])));
        const float f = M[u] == -INFINITY ? 0.f : ex2_approx((M[u] - top) * kLog2e);
        M[u] = top;
        tot[u] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float e = z[u][k] == -INFINITY ? 0.f : ex2_approx((z[u][k] - top) * kLog2e);   // 0: an empty part
          const float v[8] = {x[u][k][0].x, x[u][k][0].y, x[u][k][0].z, x[u][k][0].w,
                              x[u][k][1].x, x[u][k][1].y, x[u][k][1].z, x[u][k][1].w};
          tot[u] += e;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[u][i] = fmaf(e, v[i], acc[u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (orow[u] < 0) continue;
      const float f = tot[u] != 0.f ? 1.0f / tot[u] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[u][i] *= f;
      *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow[u] * D + 8 * c8[u]) =
          make_uint4(E::pack(acc[u][0], acc[u][1]), E::pack(acc[u][2], acc[u][3]), E::pack(acc[u][4], acc[u][5]),
                     E::pack(acc[u][6], acc[u][7]));
      if (a.lse && c8[u] == 0) a.lse[orow[u]] = tot[u] != 0.f ? M[u] + lg2_approx(tot[u]) * kLn2 : -INFINITY;
    }
  }
  if (threadIdx.x == 0) a.tickets[w.unit] = 0;
}

// Items of a call: at most one partly filled one per request.
int64_t items_of(int64_t tokens, int batch, int G, int D) { return tokens / (ways(D) * (128 / G)) + batch; }

// Items are cut into parts where they would leave half of the SMs idle (three
// requests a lane are looked over then).
bool splits(int64_t units, int batch, int ctas) { return 2 * units <= ctas && batch <= 96; }

// CTAs that run at once.
constexpr int per_sm(int D) { return 3 - ways(D); }
int resident(int D) { return sm_count() * per_sm(D); }

// Over 8 bits, items of some more units are cut into parts for several rounds of CTAs: those of one request that leave a
// fifth of the CTAs idle, and those of requests of several lengths, of which the longest would set the time (the lengths are
// looked at on the device). Measured (us) whole / so, 32 query heads over 8: of 128, 16 requests of 9 - 30 tokens behind 1000 -
// 32000 396 / 243, 32 such 585 / 447, 640 tokens behind 32000 434 / 307, 18 of 20 - 30 behind 8000 128 / 108; of 64, the 16
// 520 / 182; four prompts of 100 - 500, none of which is cut, 23.6 / 25.4.
constexpr int rounds(int D) { return D == 128 ? 3 : 2; }
bool splits_more(int64_t units, int batch, int D) {
  static_assert(rounds(64) * per_sm(64) <= kTicketsPerSm && rounds(128) * per_sm(128) <= kTicketsPerSm, "a counter for each unit");
  return batch <= 96 && (5 * units < 4 * resident(D) || (batch > 1 && units <= int64_t(rounds(D)) * resident(D)));
}

struct WsLayout {
  size_t part_lse, part_o, total;
};
WsLayout ws_layout(int64_t ctas, int D) {
  static_assert(per_sm(64) <= kTicketsPerSm && per_sm(128) <= kTicketsPerSm, "a counter for each CTA");
  WsLayout w;
  w.part_lse = ticket_bytes();
  w.part_o = w.part_lse + size_t(ctas) * 128 * ways(D) * 4;
  w.total = w.part_o + size_t(ctas) * 128 * ways(D) * D * 4;
  return w;
}

int g_smem[8][64];

template <typename T, int D, bool kTma, bool kQ8>
sa_status launch(const PagedPrefillArgs& a, cudaStream_t s, const CUtensorMap& mq, const CUtensorMap& mk,
                 const CUtensorMap& mv, int* cache) {
  auto k = paged_prefill_kernel<T, D, kTma, kQ8>;
  constexpr int smem = Cfg<D, kTma, kQ8>::kSharedAt + int(sizeof(Shared));
  if (!ensure_smem(k, smem, cache)) return SA_ERR_CUDA;
  const unsigned ctas = a.split ? unsigned(a.split * resident(D)) : unsigned(a.whole + (a.items * a.H_kv - a.whole) * a.tail_parts);
  return launch_ex(k, dim3(ctas), dim3(Cfg<D, kTma, kQ8>::kThreads), smem, s, false, 1, a, mq, mk, mv) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

template <typename T, int D, bool kQ8>
sa_status dispatch(const PagedPrefillArgs& a, cudaStream_t s, const sa_cache* c, const void* q, int slot) {
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (!make_query_map(&mq, q, D, a.H_q, a.T, a.G, 128 / a.G)) return SA_ERR_CUDA;
  if constexpr (kQ8) return launch<T, D, false, true>(a, s, mq, mk, mv, g_smem[slot]);
  else if (c->page_size >= 8 && make_group_map(&mk, c->k, c, c->page_size / 8) && make_group_map(&mv, c->v, c, c->page_size / 8))
    return launch<T, D, true, false>(a, s, mq, mk, mv, g_smem[2 * slot + 1]);
  else return launch<T, D, false, false>(a, s, mq, mk, mv, g_smem[2 * slot]);
}

size_t prefill_workspace(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads, int32_t head_dim, int32_t num_tokens) {
  if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || head_dim <= 0 || num_tokens < 0 ||
      num_q_heads % num_kv_heads)
    return 0;
  return ws_layout(resident(head_dim), head_dim).total;           // a part each of the CTAs that run at once
}

// Workspace of the calls of up to `tokens` rows over 8 bits but for the pages of many rows.
size_t few_workspace(int64_t tokens, int batch, int G, int D, int H) {
  const bool one = splits(items_of(tokens, batch, G, D) * H, batch, resident(D));
  const size_t n = ws_layout((one ? 1 : rounds(D)) * resident(D), D).total, draft = draft8_workspace(G, D);
  return n > draft ? n : draft;
}

// Calls over 8 bits whose requests have on the mean no more rows (token, query head) of a KV head than a warp holds sums for
// in registers go to the decode kernel, which turns no codes into values in shared memory; with 17 to 32 rows of 128 columns
// only where there are units enough that each is cut into few parts. Measured (us) there / here, 32 query heads of 128 over 8
// KV heads, four requests over 8000 - 30000: 1 - 2 tokens 44 / 78, 2 - 4 tokens 51 / 78, 3 - 8 tokens 64 / 77; one request over
// 30000, 4 tokens 31 / 37, 8 tokens 43 / 37; heads of 64, 3 - 8 tokens of four 45 / 61, 8 of one 31 / 36. A mean does not see
// a long request among short ones: 512 tokens behind 32000 beside 63 / 255 single tokens behind 1000 - 2000 take 529 / 1570
// here, in a call of their own 234 and the single ones 54 / 154; 2048 tokens 975 / 1203 against 889 and 54 / 155.
bool few_rows(int64_t tokens, int G, int D, int H, int batch) {
  const int most = D == 64 || batch * H >= 16 ? 32 : 16;
  return tokens * G <= most * int64_t(batch) && batch <= 1024;
}

// Calls over 8 bits with many products turn the codes into 16-bit pages of 128 tokens once, where the workspace has room for
// those, and run on them; a CTA's own turning of its tiles slows its products by a fifth, at head dim 64 to half. Worth it
// where that (`pairs`: of queries and keys that they see) takes longer than the pages do: their bytes, three for each code, and
// 8 us of launches. Measured (us) there / here, 32 query heads over 8 KV heads: of 128, 16384 tokens 1560 / 1280, 4096 147 / 136,
// 3000 94 / 107, eight prompts of 500 - 1200 106 / 109; of 64, 16384 tokens 2035 / 941, 2048 64 / 46, 1500 39 / 49, 2048 behind
// 32000 1168 / 550; 2048 behind 64000 with 64 heads of 128 2970 / 2370.
__host__ __device__ inline bool worth_pages(float pairs, float tokens, int Hq, int H, int D) {
  const float turning = (D == 128 ? 4.7e-10f : 2.6e-9f) * pairs * float(Hq * D), pages = 8.f + 1e-6f * tokens * float(H * D);
  return turning > pages;
}
// Of requests alike with `tokens` new ones in all and `cached` with them.
inline bool worth_pages(int64_t tokens, int64_t cached, int batch, int64_t seen, int Hq, int H, int D) {
  const double all = double(max(cached, tokens)), mean = min(double(seen), (all - 0.5 * double(tokens)) / batch);
  return worth_pages(float(double(tokens) * mean), float(min(all, double(seen) * batch + double(tokens))), Hq, H, D);
}

// A workspace's part for that behind the first `base` bytes: the two words of `turn`, a table of `pages` for each request, the
// pages.
struct Laid {
  size_t table, k, v, total;
};
inline Laid laid_layout(size_t base, int64_t pages, int batch, int H, int D) {
  Laid w;
  w.table = align256(base) + 256;
  w.k = w.table + align256(size_t(batch) * pages * 4);
  w.v = w.k + size_t(pages) * H * 128 * D * 2;
  w.total = w.v + size_t(pages) * H * 128 * D * 2;
  return w;
}

// Either call, on a checked cache; laid_call: of many rows over 8 bits (paged_prefill8.cu).
template <bool kQ8, typename LaidCall>
sa_status prefill_call(const sa_cache* cache, const sa_cache8* cache8, const sa_batch* batch, const void* q, int32_t num_q_heads,
                       const int32_t* new_cu, int32_t num_tokens, int32_t window, int32_t n_sink, float scale, void* out,
                       float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream,
                       LaidCall laid_call) {
  sa_status st = check_batch(batch);
  if (st != SA_OK) return st;
  if (!new_cu || num_tokens < 0 || (num_tokens > 0 && (!q || !out)) || num_q_heads <= 0 || num_q_heads % cache->num_kv_heads)
    return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || window < 0 || n_sink < 0) return SA_ERR_INVALID_ARG;
  const int G = num_q_heads / cache->num_kv_heads, D = cache->head_dim, H = cache->num_kv_heads;
  if (G > 16) return SA_ERR_UNSUPPORTED;
  // pool rows are counted in 32 bits
  if (kQ8 && uint64_t(cache->num_blocks) * H * cache->page_size >= 0xffffffffull) return SA_ERR_UNSUPPORTED;
  // (over 8 bits room for pages is no need: a workspace for more requests may have none where fewer of as many tokens want it)
  const size_t need = kQ8 ? few_workspace(num_tokens, batch->batch, G, D, H)
                          : sa_paged_prefill_workspace_size(batch->batch, H, num_q_heads, D, num_tokens);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return SA_ERR_WORKSPACE;
  if (num_tokens == 0) return SA_OK;
  if (kQ8 && few_rows(num_tokens, G, D, H, batch->batch)) {
    const sa_status few = draft8_call(cache8, batch, q, num_q_heads, new_cu, num_tokens, window, n_sink, scale, out, lse,
                                      workspace, dev_status, stream);
    if (few != SA_ERR_UNSUPPORTED) return few;
  }
  PagedPrefillArgs a = {};
  a.k = cache->k; a.v = cache->v; a.scale = kQ8 ? cache8->scale : nullptr; a.bt = batch->block_table; a.seq_lens = batch->seq_lens; a.new_cu = new_cu;
  a.out = out; a.lse = lse; a.status = dev_status;
  a.H_kv = H; a.H_q = num_q_heads; a.G = G; a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks;
  a.bt_stride = batch->bt_stride; a.batch = batch->batch; a.T = num_tokens; a.n_sink = n_sink;
  // a window of the table's length hides nothing
  a.window = window < int64_t(batch->bt_stride) * cache->page_size ? window : 0;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf(float(D))) * kLog2e;
  const int64_t items = items_of(num_tokens, batch->batch, G, D), units = items * H;
  if (units > 0x7fffffff) return SA_ERR_UNSUPPORTED;
  a.items = int(items);
  a.split = splits(units, batch->batch, resident(D)) ? 1 : kQ8 && splits_more(units, batch->batch, D) ? rounds(D) : 0;
  // The units behind the last full round of CTAs in parts that fill one more, where the table and the window leave room
  // for two parts' keys. Measured (us) without / with: a chunk of 2048 tokens x 64 heads behind 64000 (512 units) 2730 /
  // 2510, three requests of 700 - 900 behind 3000 - 4500 153 / 147; five of 100 - 900 behind 300 - 1500, whose parts would
  // all be empty, 65.5 / 68.
  const int ctas = resident(D), rest = int(units % ctas);
  const int64_t keys = min(int64_t(batch->bt_stride) * cache->page_size,
                           a.window > 0 ? int64_t(a.window) + n_sink : int64_t(0x7fffffff));
  a.tail_parts = !a.split && rest && keys >= 2 * kTailPart * kKeys ? max(1, min(ctas / rest, kMostTail)) : 1;
  a.whole = int(a.tail_parts > 1 ? units - rest : units);
  const WsLayout w = ws_layout((a.split > 1 ? a.split : 1) * ctas, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.tickets = reinterpret_cast<int32_t*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.part_o = reinterpret_cast<float4*>(ws + w.part_o);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if constexpr (kQ8) {
    st = laid_call(cache8, batch, q, a, workspace, workspace_bytes, need, s);
    if (st != SA_OK) return st;
  }
  const bool bf = cache->dtype == SA_BF16;
  if (D == 128)
    return bf ? dispatch<__nv_bfloat16, 128, kQ8>(a, s, cache, q, 0) : dispatch<__half, 128, kQ8>(a, s, cache, q, 1);
  return bf ? dispatch<__nv_bfloat16, 64, kQ8>(a, s, cache, q, 2) : dispatch<__half, 64, kQ8>(a, s, cache, q, 3);
}

}  // namespace
}  // namespace sa
