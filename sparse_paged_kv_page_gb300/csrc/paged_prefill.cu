// sa_paged_prefill: causal softmax attention of new tokens (a prompt, a chunk of
// one, a few drafted tokens) over the paged cache that already holds them.
//
// Mathematics: o = sum_j p_j v_j, p = softmax(scale q . k_j) over the visible
// positions j, in one pass with a running maximum m and sum l. O is rescaled only
// where m has grown by more than 2^8 since it was last used (p stays below 2^8,
// exact in float32 sums and inside both 16-bit types); the quotient o / l at the
// end makes any m right.
//
// A CTA owns 2 x 128 packed rows (token, query head of one KV head's group), so a
// key is read once for all G heads, and walks the visible keys 128 at a time. The
// products run on the 5th-generation tensor cores, accumulators in TMEM: S = Q K^T
// (128 x 128, one per half), P over S's columns as the A operand from TMEM, O += P V.
// Two warpgroups take the two halves, one row a thread (no shuffles): while one
// turns S into P the tensor cores work for the other. One warp issues the products,
// one the copies: keys and values in a ring of 128-row slots, page by page through
// a tensor map (pages of 8 tokens and more), or row by row with cp.async (smaller
// pages, and tiles with rows that must not be read: those get zeros).
//
// Bound by the tensor cores for prompts; for a few rows over a long cache by HBM,
// where the keys are split over CTAs and the last of an item's CTAs merges the
// parts in order.
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "paged.cuh"
#include "tc5.cuh"
#include "tma_map.h"

namespace sa {
namespace {

constexpr int kKeys = 128;                // positions per step
constexpr int kMmaWarp = 8;               // warps 0-3 and 4-7: the softmax of the two halves
constexpr int kSoftmaxThreads = 32 * kMmaWarp;
constexpr int kThreads = kSoftmaxThreads + 128;
// Registers: 384 threads are launched with 168 each; the softmax warpgroups take
// 208 (a row of 128 scores a thread) of what the third one gives back:
// 256 x 208 + 128 x 88 = 384 x 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kTileRing = 8;              // steps whose row masks are kept
constexpr float kGrow = 8.0f;             // log2 of the growth of the maximum that O does not follow
constexpr int kMaxSplit = 64;

struct PagedPrefillArgs {
  const void* k;
  const void* v;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* new_cu;
  void* out;
  float* lse;
  float* part_o;        // [items * H_kv][splits][256][D]
  float* part_lse;      // [items * H_kv][splits][256]
  int32_t* tickets;     // [items * H_kv]
  int32_t* status;
  int H_kv, H_q, G, ps_shift, num_blocks, bt_stride, batch, T, window, n_sink, items;
  float scale_log2;
};

template <int D, bool kTma>
struct Cfg {
  static constexpr int kProducers = kTma ? 1 : 3;                  // copy warps
  static constexpr int kHalves = D / 64;                           // 64-column halves of a row
  static constexpr int kGroupBytes = kHalves * 1024;               // 8 rows of a slot: [half][8 rows of 128 bytes]
  static constexpr int kSlotBytes = kKeys / 8 * kGroupBytes;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kQBytes = 2 * kSlotBytes;
  static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + 1024;
};

struct Shared {
  uint64_t full[8], empty[8], q, s[2], p[2], o[2];
  uint32_t tile[kTileRing][1 + kKeys / 32];   // [0]: rows of the step are masked by the words that follow
  int64_t off[kKeys];                         // pool row of each position of a gathered step, -1: none
  uint32_t tmem;
  int abort, last;
};

// Wait for a phase; false once any wait of the CTA has given up. The clock is read
// only after many tries (each try suspends the thread for a while by itself).
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, Shared& sh, int32_t* status) {
  const uint32_t b = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sh.abort)) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      flag(status, SA_DEV_TIMEOUT);
      *reinterpret_cast<volatile int*>(&sh.abort) = 1;
      return false;
    }
  }
}

template <typename T, int D, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ PagedPrefillArgs a, const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
  using E = Elem<T>;
  using C = Cfg<D, kTma>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = smem + C::kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.G, pss = a.ps_shift, half_tokens = 128 / G;

  // heads outermost: the CTAs of a wave share one head's keys in L2; long items first
  const int h = blockIdx.x / a.items, idx = a.items - 1 - blockIdx.x % a.items;
  int b, item;
  if (!find_item(a.new_cu, a.batch, 2 * half_tokens, idx, b, item)) return;
  const int c0 = a.new_cu[b], n = a.new_cu[b + 1] - c0, L = a.seq_lens[b];
  const int cap = int(min(int64_t(a.bt_stride) << pss, int64_t(0x7fffffff)));
  if (threadIdx.x == 0 && item == 0 && h == 0 && blockIdx.y == 0) {
    if (c0 < 0 || int64_t(c0) + n > a.T || L < n) flag(a.status, SA_DEV_BAD_COUNT);
    if (L > cap) flag(a.status, SA_DEV_OVERFLOW);
  }
  if (c0 < 0 || int64_t(c0) + n > a.T) return;
  const int t0 = item * 2 * half_tokens, nt = min(2 * half_tokens, n - t0);
  const int first = L - n + t0, last = first + nt - 1, len = min(max(L, 0), cap);
  const Span<kKeys> sp(first, last, len, a.window, a.n_sink);
  const bool two = nt > half_tokens;                              // the second half has rows
  const int ns = gridDim.y, per = (sp.tiles + ns - 1) / ns;
  const int tb = min(sp.tiles, int(blockIdx.y) * per), steps = min(sp.tiles, tb + per) - tb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.q), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s[i]), 1);
      mbar_init(smem_u32(&sh.p[i]), 4);
      mbar_init(smem_u32(&sh.o[i]), 1);
    }
    mbar_init_fence();
    sh.abort = 0;
  }
  if (warp == kMmaWarp) tc5_alloc(smem_u32(&sh.tmem), 512);
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = sh.tmem;                                  // columns: S/P of the halves, then O of the halves

  if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------- softmax: one row a thread
    const int tile = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(warp & 3) << 21;              // TMEM lane 32 * (warp % 4)
    const uint32_t s_col = tmem + lanes + tile * 128, o_col = tmem + lanes + 256 + tile * 128;
    const int t = tile * half_tokens + row / G;
    const bool in = row / G < half_tokens && t < nt;
    const int pos = in ? first + t : -1;
    const int64_t orow = in ? int64_t(c0 + t0 + t) * a.H_q + int64_t(h) * G + row % G : -1;
    float m = -INFINITY, l = 0.f;
    const bool act = tile == 0 || two;
    for (int j = 0; act && j < steps; ++j) {
      if (!__all_sync(kFull, wait_on(&sh.s[tile], j & 1, sh, a.status))) break;
      tc5_fence_after();
      float s[kKeys];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc5_ld32(reinterpret_cast<uint32_t*>(s) + 32 * c, s_col + 32 * c);
      const int j0 = sp.start(tb + j);
      const uint32_t* words = sh.tile[j % kTileRing];
      const uint32_t masked = *reinterpret_cast<const volatile uint32_t*>(words);
      // columns seen: up to hi, from lo on or below sk
      const int hi = min(pos, len - 1) - j0;
      const int lo = a.window > 0 ? pos - a.window + 1 - j0 : 0, sk = a.n_sink - j0;
      tc5_wait_ld();
      if (__any_sync(kFull, hi < kKeys - 1 || (lo > 0 && sk < kKeys) || masked)) {
#pragma unroll
        for (int c = 0; c < kKeys; ++c)
          if (c > hi || (c < lo && c >= sk)) s[c] = -INFINITY;
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t bits = reinterpret_cast<const volatile uint32_t*>(words)[1 + w];
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((bits >> c) & 1u)) s[32 * w + c] = -INFINITY;
          }
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < kKeys - 4; c += 8) {
#pragma unroll
        for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], s[c + x], s[c + 4 + x]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], s[kKeys - 4 + x]);
      const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      if (j == 0) {
        m = m_new;
      } else if (__any_sync(kFull, (m_new - m) * a.scale_log2 > kGrow)) {
        // S of this step is complete, so the products into O before it are too
        const float f = m_new == m ? 1.f : ex2_approx((m - m_new) * a.scale_log2);
        l *= f;
        m = m_new;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc5_ld32(reinterpret_cast<uint32_t*>(o), o_col + 32 * c);
          tc5_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] *= f;
          tc5_st32(o_col + 32 * c, reinterpret_cast<uint32_t*>(o));
        }
      }
      const float base = m == -INFINITY ? 0.f : -m * a.scale_log2;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          float p0, p1;
          fma2(p0, p1, s[32 * c + 2 * x], s[32 * c + 2 * x + 1], a.scale_log2, base);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          add2(sum[2 * (x & 1)], sum[2 * (x & 1) + 1], p0, p1);
          w[x] = E::pack(p0, p1);
        }
        tc5_st16(s_col + 16 * c, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc5_wait_st();
      tc5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.p[tile]));
    }
    // ------------------------------------------------------------- outputs
    if (act) {
      bool ok = steps == 0 || wait_on(&sh.o[tile], 0, sh, a.status);
      ok = __all_sync(kFull, ok) && steps > 0;
      tc5_fence_after();
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      const float row_lse = l > 0.f ? (m * a.scale_log2 + lg2_approx(l)) * kLn2 : -INFINITY;
      const int64_t prow = ((int64_t(blockIdx.x) * ns + blockIdx.y) * 2 + tile) * 128 + row;
      if (in) {
        if (ns > 1) a.part_lse[prow] = row_lse;
        else if (a.lse) a.lse[orow] = row_lse;
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        __syncwarp();
        if (ok) {
          tc5_ld32(reinterpret_cast<uint32_t*>(o), o_col + 32 * c);
          tc5_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = l > 0.f ? o[x] * inv : 0.f;
        if (in && ns > 1) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + prow * D + 32 * c);
#pragma unroll
          for (int x = 0; x < 8; ++x) dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        } else if (in) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * D + 32 * c);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            dst[x] = make_uint4(E::pack(o[8 * x], o[8 * x + 1]), E::pack(o[8 * x + 2], o[8 * x + 3]),
                                E::pack(o[8 * x + 4], o[8 * x + 5]), E::pack(o[8 * x + 6], o[8 * x + 7]));
        }
      }
      tc5_fence_before();
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
  if (warp == kMmaWarp) {
    // ------------------------------------------------------------- products, issued by one thread
    if (steps > 0 && elect_one()) {
      constexpr uint32_t id_s = tc5_idesc(kBf16, 128, kKeys, false), id_o = tc5_idesc(kBf16, 128, D, true);
      const uint64_t q_desc = tc5_desc(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = tc5_desc(smem_u32(ring), 16, C::kGroupBytes);
      const uint64_t v_desc = tc5_desc(smem_u32(ring), 1024, C::kGroupBytes);
      auto scores = [&](int tile, int slot) {                       // S = Q K^T
        const uint64_t qd = q_desc + uint32_t(tile * C::kSlotBytes / 16), kd = k_desc + uint32_t(slot * C::kSlotBytes / 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t q_at = (kk >> 2) * (128 * 128) + (kk & 3) * 32, k_at = (kk >> 2) * 1024 + (kk & 3) * 32;
          tc5_mma_ss(tmem + tile * 128, qd + q_at / 16, kd + k_at / 16, id_s, kk > 0);
        }
      };
      auto outputs = [&](int tile, int slot, bool add, uint32_t parity) {   // O += P V once P is there
        if (!wait_on(&sh.p[tile], parity, sh, a.status)) return false;
        tc5_fence_after();
        const uint64_t vd = v_desc + uint32_t(slot * C::kSlotBytes / 16);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc5_mma_ts(tmem + 256 + tile * 128, tmem + tile * 128 + kk * 8, vd + uint32_t(kk * 2 * C::kGroupBytes / 16), id_o,
                     add || kk > 0);
        return true;
      };
      auto wait_full = [&](int seq) { return wait_on(&sh.full[seq % C::kSlots], (seq / C::kSlots) & 1, sh, a.status); };
      bool ok = wait_on(&sh.q, 0, sh, a.status) && wait_full(0);
      if (ok) {
        tc5_fence_after();
        scores(0, 0);
        tc5_commit(smem_u32(&sh.s[0]));
        if (two) {
          scores(1, 0);
          tc5_commit(smem_u32(&sh.s[1]));
        }
        tc5_commit(smem_u32(&sh.empty[0]));
      }
      for (int j = 0; ok && j < steps; ++j) {
        const int sv = 2 * j + 1, sk = 2 * j + 2;
        const bool more = j + 1 < steps;
        if (!(ok = wait_full(sv) && outputs(0, sv % C::kSlots, j > 0, j & 1))) break;
        if (!more) tc5_commit(smem_u32(&sh.o[0]));
        if (more) {
          if (!(ok = wait_full(sk))) break;
          tc5_fence_after();
          scores(0, sk % C::kSlots);
          tc5_commit(smem_u32(&sh.s[0]));
        }
        if (two) {
          if (!(ok = outputs(1, sv % C::kSlots, j > 0, j & 1))) break;
          if (!more) tc5_commit(smem_u32(&sh.o[1]));
        }
        tc5_commit(smem_u32(&sh.empty[sv % C::kSlots]));
        if (more) {
          if (two) {
            scores(1, sk % C::kSlots);
            tc5_commit(smem_u32(&sh.s[1]));
          }
          tc5_commit(smem_u32(&sh.empty[sk % C::kSlots]));
        }
      }
      if (!ok) {                                                    // let what was issued finish
        tc5_commit(smem_u32(&sh.o[0]));
        mbar_wait(smem_u32(&sh.o[0]), 0, a.status);
      }
    }
    __syncwarp();
  } else if (warp <= kMmaWarp + C::kProducers) {
    // ------------------------------------------------------------- copies
    constexpr int kCopyThreads = 32 * C::kProducers;
    const int ct = threadIdx.x - 32 * (kMmaWarp + 1);
    auto copy_sync = [&]() {
      if (C::kProducers == 1) __syncwarp();
      else asm volatile("bar.sync 1, %0;\n" ::"n"(kCopyThreads) : "memory");
    };
    const int w0 = a.window > 0 ? max(0, first - a.window + 1) : 0;
    const int32_t* btb = a.bt + int64_t(b) * a.bt_stride;
    const int ps = 1 << pss;
    if (steps > 0 && ct == 0) {
      const uint32_t bar = smem_u32(&sh.q);
      mbar_arrive_expect_tx(bar, uint32_t((two ? 2 : 1) * C::kHalves * G * half_tokens * 128));
      for (int tile = 0; tile < (two ? 2 : 1); ++tile)
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem_u32(smem) + tile * C::kSlotBytes + hf * kKeys * 128, &tmq, hf * 64, h * G,
                      c0 + t0 + tile * half_tokens, bar);
    }
    // The block ids of a step through the tensor map, one a lane; -1 where there is none.
    auto page_ids = [&](int j) {
      int id = -1;
      if (kTma && j < steps) {
        const int at = sp.start(tb + j) + (lane << pss);
        if (lane < (kKeys >> pss) && at < len) id = btb[at >> pss];
      }
      return id;
    };
    int pending = -1;                                              // slot whose gathered rows are still under way
    auto finish = [&](int slot) {
      fence_proxy_async_smem();
      copy_sync();
      if (ct == 0) mbar_arrive(smem_u32(&sh.full[slot]));
    };
    int ids = page_ids(0);
    bool ok = true;
    int seq = 0;
    for (int j = 0; ok && j < steps; ++j) {
      const int j0 = sp.start(tb + j);
      const int cur = ids;
      ids = page_ids(j + 1);
      // every row of the step may be read, and comes from a page that exists
      bool clean = false;
      if (kTma) {
        clean = j0 + kKeys <= len && (j0 >= w0 || j0 + kKeys <= a.n_sink);
        clean = clean && __all_sync(kFull, lane >= (kKeys >> pss) || (cur >= 0 && cur < a.num_blocks));
      }
      if (!clean) {
        copy_sync();                                               // the offsets of the step before are used up
        for (int r0 = 0; r0 < kKeys; r0 += kCopyThreads) {
          const int r = r0 + ct, p = j0 + r;
          if (r >= kKeys) break;                                   // (whole warps)
          int64_t off = -1;
          if (p < len && (p >= w0 || p < a.n_sink)) {
            const int blk = btb[p >> pss];
            if (blk < 0 || blk >= a.num_blocks) flag(a.status, SA_DEV_BAD_BLOCK);
            else off = ((int64_t(blk) * a.H_kv + h) << pss) + (p & (ps - 1));
          }
          sh.off[r] = off;
          const uint32_t bits = __ballot_sync(kFull, off >= 0);
          if (lane == 0) sh.tile[j % kTileRing][1 + r / 32] = bits;
        }
      }
      if (ct == 0) sh.tile[j % kTileRing][0] = !clean;
      copy_sync();
#pragma unroll 1
      for (int part = 0; part < 2; ++part, ++seq) {
        const int slot = seq % C::kSlots;
        if (seq >= C::kSlots) {
          ok = wait_on(&sh.empty[slot], (seq / C::kSlots - 1) & 1, sh, a.status);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
        }
        const uint32_t dst = smem_u32(ring) + slot * C::kSlotBytes;
        if (clean) {
          const uint32_t bar = smem_u32(&sh.full[slot]);
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kSlotBytes);
          __syncwarp();
          if (lane < (kKeys >> pss)) {
            const int group = int(((int64_t(cur) * a.H_kv + h) << pss) >> 3);
            tma_load_4d(dst + (uint32_t(lane * C::kGroupBytes) << (pss - 3)), part ? &tmv : &tmk, 0, 0, 0, group, bar);
          }
        } else {
          const uint8_t* pool = static_cast<const uint8_t*>(part ? a.v : a.k);
          constexpr int kChunks = D / 8;
          const int c = ct % kChunks;
#pragma unroll 8
          for (int r = ct / kChunks; r < kKeys; r += kCopyThreads / kChunks) {
            const int64_t off = sh.off[r];
            cp_async_16(dst + (r >> 3) * C::kGroupBytes + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4),
                        off >= 0 ? pool + off * (D * 2) + c * 16 : pool, off >= 0 ? 16 : 0);
          }
          cp_async_commit();
          if (kTma) {
            cp_async_wait<0>();
            finish(slot);
          } else {
            if (pending >= 0) {
              cp_async_wait<1>();
              finish(pending);
            }
            pending = slot;
          }
        }
      }
    }
    cp_async_wait<0>();
    if (pending >= 0) finish(pending);
    if (!ok && steps > 0) {                                        // leave no copy under way (bounded waits)
      mbar_wait(smem_u32(&sh.q), 0, a.status);
      for (int x = max(0, seq - C::kSlots); x < seq; ++x)
        mbar_wait(smem_u32(&sh.full[x % C::kSlots]), (x / C::kSlots) & 1, a.status);
    }
  }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc5_fence_after();
    tc5_dealloc(tmem, 512);
  }
  if (ns == 1 || warp >= kMmaWarp) return;

  // ------------------------------------------------------------- merge the parts of the item
  auto merge_sync = [] { asm volatile("bar.sync 2, %0;\n" ::"n"(kSoftmaxThreads) : "memory"); };
  if (threadIdx.x == 0) sh.last = ticket(&a.tickets[blockIdx.x]) == ns - 1;
  merge_sync();
  if (!sh.last) return;
  float* wgt = reinterpret_cast<float*>(smem);                     // [256][ns], then 1 / sum in [256]
  float* inv = wgt + 256 * ns;
  const int64_t part0 = int64_t(blockIdx.x) * ns * 256;
  auto row_of = [&](int r) -> int64_t {                            // row of q and out, -1: none
    const int t = (r >> 7) * half_tokens + (r & 127) / G;
    if ((r & 127) / G >= half_tokens || t >= nt) return -1;
    return int64_t(c0 + t0 + t) * a.H_q + int64_t(h) * G + (r & 127) % G;
  };
  const int mine = threadIdx.x;
  if (const int64_t orow = row_of(mine); orow >= 0) {
    const int r = mine;
    float M = -INFINITY, tot = 0.f;
    for (int s = 0; s < ns; ++s) {
      const float x = __ldcg(a.part_lse + part0 + s * 256 + r);
      wgt[r * ns + s] = x;
      M = fmaxf(M, x);
    }
    for (int s = 0; s < ns; ++s) {
      const float x = wgt[r * ns + s], w = x == -INFINITY ? 0.f : ex2_approx((x - M) * kLog2e);
      wgt[r * ns + s] = w;
      tot += w;
    }
    inv[r] = tot > 0.f ? 1.0f / tot : 0.f;
    if (a.lse) a.lse[orow] = tot > 0.f ? M + lg2_approx(tot) * kLn2 : -INFINITY;
  }
  merge_sync();
  for (int i = threadIdx.x; i < 256 * (D / 4); i += kSoftmaxThreads) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    const int64_t orow = row_of(r);
    if (orow < 0) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < ns; ++s) {
      const float w = wgt[r * ns + s];
      const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + (part0 + s * 256 + r) * D + d));
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
    const float f = inv[r];
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + orow * D + d) =
        make_uint2(E::pack(acc.x * f, acc.y * f), E::pack(acc.z * f, acc.w * f));
  }
  if (threadIdx.x == 0) a.tickets[blockIdx.x] = 0;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Items of a call: at most one partly filled one per request.
int64_t items_of(int64_t tokens, int batch, int G) { return tokens / (2 * (128 / G)) + batch; }

// CTAs that share an item's keys: as many as fill the SMs once, where the items
// alone would leave half of them idle.
int splits_of(int64_t ctas, int64_t cap_tokens, int sms) {
  if (2 * ctas > sms) return 1;
  int64_t s = sms / ctas;
  const int64_t steps = (cap_tokens + kKeys - 1) / kKeys;
  if (s > steps) s = steps;
  if (s > kMaxSplit) s = kMaxSplit;
  return s < 1 ? 1 : int(s);
}

struct WsLayout {
  size_t part_lse, part_o, total;
};
// For `ctas` (item, split) pairs. Where a call splits, items x splits <= SMs, so
// this depends on the call's tokens only through whether it can split at all.
WsLayout ws_layout(int64_t ctas, int D) {
  WsLayout w;
  w.part_lse = align256(size_t(ctas) * 4);
  w.part_o = w.part_lse + size_t(ctas) * 256 * 4;
  w.total = w.part_o + size_t(ctas) * 256 * D * 4;
  return w;
}

int g_smem[8][64];

template <typename T, int D, bool kTma>
sa_status launch(const PagedPrefillArgs& a, int splits, cudaStream_t s, const CUtensorMap& mq, const CUtensorMap& mk,
                 const CUtensorMap& mv, int* cache) {
  auto k = paged_prefill_kernel<T, D, kTma>;
  if (!ensure_smem(k, Cfg<D, kTma>::kSmem, cache)) return SA_ERR_CUDA;
  return launch_ex(k, dim3(unsigned(a.items) * a.H_kv, splits), dim3(kThreads), Cfg<D, kTma>::kSmem, s,
                   false, 1, a, mq, mk, mv) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

template <typename T, int D>
sa_status dispatch(const PagedPrefillArgs& a, int splits, cudaStream_t s, const sa_cache* c, const void* q, int slot) {
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (!make_query_map(&mq, q, D, a.H_q, a.T, a.G, 128 / a.G)) return SA_ERR_CUDA;
  if (c->page_size >= 8 && make_group_map(&mk, c->k, c, c->page_size / 8) && make_group_map(&mv, c->v, c, c->page_size / 8))
    return launch<T, D, true>(a, splits, s, mq, mk, mv, g_smem[2 * slot + 1]);
  return launch<T, D, false>(a, splits, s, mq, mk, mv, g_smem[2 * slot]);
}

}  // namespace
}  // namespace sa

extern "C" size_t sa_paged_prefill_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads,
                                                  int32_t head_dim, int32_t num_tokens) {
  using namespace sa;
  if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || head_dim <= 0 || num_tokens < 0 ||
      num_q_heads % num_kv_heads)
    return 0;
  const int64_t least = int64_t(batch) * num_kv_heads;             // items of a call of few tokens
  return 2 * least > sm_count() ? 256 : ws_layout(sm_count(), head_dim).total;
}

extern "C" sa_status sa_paged_prefill(const sa_cache* cache, const sa_batch* batch, const void* q, int32_t num_q_heads,
                                      const int32_t* new_cu, int32_t num_tokens, int32_t window, int32_t n_sink,
                                      float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                      int32_t* dev_status, void* stream) {
  using namespace sa;
  sa_status st = check_cache(cache, true, false);
  if (st != SA_OK) return st;
  if ((st = check_batch(batch)) != SA_OK) return st;
  if (!q || !out || !new_cu || num_tokens < 0 || num_q_heads <= 0 || num_q_heads % cache->num_kv_heads)
    return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || window < 0 || n_sink < 0) return SA_ERR_INVALID_ARG;
  const int G = num_q_heads / cache->num_kv_heads, D = cache->head_dim, H = cache->num_kv_heads;
  if (G > 16) return SA_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < sa_paged_prefill_workspace_size(batch->batch, H, num_q_heads, D, num_tokens))
    return SA_ERR_WORKSPACE;
  if (num_tokens == 0) return SA_OK;
  PagedPrefillArgs a = {};
  a.k = cache->k; a.v = cache->v; a.bt = batch->block_table; a.seq_lens = batch->seq_lens; a.new_cu = new_cu;
  a.out = out; a.lse = lse; a.status = dev_status;
  a.H_kv = H; a.H_q = num_q_heads; a.G = G; a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks;
  a.bt_stride = batch->bt_stride; a.batch = batch->batch; a.T = num_tokens; a.window = window; a.n_sink = n_sink;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf(float(D))) * kLog2e;
  const int64_t items = items_of(num_tokens, batch->batch, G), ctas = items * H;
  if (ctas > 0x7fffffff) return SA_ERR_UNSUPPORTED;
  a.items = int(items);
  const int64_t seen = window > 0 ? int64_t(window) + n_sink + 3 * kKeys : int64_t(1) << 40;
  const int64_t cap = int64_t(batch->bt_stride) * cache->page_size;
  const int splits = splits_of(ctas, cap < seen ? cap : seen, sm_count());
  if (splits > 1) {
    const WsLayout w = ws_layout(sm_count(), D);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.tickets = reinterpret_cast<int32_t*>(ws);
    a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SA_BF16;
  if (D == 128)
    return bf ? dispatch<__nv_bfloat16, 128>(a, splits, s, cache, q, 0) : dispatch<__half, 128>(a, splits, s, cache, q, 1);
  return bf ? dispatch<__nv_bfloat16, 64>(a, splits, s, cache, q, 2) : dispatch<__half, 64>(a, splits, s, cache, q, 3);
}
