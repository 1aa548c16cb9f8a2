// sa_paged_decode: softmax attention of one new token per request over its whole
// paged cache, or over a sliding window of it and its first tokens.
//
// Mathematics: o = sum_j p_j v_j with p = softmax(scale q . k_j) over the visible
// positions j, in one pass: running maximum m and sum l, o rescaled when m grows.
// Parts over disjoint ranges with (o_s, lse_s) merge exactly to
// lse = log sum_s exp(lse_s), o = sum_s exp(lse_s - lse) o_s.
//
// Bound by HBM: every visible key and value is read once for the G <= 16 query
// heads of its KV head (4 G flops per 4 bytes at most). All requests' visible
// tokens, in groups of 64, are one line that the CTAs cut into equal parts (the
// lengths are read on the device), so a ragged batch keeps every SM busy. A CTA's
// part covers the end of one (request, KV head), whole ones, and the beginning of
// another; a unit cut into parts is merged by the last of its CTAs to finish, in
// the order of the parts, so results do not depend on timing.
//
// Each of the 4 warps takes every fourth tile of 16 tokens through a private ring
// of stages filled by the TMA engine (pages of 16 tokens and more) or by 16-byte
// cp.async row by row (smaller pages): S = Q K^T and O += P V with mma.sync
// m16n8k16 (rows: the query heads, padded to 16), P rounded to the element type as
// the operand, sums in float32.
//
// Measured in replayed graphs: 4 requests of 131072 tokens, 64 / 8 heads of 128, 312 us,
// 6.9 TB/s (more than a copy's 6.8: reads alone); 16 of 2048 - 32768, 178 us, 6.5 TB/s;
// pages of one token behind a window of 4096, 81 us, bound by the rows' copies; one request
// of 1024, 7.4 us, bound by the launch, three dependent loads and the merge.
#include "common.cuh"
#include "host.h"
#include "paged.cuh"
#include "tma_map.h"

namespace sa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;              // 241 registers a thread
constexpr int kMaxBatch = 1024;
constexpr int kFlight = 8;                 // parts a merging thread has in flight

struct PagedDecodeArgs {
  const void* k;
  const void* v;
  const void* q;
  const int32_t* bt;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  float* part_o;        // [CTAs][2][G][D]
  float* part_lse;      // [CTAs][2][G]
  int32_t* tickets;     // [CTAs]: of the cut unit that begins in a CTA
  int32_t* status;
  int H_kv, H_q, G, ps_shift, num_blocks, bt_stride, batch, window, n_sink;
  float scale_log2;
};

template <int D>
struct Tile {
  // Tiles a warp has under way or at work. D = 128, 128 k tokens of 4 requests: 319 us with 3, 307 with 2.
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kBytes = 16 * D * 2;
  static constexpr int kChunks = D / 8;
  static constexpr int kRowsPerOp = 32 / kChunks;
  static constexpr int kOps = 16 / kRowsPerOp;
  static constexpr int kStageBytes = 2 * kBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMerge = 4 * (kWarps * 32 + kWarps * 16 * (D + 4));
  static constexpr int kSmem = kRing + kMerge + 1024;
};

template <typename T, int D, bool kTma>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  using E = Elem<T>;
  using TL = Tile<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int kStages = TL::kStages;
  __shared__ uint32_t s_mask[kWarps][kStages];
  __shared__ __align__(8) uint64_t s_bar[kWarps][kStages];
  __shared__ int s_last;
  __shared__ float s_sf[kWarps][16], s_rl[16];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int G = a.G, pss = a.ps_shift;
  const int cap = int(min(int64_t(a.bt_stride) << pss, int64_t(0x7fffffff)));
  auto length = [&](int b) { return max(0, a.seq_lens[b]); };
  auto span = [&](int L) { return Span<16>(L - 1, L - 1, min(L, cap), a.window, a.n_sink); };

  // A warp's barriers are its own: its first lane makes them, and the warp meets before any lane arms or waits on one
  // (no barrier of the block stands between this and a warp's first copies).
  if constexpr (kTma) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&s_bar[warp][s]), 1);
      mbar_init_fence();
    }
    __syncwarp();
  }
  // Groups of a request (an empty one has a group per head too: its outputs are written). Every warp finds its
  // places by itself, 32 requests at a time.
  auto groups_of = [&](int b0) {
    if (b0 + lane >= a.batch) return 0;
    const int L = a.seq_lens[b0 + lane];
    if (blockIdx.x == 0 && threadIdx.x < 32) {
      if (L < 0) flag(a.status, SA_DEV_BAD_COUNT);
      if (L > cap) flag(a.status, SA_DEV_OVERFLOW);
    }
    return a.H_kv * max(1, (span(max(0, L)).tiles + 3) >> 2);
  };
  const int head_groups = groups_of(0);          // of requests 0 .. 31
  int all = head_groups;
#pragma unroll 4
  for (int b0 = 32; b0 < a.batch; b0 += 32) all += groups_of(b0);
  const int64_t total = __reduce_add_sync(kFull, all), N = min(int64_t(gridDim.x), total);   // every CTA has a group
  if (blockIdx.x >= N) return;
  int at = int(total * blockIdx.x / N);
  const int stop = int(total * (int64_t(blockIdx.x) + 1) / N);

  uint8_t* wbuf = smem + warp * kStages * TL::kStageBytes;
  int cnt = 0;                                  // tiles this warp has issued and consumed in all
  bool alive = true;

  // The part of a unit at work: request b, KV head h, groups [gi, ge) of its `groups` (the first is group unit_at of
  // all), the lengths and the visible range, this warp's nt tiles from t_begin + warp on, every kWarps-th.
  int b = 0, h = 0, gi = 0, ge = 0, groups = 1, unit_at = 0, Lc = 0, w0 = 0, t_begin = 0, nt = 0;
  Span<16> sp(-1, -1, 0, 0, 0);
  const int32_t* btb = a.bt;
  uint32_t qa[D / 16][4];                       // Q as the A operand (rows: the query heads, zero beyond G)
  float o[D / 8][4], m_r[2], l_r[2];
  // Block ids are loaded a batch of tiles ahead, one id a lane: a tile has one page, or 16 / page_size of them.
  const int ids_shift = max(0, 4 - pss);                 // log2 of the ids of a tile
  const int per_batch = 32 >> ids_shift;
  int ids = -1, ids_next = -1;
  bool running = false;

  while (true) {
    // what the merge of the part just done needs; then the next part begins, so that its first tiles are under way
    // during the merge
    const int d_b = b, d_h = h, d_gi = gi, d_ge = ge, d_groups = groups, d_unit_at = unit_at;
    const bool more = at < stop;
    auto load_ids = [&](int i) {
      const int ti = i + (lane >> ids_shift);
      int id = -1;
      if (ti < nt) {
        const int j = sp.start(t_begin + warp + ti * kWarps) + ((lane & ((1 << ids_shift) - 1)) << pss);
        if (j < Lc) {
          id = btb[j >> pss];
          if (id < 0 || id >= a.num_blocks) {
            flag(a.status, SA_DEV_BAD_BLOCK);
            id = -1;
          }
        }
      }
      return id;
    };
    auto issue = [&](int i) {
      if ((i & (per_batch - 1)) == 0) {
        ids = ids_next;
        ids_next = load_ids(i + per_batch);
      }
      const int st = (cnt + i) % kStages;
      const int j0 = sp.start(t_begin + warp + i * kWarps);
      // rows of the tile that the query sees
      auto low = [&](int n) { return (1u << min(max(n, 0), 16)) - 1u; };
      uint32_t vmask = low(Lc - j0) & (~low(w0 - j0) | low(min(a.n_sink, w0) - j0));
      const uint32_t sk = smem_u32(wbuf + st * TL::kStageBytes), sv = sk + TL::kBytes;
      if constexpr (kTma) {
        const int blk = __shfl_sync(kFull, ids, i & 31);
        if (blk < 0) vmask = 0;
        if (lane == 0) {
          s_mask[warp][st] = vmask;
          const uint32_t bar = smem_u32(&s_bar[warp][st]);
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(bar, vmask ? uint32_t(TL::kStageBytes) : 0u);
          if (vmask) {
            const int y = int(((int64_t(blk) * a.H_kv + h) << pss) + (j0 & ((1 << pss) - 1)));
            tma_load_3d(sk, &tmk, 0, y, 0, bar);
            tma_load_3d(sv, &tmv, 0, y, 0, bar);
          }
        }
      } else {
        // lane r < 16 knows the pool row of tile row r
        const int r = lane & 15;
        const int src = (((i & (per_batch - 1)) << ids_shift) + (r >> pss)) & 31;
        const int blk = __shfl_sync(kFull, ids, pss >= 4 ? (i & 31) : src);
        const bool valid = blk >= 0 && ((vmask >> r) & 1u);
        const int64_t off = (((int64_t(blk) * a.H_kv + h) << pss) + ((j0 + r) & ((1 << pss) - 1))) * D;
        vmask = __ballot_sync(kFull, valid) & 0xffffu;
        if (lane == 0) s_mask[warp][st] = vmask;
        const T* kbase = static_cast<const T*>(a.k);
        const T* vbase = static_cast<const T*>(a.v);
        const int chunk = lane % TL::kChunks;
#pragma unroll
        for (int r0 = 0; r0 < TL::kOps; ++r0) {
          const int row = lane / TL::kChunks + r0 * TL::kRowsPerOp;
          const int64_t ro = __shfl_sync(kFull, off, row);
          const bool rv = (vmask >> row) & 1u;
          const uint32_t d = swz16<D>(row, chunk);
          cp_async_16(sk + d, rv ? static_cast<const void*>(kbase + ro + chunk * 8) : a.k, rv ? 16 : 0);
          cp_async_16(sv + d, rv ? static_cast<const void*>(vbase + ro + chunk * 8) : a.v, rv ? 16 : 0);
        }
      }
    };

    if (more) {
      // the request and head of group `at`
      int before = 0, mine = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int x = b0 ? groups_of(b0) : head_groups;
        int sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, sum, o);
          if (lane >= o) sum += y;
        }
        const int k = __popc(__ballot_sync(kFull, before + sum <= at));
        if (k < 32) {
          b = b0 + k;
          mine = __shfl_sync(kFull, x, k);
          before += __shfl_sync(kFull, sum, k) - mine;
          break;
        }
        before += __shfl_sync(kFull, sum, 31);
      }
      groups = mine / a.H_kv;
      h = (at - before) / groups, unit_at = before + h * groups;
      gi = at - unit_at, ge = min(groups, gi + stop - at);
      at += ge - gi;
      const int L = length(b);
      Lc = min(L, cap);
      sp = span(L);
      w0 = a.window > 0 ? max(0, L - a.window) : 0;
      t_begin = gi * 4;
      const int t_end = min(ge * 4, sp.tiles);
      nt = t_begin + warp < t_end ? (t_end - t_begin - warp + kWarps - 1) / kWarps : 0;
      btb = a.bt + int64_t(b) * a.bt_stride;
      ids_next = load_ids(0);
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) +
                                                             (int64_t(b) * a.H_q + int64_t(h) * G) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int c0 = (kk * 16 + 2 * tq) >> 1, c1 = c0 + 4;
        qa[kk][0] = g < G ? qp[g * (D / 2) + c0] : 0u;
        qa[kk][1] = g + 8 < G ? qp[(g + 8) * (D / 2) + c0] : 0u;
        qa[kk][2] = g < G ? qp[g * (D / 2) + c1] : 0u;
        qa[kk][3] = g + 8 < G ? qp[(g + 8) * (D / 2) + c1] : 0u;
      }
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        if (i < nt && alive) issue(i);
        if constexpr (!kTma) cp_async_commit();
      }
    }
    if (running) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l_r[r] += __shfl_xor_sync(kFull, l_r[r], 1);
      l_r[r] += __shfl_xor_sync(kFull, l_r[r], 2);
    }

    // merge the 4 warps in shared memory
    constexpr int WS = D + 4;
    float* wm = reinterpret_cast<float*>(smem + TL::kRing);
    float* wl = wm + kWarps * 16;
    float* wo = wl + kWarps * 16;
    if (tq == 0) {
      wm[warp * 16 + g] = m_r[0];
      wm[warp * 16 + g + 8] = m_r[1];
      wl[warp * 16 + g] = l_r[0];
      wl[warp * 16 + g + 8] = l_r[1];
    }
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
      const int d = x * 8 + 2 * tq;
      if (g < G) *reinterpret_cast<float2*>(&wo[(warp * G + g) * WS + d]) = make_float2(o[x][0], o[x][1]);
      if (g + 8 < G) *reinterpret_cast<float2*>(&wo[(warp * G + g + 8) * WS + d]) = make_float2(o[x][2], o[x][3]);
    }
    __syncthreads();
    if (threadIdx.x < G) {
      const int row = threadIdx.x;
      float M = -INFINITY, f[kWarps], tot = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * 16 + row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = wm[w * 16 + row];
        f[w] = mw == -INFINITY ? 0.f : ex2_approx(mw - M);
        tot = fmaf(wl[w * 16 + row], f[w], tot);
      }
      const float inv = tot != 0.f ? 1.0f / tot : 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s_sf[w][row] = f[w] * inv;
      s_rl[row] = tot != 0.f ? (M + lg2_approx(tot)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    auto merged = [&](int row, int d) {
      float acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float sf = s_sf[w][row];
        if (sf != 0.f) acc = fmaf(wo[(w * G + row) * WS + d], sf, acc);
      }
      return acc;
    };
    const int64_t row0 = int64_t(d_b) * a.H_q + int64_t(d_h) * G;
    uint16_t* outp = static_cast<uint16_t*>(a.out) + row0 * D;
    if (d_gi == 0 && d_ge == d_groups) {                       // the whole unit
      for (int idx = threadIdx.x; idx < G * D; idx += kThreads) outp[idx] = E::from_f(merged(idx / D, idx % D));
      if (a.lse && threadIdx.x < G) a.lse[row0 + threadIdx.x] = s_rl[threadIdx.x];
    } else {
      const int64_t slot = 2 * int64_t(blockIdx.x) + (d_gi == 0 ? 1 : 0);
      for (int idx = threadIdx.x; idx < G * D; idx += kThreads)
        a.part_o[slot * G * D + idx] = merged(idx / D, idx % D);
      if (threadIdx.x < G) a.part_lse[slot * G + threadIdx.x] = s_rl[threadIdx.x];
      // CTAs that hold parts of the unit: owners of its first to its last group
      const int c_first = int(((int64_t(d_unit_at) + 1) * N - 1) / total);
      const int c_last = int(((int64_t(d_unit_at) + d_groups) * N - 1) / total);
      const int parts = c_last - c_first + 1;
      __syncthreads();
      // of the units that begin in a CTA the last alone is cut
      if (threadIdx.x == 0) s_last = ticket(&a.tickets[c_first]) == parts - 1;
      __syncthreads();
      if (s_last) {
        // A thread merges four columns of a row, kFlight parts in flight, in the order of the parts; where the rows
        // leave threads over, `ways` of them take every ways-th batch of a column and meet in shared memory.
        auto slot_of = [&](int p) { return 2 * int64_t(c_first + p) + (p == 0 ? 1 : 0); };
        const int quads = G * (D / 4), ways = quads >= kThreads ? 1 : kThreads / quads;
        float* meet = wo;                                    // [ways][quads][6]
        for (int i = threadIdx.x; i < quads * ways; i += kThreads) {
          const int quad = i % quads, way = i / quads, idx = 4 * quad, row = idx / D;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float M = -INFINITY, tot = 0.f;
          for (int p0 = way * kFlight; p0 < parts; p0 += ways * kFlight) {
            float4 x[kFlight];
            float z[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
              z[k] = -INFINITY;
              if (p0 + k < parts) {
                const int64_t r = slot_of(p0 + k) * G;
                z[k] = __ldcg(a.part_lse + r + row);
                x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + r * D + idx));
              }
            }
            float m = M;
#pragma unroll
            for (int k = 0; k < kFlight; ++k) m = fmaxf(m, z[k]);
            const float f = M == -INFINITY ? 0.f : ex2_approx((M - m) * kLog2e);
            tot *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
            M = m;
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
              if (z[k] == -INFINITY) continue;             // an empty part
              const float w = ex2_approx((z[k] - M) * kLog2e);
              tot += w;
              acc.x = fmaf(w, x[k].x, acc.x);
              acc.y = fmaf(w, x[k].y, acc.y);
              acc.z = fmaf(w, x[k].z, acc.z);
              acc.w = fmaf(w, x[k].w, acc.w);
            }
          }
          if (ways > 1) {
            float* mine = meet + int64_t(i) * 6;
            mine[0] = M, mine[1] = tot, mine[2] = acc.x, mine[3] = acc.y, mine[4] = acc.z, mine[5] = acc.w;
            continue;
          }
          const float f = tot != 0.f ? 1.0f / tot : 0.f;
          *reinterpret_cast<uint2*>(outp + idx) = make_uint2(E::pack(acc.x * f, acc.y * f), E::pack(acc.z * f, acc.w * f));
          if (a.lse && idx % D == 0) a.lse[row0 + row] = tot != 0.f ? M + lg2_approx(tot) * kLn2 : -INFINITY;
        }
        if (ways > 1) {
          __syncthreads();
          if (int(threadIdx.x) < quads) {
            const int idx = 4 * threadIdx.x, row = idx / D;
            float M = -INFINITY, tot = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q = 0; q < ways; ++q) M = fmaxf(M, meet[(q * quads + threadIdx.x) * 6]);
            for (int q = 0; q < ways; ++q) {
              const float* x = meet + (q * quads + threadIdx.x) * 6;
              const float w = x[0] == -INFINITY ? 0.f : ex2_approx((x[0] - M) * kLog2e);
              tot = fmaf(w, x[1], tot);
              acc.x = fmaf(w, x[2], acc.x);
              acc.y = fmaf(w, x[3], acc.y);
              acc.z = fmaf(w, x[4], acc.z);
              acc.w = fmaf(w, x[5], acc.w);
            }
            const float f = tot != 0.f ? 1.0f / tot : 0.f;
            *reinterpret_cast<uint2*>(outp + idx) = make_uint2(E::pack(acc.x * f, acc.y * f), E::pack(acc.z * f, acc.w * f));
            if (a.lse && idx % D == 0) a.lse[row0 + row] = tot != 0.f ? M + lg2_approx(tot) * kLn2 : -INFINITY;
          }
        }
        if (threadIdx.x == 0) a.tickets[c_first] = 0;
      }
    }
    __syncthreads();                                     // the merge area is free again
    }
    if (!more) break;
    running = true;
#pragma unroll
    for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
    m_r[0] = m_r[1] = -INFINITY;
    l_r[0] = l_r[1] = 0.f;
    for (int i = 0; i < nt && alive; ++i) {
      __syncwarp();
      if (i + kStages - 1 < nt) issue(i + kStages - 1);
      const int st = (cnt + i) % kStages;
      if constexpr (kTma) {
        if (!mbar_wait(smem_u32(&s_bar[warp][st]), ((cnt + i) / kStages) & 1, a.status)) alive = false;
        alive = __all_sync(kFull, alive);
        if (!alive) break;
      } else {
        cp_async_commit();
        cp_async_wait<kStages - 1>();
      }
      __syncwarp();
      const uint32_t sk = smem_u32(wbuf + st * TL::kStageBytes), sv = sk + TL::kBytes;
      const uint32_t vmask = s_mask[warp][st];
      if (vmask == 0) continue;
      if (kTma && vmask != 0xffffu) {
        // rows the query does not see could hold anything (NaN): zero their values
        for (int idx = lane; idx < 16 * TL::kChunks; idx += 32) {
          const int row = idx / TL::kChunks, chunk = idx % TL::kChunks;
          if (!((vmask >> row) & 1u))
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};\n" ::"r"(sv + swz16<D>(row, chunk)), "r"(0u) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      // S = Q K^T, even and odd k-steps in two chains
      float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float c2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int mi = lane >> 3, rr = lane & 7;
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        const int tok = (mi >> 1) * 8 + rr;
        uint32_t r[4], r2[4];
        ldmatrix_x4(r, sk + swz16<D>(tok, kk * 2 + (mi & 1)));
        ldmatrix_x4(r2, sk + swz16<D>(tok, (kk + 1) * 2 + (mi & 1)));
        E::mma(c[0], qa[kk], r[0], r[1]);
        E::mma(c[1], qa[kk], r[2], r[3]);
        E::mma(c2[0], qa[kk + 1], r2[0], r2[1]);
        E::mma(c2[1], qa[kk + 1], r2[2], r2[3]);
      }
      float pmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n2 = 0; n2 < 2; ++n2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool ok = (vmask >> (n2 * 8 + 2 * tq + e)) & 1u;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float& z = c[n2][2 * r + e];
            z = ok ? (z + c2[n2][2 * r + e]) * a.scale_log2 : -INFINITY;
            pmax[r] = fmaxf(pmax[r], z);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        pmax[r] = fmaxf(pmax[r], __shfl_xor_sync(kFull, pmax[r], 1));
        pmax[r] = fmaxf(pmax[r], __shfl_xor_sync(kFull, pmax[r], 2));
        const float m_new = fmaxf(m_r[r], pmax[r]);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(m_r[r] - m_use);
        float rs = 0.f;
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = ex2_approx(c[n2][2 * r + e] - m_use);
            c[n2][2 * r + e] = p;
            rs += p;
          }
        }
        l_r[r] = l_r[r] * alpha + rs;
        m_r[r] = m_new;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          o[x][2 * r] *= alpha;
          o[x][2 * r + 1] *= alpha;
        }
      }
      // O += P V
      const uint32_t pa[4] = {E::pack(c[0][0], c[0][1]), E::pack(c[0][2], c[0][3]), E::pack(c[1][0], c[1][1]),
                              E::pack(c[1][2], c[1][3])};
#pragma unroll
      for (int nd = 0; nd < D / 16; ++nd) {
        uint32_t r[4];
        ldmatrix_x4_trans(r, sv + swz16<D>((mi & 1) * 8 + rr, 2 * nd + (mi >> 1)));
        E::mma(o[2 * nd], pa, r[0], r[1]);
        E::mma(o[2 * nd + 1], pa, r[2], r[3]);
      }
    }
    if (kTma && !alive) {
      // leave no copy in flight (each wait is bounded)
      for (int i = 0; i < nt && lane == 0; ++i)
        if (!mbar_wait(smem_u32(&s_bar[warp][(cnt + i) % kStages]), ((cnt + i) / kStages) & 1, a.status)) break;
    }
    cnt += nt;
  }
  if constexpr (!kTma) cp_async_wait<0>();
}

struct WsLayout {
  size_t part_lse, part_o, total;
};
WsLayout ws_layout(int G, int D, int ctas) {
  static_assert(kCtasPerSm <= kTicketsPerSm, "a counter for each CTA");
  WsLayout w;
  w.part_lse = ticket_bytes();
  w.part_o = w.part_lse + align256(size_t(ctas) * 2 * G * 4);
  w.total = w.part_o + size_t(ctas) * 2 * G * D * 4;
  return w;
}

int g_smem[8][64];

template <typename T, int D, bool kTma>
sa_status launch(const PagedDecodeArgs& a, int ctas, cudaStream_t s, const CUtensorMap& mk, const CUtensorMap& mv,
                 int* cache) {
  auto k = paged_decode_kernel<T, D, kTma>;
  if (!ensure_smem(k, Tile<D>::kSmem, cache)) return SA_ERR_CUDA;
  return launch_ex(k, dim3(ctas), dim3(kThreads), Tile<D>::kSmem, s, false, 1, a, mk, mv) == cudaSuccess ? SA_OK
                                                                                                       : SA_ERR_CUDA;
}

template <typename T, int D>
sa_status dispatch(const PagedDecodeArgs& a, int ctas, cudaStream_t s, const sa_cache* c, int slot) {
  CUtensorMap mk = {}, mv = {};
  if (c->page_size >= 16 && make_row_map(&mk, c->k, c) && make_row_map(&mv, c->v, c))
    return launch<T, D, true>(a, ctas, s, mk, mv, g_smem[2 * slot + 1]);
  return launch<T, D, false>(a, ctas, s, mk, mv, g_smem[2 * slot]);
}

}  // namespace
}  // namespace sa

extern "C" size_t sa_paged_decode_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads,
                                                 int32_t head_dim) {
  using namespace sa;
  if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || head_dim <= 0 || num_q_heads % num_kv_heads) return 0;
  return ws_layout(num_q_heads / num_kv_heads, head_dim, kCtasPerSm * sm_count()).total;
}

extern "C" sa_status sa_paged_decode(const sa_cache* cache, const sa_batch* batch, const void* q, int32_t num_q_heads,
                                     int32_t window, int32_t n_sink, float scale, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  using namespace sa;
  sa_status st = check_cache(cache, true, false);
  if (st != SA_OK) return st;
  if ((st = check_batch(batch)) != SA_OK) return st;
  if (!q || !out || num_q_heads <= 0 || num_q_heads % cache->num_kv_heads) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || window < 0 || n_sink < 0) return SA_ERR_INVALID_ARG;
  const int G = num_q_heads / cache->num_kv_heads, D = cache->head_dim, H = cache->num_kv_heads;
  if (G > 16 || batch->batch > kMaxBatch || H > 65535) return SA_ERR_UNSUPPORTED;
  // groups of 64 tokens that the batch can have
  const int64_t seen = window > 0 ? int64_t(window) + n_sink + 128 : int64_t(1) << 40;
  const int64_t cap = int64_t(batch->bt_stride) * cache->page_size;
  const int64_t most = int64_t(batch->batch) * H * (((cap < seen ? cap : seen) + 63) / 64);
  if (cap > 0x7fffffff || most > 0x3fffffff) return SA_ERR_UNSUPPORTED;
  const int sms = kCtasPerSm * sm_count();
  const int ctas = most < sms ? int(most) : sms;
  const WsLayout w = ws_layout(G, D, sms);
  if (!workspace || workspace_bytes < w.total || !aligned16(workspace)) return SA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PagedDecodeArgs a = {};
  a.k = cache->k; a.v = cache->v; a.q = q; a.bt = batch->block_table; a.seq_lens = batch->seq_lens;
  a.out = out; a.lse = lse; a.status = dev_status;
  a.tickets = reinterpret_cast<int32_t*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.H_kv = H; a.H_q = num_q_heads; a.G = G; a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks;
  a.bt_stride = batch->bt_stride; a.batch = batch->batch; a.n_sink = n_sink;
  a.window = window < cap ? window : 0;                      // a window of the table's length hides nothing
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf(float(D))) * kLog2e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SA_BF16;
  if (D == 128)
    return bf ? dispatch<__nv_bfloat16, 128>(a, ctas, s, cache, 0) : dispatch<__half, 128>(a, ctas, s, cache, 1);
  return bf ? dispatch<__nv_bfloat16, 64>(a, ctas, s, cache, 2) : dispatch<__half, 64>(a, ctas, s, cache, 3);
}
