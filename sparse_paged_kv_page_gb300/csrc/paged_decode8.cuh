// sa_paged_decode8, sa_sparse_decode8 and sa_paged_prefill8 of few tokens: softmax
// attention of one new token per request over a paged cache held in 8 bits, all of it, a
// sliding window and its first tokens, or the pages selected for each KV head; or of a
// few tokens each, causal, over all of it or a window.
//
// Mathematics: a row's codes c and scale 2^s stand for c 2^s. With z_j = scale q . c_j
// 2^(ks_j) (base 2 from here) and y_j = z_j + vs_j, in one pass with the running
// maximum m of y: l = sum_j 2^(z_j - m), o = sum_j 2^(y_j - m) cv_j, out = o / l. The
// value scales thus sit in the weights, of which the largest is 1 whatever the scales
// are, and the products see codes alone, which fp16 holds exactly. The query goes to
// fp16 too, each head times the power of two that brings its largest value to [2^14,
// 2^15): off by 2^-39 of that at most where bf16 has more range. Weights are rounded to
// fp16 (2^-11 of the weight, 2^-25 near 0). Parts over disjoint ranges merge as in
// sa_paged_decode: lse = m + log2 l. With one token, whose rows are few, the last CTA of a
// unit merges its parts; those of a few tokens are merged by a kernel behind.
//
// Bound by HBM, at half the bytes of 16 bits, so instructions per byte count twice. Each of
// a CTA's warps takes tiles of 32 tokens through a private ring filled by 16-byte cp.async,
// whatever the page size (a page of 16 tokens is 2 KB here, and a copy of the TMA engine
// costs about 100 cycles whatever its size). Both products are transposed, S^T = C Q^T and
// O^T += C^T P^T by m16n8k16, so that the query heads are padded to 8 and not to 16: half
// the products and registers. Codes become fp16 two at a time on the way
// (cvt.rn.f16x2.e4m3x2). A lane copies just the chunks of keys that it will read back: the
// order of the columns within a product is free as long as both operands share it, so lane
// (g, t) of a product holds 16 adjacent codes of token g and no swizzle or ldmatrix is
// needed. Values go through ldmatrix.trans as pairs of codes of two tokens, put in order by
// one byte permutation; the weights change places by movmatrix.
//
// A few tokens (kDraft) are rows (token, query head) in groups of 8 like the heads of one;
// tiles that some row of a unit does not see whole are masked by each row's own position.
//
// Work split as in sa_paged_decode: the tiles of all units are one line that the CTAs, each
// with a tile a warp or a unit at least, cut into equal parts.
//
// Measured in replayed graphs (us; bytes a second of the codes and scales): 4 requests of
// 128 k tokens, 64 / 8 heads of 128, 175 (6.2 TB/s, 92% of a copy; in 16 bits
// 311), 128 / 8 heads 190, heads of 64 97; 16 of 2 - 32 k, 32 / 8 heads, 100 - 102 (177): about
// 12 us of start, merge and tail beside 6.5 TB/s. One of 1024 tokens 6.2 (7.1): launch, then
// lengths -> ids -> codes -> parts, each a round trip. 256 selected pages of 16 of each of 32
// units, 17.3 (34 MB): 4 us until the first codes are asked for, 6 of codes, 2 of merge, 5 that no
// measurement names. 3 - 8 tokens of 4 requests behind 8 - 30 k 64: latency, the eight warps an SM that
// 255 registers leave have issue slots 38% busy, tensor cores 30%, HBM 36% (1 - 4 tokens 50).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "kv8.cuh"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kRows = 32;                  // tokens of a tile
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxBatch = 1024;
constexpr int kMaxUnits = 16384;           // (request, KV head) pairs of a call over selected pages
constexpr int kFlight = 8;                 // parts a merging thread has in flight
constexpr int kStages = 2;                 // tiles of a warp: one at work, one under way
// Of a tile of a unit of g groups of rows: kTileShare + g kGroupShare, as measured (6 / 8 tokens of 128
// requests behind 1000 - 32000, 32 / 8 heads, 3 / 4 groups: 985 / 1156 us). Tiles alike to the line / by shares, 3 - 8 tokens of 16
// such requests 169 / 150, 32 336 / 285.
constexpr int kTileShare = 7, kGroupShare = 3;
constexpr int kDense = 0, kList = 1, kDraft = 2;

struct Decode8Args {
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* scale;
  const void* q;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* sel;     // kList: [units][sel_stride] pages
  const int32_t* cnt;     // kList: [units]
  const int32_t* new_cu;  // kDraft: [batch + 1] rows of q
  void* out;
  float* lse;
  float* part_o;          // [CTAs][2][R][D]
  float* part_lse;        // [CTAs][2][R]
  int32_t* tickets;       // [CTAs]: of the cut unit that begins in a CTA
  int4* cut;              // kDraft, [CTAs]: of that unit, the first row of q, rows, KV head and parts (0: there is none)
  int32_t* status;
  int R;                  // rows of a unit at most: G, or (kDraft) those of `per` tokens
  int per, T, ctas;       // kDraft: tokens of a unit at most; rows of q; CTAs of the kernel before the merge
  int H_kv, H_q, G, ps_shift, num_blocks, bt_stride, batch, window, n_sink, sel_stride;
  float scale_log2;
};

// kN: groups of 8 rows, 1, 2 or (kDraft) 4.
template <int D, int kN>
struct Tile8 {
  // An SM, at 168 or 255 (head dim 128), 128 or 255 registers a thread. Two groups spill 12 to 40 words at that and still gain
  // (us, 16 query heads a KV head of 128, 4 x 128k tokens, two CTAs / three 200 / 189); four would have to spill their sums.
  static constexpr int kCtas = kN == 4 ? 2 : D == 128 ? 3 : 4;
  static constexpr int kBytes = kRows * D;
  static constexpr int kStageBytes = 2 * kBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMerge = 4 * (2 * kWarps * 8 * kN + kWarps * 8 * kN * (D + 4));   // in place of the ring, between parts
  static constexpr int kQAt = kMerge > kRing ? kMerge : kRing;
  static constexpr bool kQShared = kN >= 2;   // Q's operands in shared memory, a group of rows made by each of the first kN warps
  static constexpr int kSmem = kQAt + (kQShared ? D / 16 * kN * 32 * 8 + 8 * kN * 4 : 0);
  static constexpr int kHalves = D / 64;   // 64 columns of keys are one 16-byte chunk a lane
};

// 16-byte chunk of row r of a tile of values: the rows that ldmatrix reads together lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t value_at(int r, int chunk) {
  return uint32_t(r * D + ((D == 128 ? chunk ^ (r & 7) : chunk ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}

template <typename T, int D, int kN, int kMode>
__global__ void __launch_bounds__(kThreads, Tile8<D, kN>::kCtas) decode8_kernel(const __grid_constant__ Decode8Args a) {
  using E = Elem<T>;
  using F = Elem<__half>;
  using TL = Tile8<D, kN>;
  constexpr int kHalves = TL::kHalves, kR = 8 * kN;
  constexpr bool kSel = kMode == kList;
  static_assert(kN == 1 || kN == 2 || (kN == 4 && kMode == kDraft), "groups of rows");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float4 s_tok[kWarps][kRows];       // of a tile's tokens: key factor, 0 or -inf, exponent and factor of the values
  __shared__ int s_last;
  __shared__ float s_sf[kWarps][kR], s_rl[kR];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int G = a.G, pss = a.ps_shift, ps = 1 << pss;
  const int cap = int(min(int64_t(a.bt_stride) << pss, int64_t(0x7fffffff)));
  // The line of work is of owners: requests, whose units (KV heads, and with kDraft runs of tokens) have the same tiles, or
  // (kList) single units. Of owner u0 + lane: units, tiles of each (an empty one has one too: its outputs are written), length,
  // listed pages or new tokens, first row of q. Every warp finds its places by itself, 32 owners at a time.
  const int owners = kSel ? a.batch * a.H_kv : a.batch;
  struct Owner {
    int units, tiles, len, count, c0;
  };
  auto owner = [&](int u0) {
    Owner x = {0, 0, 0, 0, 0};
    const int u = u0 + lane;
    if (u >= owners) return x;
    const bool report = blockIdx.x == 0 && threadIdx.x < 32;
    x.len = a.seq_lens[kSel ? u / a.H_kv : u];
    if (kSel) {
      const int c = a.cnt[u];
      if (report && (c < 0 || c > a.sel_stride)) flag(a.status, SA_DEV_BAD_COUNT);
      x.count = min(max(c, 0), a.sel_stride);
      x.tiles = ((x.count << pss) + kRows - 1) / kRows;
      x.units = 1;
    } else if (kMode == kDense) {
      if (report && x.len < 0) flag(a.status, SA_DEV_BAD_COUNT);
      if (report && x.len > cap) flag(a.status, SA_DEV_OVERFLOW);
      x.len = max(0, x.len);
      x.tiles = Span<kRows>(x.len - 1, x.len - 1, min(x.len, cap), a.window, a.n_sink).tiles;
      x.units = a.H_kv;
    } else {
      x.c0 = a.new_cu[u], x.count = a.new_cu[u + 1] - x.c0;
      const bool rows = x.c0 >= 0 && int64_t(x.c0) + x.count <= a.T;
      if (report && (!rows || x.len < x.count)) flag(a.status, SA_DEV_BAD_COUNT);
      if (report && x.len > cap) flag(a.status, SA_DEV_OVERFLOW);
      x.count = rows ? max(0, x.count) : 0;
      x.len = max(0, x.len);
      // as many as any run of its tokens has: the last has the most, but for where a window's ends lie in their tiles
      x.tiles = Span<kRows>(x.len - min(x.count, a.per), x.len - 1, min(max(x.len, 0), cap), a.window, a.n_sink).tiles +
                (a.window > 0 ? 2 : 0);
      x.units = (x.count + a.per - 1) / a.per * a.H_kv;
    }
    x.tiles = max(1, x.tiles);
    return x;
  };
  pdl_wait();
  // A tile's share of the line: what one of units of 2, 3 or 4 groups of rows takes.
  constexpr bool kWeigh = kMode == kDraft && kN == 4;
  auto groups_of = [&](int rows) { return rows <= 16 ? 2 : rows <= 24 ? 3 : 4; };
  auto share = [&](int count) { return kWeigh ? kTileShare + kGroupShare * groups_of(min(count, a.per) * G) : 1; };
  auto line = [&](const Owner& x) { return x.units * x.tiles * share(x.count); };
  // Lengths on the line of all owners, 32 a batch; a lane keeps those of `run` batches, where a CTA looks for its first owner.
  const int batches = (owners + 31) >> 5, run = (batches + 31) >> 5;
  int of_run = 0, units = 0, rows = 0;
  Owner ow;                                      // of owners ow0 .. ow0 + 31, which the CTA is at
#pragma unroll 4
  for (int i = batches - 1; i >= 0; --i) {
    ow = owner(32 * i);
    const int t = __reduce_add_sync(kFull, line(ow));
    if (unsigned(i - lane * run) < unsigned(run)) of_run += t;
    units += ow.units, rows += ow.count;
  }
  if (kMode == kDraft) {
    units = __reduce_add_sync(kFull, units), rows = __reduce_add_sync(kFull, rows);
    if (rows > a.T) {                            // not a list of offsets within the rows
      if (blockIdx.x == 0 && threadIdx.x == 0) flag(a.status, SA_DEV_BAD_COUNT);
      if (threadIdx.x == 0) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
  } else {
    units = a.batch * a.H_kv;
  }
  constexpr unsigned kPerCta = kWarps * (kWeigh ? kTileShare + 4 * kGroupShare : 1);
  const unsigned total = __reduce_add_sync(kFull, of_run), N0 = min(gridDim.x, max(unsigned(units), (total + kPerCta - 1) / kPerCta));
  // A few CTAs less where those of units alike have one part each then: 4 x 128k tokens, 64 / 8 heads, 456 / 448 CTAs 180.5 / 175
  // us, 64 / 4 heads 112 / 107 (in pages of one token, bound by the places to read from, 387 / 398).
  const unsigned over = N0 % unsigned(max(units, 1)), N = 50 * over <= N0 ? N0 - over : N0;
  if (blockIdx.x >= N) {
    if (kMode == kDraft && threadIdx.x == 0) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  // Neighbours on the line, whose units have the same rows, on one SM, so that its CTAs run the same instructions (128 requests as
  // above 1160 -> 1049 us). (Which SM a CTA is on is a guess that only the time depends on.)
  const unsigned sms = gridDim.x / TL::kCtas, cta = kWeigh && N == sms * TL::kCtas ? blockIdx.x % sms * TL::kCtas + blockIdx.x / sms : blockIdx.x;
  // CTA c has shares c q + min(c, r) and on: q or, the first r, q + 1 of them
  const unsigned q_ = total / N, r_ = total - q_ * N;
  auto cta_of = [&](unsigned t) { return int(t < r_ * (q_ + 1) ? t / (q_ + 1) : r_ + (t - r_ * (q_ + 1)) / q_); };
  int at = int(cta * q_ + min(cta, r_));
  const int stop = at + int(q_) + (cta < r_ ? 1 : 0);
  auto sum_to = [&](int x) {                     // of lanes 0 .. lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  int ow0 = 0, ow_before = 0, ow_sum;            // shares of the owners before; of owners ow0 .. ow0 + lane
  if (batches > 1) {
    const int to = sum_to(of_run), k = __popc(__ballot_sync(kFull, to <= at));
    ow0 = 32 * run * k, ow_before = __shfl_sync(kFull, to - of_run, k);
    if (ow0 > 0) ow = owner(ow0);
  }
  if (kN == 1) ow_sum = sum_to(line(ow));

  const uint8_t* k_lane = a.k + tq * 16;
  const uint8_t* v_lane = a.v + tq * 16;
  const uint32_t wbuf = smem_u32(smem) + warp * kStages * TL::kStageBytes;
  int cnt = 0;                                  // tiles this warp has consumed in all

  // The part of a unit at work: request b, KV head h, its first row of q and its rows R, tiles [ti, te) of its `tiles` (the
  // shares begin at unit_at and are unit_len), the lengths and the visible range, positions of its first and last token, this warp's nt tiles
  // from ti + warp on, every kWarps-th.
  int b = 0, h = 0, row0 = 0, R = 0, ti = 0, te = 0, tiles = 1, unit_at = 0, unit_len = 1, Lc = 0, w0 = 0, nt = 0, listed = 0, first = 0, last = 0;
  Span<kRows> sp(-1, -1, 0, 0, 0);
  const int32_t* btb = a.bt;
  const int32_t* sel = a.sel;
  uint32_t qb[TL::kQShared ? 1 : D / 16][kN][2];   // Q as the B operand (columns: 8 rows each, zero beyond R)
  uint2* s_q = reinterpret_cast<uint2*>(smem + TL::kQAt);                      // kQShared: [D / 16][kN][32 lanes]
  float* s_down = reinterpret_cast<float*>(s_q + D / 16 * kN * 32);            // [8 kN]
  float z_scale[TL::kQShared ? 1 : kN][2];      // of rows 8 n + 2 tq + e: q . c to base-2 logits, but for the key's scale
  // of rows 8 n + 2 tq + e: O of columns 16 x + 2 g + {0, 1} in o[x][n][{0, 2} + e]; maximum; sum over this lane's tokens
  float o[D / 16][kN][4], m_r[kN][2], l_r[kN][2];
  // Block ids are loaded a batch of tiles ahead, one id a lane: a tile has one page, or 32 / page_size of them.
  const int ids_shift = max(0, 5 - pss);                 // log2 of the ids of a tile
  const int per_batch = 32 >> ids_shift;
  int ids = -1, ids_next = -1, fill = 0, fill_next = 0;  // fill (kSel): valid tokens of the page
  uint32_t next_mask = 0, next_scales = 0;               // of the tile under way: rows that are seen, this lane's token's scales
  bool running = false;

  int4 cut = make_int4(0, 0, 0, 0);

  while (true) {
    // what the merge of the part just done needs; then the next part begins, so that its first tiles are under way
    // during the merge
    const int d_row0 = row0, d_R = R, d_h = h, d_ti = ti, d_te = te, d_tiles = tiles, d_unit_at = unit_at, d_unit_end = unit_at + unit_len;
    const bool more = at < stop;
    // first token of tile i of this warp: of the sequence, or (kSel) of the listed pages in a line
    auto tile_start = [&](int i) {
      const int t = ti + warp + i * kWarps;
      return kSel ? t * kRows : sp.start(t);
    };
    auto load_ids = [&](int i, int& id, int& full) {
      const int x = i + (lane >> ids_shift);
      id = -1, full = 0;
      if (x >= nt) return;
      const int j = tile_start(x) + ((lane & ((1 << ids_shift) - 1)) << pss);
      int page = j >> pss;
      if (kSel) {
        if (page >= listed) return;
        page = sel[page];
        if (page < 0 || page >= a.bt_stride || page > (Lc - 1) >> pss) {
          flag(a.status, SA_DEV_BAD_BLOCK);
          return;
        }
        full = min(ps, Lc - (page << pss));
      } else if (j >= Lc) {
        return;
      }
      id = btb[page];
      if (id < 0 || id >= a.num_blocks) {
        flag(a.status, SA_DEV_BAD_BLOCK);
        id = -1;
      }
    };
    auto issue = [&](int i) {
      if ((i & (per_batch - 1)) == 0) {
        ids = ids_next, fill = fill_next;
        load_ids(i + per_batch, ids_next, fill_next);
      }
      const int j0 = tile_start(i), j = j0 + lane, slot = j & (ps - 1);
      const int src = (((i & (per_batch - 1)) << ids_shift) + (pss >= 5 ? 0 : lane >> pss)) & 31;
      const int blk = __shfl_sync(kFull, ids, src);
      const int full = kSel ? __shfl_sync(kFull, fill, src) : 0;
      const bool seen = blk >= 0 && (kSel ? slot < full : j < Lc && (j >= w0 || j < a.n_sink));
      // lane l knows the pool row of token l (0 where nothing is read), and its scales
      const uint32_t tile = seen ? uint32_t(blk) * a.H_kv + h : 0u, row = seen ? (tile << pss) + slot : 0u;
      next_mask = __ballot_sync(kFull, seen);
      next_scales = 0;
      if (seen) {
        const uint8_t* sc = a.scale + (uint64_t(tile) << (pss + 1)) + slot;
        next_scales = uint32_t(sc[0]) | uint32_t(sc[ps]) << 8;
      }
      const uint32_t sk = wbuf + ((cnt + i) % kStages) * TL::kStageBytes, sv = sk + TL::kBytes;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int r = 8 * n + g;
        const uint64_t off = uint64_t(__shfl_sync(kFull, row, r)) * D;
        const uint8_t* kr = k_lane + off;
        const uint8_t* vr = v_lane + off;
        const int bytes = (next_mask >> r) & 1u ? 16 : 0;
#pragma unroll
        for (int c = 0; c < kHalves; ++c) {
          cp_async_16(sk + ((n * kHalves + c) * 32 + lane) * 16, kr + 64 * c, bytes);
          cp_async_16(sv + value_at<D>(r, tq + 4 * c), vr + 64 * c, bytes);
        }
      }
    };

    // Q: lane (g, tq) takes columns 64 c + 16 tq + 4 w .. + 3 of row g of each group as k-step 4 c + w
    auto query = [&](int row, int kk) {
      if (row >= R) return make_uint2(0u, 0u);
      const int t = kMode == kDraft ? row / G : 0;
      const int64_t at = (int64_t(row0 + t) * a.H_q + int64_t(h) * G + (row - t * G)) * D + 16 * tq + (kk >> 2) * 64 + (kk & 3) * 4;
      return *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
    };
    if (more) {
      // the owner and unit of tile `at`
      if (kN > 1) ow = owner(ow0), ow_sum = sum_to(line(ow));   // (has no registers to keep them in)
      int k;
      while ((k = __popc(__ballot_sync(kFull, ow_before + ow_sum <= at))) == 32) {
        ow_before += __shfl_sync(kFull, ow_sum, 31);
        ow0 += 32;
        ow = owner(ow0);
        ow_sum = sum_to(line(ow));
      }
      const int u = ow0 + k, before = ow_before + __shfl_sync(kFull, ow_sum - line(ow), k);
      const int L = __shfl_sync(kFull, ow.len, k), count = __shfl_sync(kFull, ow.count, k), c0 = __shfl_sync(kFull, ow.c0, k);
      const int mine = __shfl_sync(kFull, ow.units, k);
      tiles = __shfl_sync(kFull, ow.tiles, k);
      const int w = share(count);
      unit_len = tiles * w;
      const int in = kSel ? 0 : (at - before) / unit_len;
      unit_at = before + in * unit_len;
      b = kSel ? u / a.H_kv : u, h = kSel ? u - b * a.H_kv : in;
      row0 = b, R = G;
      // the tiles that begin in the CTA's shares (there may be none)
      ti = (at - unit_at + w - 1) / w, te = min(tiles, (stop - unit_at + w - 1) / w);
      at = min(stop, unit_at + unit_len);
      Lc = min(max(L, 0), cap);
      int full;                                            // 0 of an empty unit
      if (kSel) {
        listed = count;
        sel = a.sel + int64_t(u) * a.sel_stride;
        full = ((listed << pss) + kRows - 1) / kRows;
      } else {
        first = last = L - 1;
        if (kMode == kDraft) {
          const int runs = mine / a.H_kv, t0 = (in % runs) * a.per, n = min(a.per, count - t0);
          h = in / runs, row0 = c0 + t0, R = n * G;
          first = L - count + t0, last = first + n - 1;
        }
        sp = Span<kRows>(first, last, Lc, a.window, a.n_sink);
        w0 = a.window > 0 ? max(0, first - a.window + 1) : 0;
        Lc = min(Lc, last + 1);
        full = sp.tiles;
      }
      const int t_end = min(te, full);
      nt = ti + warp < t_end ? (t_end - ti - warp + kWarps - 1) / kWarps : 0;
      btb = a.bt + int64_t(b) * a.bt_stride;
      if constexpr (!TL::kQShared) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const uint2 x = query(g + 8 * n, kk);
            qb[kk][n][0] = x.x, qb[kk][n][1] = x.y;
          }
        }
      }
      load_ids(0, ids_next, fill_next);
    }
    if (running) {
      // merge the warps in shared memory, in place of the ring
      constexpr int WS = D + 4;
      float* wm = reinterpret_cast<float*>(smem);
      float* wl = wm + kWarps * kR;
      float* wo = wl + kWarps * kR;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l_r[n][e] += __shfl_xor_sync(kFull, l_r[n][e], x);
        }
      }
      __syncthreads();                                     // every warp's tiles are used up
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * tq + e;
          if (row >= d_R) continue;
          if (g == 0) wm[warp * kR + row] = m_r[n][e], wl[warp * kR + row] = l_r[n][e];
          float* to = &wo[(warp * d_R + row) * WS + 2 * g];
#pragma unroll
          for (int x = 0; x < D / 16; ++x) *reinterpret_cast<float2*>(to + 16 * x) = make_float2(o[x][n][e], o[x][n][2 + e]);
        }
      }
      __syncthreads();
      if (int(threadIdx.x) < d_R) {
        const int row = threadIdx.x;
        float M = -INFINITY, f[kWarps], tot = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * kR + row]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = wm[w * kR + row];
          f[w] = mw == -INFINITY ? 0.f : ex2_approx(mw - M);
          tot = fmaf(wl[w * kR + row], f[w], tot);
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
          if (sf != 0.f) acc = fmaf(wo[(w * d_R + row) * WS + d], sf, acc);
        }
        return acc;
      };
      // row of out
      auto out_row = [&](int row) {
        const int t = kMode == kDraft ? row / G : 0;
        return int64_t(d_row0 + t) * a.H_q + int64_t(d_h) * G + (row - t * G);
      };
      uint16_t* outp = static_cast<uint16_t*>(a.out);
      if (d_ti == 0 && d_te == d_tiles) {                       // the whole unit
        for (int idx = threadIdx.x; idx < d_R * D; idx += kThreads)
          outp[out_row(idx / D) * D + idx % D] = E::from_f(merged(idx / D, idx % D));
        if (a.lse && int(threadIdx.x) < d_R) a.lse[out_row(threadIdx.x)] = s_rl[threadIdx.x];
      } else {
        const int64_t slot = 2 * int64_t(cta) + (d_ti == 0 ? 1 : 0);
        for (int idx = threadIdx.x; idx < d_R * D; idx += kThreads)
          a.part_o[slot * a.R * D + idx] = merged(idx / D, idx % D);
        if (int(threadIdx.x) < d_R) a.part_lse[slot * a.R + threadIdx.x] = s_rl[threadIdx.x];
        // CTAs that hold parts of the unit: owners of its first to its last tile
        const int c_first = cta_of(unsigned(d_unit_at)), c_last = cta_of(unsigned(d_unit_end - 1));
        const int parts = c_last - c_first + 1;
        if constexpr (kMode == kDraft) {
          if (d_ti == 0) cut = make_int4(d_row0, d_R, d_h, parts);
        } else {
        __syncthreads();
        // of the units that begin in a CTA the last alone is cut
        if (threadIdx.x == 0) s_last = ticket(&a.tickets[c_first]) == parts - 1;
        __syncthreads();
        if (s_last) {
          // A thread merges four columns of a row, kFlight parts in flight, in the order of the parts; where the rows
          // leave threads over, `ways` of them take every ways-th batch of a column and meet in shared memory.
          auto slot_of = [&](int p) { return 2 * int64_t(c_first + p) + (p == 0 ? 1 : 0); };
          const int quads = d_R * (D / 4), ways = quads >= kThreads ? 1 : kThreads / quads;
          float* meet = wo;                                    // [ways][quads][6]
          auto store = [&](int idx, float4 acc, float M, float tot) {
            const float f = tot != 0.f ? 1.0f / tot : 0.f;
            const int64_t row = out_row(idx / D);
            *reinterpret_cast<uint2*>(outp + row * D + idx % D) = make_uint2(E::pack(acc.x * f, acc.y * f), E::pack(acc.z * f, acc.w * f));
            if (a.lse && idx % D == 0) a.lse[row] = tot != 0.f ? M + lg2_approx(tot) * kLn2 : -INFINITY;
          };
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
                  const int64_t r = slot_of(p0 + k) * a.R;
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
            } else {
              store(idx, acc, M, tot);
            }
          }
          if (ways > 1) {
            __syncthreads();
            if (int(threadIdx.x) < quads) {
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
              store(4 * threadIdx.x, acc, M, tot);
            }
          }
          if (threadIdx.x == 0) a.tickets[c_first] = 0;
        }
        }
      }
      __syncthreads();                                     // the ring is free again
    }
    if (!more) break;
    running = true;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      m_r[n][0] = m_r[n][1] = -INFINITY;
      l_r[n][0] = l_r[n][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o[x][n][0] = o[x][n][1] = o[x][n][2] = o[x][n][3] = 0.f;
    }
    if (nt > 0) issue(0);
    cp_async_commit();
    // Q to fp16 while the first tile is under way: each row by the power of two that its largest finite value says
    auto finite = [](float x) {                              // bits of the magnitude
      const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
      return u < 0x7f800000u ? u : 0u;
    };
    auto largest = [&](uint32_t big, uint2 x) {
      return max(max(big, max(finite(E::lo(x.x)), finite(E::hi(x.x)))), max(finite(E::lo(x.y)), finite(E::hi(x.y))));
    };
    auto factors = [&](uint32_t big, float& up, float& down) {
      big = max(big, __shfl_xor_sync(kFull, big, 1));
      big = max(big, __shfl_xor_sync(kFull, big, 2));
      const int e = max(int(big >> 23), 15);
      up = __uint_as_float(uint32_t(268 - e) << 23);                      // 2^14 / 2^(e - 127)
      down = a.scale_log2 * __uint_as_float(uint32_t(e - 14) << 23);
    };
    auto scaled = [&](uint2 x, float up) {
      return make_uint2(F::pack(E::lo(x.x) * up, E::hi(x.x) * up), F::pack(E::lo(x.y) * up, E::hi(x.y) * up));
    };
    if constexpr (TL::kQShared) {                            // (the merge's last barrier, or none before: nobody reads these now)
      if (warp < kN) {
        uint2 x[D / 16];
        uint32_t big = 0;
        float up, down;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) x[kk] = query(8 * warp + g, kk), big = largest(big, x[kk]);
        factors(big, up, down);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) s_q[(kk * kN + warp) * 32 + lane] = scaled(x[kk], up);
        if (tq == 0) s_down[8 * warp + g] = down;
      }
      __syncthreads();
    }
    if constexpr (!TL::kQShared) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        uint32_t big = 0;
        float up, down;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) big = largest(big, make_uint2(qb[kk][n][0], qb[kk][n][1]));
        factors(big, up, down);
        z_scale[n][0] = __shfl_sync(kFull, down, 8 * tq);
        z_scale[n][1] = __shfl_sync(kFull, down, 8 * tq + 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint2 x = scaled(make_uint2(qb[kk][n][0], qb[kk][n][1]), up);
          qb[kk][n][0] = x.x, qb[kk][n][1] = x.y;
        }
      }
    }
    // tiles of units of kG groups of rows
    auto work = [&](auto groups) {
      constexpr int kG = decltype(groups)::value;
      for (int i = 0; i < nt; ++i) {
        const uint32_t mask = next_mask, scales = next_scales;
        __syncwarp();                                        // the tile before is used up
        if (i + 1 < nt) issue(i + 1);
        cp_async_commit();
        // the tokens' factors, for all lanes
        {
          const uint32_t ks = scales & 0xffu, vs = scales >> 8;
          const bool seen = (mask >> lane) & 1u;
          const float nan = __uint_as_float(0x7fc00000u);
          s_tok[warp][lane] = make_float4(seen ? (ks == kScaleNan ? nan : __uint_as_float(ks << 23)) : 0.f,
                                          seen ? 0.f : -INFINITY, seen && vs != kScaleNan ? float(int(vs) - 127) : 0.f,
                                          vs == kScaleNan ? nan : __uint_as_float(vs << 23));
        }
        cp_async_wait<1>();
        __syncwarp();
        if (mask == 0) continue;
        const uint32_t sk = wbuf + ((cnt + i) % kStages) * TL::kStageBytes, sv = sk + TL::kBytes;
        // S^T = C Q^T of 16 tokens twice: this lane's are tokens 8 t + g, t = 2 y and 2 y + 1 in c[y][n][{0, 2} + e]
        float c[2][kG][4];
#pragma unroll
        for (int n = 0; n < kG; ++n) {
#pragma unroll
          for (int x = 0; x < 4; ++x) c[0][n][x] = c[1][n][x] = 0.f;
        }
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
          uint4 w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = lds128(sk + ((t * kHalves + hf) * 32 + lane) * 16);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint4 u = w[2 * y], v = w[2 * y + 1];
              const uint32_t p = x == 0 ? u.x : x == 1 ? u.y : x == 2 ? u.z : u.w, q = x == 0 ? v.x : x == 1 ? v.y : x == 2 ? v.z : v.w;
              const uint32_t ka[4] = {codes_f16(p, false), codes_f16(q, false), codes_f16(p, true), codes_f16(q, true)};
#pragma unroll
              for (int n = 0; n < kG; ++n) {
                if constexpr (TL::kQShared) {
                  const uint2 b = s_q[((4 * hf + x) * kN + n) * 32 + lane];
                  F::mma(c[y][n], ka, b.x, b.y);
                } else {
                  F::mma(c[y][n], ka, qb[4 * hf + x][n][0], qb[4 * hf + x][n][1]);
                }
              }
            }
          }
        }
        float4 f[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) f[t] = s_tok[warp][8 * t + g];
        float top[kG][2];
#pragma unroll
        for (int n = 0; n < kG; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float zs;
            if constexpr (TL::kQShared) zs = s_down[8 * n + 2 * tq + e];
            else zs = z_scale[n][e];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              float& z = c[t >> 1][n][2 * (t & 1) + e];
              z = fmaf(z, f[t].x * zs, f[t].y);
            }
          }
        }
        if constexpr (kMode == kDraft) {
          // a tile that some row of the unit does not see whole
          const int j0 = tile_start(i);
          if (j0 + kRows - 1 > first || (a.window > 0 && j0 <= last - a.window && j0 + kRows > a.n_sink)) {
#pragma unroll
            for (int n = 0; n < kG; ++n) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int at = first + (8 * n + 2 * tq + e) / G;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                  const int j = j0 + 8 * t + g;
                  if (j > at || (a.window > 0 && j <= at - a.window && j >= a.n_sink)) c[t >> 1][n][2 * (t & 1) + e] = -INFINITY;
                }
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < kG; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[n][e] = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t) top[n][e] = fmaxf(top[n][e], c[t >> 1][n][2 * (t & 1) + e] + f[t].z);
          }
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < kG; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(kFull, top[n][e], x));
            top[n][e] = fmaxf(m_r[n][e], top[n][e]);
            grow = grow || top[n][e] != m_r[n][e];
          }
        }
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int n = 0; n < kG; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float alpha = top[n][e] == -INFINITY ? 1.f : ex2_approx(m_r[n][e] - top[n][e]);
              l_r[n][e] *= alpha;
              m_r[n][e] = top[n][e];
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                o[x][n][e] *= alpha;
                o[x][n][2 + e] *= alpha;
              }
            }
          }
        }
        // weights: 2^(z - m) into l, times the values' scale into the product
        uint32_t pb[4][kG];
#pragma unroll
        for (int n = 0; n < kG; ++n) {
          const float m0 = m_r[n][0] == -INFINITY ? 0.f : m_r[n][0], m1 = m_r[n][1] == -INFINITY ? 0.f : m_r[n][1];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float p0 = ex2_approx(c[t >> 1][n][2 * (t & 1)] - m0), p1 = ex2_approx(c[t >> 1][n][2 * (t & 1) + 1] - m1);
            l_r[n][0] += p0;
            l_r[n][1] += p1;
            pb[t][n] = transpose8x8(F::pack(p0 * f[t].w, p1 * f[t].w));
          }
        }
        // O^T += C^T P^T: a register of ldmatrix.trans has two columns of two tokens, here rows g and g + 8 of a product
        const int mi = lane >> 3, rr = lane & 7;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t w[4];
            ldmatrix_x4_trans(w, sv + value_at<D>(kt * 16 + (mi & 1) * 8 + rr, 2 * x + (mi >> 1)));
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = __byte_perm(w[y], 0u, 0x3120);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t va[4] = {codes_f16(w[2 * y], false), codes_f16(w[2 * y], true), codes_f16(w[2 * y + 1], false),
                                      codes_f16(w[2 * y + 1], true)};
#pragma unroll
              for (int n = 0; n < kG; ++n) F::mma(o[2 * x + y][n], va, pb[2 * kt][n], pb[2 * kt + 1][n]);
            }
          }
        }
      }
    };
    // A group less is products and exponentials less (all as 4 groups / so, 16 requests as above 174 / 169 us).
    if constexpr (kMode == kDraft && kN == 4) {
      const int groups = groups_of(R);
      if (groups == 2) work(std::integral_constant<int, 2>());
      else if (groups == 3) work(std::integral_constant<int, 3>());
      else work(std::integral_constant<int, 4>());
    } else {
      work(std::integral_constant<int, kN>());
    }
    cnt += nt;
  }
  cp_async_wait<0>();
  if (kMode == kDraft && threadIdx.x == 0) a.cut[cta] = cut;
}

// kDraft: merges the parts of the units that are cut, four rows of a unit a block or, where that would be more than a block each,
// more of them. Every block lists the units for itself; a warp has a row and every ways-th batch of its parts, and the ways meet
// in shared memory. Measured (us) with a block for each CTA before and all rows of its unit / so: 3 - 8 tokens of 4 requests
// behind 8000 - 30000, 32 / 8 heads, 67 / 64, 4 of one 35 / 31, 3 - 8 of 16 150 / 151.
constexpr int kMergeWarps = 32, kBatch = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge8_kernel(const __grid_constant__ Decode8Args a) {
  using E = Elem<T>;
  constexpr int kCols = D / 32;                 // columns of a lane
  __shared__ float s_acc[kMergeWarps][D], s_m[kMergeWarps], s_tot[kMergeWarps];
  __shared__ int s_cut[32 * kMergeWarps], s_count[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.G;
  pdl_wait();
  for (int c0 = 0; c0 < a.ctas; c0 += 32 * kMergeWarps) {
    const int c = c0 + int(threadIdx.x);
    const unsigned cuts = __ballot_sync(kFull, c < a.ctas && a.cut[c].w > 0);
    if (lane == 0) s_count[warp] = __popc(cuts);
    __syncthreads();
    const int count = s_count[lane], before = __reduce_add_sync(kFull, lane < warp ? count : 0);
    const int units = __reduce_add_sync(kFull, count);
    int shift = 2;                              // log2 of the rows of an item
    while (shift < 5 && units * ((a.R - 1 >> shift) + 1) > int(gridDim.x)) ++shift;
    const int slices = (a.R - 1 >> shift) + 1, all_ways = kMergeWarps >> shift;
    if ((cuts >> lane) & 1u) s_cut[before + __popc(cuts & ((1u << lane) - 1u))] = c;
    __syncthreads();
    for (int item = blockIdx.x; item < units * slices; item += gridDim.x) {
      const int c_first = s_cut[item / slices], r0 = item % slices << shift;
      const int4 cut = a.cut[c_first];
      const int R = cut.y, parts = cut.w, row = r0 + (warp & ((1 << shift) - 1)), way = warp >> shift;
      if (r0 >= R) continue;
      float acc[kCols], M = -INFINITY, tot = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
      auto join = [&](float m, float t, const float (&x)[kCols]) {   // one more state: sums relative to e^m
        if (m == -INFINITY && t == t) return;   // empty (states of NaN alone have no maximum, but a NaN sum)
        const float top = fmaxf(M, m), f = M == -INFINITY ? 0.f : ex2_approx((M - top) * kLog2e), w = ex2_approx((m - top) * kLog2e);
        tot = fmaf(t, w, tot * f);
        M = top;
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = fmaf(x[i], w, acc[i] * f);
      };
      for (int p0 = way * kBatch; row < R && p0 < parts; p0 += all_ways * kBatch) {
        float x[kBatch][kCols], z[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          z[k] = -INFINITY;
          if (p0 + k < parts) {
            const int64_t at = (2 * int64_t(c_first + p0 + k) + (p0 + k == 0 ? 1 : 0)) * a.R + row;
            z[k] = __ldcg(a.part_lse + at);
#pragma unroll
            for (int i = 0; i < kCols; i += 2) {
              const float2 y = __ldcg(reinterpret_cast<const float2*>(a.part_o + at * D + kCols * lane + i));
              x[k][i] = y.x, x[k][i + 1] = y.y;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) join(z[k], 1.f, x[k]);
      }
      const int ways = min(all_ways, (parts + kBatch - 1) / kBatch);
      if (ways > 1) {
        __syncthreads();                        // what the item before left there is used up
        if (way > 0 && way < ways) {
#pragma unroll
          for (int i = 0; i < kCols; ++i) s_acc[warp][kCols * lane + i] = acc[i];
          if (lane == 0) s_m[warp] = M, s_tot[warp] = tot;
        }
        __syncthreads();
        for (int w = 1; w < ways && way == 0; ++w) {
          float x[kCols];
#pragma unroll
          for (int i = 0; i < kCols; ++i) x[i] = s_acc[(w << shift) + warp][kCols * lane + i];
          join(s_m[(w << shift) + warp], s_tot[(w << shift) + warp], x);
        }
      }
      if (way > 0 || row >= R) continue;
      const float f = tot != 0.f ? 1.0f / tot : 0.f;
      const int t = row / G;
      const int64_t to = int64_t(cut.x + t) * a.H_q + int64_t(cut.z) * G + (row - t * G);
#pragma unroll
      for (int i = 0; i < kCols; i += 2)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to * D + kCols * lane + i) = E::pack(acc[i] * f, acc[i + 1] * f);
      if (a.lse && lane == 0) a.lse[to] = tot != 0.f ? M + lg2_approx(tot) * kLn2 : -INFINITY;
    }
    __syncthreads();
  }
}

struct WsLayout {
  size_t cut, part_lse, part_o, total;
};
// Of units of R rows in kN groups.
template <int kN>
WsLayout ws_layout(int R, int D) {
  constexpr int kCtas64 = Tile8<64, kN>::kCtas, kCtas128 = Tile8<128, kN>::kCtas;
  static_assert(kCtas64 <= kTicketsPerSm && kCtas128 <= kTicketsPerSm, "a counter for each CTA");
  const int ctas = (D == 128 ? kCtas128 : kCtas64) * sm_count();
  WsLayout w;
  w.cut = ticket_bytes();
  w.part_lse = w.cut + align256(size_t(ctas) * sizeof(int4));
  w.part_o = w.part_lse + align256(size_t(ctas) * 2 * R * 4);
  w.total = w.part_o + size_t(ctas) * 2 * R * D * 4;
  return w;
}

template <typename T, int D, int kN, int kMode>
sa_status launch(const Decode8Args& a, int64_t most, cudaStream_t s) {
  using TL = Tile8<D, kN>;
  static int smem_set[64];
  auto k = decode8_kernel<T, D, kN, kMode>;
  if (!ensure_smem(k, TL::kSmem, smem_set)) return SA_ERR_CUDA;
  const int64_t sms = TL::kCtas * sm_count();
  const unsigned ctas = unsigned(most < sms ? most : sms);
  if (launch_ex(k, dim3(ctas), dim3(kThreads), TL::kSmem, s, true, 1, a) != cudaSuccess) return SA_ERR_CUDA;
  if (kMode != kDraft) return SA_OK;
  Decode8Args m = a;
  m.ctas = int(ctas);
  return launch_ex(merge8_kernel<T, D>, dim3(sm_count()), dim3(32 * kMergeWarps), 0, s, true, 1, m) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int kN, int kMode>
sa_status dispatch(const Decode8Args& a, int dtype, int D, int64_t most, cudaStream_t s) {
  const bool bf = dtype == SA_BF16;
  if (D == 128) return bf ? launch<__nv_bfloat16, 128, kN, kMode>(a, most, s) : launch<__half, 128, kN, kMode>(a, most, s);
  return bf ? launch<__nv_bfloat16, 64, kN, kMode>(a, most, s) : launch<__half, 64, kN, kMode>(a, most, s);
}

// What every call passes on, of a checked cache and batch and an aligned workspace of enough bytes.
template <int kN>
void fill_args(Decode8Args& a, const sa_cache8* cache, const sa_batch* batch, const void* q, int32_t num_q_heads, int R,
               float scale, void* out, float* lse, void* workspace, int32_t* dev_status) {
  const int D = cache->head_dim;
  const WsLayout w = ws_layout<kN>(R, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.k = static_cast<const uint8_t*>(cache->k); a.v = static_cast<const uint8_t*>(cache->v); a.scale = cache->scale;
  a.q = q; a.bt = batch->block_table; a.seq_lens = batch->seq_lens; a.out = out; a.lse = lse; a.status = dev_status;
  a.tickets = reinterpret_cast<int32_t*>(ws);
  a.cut = reinterpret_cast<int4*>(ws + w.cut);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.R = R; a.H_kv = cache->num_kv_heads; a.H_q = num_q_heads; a.G = num_q_heads / cache->num_kv_heads;
  a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks; a.bt_stride = batch->bt_stride;
  a.batch = batch->batch;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf(float(D))) * kLog2e;
}

}  // namespace
}  // namespace sa
