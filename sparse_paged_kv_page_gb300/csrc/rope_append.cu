// sa_append_kv_rope: RMS norm and rotation of the queries and keys of new
// tokens, the rotated keys and the values written into the paged pools, and the
// statistics of every page touched recomputed.
//
// Mathematics, per head row x of D values: r = x / sqrt(mean(x^2) + eps) * w (if
// there are weights), then for each of the rot / 2 pairs (u, v) of its first rot
// columns, turned by the angle a of the token's position on the pair's axis,
// (u cos a - v sin a, u sin a + v cos a). All in float32, rounded once to the
// element type. The statistics are those of sa_append_kv, over the rounded keys.
//
// Work split, all in one launch: one warp per (page, group of KV heads) of the new
// tokens, or up to four that share a large page's tokens and join their statistics in
// shared memory (pages of 128, 35,000 tokens: 281 -> 91 us); one warp per (token, chunk
// of query heads). Lane l of a row holds its pairs N l .. N l + N - 1, N = 8 for queries
// and 4 for keys (whose statistics take registers), so a rotation needs no other lane and
// the norm is a butterfly over few of them. The rows that a warp works on at once are
// heads of one token: they share its angles, and the page statistics of a column stay
// with the lane that owns it.
//
// Every value is read once and written once. Prompts are bound by HBM, where the few
// registers left for loads in flight keep it from more (4 x 8192 tokens, 64 / 8 heads of
// 128: 246 us, 5.6 TB/s, 82% of a copy's rate); ragged prompts of a few thousand tokens
// by a page's rows following one another (5 requests of 17 - 2501 tokens, 28 / 4 heads:
// 31 us); single tokens by the launch and the dependent loads of lengths, table and page
// (16 requests: 5.7 us). Queries in a launch of their own behind the keys': 250 us, 34 us.
#include "common.cuh"
#include "host.h"
#include "page_stats.cuh"

namespace sa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKeyPairs = 4, kQueryPairs = 8;   // pairs of columns of a lane
constexpr int kQueryBatch = 2;                  // rows of queries a lane has in flight beside those at work

// Calls whose warps fit the SMs at once wait for loads: many rows in flight a lane,
// three blocks an SM. Others need warps: five blocks an SM. Measured (us) as few / many:
// 16 requests' single tokens with 2048 - 8192 cached 5.7 / 7.7, 4 x 8192 tokens 329 / 246
// (1.37 GB: 82% of the measured copy bandwidth). Five blocks leave 96 registers a thread:
// bf16 spills 4 or 5 words there, fp16 none.
template <bool kFew>
struct Depth {
  static constexpr int kBlocks = kFew ? 3 : 5;
  static constexpr int kOld = kFew ? 8 : 4;     // cached rows
  static constexpr int kNew = kFew ? 2 : 1;     // tokens of new keys and values beside those at work
};

struct RopeArgs {
  void* k;
  void* v;
  void* meta;
  void* kstd;
  const void* q_in;
  const void* k_new;
  const void* v_new;
  void* q_out;
  int64_t q_stride, k_stride, v_stride;    // elements from one token to the next
  const int32_t* new_cu;
  const int32_t* bt;
  int32_t* seq_lens;
  const float* table;
  const int32_t* positions;
  const void* q_weight;
  const void* k_weight;
  uint16_t* hh;
  int32_t* ret_pos;
  int32_t* ret_cnt;
  int32_t* status;
  int H, H_q, ps_shift, num_blocks, bt_stride, batch, T, max_new, ret_cap, advanced;
  int max_pos, rot, axes, sec[4];          // sec: first pair of each axis's section
  float eps;
  int k_units, pages, k_groups;            // requests x pages each can touch x groups of KV heads
  int page_warps;                          // warps that share a unit
  int q_chunk, q_chunks;                   // query heads per warp
};

// Request with length L and new rows c0 .. c1: old length, tokens kept, first row.
// False if nothing is to be done for it.
__device__ __forceinline__ bool plan(const RopeArgs& a, int L, int c0, int c1, bool report, int& L_old, int& n) {
  n = c1 - c0;
  if (n < 0 || c0 < 0 || c1 > a.T || (L_old = a.advanced ? L - n : L) < 0) {
    if (report) flag(a.status, SA_DEV_BAD_COUNT);
    return false;
  }
  const int64_t cap = int64_t(a.bt_stride) << a.ps_shift;
  if (n > a.max_new || L_old + int64_t(n) > cap) {
    if (report) flag(a.status, SA_DEV_OVERFLOW);
    n = int(max(int64_t(0), min(int64_t(min(n, a.max_new)), cap - L_old)));
  }
  return n > 0;
}

// N words (two elements each, N = 2 or 4) in one access.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const void* p) {
  if constexpr (N == 4) {
    const uint4 x = *static_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else {
    const uint2 x = *static_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  if constexpr (N == 4) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <int NP>
struct Turn {
  float c[NP], s[NP];
};

// A lane's share of a row: two runs of NP columns, as words of two.
template <int NP>
struct Row {
  uint32_t w[NP];
};

// The columns of one lane: pairs e .. e + NP - 1 of the row, as NP adjacent columns
// at ca and NP at cb. Half layout: the u's and the v's of the pairs; interleaved and
// beyond the rotated columns: 2 NP adjacent columns, pair by pair.
template <bool kInter, int NP>
struct Lane {
  int e, ca, cb;
  int first[NP / 4], last[NP / 4];           // axes of the ends of each four pairs
  bool turned, split;
  __device__ __forceinline__ Lane(const RopeArgs& a, int l) {
    const int r = a.rot >> 1;
    e = NP * l;
    turned = e < r;
    split = !kInter && turned;
    ca = split ? e : 2 * e;
    cb = split ? e + r : 2 * e + NP;
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      first[i] = axis(a, e + 4 * i);
      last[i] = axis(a, e + 4 * i + 3);
    }
  }
  static __device__ __forceinline__ int axis(const RopeArgs& a, int e) {
    int x = 0;
    for (int i = 1; i < a.axes; ++i) x += e >= a.sec[i];
    return x;
  }
  __device__ __forceinline__ Row<NP> load(const uint16_t* row) const {
    Row<NP> r;
    load_words<NP / 2>(r.w, row + ca);
    load_words<NP / 2>(r.w + NP / 2, row + cb);
    return r;
  }
  __device__ __forceinline__ void store(uint16_t* row, const Row<NP>& r) const {
    store_words<NP / 2>(row + ca, r.w);
    store_words<NP / 2>(row + cb, r.w + NP / 2);
  }
  // Angles at the positions p of a token on each axis, four pairs at a time where they share one.
  __device__ __forceinline__ void angles(const RopeArgs& a, const int (&p)[4], Turn<NP>& g) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) g.c[i] = 1.f, g.s[i] = 0.f;
    if (!turned) return;
#pragma unroll
    for (int i = 0; i < NP; i += 4) {
      if (first[i / 4] == last[i / 4]) {
        const int pos = pick(p, first[i / 4]);
        if (pos < 0 || pos >= a.max_pos) {
          flag(a.status, SA_DEV_BAD_POSITION);
          continue;
        }
        const float* f = a.table + int64_t(pos) * a.rot + e + i;
        const float4 c = __ldg(reinterpret_cast<const float4*>(f));
        const float4 s = __ldg(reinterpret_cast<const float4*>(f + (a.rot >> 1)));
        g.c[i] = c.x, g.c[i + 1] = c.y, g.c[i + 2] = c.z, g.c[i + 3] = c.w;
        g.s[i] = s.x, g.s[i + 1] = s.y, g.s[i + 2] = s.z, g.s[i + 3] = s.w;
      } else {                               // a section ends inside them
#pragma unroll
        for (int x = i; x < i + 4; ++x) {
          const int pos = pick(p, axis(a, e + x));
          if (pos < 0 || pos >= a.max_pos) {
            flag(a.status, SA_DEV_BAD_POSITION);
            continue;
          }
          const float* f = a.table + int64_t(pos) * a.rot + e + x;
          g.c[x] = __ldg(f);
          g.s[x] = __ldg(f + (a.rot >> 1));
        }
      }
    }
  }
  static __device__ __forceinline__ int pick(const int (&p)[4], int x) {
    return x == 0 ? p[0] : x == 1 ? p[1] : x == 2 ? p[2] : p[3];
  }
};

// Positions of row t of the call on each axis, where the call gives them.
__device__ __forceinline__ void load_positions(const RopeArgs& a, int t, int (&p)[4]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) p[x] = a.positions && x < a.axes ? __ldg(a.positions + int64_t(x) * a.T + t) : 0;
}

template <typename T, int NP>
__device__ __forceinline__ void unpack(float (&x)[2 * NP], const Row<NP>& r) {
#pragma unroll
  for (int i = 0; i < NP; ++i) x[2 * i] = Elem<T>::lo(r.w[i]), x[2 * i + 1] = Elem<T>::hi(r.w[i]);
}

// One row: norm over its lanes (w: the weights of this lane's columns), rotation, rounding.
template <typename T, int D, bool kInter, int NP>
__device__ __forceinline__ Row<NP> transform(const Lane<kInter, NP>& ln, const Row<NP>& r, const Turn<NP>& g, bool norm,
                                             const Row<NP>& w, float eps) {
  if (!norm && !ln.turned) return r;
  float x[2 * NP];
  unpack<T, NP>(x, r);
  if (norm) {
    float ss = 0.f, wt[2 * NP];
    unpack<T, NP>(wt, w);
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < D / (2 * NP); o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float f = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) x[i] *= f * wt[i];
  }
  if (ln.split) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float u = x[i], v = x[NP + i];
      x[i] = u * g.c[i] - v * g.s[i];
      x[NP + i] = u * g.s[i] + v * g.c[i];
    }
  } else if (ln.turned) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float u = x[2 * i], v = x[2 * i + 1];
      x[2 * i] = u * g.c[i] - v * g.s[i];
      x[2 * i + 1] = u * g.s[i] + v * g.c[i];
    }
  }
  Row<NP> y;
#pragma unroll
  for (int i = 0; i < NP; ++i) y.w[i] = Elem<T>::pack(x[2 * i], x[2 * i + 1]);
  return y;
}

template <bool kInter, int NP>
__device__ __forceinline__ Row<NP> weights(const Lane<kInter, NP>& ln, const void* w) {
  return w ? ln.load(static_cast<const uint16_t*>(w)) : Row<NP>{};
}

// Packed minimum and maximum of two elements; a NaN loses to a number.
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y, __half) {
  const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y, __half) {
  const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Running statistics of a lane's columns; minimum and maximum in the elements' own type, the sum in float32 with the
// exact errors of its additions summed beside it.
template <typename T, int NP>
struct Columns {
  uint32_t mn[NP], mx[NP];
  float sum[2 * NP], err[2 * NP];
  uint32_t rounded = 0;                      // bit i: an addition of column i's sum has rounded
  __device__ __forceinline__ Columns() {
    const uint32_t inf = Elem<T>::pack(INFINITY, INFINITY);
#pragma unroll
    for (int i = 0; i < NP; ++i) mn[i] = inf, mx[i] = inf | 0x80008000u;
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) sum[i] = err[i] = 0.f;
  }
  __device__ __forceinline__ void add_to(int i, float x) {
    const float t = sum[i] + x, y = t - sum[i];
    const float e = (sum[i] - (t - y)) + (x - y);
    sum[i] = t;
    err[i] += e;
    rounded |= uint32_t(e != 0.f) << i;
  }
  __device__ __forceinline__ void add(const Row<NP>& r) {
    float x[2 * NP];
    unpack<T, NP>(x, r);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      mn[i] = min2(mn[i], r.w[i], T());
      mx[i] = max2(mx[i], r.w[i], T());
    }
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) add_to(i, x[i]);
  }
  // To and from shared memory, a lane's words 32 apart.
  static constexpr int kWords = 6 * NP + 1;
  __device__ __forceinline__ void save(uint32_t* p) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) p[32 * i] = mn[i], p[32 * (NP + i)] = mx[i];
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      p[32 * (2 * NP + i)] = __float_as_uint(sum[i]);
      p[32 * (4 * NP + i)] = __float_as_uint(err[i]);
    }
    p[32 * 6 * NP] = rounded;
  }
  __device__ __forceinline__ void join(const uint32_t* p) {
    rounded |= p[32 * 6 * NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      mn[i] = min2(mn[i], p[32 * i], T());
      mx[i] = max2(mx[i], p[32 * (NP + i)], T());
    }
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      add_to(i, __uint_as_float(p[32 * (2 * NP + i)]));
      err[i] += __uint_as_float(p[32 * (4 * NP + i)]);
    }
  }
};

// The float64 mean of a column, rounded once, where its float32 sum has rounded: from the sum and its errors. The sum of
// the n errors, each at most 2^-24 n |x|, is off by at most n 2^-24 of theirs, n^3 2^-48 |x| with |x| the column's
// largest value (and float64 by 2^-50 of the mean); where it could round two ways within that (or is not finite), from
// the pool's rows
// (half `hi` of words p, p + C, ..).
template <typename T>
__device__ __noinline__ uint16_t mean_f64(float sum, float err, float big, const uint32_t* p, int C, int fill, bool hi) {
  const double n = double(fill), mean = (double(sum) + double(err)) / n, off = n * n * 0x1p-48 * double(big) + 0x1p-50 * fabs(mean);
  const uint16_t lo = Elem<T>::from_f64(mean - off);
  if (lo == Elem<T>::from_f64(mean + off) && fabsf(sum) < 0x1p126f) return lo;
  double d = 0.0;
  for (int s = 0; s < fill; ++s) {
    const uint32_t w = p[int64_t(s) * C];
    d += double(hi ? Elem<T>::hi(w) : Elem<T>::lo(w));
  }
  return Elem<T>::from_f64(d / n);
}

// Statistics of the lane's columns of (block, head), written; the page's rows are in the pool.
template <typename T, int D, int NP>
__device__ __forceinline__ void write_stats(const RopeArgs& a, const Columns<T, NP>& st, int64_t tile, int blk, int h,
                                            int ca, int cb, int fill) {
  using E = Elem<T>;
  constexpr int C = D / 2;
  const uint32_t* kp = static_cast<const uint32_t*>(a.k) + tile * C;
  uint32_t* m = static_cast<uint32_t*>(a.meta) + (int64_t(blk) * a.H + h) * 3 * C;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t mean[NP / 2];
    const int c0 = (half ? cb : ca) >> 1;    // first column pair
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      const int x = NP * half + 2 * i, w = NP / 2 * half + i;
      uint16_t m0 = 0, m1 = 0;
      if (((st.rounded >> x) & 1u) || !mean_f32<T>(st.sum[x], fill, m0))
        m0 = mean_f64<T>(st.sum[x], st.err[x], fmaxf(fabsf(E::lo(st.mn[w])), fabsf(E::lo(st.mx[w]))), kp + c0 + i, C, fill, false);
      if (((st.rounded >> (x + 1)) & 1u) || !mean_f32<T>(st.sum[x + 1], fill, m1))
        m1 = mean_f64<T>(st.sum[x + 1], st.err[x + 1], fmaxf(fabsf(E::hi(st.mn[w])), fabsf(E::hi(st.mx[w]))), kp + c0 + i, C,
                         fill, true);
      mean[i] = uint32_t(m0) | (uint32_t(m1) << 16);
    }
    store_words<NP / 2>(m + c0, st.mn + NP / 2 * half);
    store_words<NP / 2>(m + C + c0, st.mx + NP / 2 * half);
    store_words<NP / 2>(m + 2 * C + c0, mean);
    if (a.kstd)
      for (int i = 0; i < NP / 2; ++i)
        page_std_pair<T>(a.kstd, static_cast<const uint32_t*>(a.k), tile, fill, blk, a.H, C, h, c0 + i);
  }
}

// The rows of unit `u` (a group of KV heads on one page) that warp `part` of the a.page_warps that share it has.
template <int RPW>
struct PageRows {
  int h, b, start, blk, fill;          // head of this lane, request, first position of the page, its block and rows
  int lo, s_old, s_new, hi;            // this warp's slots: [lo, s_old) cached before, [s_new, hi) new
  int row0, pos0;                      // row of the call at slot 0; old length
  bool on, live;                       // there is such a head; there is something to do
  __device__ __forceinline__ PageRows(const RopeArgs& a, int u, int part, bool unit, int sub, bool report) {
    live = unit;
    if (!unit) u = 0;
    h = (u % a.k_groups) * RPW + sub;
    on = h < a.H;
    const int rest = u / a.k_groups, i = rest % a.pages;
    b = rest / a.pages;
    const int c0 = a.new_cu[b], c1 = a.new_cu[b + 1], L = a.seq_lens[b];
    int L_old = 0, n = 0;
    live = live && plan(a, L, c0, c1, report && part == 0 && u % a.k_groups == 0 && i == 0, L_old, n);
    const int ps = 1 << a.ps_shift, p = (L_old >> a.ps_shift) + i;
    live = live && p <= ((L_old + n - 1) >> a.ps_shift);
    start = p << a.ps_shift;
    blk = live ? a.bt[int64_t(b) * a.bt_stride + p] : -1;
    if (live && (blk < 0 || blk >= a.num_blocks)) {
      if (report) flag(a.status, SA_DEV_BAD_BLOCK);
      live = false;
    }
    pos0 = L_old;
    row0 = c0 + start - L_old;
    fill = min(ps, L_old + n - start);
    const int first = max(0, L_old - start);
    lo = part * (ps / a.page_warps);
    hi = live ? min(fill, lo + ps / a.page_warps) : 0;
    s_new = max(lo, first);
    s_old = min(first, hi);
  }
};

// The new keys and values of unit `u` and the statistics of its page. All warps of a block call it.
template <typename T, int D, bool kInter, bool kFew>
__device__ __forceinline__ void key_unit(const RopeArgs& a, int u, int part, bool live, uint32_t* joint) {
  constexpr int NP = kKeyPairs, LPR = D / (2 * NP), RPW = 32 / LPR, kKeyBatch = Depth<kFew>::kNew, kOldBatch = Depth<kFew>::kOld;
  const int lane = threadIdx.x & 31, col = 2 * NP * (lane % LPR);
  const PageRows<RPW> r(a, u, part, live, lane / LPR, lane == 0);
  const Lane<kInter, NP> ln(a, lane % LPR);
  const int h = r.h, start = r.start, blk = r.blk, fill = r.fill, ps = 1 << a.ps_shift;
  const int lo = r.lo, s_old = r.s_old, s_new = r.s_new, hi = r.hi, row0 = r.row0;
  const bool on = r.on;
  live = r.live;
  const uint16_t* kn = static_cast<const uint16_t*>(a.k_new) + h * D;
  const uint16_t* vn = static_cast<const uint16_t*>(a.v_new) + h * D + col;
  Row<NP> x[kKeyBatch], v[kKeyBatch];
  Turn<NP> g[kKeyBatch];
  int at[4] = {0, 0, 0, 0};                  // positions of the page's token 32 m + lane, on each axis
  auto fetch = [&](int s0) {
#pragma unroll
    for (int j = 0; j < kKeyBatch; ++j) {
      const int s = s0 + j, t = row0 + s;
      if (a.positions && (s == s_new || (s & 31) == 0)) {
        const int mine = (s & ~31) + lane;
        if (mine >= s_new && mine < hi) load_positions(a, row0 + mine, at);
      }
      int pos[4] = {start + s, 0, 0, 0};
      if (a.positions) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < a.axes) pos[x] = __shfl_sync(kFull, at[x], s & 31);
      }
      x[j] = v[j] = Row<NP>{};
      if (s < hi) {
        if (on) {
          x[j] = ln.load(kn + t * a.k_stride);
          load_words<NP>(v[j].w, vn + t * a.v_stride);
        }
        ln.angles(a, pos, g[j]);
      }
    }
  };
  fetch(s_new);
  const Row<NP> w = weights(ln, a.k_weight);
  const int64_t tile = (int64_t(blk) * a.H + h) * ps;
  uint16_t* kp = static_cast<uint16_t*>(a.k) + tile * D;
  uint16_t* vp = static_cast<uint16_t*>(a.v) + tile * D + col;
  Columns<T, NP> st;
  if (a.meta && on) {
    for (int s0 = lo; s0 < s_old; s0 += kOldBatch) {
      Row<NP> old[kOldBatch];
#pragma unroll
      for (int j = 0; j < kOldBatch; ++j)
        if (s0 + j < s_old) old[j] = ln.load(kp + (s0 + j) * D);
#pragma unroll
      for (int j = 0; j < kOldBatch; ++j)
        if (s0 + j < s_old) st.add(old[j]);
    }
  }
  __syncwarp();
  for (int s0 = s_new; s0 < hi; s0 += kKeyBatch) {
    Row<NP> y[kKeyBatch], z[kKeyBatch];
#pragma unroll
    for (int j = 0; j < kKeyBatch; ++j) {
      y[j] = transform<T, D, kInter, NP>(ln, x[j], g[j], a.k_weight != nullptr, w, a.eps);
      z[j] = v[j];
    }
    if (s0 + kKeyBatch < hi) fetch(s0 + kKeyBatch);
#pragma unroll
    for (int j = 0; j < kKeyBatch; ++j) {
      const int s = s0 + j;
      if (s < hi && on) {
        ln.store(kp + s * D, y[j]);
        store_words<NP>(vp + s * D, z[j].w);
        if (a.meta) st.add(y[j]);
      }
    }
  }
  if (a.page_warps > 1 && a.meta) {          // the page's statistics meet in its first warp
    uint32_t* mine = joint + (threadIdx.x >> 5) * 32 * Columns<T, NP>::kWords + lane;
    if (part > 0) st.save(mine);
    __syncthreads();
    if (part == 0)
      for (int q = 1; q < a.page_warps; ++q) st.join(mine + q * 32 * Columns<T, NP>::kWords);
  }
  if (!on || !live) return;
  if (a.meta && part == 0) write_stats<T, D, NP>(a, st, tile, blk, h, ln.ca, ln.cb, fill);
  for (int s = s_new + lane % LPR; s < hi; s += LPR) {
    if (a.hh) a.hh[(int64_t(blk) * ps + s) * a.H + h] = 0;
    if (a.ret_pos) {
      const int cpos = a.ret_cnt[r.b * a.H + h] + (start + s - r.pos0);
      if (cpos < 0 || cpos >= a.ret_cap) flag(a.status, SA_DEV_OVERFLOW);
      else a.ret_pos[(int64_t(r.b) * a.H + h) * a.ret_cap + cpos] = start + s;
    }
  }
}

// Warp `u`: a chunk of the query heads of one token.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void query_unit(const RopeArgs& a, int u) {
  constexpr int NP = kQueryPairs, LPR = D / (2 * NP), RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const int t = u / a.q_chunks, h0 = (u % a.q_chunks) * a.q_chunk, h1 = min(a.H_q, h0 + a.q_chunk);
  const Lane<kInter, NP> ln(a, lane % LPR);
  const uint16_t* qi = static_cast<const uint16_t*>(a.q_in) + t * a.q_stride;
  uint16_t* qo = static_cast<uint16_t*>(a.q_out) + int64_t(t) * a.H_q * D;
  Row<NP> x[kQueryBatch];
  auto fetch = [&](int h) {
#pragma unroll
    for (int j = 0; j < kQueryBatch; ++j) {
      const int hh = h + j * RPW + sub;
      x[j] = hh < h1 ? ln.load(qi + hh * D) : Row<NP>{};
    }
  };
  fetch(h0);
  int pos[4];
  load_positions(a, t, pos);
  const Row<NP> w = weights(ln, a.q_weight);
  // the token's request: the first whose rows end behind t
  int b = 0, c0 = 0, c1 = 0, L = 0, from = 0;
  if (a.batch > 32) {                        // first among 32 evenly spaced ones: two rounds of loads for 1024 requests
    const int step = (a.batch + 31) / 32;
    from = step * __popc(__ballot_sync(kFull, a.new_cu[min((lane + 1) * step, a.batch)] <= t));
  }
  for (int b0 = from; b0 < a.batch; b0 += 32) {
    const int i = min(b0 + lane, a.batch - 1);
    const int end = a.new_cu[i + 1], beg = a.new_cu[i], len = a.seq_lens[i];
    const int k = __popc(__ballot_sync(kFull, b0 + lane < a.batch && end <= t));
    b = b0 + k;
    c1 = __shfl_sync(kFull, end, k & 31);
    c0 = __shfl_sync(kFull, beg, k & 31);
    L = __shfl_sync(kFull, len, k & 31);
    if (k < 32) break;
  }
  int L_old, n;
  if (b >= a.batch || t < c0 || !plan(a, L, c0, c1, false, L_old, n) || t - c0 >= n) return;
  Turn<NP> g;
  if (!a.positions) pos[0] = L_old + t - c0;
  ln.angles(a, pos, g);
  __syncwarp();
  for (int h = h0; h < h1; h += kQueryBatch * RPW) {
    Row<NP> y[kQueryBatch];
#pragma unroll
    for (int j = 0; j < kQueryBatch; ++j) y[j] = transform<T, D, kInter, NP>(ln, x[j], g, a.q_weight != nullptr, w, a.eps);
    if (h + kQueryBatch * RPW < h1) fetch(h + kQueryBatch * RPW);
#pragma unroll
    for (int j = 0; j < kQueryBatch; ++j) {
      const int hh = h + j * RPW + sub;
      if (hh < h1) ln.store(qo + hh * D, y[j]);
    }
  }
}

template <typename T, int D, bool kInter, bool kFew>
__global__ void __launch_bounds__(kThreads, Depth<kFew>::kBlocks) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ uint32_t joint[];        // a block's column statistics, where warps share pages
  const int per_block = kWarps / a.page_warps, k_blocks = (a.k_units + per_block - 1) / per_block;
  const int warp = threadIdx.x >> 5;
  if (int(blockIdx.x) < k_blocks) {
    const int u = blockIdx.x * per_block + warp / a.page_warps;
    key_unit<T, D, kInter, kFew>(a, u, warp % a.page_warps, u < a.k_units, joint);
  } else {
    const int u = (blockIdx.x - k_blocks) * kWarps + warp;
    if (u < a.T * a.q_chunks) query_unit<T, D, kInter>(a, u);
  }
}

// Advances lengths and retained counts once the kernel before it has read them.
__global__ void rope_advance_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.batch; b += gridDim.x * blockDim.x) {
    int L_old, n;
    if (!plan(a, a.seq_lens[b], a.new_cu[b], a.new_cu[b + 1], false, L_old, n)) continue;
    if (a.ret_cnt)
      for (int h = 0; h < a.H; ++h) a.ret_cnt[b * a.H + h] = min(max(a.ret_cnt[b * a.H + h] + n, 0), a.ret_cap);
    if (!a.advanced) a.seq_lens[b] = L_old + n;
  }
}

template <typename T, int D>
cudaError_t launch(const RopeArgs& a, unsigned blocks, bool inter, cudaStream_t s) {
  const size_t smem = a.page_warps > 1 ? sizeof(uint32_t) * kWarps * 32 * Columns<T, kKeyPairs>::kWords : 0;
  const bool few = blocks <= unsigned(Depth<true>::kBlocks * sm_count());
  auto k = few ? (inter ? rope_append_kernel<T, D, true, true> : rope_append_kernel<T, D, false, true>)
               : (inter ? rope_append_kernel<T, D, true, false> : rope_append_kernel<T, D, false, false>);
  return launch_ex(k, dim3(blocks), dim3(kThreads), smem, s, false, 1, a);
}

bool bad_stride(int64_t stride, int64_t row) { return stride < row || stride % 8; }

}  // namespace
}  // namespace sa

extern "C" sa_status sa_append_kv_rope(const sa_cache* cache, const sa_batch* batch, const sa_rope* rope, const void* q,
                                       int64_t q_stride, int32_t num_q_heads, const void* k_new, int64_t k_stride,
                                       const void* v_new, int64_t v_stride, const int32_t* new_cu, int32_t num_tokens,
                                       int32_t max_new_per_req, int32_t advanced, void* q_out, void* hh,
                                       int32_t* ret_pos, int32_t* ret_cnt, int32_t ret_cap, int32_t* dev_status,
                                       void* stream) {
  using namespace sa;
  sa_status st = check_cache(cache, true, false);
  if (st != SA_OK) return st;
  if ((st = check_batch(batch)) != SA_OK) return st;
  if (!rope || !new_cu || num_tokens < 0 || max_new_per_req < 0) return SA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!k_new || !v_new)) return SA_ERR_INVALID_ARG;   // (no rows: they may have no address)
  if ((q == nullptr) != (q_out == nullptr) || (q && num_q_heads <= 0)) return SA_ERR_INVALID_ARG;
  if ((ret_pos == nullptr) != (ret_cnt == nullptr) || (ret_pos && ret_cap <= 0)) return SA_ERR_INVALID_ARG;
  if (cache->kstd && !cache->meta) return SA_ERR_INVALID_ARG;
  const int D = cache->head_dim, H = cache->num_kv_heads;
  if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 16) return SA_ERR_INVALID_ARG;
  if (rope->rot_dim && (!rope->table || rope->max_pos <= 0)) return SA_ERR_INVALID_ARG;
  if (rope->num_axes < 1 || rope->num_axes > 4 || (rope->num_axes > 1 && num_tokens > 0 && !rope->positions)) return SA_ERR_INVALID_ARG;
  if (!(rope->eps >= 0.f)) return SA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(rope->table) ||
      !aligned16(rope->q_weight) || !aligned16(rope->k_weight))
    return SA_ERR_INVALID_ARG;
  if ((q && bad_stride(q_stride, int64_t(num_q_heads) * D)) || bad_stride(k_stride, int64_t(H) * D) ||
      bad_stride(v_stride, int64_t(H) * D))
    return SA_ERR_INVALID_ARG;
  RopeArgs a = {};
  int pairs = 0;
  for (int x = 0; x < rope->num_axes; ++x) {
    if (rope->num_axes > 1 && rope->sections[x] < 0) return SA_ERR_INVALID_ARG;
    a.sec[x] = pairs;
    pairs += rope->num_axes > 1 ? rope->sections[x] : rope->rot_dim / 2;
    if (pairs > rope->rot_dim / 2) return SA_ERR_INVALID_ARG;
  }
  if (pairs != rope->rot_dim / 2) return SA_ERR_INVALID_ARG;
  if (num_tokens == 0 || max_new_per_req == 0) return SA_OK;
  a.k = cache->k; a.v = cache->v; a.meta = cache->meta; a.kstd = cache->kstd;
  a.q_in = q; a.k_new = k_new; a.v_new = v_new; a.q_out = q_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.new_cu = new_cu; a.bt = batch->block_table; a.seq_lens = batch->seq_lens;
  a.table = rope->table; a.positions = rope->positions; a.q_weight = rope->q_weight; a.k_weight = rope->k_weight;
  a.hh = static_cast<uint16_t*>(hh); a.ret_pos = ret_pos; a.ret_cnt = ret_cnt; a.status = dev_status;
  a.H = H; a.H_q = num_q_heads; a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks;
  a.bt_stride = batch->bt_stride; a.batch = batch->batch; a.T = num_tokens;
  a.max_new = max_new_per_req < num_tokens ? max_new_per_req : num_tokens;
  a.ret_cap = ret_pos ? ret_cap : 0; a.advanced = advanced ? 1 : 0;
  a.max_pos = rope->max_pos; a.rot = rope->rot_dim; a.axes = rope->num_axes; a.eps = rope->eps;
  // n tokens from any slot touch at most (n + ps - 2) / ps + 1 pages
  a.pages = int((int64_t(a.max_new) + cache->page_size - 2) / cache->page_size) + 1;
  const int k_rows = 64 * kKeyPairs / D, rows = 64 * kQueryPairs / D;   // heads a warp works on at once
  a.k_groups = (H + k_rows - 1) / k_rows;
  const int64_t k_units = int64_t(batch->batch) * a.pages * a.k_groups;
  // query heads per warp: one batch where tokens are few, more where one read of the angles can serve them
  a.q_chunk = rows;
  const int64_t full = int64_t(sm_count()) * 64;
  while (q && a.q_chunk < 32 && a.q_chunk < num_q_heads && int64_t(num_tokens) * num_q_heads / (2 * a.q_chunk) >= full)
    a.q_chunk *= 2;
  a.q_chunks = q ? (num_q_heads + a.q_chunk - 1) / a.q_chunk : 0;
  const int64_t q_units = int64_t(num_tokens) * a.q_chunks;
  if (k_units > 0x1fffff00 || q_units > 0x7fffff00) return SA_ERR_UNSUPPORTED;
  a.k_units = int(k_units);
  // warps that share a page's rows: as many as give each at least 8 of them, while the pages alone leave SMs waiting
  // (us with 1 / 2 / 4 warps a page of 32 and 128 tokens: 56 / 27 / 21 and 207 / 182 / 91 for 3 k and 35 k tokens of
  // 4 KV heads; 4 x 8192 tokens in pages of 16: 247 / 254)
  a.page_warps = 1;
  while (a.page_warps < kWarps && cache->page_size >= 16 * a.page_warps && k_units * a.page_warps < int64_t(24) * sm_count())
    a.page_warps *= 2;
  const int per_block = kWarps / a.page_warps;
  const unsigned blocks = unsigned((k_units + per_block - 1) / per_block + (q_units + kWarps - 1) / kWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SA_BF16, inter = rope->interleaved != 0;
  const cudaError_t e = D == 128 ? (bf ? launch<__nv_bfloat16, 128>(a, blocks, inter, s) : launch<__half, 128>(a, blocks, inter, s))
                                 : (bf ? launch<__nv_bfloat16, 64>(a, blocks, inter, s) : launch<__half, 64>(a, blocks, inter, s));
  if (e != cudaSuccess) return SA_ERR_CUDA;
  if (advanced && !ret_cnt) return SA_OK;
  const unsigned ab = unsigned((batch->batch + 127) / 128);
  return launch_ex(rope_advance_kernel, dim3(ab), dim3(128), 0, s, true, 1, a) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
