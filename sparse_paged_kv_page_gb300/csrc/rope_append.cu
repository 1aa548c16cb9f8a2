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
// Work split: one warp per (page, KV head) of the new tokens, one warp per
// (token, chunk of query heads), all in one launch. A row is D / 4 lanes of
// four columns: lane l holds pairs 2l and 2l + 1, so a rotation needs no other
// lane, the norm is one butterfly sum, and the page statistics of a column stay
// in the registers of the lane that owns it. Rows are loaded four at a time.
// Every value is read once and written once: HBM bound for prompts, bound by the
// launch and two dependent loads (lengths, then angles) for single tokens.
#include "common.cuh"
#include "host.h"
#include "page_stats.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;                  // rows a lane has in flight

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
  int k_units, pages, q_chunk, q_chunks;   // K warps, pages a request can touch, query heads per warp
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

struct Turn {
  float c0, c1, s0, s1;
};

// The columns of one lane: pairs e and e + 1 of the row, as two adjacent column
// pairs at ca and cb. Half layout: (ca, cb) = (u's, v's); interleaved and beyond
// the rotated columns: (ca, cb) = (pair e, pair e + 1).
template <bool kInter>
struct Lane {
  int e, ca, cb, ax0, ax1;
  bool turned, split;
  __device__ __forceinline__ Lane(const RopeArgs& a, int l) {
    const int r = a.rot >> 1;
    e = 2 * l;
    turned = e < r;
    split = !kInter && turned;
    ca = split ? e : 2 * e;
    cb = split ? e + r : 2 * e + 2;
    ax0 = ax1 = 0;
    for (int x = 1; x < a.axes; ++x) {
      ax0 += e >= a.sec[x];
      ax1 += e + 1 >= a.sec[x];
    }
  }
  __device__ __forceinline__ uint2 load(const uint16_t* row) const {
    if (kInter) return *reinterpret_cast<const uint2*>(row + ca);
    return make_uint2(*reinterpret_cast<const uint32_t*>(row + ca), *reinterpret_cast<const uint32_t*>(row + cb));
  }
  __device__ __forceinline__ void store(uint16_t* row, uint2 w) const {
    if (kInter) {
      *reinterpret_cast<uint2*>(row + ca) = w;
    } else {
      *reinterpret_cast<uint32_t*>(row + ca) = w.x;
      *reinterpret_cast<uint32_t*>(row + cb) = w.y;
    }
  }
  // Angles of row t of the call (position `pos` where the call gives none).
  __device__ __forceinline__ Turn angles(const RopeArgs& a, int t, int pos) const {
    Turn g = {1.f, 1.f, 0.f, 0.f};
    if (!turned) return g;
    int p0 = pos, p1 = pos;
    if (a.positions) {
      p0 = __ldg(a.positions + int64_t(ax0) * a.T + t);
      p1 = ax1 == ax0 ? p0 : __ldg(a.positions + int64_t(ax1) * a.T + t);
    }
    if (p0 < 0 || p0 >= a.max_pos || p1 < 0 || p1 >= a.max_pos) {
      flag(a.status, SA_DEV_BAD_POSITION);
      return g;
    }
    const float* f0 = a.table + int64_t(p0) * a.rot + e;
    if (p0 == p1) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(f0));
      const float2 s = __ldg(reinterpret_cast<const float2*>(f0 + (a.rot >> 1)));
      g = {c.x, c.y, s.x, s.y};
    } else {
      const float* f1 = a.table + int64_t(p1) * a.rot + e + 1;
      g = {__ldg(f0), __ldg(f1), __ldg(f0 + (a.rot >> 1)), __ldg(f1 + (a.rot >> 1))};
    }
    return g;
  }
};

// One row: norm over its LPR lanes (weights w of this lane's columns), rotation, rounding.
template <typename T, int D, bool kInter>
__device__ __forceinline__ uint2 transform(const Lane<kInter>& ln, uint2 x, const Turn& g, bool norm, const float4& w,
                                           float eps) {
  using E = Elem<T>;
  float a0 = E::lo(x.x), a1 = E::hi(x.x), b0 = E::lo(x.y), b1 = E::hi(x.y);
  if (norm) {
    float ss = fmaf(a0, a0, a1 * a1) + fmaf(b0, b0, b1 * b1);
#pragma unroll
    for (int o = 1; o < D / 4; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float f = rsqrtf(ss * (1.0f / D) + eps);
    a0 *= f * w.x;
    a1 *= f * w.y;
    b0 *= f * w.z;
    b1 *= f * w.w;
  }
  if (ln.split)
    return make_uint2(E::pack(a0 * g.c0 - b0 * g.s0, a1 * g.c1 - b1 * g.s1),
                      E::pack(a0 * g.s0 + b0 * g.c0, a1 * g.s1 + b1 * g.c1));
  if (ln.turned)
    return make_uint2(E::pack(a0 * g.c0 - a1 * g.s0, a0 * g.s0 + a1 * g.c0),
                      E::pack(b0 * g.c1 - b1 * g.s1, b0 * g.s1 + b1 * g.c1));
  return norm ? make_uint2(E::pack(a0, a1), E::pack(b0, b1)) : x;
}

template <typename T, bool kInter>
__device__ __forceinline__ float4 weights(const Lane<kInter>& ln, const void* w) {
  if (!w) return make_float4(1.f, 1.f, 1.f, 1.f);
  const uint2 x = ln.load(static_cast<const uint16_t*>(w));
  return make_float4(Elem<T>::lo(x.x), Elem<T>::hi(x.x), Elem<T>::lo(x.y), Elem<T>::hi(x.y));
}

// Running statistics of one column.
struct Column {
  float mn = INFINITY, mx = -INFINITY, sum = 0.f;
  bool exact = true;
  __device__ __forceinline__ void add(float x) {
    mn = fminf(mn, x);
    mx = fmaxf(mx, x);
    two_sum(sum, x, exact);
  }
  __device__ __forceinline__ void join(int lanes) {
    mn = fminf(mn, __shfl_xor_sync(kFull, mn, lanes));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, lanes));
    const bool both = __shfl_xor_sync(kFull, exact, lanes) && exact;
    const float other = __shfl_xor_sync(kFull, sum, lanes);
    exact = both;
    two_sum(sum, other, exact);            // an exact sum is the same in either order
  }
};

// Statistics of the adjacent columns (2c, 2c + 1) of (block, head), written; rows already in the pool.
template <typename T>
__device__ __forceinline__ void write_stats(const RopeArgs& a, const Column& x, const Column& y, int64_t tile, int blk,
                                            int h, int D, int c, int fill) {
  using E = Elem<T>;
  const int C = D / 2;
  const uint32_t* kp = static_cast<const uint32_t*>(a.k);
  uint16_t m0 = 0, m1 = 0;
  const bool ok0 = x.exact && mean_f32<T>(x.sum, fill, m0);
  const bool ok1 = y.exact && mean_f32<T>(y.sum, fill, m1);
  if (!ok0 || !ok1) {                      // rare: float64 over the pool's rows
    double d0 = 0.0, d1 = 0.0;
    for (int s = 0; s < fill; ++s) {
      const uint32_t w = kp[(tile + s) * C + c];
      d0 += double(E::lo(w));
      d1 += double(E::hi(w));
    }
    if (!ok0) m0 = E::from_f64(d0 / double(fill));
    if (!ok1) m1 = E::from_f64(d1 / double(fill));
  }
  uint32_t* m = static_cast<uint32_t*>(a.meta) + (int64_t(blk) * a.H + h) * 3 * C + c;
  m[0] = E::pack(x.mn, y.mn);
  m[C] = E::pack(x.mx, y.mx);
  m[2 * C] = uint32_t(m0) | (uint32_t(m1) << 16);
  if (a.kstd) page_std_pair<T>(a.kstd, kp, tile, fill, blk, a.H, C, h, c);
}

// Warp `u`: the new keys and values of one KV head on one page.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void key_unit(const RopeArgs& a, int u) {
  using E = Elem<T>;
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, col = 4 * (lane % LPR);
  const int h = u % a.H, rest = u / a.H, b = rest / a.pages, i = rest % a.pages;
  const int c0 = a.new_cu[b], c1 = a.new_cu[b + 1], L = a.seq_lens[b];
  int L_old, n;
  if (!plan(a, L, c0, c1, lane == 0 && h == 0 && i == 0, L_old, n)) return;
  const int ps = 1 << a.ps_shift;
  const int p = (L_old >> a.ps_shift) + i;
  if (p > ((L_old + n - 1) >> a.ps_shift)) return;
  const int blk = a.bt[int64_t(b) * a.bt_stride + p];
  if (blk < 0 || blk >= a.num_blocks) {
    if (lane == 0) flag(a.status, SA_DEV_BAD_BLOCK);
    return;
  }
  const Lane<kInter> ln(a, lane % LPR);
  const float4 w = weights<T>(ln, a.k_weight);
  const int start = p << a.ps_shift;
  const int s_new = max(0, L_old - start), fill = min(ps, L_old + n - start);
  const int64_t tile = (int64_t(blk) * a.H + h) * ps;
  uint16_t* kp = static_cast<uint16_t*>(a.k) + tile * D;
  uint16_t* vp = static_cast<uint16_t*>(a.v) + tile * D;
  const uint16_t* kn = static_cast<const uint16_t*>(a.k_new) + int64_t(h) * D;
  const uint16_t* vn = static_cast<const uint16_t*>(a.v_new) + int64_t(h) * D + col;
  Column st[4];
  for (int s0 = a.meta ? 0 : s_new / RPW * RPW; s0 < fill; s0 += kBatch * RPW) {
    uint2 x[kBatch], v[kBatch];
    Turn g[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = s0 + j * RPW + sub, t = c0 + start + s - L_old;
      x[j] = v[j] = make_uint2(0u, 0u);
      g[j] = {1.f, 1.f, 0.f, 0.f};
      if (s >= s_new && s < fill) {
        x[j] = ln.load(kn + t * a.k_stride);
        v[j] = __ldg(reinterpret_cast<const uint2*>(vn + t * a.v_stride));
        g[j] = ln.angles(a, t, start + s);
      } else if (s < s_new && a.meta) {
        x[j] = ln.load(kp + s * D);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = s0 + j * RPW + sub;
      const uint2 y = transform<T, D, kInter>(ln, x[j], g[j], a.k_weight != nullptr, w, a.eps);
      if (s >= s_new && s < fill) {
        x[j] = y;
        ln.store(kp + s * D, y);
        *reinterpret_cast<uint2*>(vp + s * D + col) = v[j];
      }
      if (s < fill) {
        st[0].add(E::lo(x[j].x));
        st[1].add(E::hi(x[j].x));
        st[2].add(E::lo(x[j].y));
        st[3].add(E::hi(x[j].y));
      }
    }
  }
  __syncwarp();                            // the other lanes' rows are in the pool
  if (a.meta) {
    if (RPW == 2) {
#pragma unroll
      for (int x = 0; x < 4; ++x) st[x].join(LPR);
    }
    if (sub == 0) {
      write_stats<T>(a, st[0], st[1], tile, blk, h, D, ln.ca >> 1, fill);
      write_stats<T>(a, st[2], st[3], tile, blk, h, D, ln.cb >> 1, fill);
    }
  }
  for (int s = s_new + lane; s < fill; s += 32) {
    if (a.hh) a.hh[(int64_t(blk) * ps + s) * a.H + h] = 0;
    if (a.ret_pos) {
      const int cpos = a.ret_cnt[b * a.H + h] + (start + s - L_old);
      if (cpos < 0 || cpos >= a.ret_cap) flag(a.status, SA_DEV_OVERFLOW);
      else a.ret_pos[(int64_t(b) * a.H + h) * a.ret_cap + cpos] = start + s;
    }
  }
}

// Warp `u`: a chunk of the query heads of one token.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void query_unit(const RopeArgs& a, int u) {
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const int t = u / a.q_chunks, h0 = (u % a.q_chunks) * a.q_chunk, h1 = min(a.H_q, h0 + a.q_chunk);
  const Lane<kInter> ln(a, lane % LPR);
  const uint16_t* qi = static_cast<const uint16_t*>(a.q_in) + t * a.q_stride;
  uint16_t* qo = static_cast<uint16_t*>(a.q_out) + int64_t(t) * a.H_q * D;
  uint2 x[kBatch];
  auto fetch = [&](int h) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int hh = h + j * RPW + sub;
      x[j] = hh < h1 ? ln.load(qi + hh * D) : make_uint2(0u, 0u);
    }
  };
  fetch(h0);
  const float4 w = weights<T>(ln, a.q_weight);
  // the token's request: the first whose rows end behind t
  int b = 0, c0 = 0, c1 = 0, L = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
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
  const Turn g = ln.angles(a, t, L_old + t - c0);
  for (int h = h0; h < h1; h += kBatch * RPW) {
    uint2 y[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) y[j] = transform<T, D, kInter>(ln, x[j], g, a.q_weight != nullptr, w, a.eps);
    if (h + kBatch * RPW < h1) fetch(h + kBatch * RPW);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int hh = h + j * RPW + sub;
      if (hh < h1) ln.store(qo + hh * D, y[j]);
    }
  }
}

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  const int k_blocks = (a.k_units + kWarps - 1) / kWarps;
  const int warp = threadIdx.x >> 5;
  if (int(blockIdx.x) < k_blocks) {
    const int u = blockIdx.x * kWarps + warp;
    if (u < a.k_units) key_unit<T, D, kInter>(a, u);
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
  auto k = inter ? rope_append_kernel<T, D, true> : rope_append_kernel<T, D, false>;
  return launch_ex(k, dim3(blocks), dim3(kThreads), 0, s, false, 1, a);
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
  if (!rope || !k_new || !v_new || !new_cu || num_tokens < 0 || max_new_per_req < 0) return SA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (q && num_q_heads <= 0)) return SA_ERR_INVALID_ARG;
  if ((ret_pos == nullptr) != (ret_cnt == nullptr) || (ret_pos && ret_cap <= 0)) return SA_ERR_INVALID_ARG;
  if (cache->kstd && !cache->meta) return SA_ERR_INVALID_ARG;
  const int D = cache->head_dim, H = cache->num_kv_heads;
  if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 4) return SA_ERR_INVALID_ARG;
  if (rope->rot_dim && (!rope->table || rope->max_pos <= 0)) return SA_ERR_INVALID_ARG;
  if (rope->num_axes < 1 || rope->num_axes > 4 || (rope->num_axes > 1 && !rope->positions)) return SA_ERR_INVALID_ARG;
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
  const int64_t k_units = int64_t(batch->batch) * a.pages * H;
  // query heads per warp: few where tokens are few, up to 32 where one read of the angles serves more heads
  a.q_chunk = 4;
  const int64_t full = int64_t(sm_count()) * 64;
  while (q && a.q_chunk < 32 && a.q_chunk < num_q_heads && int64_t(num_tokens) * num_q_heads / (2 * a.q_chunk) >= full)
    a.q_chunk *= 2;
  a.q_chunks = q ? (num_q_heads + a.q_chunk - 1) / a.q_chunk : 0;
  const int64_t q_units = int64_t(num_tokens) * a.q_chunks;
  if (k_units > 0x7fffff00 || q_units > 0x7fffff00) return SA_ERR_UNSUPPORTED;
  a.k_units = int(k_units);
  const unsigned blocks = unsigned((k_units + kWarps - 1) / kWarps + (q_units + kWarps - 1) / kWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SA_BF16, inter = rope->interleaved != 0;
  const cudaError_t e = D == 128 ? (bf ? launch<__nv_bfloat16, 128>(a, blocks, inter, s) : launch<__half, 128>(a, blocks, inter, s))
                                 : (bf ? launch<__nv_bfloat16, 64>(a, blocks, inter, s) : launch<__half, 64>(a, blocks, inter, s));
  if (e != cudaSuccess) return SA_ERR_CUDA;
  if (advanced && !ret_cnt) return SA_OK;
  const unsigned ab = unsigned((batch->batch + 127) / 128);
  return launch_ex(rope_advance_kernel, dim3(ab), dim3(128), 0, s, true, 1, a) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}
