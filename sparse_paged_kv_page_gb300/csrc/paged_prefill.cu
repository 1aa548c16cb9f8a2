// sa_paged_prefill: causal softmax attention of new tokens (a prompt, a chunk of
// one, a few drafted tokens) over the paged cache that already holds them.
#include "common.cuh"
#include "host.h"
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16 * kWarps;      // packed rows (token, query head of the group) of a CTA
constexpr int kKeys = 32;               // positions per step

struct PagedPrefillArgs {
  const void* k;
  const void* v;
  const void* q;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* new_cu;
  void* out;
  float* lse;
  int32_t* status;
  int H_kv, H_q, G, ps_shift, num_blocks, bt_stride, batch, T, window, n_sink;
  float scale_log2;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_prefill_kernel(const __grid_constant__ PagedPrefillArgs a) {
  using E = Elem<T>;
  constexpr int kTileBytes = 16 * D * 2;
  __shared__ __align__(1024) uint8_t s_kv[2][2][kKeys / 16][kTileBytes];   // [stage][K, V][tile]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int G = a.G, per = kRows / G, pss = a.ps_shift;
  const int h = blockIdx.x % a.H_kv, idx = gridDim.x / a.H_kv - 1 - blockIdx.x / a.H_kv;
  int b, item;
  if (!find_item(a.new_cu, a.batch, per, idx, b, item)) return;
  const int c0 = a.new_cu[b], n = a.new_cu[b + 1] - c0, L = a.seq_lens[b];
  const int cap = int(min(int64_t(a.bt_stride) << pss, int64_t(0x7fffffff)));
  if (threadIdx.x == 0 && item == 0 && h == 0) {
    if (c0 < 0 || c0 + n > a.T || L < n) flag(a.status, SA_DEV_BAD_COUNT);
    if (L > cap) flag(a.status, SA_DEV_OVERFLOW);
  }
  if (c0 < 0 || int64_t(c0) + n > a.T) return;
  const int t0 = item * per, nt = min(per, n - t0);           // tokens of this CTA
  const int first = L - n + t0, last = first + nt - 1;        // their positions
  const int len = min(max(L, 0), cap);
  const Span<kKeys> sp(first, last, len, a.window, a.n_sink);

  // rows of this thread: r0 = warp * 16 + g and r0 + 8
  int pos[2];
  int64_t row[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int x = warp * 16 + g + 8 * r, t = x / G;
    const bool in = t < nt;
    pos[r] = in ? first + t : -1;
    row[r] = in ? (int64_t(c0 + t0 + t) * a.H_q + int64_t(h) * G + x % G) : -1;
  }
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const int x0 = (kk * 16 + 2 * tq) >> 1;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t* qp = static_cast<const uint32_t*>(a.q) + row[r] * (D / 2);
      qa[kk][r] = row[r] >= 0 ? qp[x0] : 0u;
      qa[kk][2 + r] = row[r] >= 0 ? qp[x0 + 4] : 0u;
    }
  }
  const int32_t* btb = a.bt + int64_t(b) * a.bt_stride;
  __shared__ uint32_t s_ok[2][kThreads / 32];
  // copies of step i: thread (row, part) -> 16-byte chunks of one K and V row
  constexpr int kParts = kThreads / kKeys;
  auto issue = [&](int i) {
    if (i < sp.tiles) {
      const int r = threadIdx.x % kKeys, part = threadIdx.x / kKeys, j = sp.start(i) + r;
      int blk = -1;
      // rows that no query of the CTA sees could hold anything (NaN): zeros instead
      if (j < len && j <= last && (a.window == 0 || j > first - a.window || j < a.n_sink)) {
        blk = btb[j >> pss];
        if (blk < 0 || blk >= a.num_blocks) {
          flag(a.status, SA_DEV_BAD_BLOCK);
          blk = -1;
        }
      }
      if (part == 0) s_ok[i & 1][0] = __ballot_sync(kFull, blk >= 0);
      const int64_t off = (((int64_t(blk) * a.H_kv + h) << pss) + (j & ((1 << pss) - 1))) * D;
      const uint32_t sk = smem_u32(&s_kv[i & 1][0][r >> 4][0]), sv = smem_u32(&s_kv[i & 1][1][r >> 4][0]);
#pragma unroll
      for (int c = part; c < D / 8; c += kParts) {
        const uint32_t d = swz16<D>(r & 15, c);
        cp_async_16(sk + d, blk >= 0 ? static_cast<const T*>(a.k) + off + c * 8 : a.k, blk >= 0 ? 16 : 0);
        cp_async_16(sv + d, blk >= 0 ? static_cast<const T*>(a.v) + off + c * 8 : a.v, blk >= 0 ? 16 : 0);
      }
    }
    cp_async_commit();
  };
  float o[D / 8][4];
#pragma unroll
  for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
  float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
  issue(0);
  for (int i = 0; i < sp.tiles; ++i) {
    issue(i + 1);
    cp_async_wait<1>();
    __syncthreads();
    const uint32_t okm = s_ok[i & 1][0];
    const int j0 = sp.start(i);
    const int mi = lane >> 3, rr = lane & 7;
    float c[kKeys / 8][4];
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x) c[x][0] = c[x][1] = c[x][2] = c[x][3] = 0.f;
#pragma unroll
    for (int t = 0; t < kKeys / 16; ++t) {
      const uint32_t sk = smem_u32(&s_kv[i & 1][0][t][0]);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t r[4];
        ldmatrix_x4(r, sk + swz16<D>((mi >> 1) * 8 + rr, kk * 2 + (mi & 1)));
        E::mma(c[2 * t], qa[kk], r[0], r[1]);
        E::mma(c[2 * t + 1], qa[kk], r[2], r[3]);
      }
    }
    float pmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int jj = x * 8 + 2 * tq + (e & 1), j = j0 + jj, r = e >> 1;
        const bool ok = ((okm >> jj) & 1u) && j <= pos[r] &&
                        (a.window == 0 || j > pos[r] - a.window || j < a.n_sink);
        c[x][e] = ok ? c[x][e] * a.scale_log2 : -INFINITY;
        pmax[r] = fmaxf(pmax[r], c[x][e]);
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
      for (int x = 0; x < kKeys / 8; ++x) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = ex2_approx(c[x][2 * r + e] - m_use);
          c[x][2 * r + e] = p;
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
#pragma unroll
    for (int t = 0; t < kKeys / 16; ++t) {
      const uint32_t sv = smem_u32(&s_kv[i & 1][1][t][0]);
      const uint32_t pa[4] = {E::pack(c[2 * t][0], c[2 * t][1]), E::pack(c[2 * t][2], c[2 * t][3]),
                              E::pack(c[2 * t + 1][0], c[2 * t + 1][1]), E::pack(c[2 * t + 1][2], c[2 * t + 1][3])};
#pragma unroll
      for (int nd = 0; nd < D / 16; ++nd) {
        uint32_t r[4];
        ldmatrix_x4_trans(r, sv + swz16<D>((mi & 1) * 8 + rr, 2 * nd + (mi >> 1)));
        E::mma(o[2 * nd], pa, r[0], r[1]);
        E::mma(o[2 * nd + 1], pa, r[2], r[3]);
      }
    }
    __syncthreads();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l_r[r] += __shfl_xor_sync(kFull, l_r[r], 1);
    l_r[r] += __shfl_xor_sync(kFull, l_r[r], 2);
    if (row[r] < 0) continue;
    const float inv = l_r[r] > 0.f ? 1.0f / l_r[r] : 0.f;
    uint32_t* op = static_cast<uint32_t*>(a.out) + row[r] * (D / 2);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) op[x * 4 + tq] = E::pack(o[x][2 * r] * inv, o[x][2 * r + 1] * inv);
    if (a.lse && tq == 0) a.lse[row[r]] = l_r[r] > 0.f ? (m_r[r] + lg2_approx(l_r[r])) * kLn2 : -INFINITY;
  }
}

template <typename T, int D>
sa_status launch(const PagedPrefillArgs& a, unsigned blocks, cudaStream_t s) {
  paged_prefill_kernel<T, D><<<blocks, kThreads, 0, s>>>(a);
  return launch_status();
}

}  // namespace
}  // namespace sa

extern "C" size_t sa_paged_prefill_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads,
                                                  int32_t head_dim, int32_t num_tokens) {
  if (batch <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || head_dim <= 0 || num_tokens < 0 ||
      num_q_heads % num_kv_heads)
    return 0;
  return 256;
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
  a.k = cache->k; a.v = cache->v; a.q = q; a.bt = batch->block_table; a.seq_lens = batch->seq_lens; a.new_cu = new_cu;
  a.out = out; a.lse = lse; a.status = dev_status;
  a.H_kv = H; a.H_q = num_q_heads; a.G = G; a.ps_shift = log2i(cache->page_size); a.num_blocks = cache->num_blocks;
  a.bt_stride = batch->bt_stride; a.batch = batch->batch; a.T = num_tokens; a.window = window; a.n_sink = n_sink;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf(float(D))) * kLog2e;
  // items of kRows / G tokens: at most one partly filled one per request
  const int per = kRows / G;
  const int64_t blocks = (num_tokens / per + int64_t(batch->batch)) * H;
  if (blocks > 0x7fffffff) return SA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = cache->dtype == SA_BF16;
  if (D == 128) return bf ? launch<__nv_bfloat16, 128>(a, unsigned(blocks), s) : launch<__half, 128>(a, unsigned(blocks), s);
  return bf ? launch<__nv_bfloat16, 64>(a, unsigned(blocks), s) : launch<__half, 64>(a, unsigned(blocks), s);
}
