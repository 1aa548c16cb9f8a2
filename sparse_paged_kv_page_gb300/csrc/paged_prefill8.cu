// sa_paged_prefill8: the C entry, and the pages that calls with many products run on (kernels in
// paged_prefill.cuh, few rows in paged_decode8.cuh).
//
// A product of the tensor cores needs 16-bit operands in shared memory. A CTA that turns its own
// tiles of codes into them does it once for its 256 rows: a prompt of n tokens turns each of its
// codes n G / 512 times on the mean, beside a softmax that wants the same issue slots. One pass
// over HBM before (3 bytes read or written a code, here one page and head a block) does it once,
// and the kernel over 16-bit pages then runs as it does for sa_paged_prefill, on pages of 128
// whatever the cache's are: 16384 tokens, 32 / 8 heads of 128, 1270 - 1310 us, 1.68 - 1.73 PFLOP/s
// (a CTA's own turning 1550; over a 16-bit cache with pages of 16, 1315 - 1330), heads of 64 941
// (2035; 1161); a chunk of 2048 tokens x 64 heads behind 64000 in a workspace with room 2370
// (2970; 2510). The two decide on the device which of them runs: lengths are known there alone.
#include "paged_prefill.cuh"

namespace sa {
namespace {

struct LayArgs {
  const uint8_t* pool[2];
  const uint8_t* scale;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* new_cu;
  int32_t* turn;
  int32_t* table;
  uint16_t* out[2];
  int H, ps_shift, num_blocks, bt_stride, batch, pages, window, n_sink, Hq;
};

constexpr int kLayThreads = 256;

// Pages blockIdx.x, blockIdx.x + gridDim.x, .. of 128 tokens and KV head blockIdx.y of the tokens of all requests, one after the
// other, as 16-bit values, where some query sees one of them; their places in their requests' tables. turn[0]: all pages have
// room and are worth it; turn[1]: some token has no place in the cache (then the kernel that reads codes runs, which says what
// is wrong).
template <typename T, int D>
__global__ void __launch_bounds__(kLayThreads) lay8_kernel(const __grid_constant__ LayArgs a) {
  constexpr int kChunks = D / 8, kRows = kLayThreads / kChunks, kSteps = 128 / kRows;
  __shared__ int s_b, s_page;
  __shared__ int64_t s_row[128];
  const int h = blockIdx.y, ps = 1 << a.ps_shift, lane = threadIdx.x & 31;
  int from = 0, from_before = 0;                           // requests that the search goes on from, pages before them
  for (int page = blockIdx.x; page < a.pages; page += gridDim.x) {
    const bool all_of = page == int(blockIdx.x);           // the first time all requests are looked at
    __syncthreads();                                       // the page before is done
    if (threadIdx.x < 32) {
      int before = from_before, b = -1, at = 0;
      bool bad = false;
      float pairs = 0.f, tokens = 0.f;
      for (int b0 = from; b0 < a.batch && (all_of || b < 0); b0 += 32) {
        const bool there = b0 + lane < a.batch;
        const int L = there ? a.seq_lens[b0 + lane] : 0, n_new = there ? a.new_cu[b0 + lane + 1] - a.new_cu[b0 + lane] : 0;
        bad = bad || L < 0 || (L > 0 && ((L - 1) >> a.ps_shift) >= a.bt_stride);
        if (n_new > 0) {
          const float all = float(L) - 0.5f * float(n_new), seen = a.window > 0 ? float(a.window) + float(a.n_sink) : all;
          pairs += float(n_new) * fminf(all, seen);
          tokens += fminf(float(L), seen + float(n_new));
        }
        const int n = L > 0 ? ((L - 1) >> 7) + 1 : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, sum, o);
          if (lane >= o) sum = min(sum + y, 1 << 28);      // (garbage lengths)
        }
        const int k = __popc(__ballot_sync(kFull, before + sum <= page));
        if (b < 0 && k < 32) {
          b = b0 + k, at = page - before - (__shfl_sync(kFull, sum, k) - __shfl_sync(kFull, n, k));
          from = b0, from_before = before;
        }
        before = min(before + __shfl_sync(kFull, sum, 31), 1 << 28);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) pairs += __shfl_xor_sync(kFull, pairs, o), tokens += __shfl_xor_sync(kFull, tokens, o);
      if (all_of) {
        bad = __any_sync(kFull, bad);
        const bool go = before <= a.pages && worth_pages(pairs, tokens, a.Hq, a.H, D);
        if (page == 0 && h == 0 && lane == 0) {
          a.turn[0] = go ? 1 : 0;
          if (bad) a.turn[1] = 1;
        }
        if (!go || bad) b = -1;
      }
      if (lane == 0) s_b = b, s_page = at;
    }
    __syncthreads();
    const int b = s_b, first = s_page * 128;
    if (b < 0 || b >= a.batch) return;                     // no such page: none behind it either
    const int L = a.seq_lens[b], n = a.new_cu[b + 1] - a.new_cu[b];
    const int64_t w0 = a.window > 0 ? int64_t(L) - n - a.window + 1 : 0;   // the first token within the window of the first query
    if (n <= 0 || (first + 128 <= w0 && first >= a.n_sink)) continue;
    if (h == 0 && threadIdx.x == 0) a.table[int64_t(b) * a.pages + s_page] = page;
    if (threadIdx.x < 128) {
      const int p = first + threadIdx.x;
      int64_t row = -1;
      if (p < L && (p >= w0 || p < a.n_sink)) {
        const int blk = a.bt[int64_t(b) * a.bt_stride + (p >> a.ps_shift)];
        if (blk < 0 || blk >= a.num_blocks) a.turn[1] = 1;
        else row = ((int64_t(blk) * a.H + h) << a.ps_shift) + (p & (ps - 1));
      }
      s_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int c = threadIdx.x % kChunks;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint16_t* out = a.out[kv] + (int64_t(page) * a.H + h) * 128 * D;
#pragma unroll
      for (int i0 = 0; i0 < kSteps; i0 += 4) {
        uint2 codes[4];
        uint32_t scale[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t row = s_row[(i0 + u) * kRows + threadIdx.x / kChunks];
          codes[u] = make_uint2(0u, 0u), scale[u] = 127;
          if (row < 0) continue;
          codes[u] = *reinterpret_cast<const uint2*>(a.pool[kv] + row * D + c * 8);
          scale[u] = a.scale[((2 * (row >> a.ps_shift) + kv) << a.ps_shift) + (row & (ps - 1))];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const Factor<T> f(scale[u]);
          uint4 w;
          values4<T, true>(codes[u].x, f, w.x, w.y);
          values4<T, true>(codes[u].y, f, w.z, w.w);
          *reinterpret_cast<uint4*>(out + ((i0 + u) * kRows + threadIdx.x / kChunks) * D + c * 8) = w;
        }
      }
    }
  }
}

// The kernel over 16-bit pages of 128 tokens.
template <typename T, int D>
sa_status launch_laid(const PagedPrefillArgs& a, const LayArgs& lay, const sa_cache& pages, const void* q, cudaStream_t s) {
  static int smem_set[64];
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (!make_query_map(&mq, q, D, a.H_q, a.T, a.G, 128 / a.G) || !make_group_map(&mk, pages.k, &pages, 16) ||
      !make_group_map(&mv, pages.v, &pages, 16))
    return SA_ERR_CUDA;
  if (launch_ex(lay8_kernel<T, D>, dim3(min(lay.pages, (8 * sm_count() + lay.H - 1) / lay.H), lay.H), dim3(kLayThreads), 0, s, false, 1, lay) != cudaSuccess) return SA_ERR_CUDA;
  return launch<T, D, true, false>(a, s, mq, mk, mv, smem_set);
}

// Codes into pages and the kernel over those, where they have room (else neither does anything, and a.turn says so to the
// kernel that is launched behind: that over codes).
sa_status laid_call(const sa_cache8* cache, const sa_batch* batch, const void* q, PagedPrefillArgs& a, void* workspace,
                    size_t workspace_bytes, size_t base, cudaStream_t s) {
  const int D = cache->head_dim, H = cache->num_kv_heads, B = batch->batch;
  const size_t page = size_t(H) * 128 * D * 4, least = laid_layout(base, 0, B, H, D).total;
  int64_t pages = workspace_bytes > least ? int64_t((workspace_bytes - least) / (page + 4 * size_t(B))) : 0;
  const int64_t most = min(int64_t(B) * ((int64_t(batch->bt_stride) * cache->page_size + 127) / 128), int64_t(1) << 22);
  if (pages > most) pages = most;                                   // (no request has more)
  while (pages > 0 && laid_layout(base, pages, B, H, D).total > workspace_bytes) --pages;
  const int64_t seen = a.window > 0 ? int64_t(a.window) + a.n_sink : int64_t(1) << 40;
  // pool rows are below 2^31, blocks of a launch in y below 65536
  if (pages <= 0 || !worth_pages(a.T, pages * 128, B, seen, a.H_q, H, D) || pages * H * 128 >= (int64_t(1) << 31) || H > 65535) return SA_OK;
  const Laid w = laid_layout(base, pages, B, H, D);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LayArgs lay = {};
  lay.pool[0] = static_cast<const uint8_t*>(cache->k); lay.pool[1] = static_cast<const uint8_t*>(cache->v);
  lay.scale = cache->scale; lay.bt = batch->block_table; lay.seq_lens = batch->seq_lens; lay.new_cu = a.new_cu;
  lay.turn = reinterpret_cast<int32_t*>(ws + align256(base)); lay.table = reinterpret_cast<int32_t*>(ws + w.table);
  lay.out[0] = reinterpret_cast<uint16_t*>(ws + w.k); lay.out[1] = reinterpret_cast<uint16_t*>(ws + w.v);
  lay.H = H; lay.ps_shift = log2i(cache->page_size); lay.num_blocks = cache->num_blocks; lay.bt_stride = batch->bt_stride;
  lay.batch = B; lay.pages = int(pages); lay.window = a.window; lay.n_sink = a.n_sink; lay.Hq = a.H_q;
  if (cudaMemsetAsync(lay.turn, 0, 2 * sizeof(int32_t), s) != cudaSuccess) return SA_ERR_CUDA;
  const sa_cache c = {lay.out[0], lay.out[1], nullptr, cache->dtype, int32_t(pages), H, 128, D, nullptr};
  PagedPrefillArgs x = a;
  x.k = c.k; x.v = c.v; x.bt = lay.table; x.bt_stride = int(pages); x.num_blocks = int(pages); x.ps_shift = 7;
  x.turn = lay.turn;
  x.window = x.window < pages * 128 ? x.window : 0;
  a.turn = lay.turn;
  a.otherwise = 1;
  const bool bf = cache->dtype == SA_BF16;
  if (D == 128) return bf ? launch_laid<__nv_bfloat16, 128>(x, lay, c, q, s) : launch_laid<__half, 128>(x, lay, c, q, s);
  return bf ? launch_laid<__nv_bfloat16, 64>(x, lay, c, q, s) : launch_laid<__half, 64>(x, lay, c, q, s);
}

}  // namespace
}  // namespace sa

extern "C" size_t sa_paged_prefill8_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t num_q_heads,
                                                  int32_t head_dim, int32_t num_tokens) {
  using namespace sa;
  if (prefill_workspace(batch, num_kv_heads, num_q_heads, head_dim, num_tokens) == 0) return 0;
  const int G = num_q_heads / num_kv_heads;
  if (G > 16) return prefill_workspace(batch, num_kv_heads, num_q_heads, head_dim, num_tokens);
  const size_t n = few_workspace(num_tokens, batch, G, head_dim, num_kv_heads);
  if (!worth_pages(num_tokens, num_tokens, batch, int64_t(1) << 40, num_q_heads, num_kv_heads, head_dim)) return n;
  return laid_layout(n, int64_t(num_tokens) / 128 + batch, batch, num_kv_heads, head_dim).total;
}

extern "C" sa_status sa_paged_prefill8(const sa_cache8* cache, const sa_batch* batch, const void* q, int32_t num_q_heads,
                                      const int32_t* new_cu, int32_t num_tokens, int32_t window, int32_t n_sink,
                                      float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                      int32_t* dev_status, void* stream) {
  using namespace sa;
  sa_cache sizes;
  const sa_status st = check_cache8(cache, &sizes);
  if (st != SA_OK) return st;
  return prefill_call<true>(&sizes, cache, batch, q, num_q_heads, new_cu, num_tokens, window, n_sink, scale, out,
                            lse, workspace, workspace_bytes, dev_status, stream, laid_call);
}
