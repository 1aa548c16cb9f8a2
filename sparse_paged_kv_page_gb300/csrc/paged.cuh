// Pieces shared by the attention kernels over the whole paged cache
// (sa_paged_decode, sa_paged_prefill): the visible range of a query, shared-memory
// tiles of 16 rows, and the search for a work item's request.
#pragma once

#include "common.cuh"
#include "host.h"

namespace sa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Tiles of R positions that queries at positions [first, last] see of a cache of
// `len` readable tokens: the n_sink first ones and the `window` most recent ones
// (window <= 0: all). Tile t < sink_tiles is tile t of the sequence, the others
// continue at win_tile; the two ranges are disjoint.
template <int R>
struct Span {
  int sink_tiles, win_tile, tiles;
  __device__ __forceinline__ Span(int first, int last, int len, int window, int n_sink) {
    const int end = max(0, min(last + 1, len));
    const int w0 = window > 0 ? max(0, min(first - window + 1, end)) : 0;
    sink_tiles = (min(n_sink, w0) + R - 1) / R;
    win_tile = w0 / R;
    if (win_tile <= sink_tiles) sink_tiles = win_tile = 0;
    tiles = sink_tiles + (end + R - 1) / R - win_tile;
  }
  __device__ __forceinline__ int start(int t) const { return (t < sink_tiles ? t : t - sink_tiles + win_tile) * R; }
};

// A workspace of either call begins with the counters of units that are cut into parts, one for each CTA that runs at
// once: a region of the same size whatever the call's, so that no partial result of one call lies where another call,
// or the other operator, counts.
constexpr int kTicketsPerSm = 2;
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline size_t ticket_bytes() { return align256(size_t(kTicketsPerSm) * sm_count() * sizeof(int32_t)); }

// One more part of a unit is in memory: parts counted before it. Called by one
// thread after the block's barrier; publishes the block's writes, and makes the
// other parts' visible to the block after its next barrier.
__device__ __forceinline__ int ticket(int32_t* counter) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

// 16 rows x D columns of 2-byte elements in shared memory: 64-column halves of
// 16 x 128 bytes, 16-byte chunk c of row r at chunk c ^ (r & 7), the TMA engine's
// 128-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t swz16(int row, int chunk) {
  return uint32_t((chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// 3-D and 4-D tiled TMA loads (tensor map in kernel-parameter space), completion on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// Work item `idx` of a ragged batch in which request b has ceil(n_b / per) items
// (n_b = new_cu[b+1] - new_cu[b]): its request, its place there, the request's first
// row, rows and length. All lanes of a warp call it. False behind the last item.
__device__ __forceinline__ bool find_item(const int32_t* new_cu, const int32_t* seq_lens, int batch, int per, int idx,
                                          int& b, int& i, int& c0, int& n, int& L) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < batch; b0 += 128) {            // 128 requests a round of loads
    int first[4], rows[4], len[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = min(b0 + 32 * j + lane, batch - 1);
      first[j] = new_cu[at], rows[j] = new_cu[at + 1] - first[j], len[j] = seq_lens[at];
      if (b0 + 32 * j + lane >= batch) rows[j] = 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int items = rows[j] > 0 ? (rows[j] + per - 1) / per : 0;
      int x = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      const int k = __popc(__ballot_sync(kFull, before + x <= idx));
      if (k < 32) {
        i = idx - before - (__shfl_sync(kFull, x, k) - __shfl_sync(kFull, items, k));
        b = b0 + 32 * j + k;
        c0 = __shfl_sync(kFull, first[j], k), n = __shfl_sync(kFull, rows[j], k), L = __shfl_sync(kFull, len[j], k);
        return true;
      }
      before += __shfl_sync(kFull, x, 31);
    }
  }
  return false;
}

}  // namespace sa
