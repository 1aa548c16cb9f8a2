// Element-wise key statistics of one page column: the exactly rounded mean and
// the population standard deviation, shared by the append kernels.
#pragma once

#include "common.cuh"

namespace sa {

constexpr int kRowBatch = 16;     // rows of a page loaded per batch (independent loads)

// exact float32 sum step: s += x, clears `exact` if the addition rounded
__device__ __forceinline__ void two_sum(float& s, float x, bool& exact) {
  const float t = s + x;
  const float bb = t - s;
  const float err = (s - (t - bb)) + (x - bb);
  exact &= (err == 0.f);
  s = t;
}

// Round S / f (S exact) once to the element type; false if float32 cannot decide.
template <typename T>
__device__ __forceinline__ bool mean_f32(float S, int f, uint16_t& out) {
  using E = Elem<T>;
  const float aS = fabsf(S);
  if (S == 0.f) { out = E::from_f(S); return true; }
  if (!(aS >= 0x1p-100f)) return false;                       // float32 underflow risk
  if ((f & (f - 1)) == 0) {                                    // power of two: exact scaling
    const float q = S * (1.0f / float(f));
    if (E::midpoint(q) < 0) return false;
    out = E::from_f(q);
    return true;
  }
  const float q = S / float(f);                                // correctly rounded
  const int mid = E::midpoint(q);
  if (mid < 0) return false;
  if (mid == 0) { out = E::from_f(q); return true; }
  const float prod = q * float(f);                             // exact: few significant bits
  if (S == prod) { out = E::from_f(q); return true; }          // a true tie: to even
  const uint16_t lo = E::from_f_rz(fabsf(q));                  // smaller-magnitude neighbour
  const uint16_t mag = fabsf(S) > fabsf(prod) ? uint16_t(lo + 1) : lo;
  out = uint16_t(mag | (S < 0.f ? 0x8000u : 0u));
  return true;
}

// k_std of one column over its f rows: the population std sqrt((1/f) sum
// (x - mean)^2) around the exact mean, rounded once to the element type.
// float32 two-pass: with m the float32 mean (error dm <= (f + 1) eps sum|x| / f)
// the computed sum of squared deviations q differs from the true one by at
// most f dm^2 (the centre's error enters squared, the deviations summing to
// zero) plus (f + 3) eps q of rounding, so the std's relative error is below
// half that (+ eps). The float32 result is kept when every value within twice
// that bound rounds to the same element; otherwise float64 decides. x: the
// column's values (half kHi of each word), f <= kRowBatch of them.
template <typename T, bool kHi>
__device__ __forceinline__ uint16_t std_column(const uint32_t (&w)[kRowBatch], int fill) {
  using E = Elem<T>;
  constexpr float eps = 0x1p-24f;
  float sum = 0.f, sabs = 0.f, xmin = INFINITY, xmax = -INFINITY;
#pragma unroll
  for (int s = 0; s < kRowBatch; ++s) {
    if (s < fill) {
      const float x = kHi ? E::hi(w[s]) : E::lo(w[s]);
      sum += x;
      sabs += fabsf(x);
      xmin = fminf(xmin, x);
      xmax = fmaxf(xmax, x);
    }
  }
  if (xmin == xmax) return E::from_f(0.f);                 // every row equal
  const float f = float(fill);
  const float m = sum / f;
  float q = 0.f;
#pragma unroll
  for (int s = 0; s < kRowBatch; ++s) {
    if (s < fill) {
      const float d = (kHi ? E::hi(w[s]) : E::lo(w[s])) - m;
      q = fmaf(d, d, q);
    }
  }
  const float dm = (f + 1.f) * eps * sabs / f;
  const float rel = 0.5f * (f * dm * dm / q + (f + 3.f) * eps) + eps;
  const float sd = sqrtf(q / f);
  if (q > 0x1p-100f && rel < 0x1p-12f) {
    const uint16_t lo = E::from_f(sd * (1.f - 2.f * rel)), hi = E::from_f(sd * (1.f + 2.f * rel));
    if (lo == hi) return lo;
  }
  double s64 = 0.0;                                        // undecided: float64
#pragma unroll
  for (int s = 0; s < kRowBatch; ++s)
    if (s < fill) s64 += double(kHi ? E::hi(w[s]) : E::lo(w[s]));
  const double m64 = s64 / double(fill);
  double q64 = 0.0;
#pragma unroll
  for (int s = 0; s < kRowBatch; ++s) {
    if (s < fill) {
      const double d = double(kHi ? E::hi(w[s]) : E::lo(w[s])) - m64;
      q64 = fma(d, d, q64);
    }
  }
  return E::from_f64(sqrt(q64 / double(fill)));
}

// float64 k_std of one column over more rows than one batch (pages above 16 tokens)
template <typename T, bool kHi>
__device__ uint16_t std_column_long(const uint32_t* rows, int C, int fill) {
  using E = Elem<T>;
  double s64 = 0.0;
  for (int s = 0; s < fill; ++s) s64 += double(kHi ? E::hi(rows[int64_t(s) * C]) : E::lo(rows[int64_t(s) * C]));
  const double m64 = s64 / double(fill);
  double q64 = 0.0;
  for (int s = 0; s < fill; ++s) {
    const double d = double(kHi ? E::hi(rows[int64_t(s) * C]) : E::lo(rows[int64_t(s) * C])) - m64;
    q64 = fma(d, d, q64);
  }
  return E::from_f64(sqrt(q64 / double(fill)));
}

// k_std of the column pair [2c, 2c+1] of (block, head), C = head_dim / 2 pairs a row; the f rows, new ones
// included, are this thread's own pool writes or untouched. Only for caches
// that keep k_std; kept out of line so the common path keeps its registers.
template <typename T>
__device__ __noinline__ void page_std_pair(void* kstd, const uint32_t* kp, int64_t tile, int fill, int blk,
                                           int H, int C, int h, int c) {
  const uint32_t* rows = kp + tile * C + c;
  uint16_t v0, v1;
  if (fill <= kRowBatch) {
    uint32_t w[kRowBatch];
#pragma unroll
    for (int s = 0; s < kRowBatch; ++s) w[s] = s < fill ? rows[int64_t(s) * C] : 0u;   // one batch of loads
    v0 = std_column<T, false>(w, fill);
    v1 = std_column<T, true>(w, fill);
  } else {
    v0 = std_column_long<T, false>(rows, C, fill);
    v1 = std_column_long<T, true>(rows, C, fill);
  }
  static_cast<uint32_t*>(kstd)[(int64_t(blk) * H + h) * C + c] = uint32_t(v0) | (uint32_t(v1) << 16);
}

}  // namespace sa
