// One row of the windowed attention from its visible tokens alone, by a warp on the
// CUDA cores: for rows that a tensor-core kernel left with a result that is not
// finite.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace skv {

// The row's result is in `out` already.  What of it is not finite may come from
//   - a visible value that is a NaN or an infinity: it stands;
//   - a hidden one of a shared tile, which entered a product with weight 0;
//   - sums of large weighted values that overflowed, where their mean does not;
//   - a sum of weights that is 0, of huge logits (reference_of).
// The first is looked for beforehand, so that inputs with NaNs cost one pass over
// the values at most; the others are computed again, weights in units of 2^24 (as
// many tokens as a sequence can have).
template <typename T, int D>
__device__ __noinline__ void window_row_again(const WindowArgs& a, int s, int h, int i) {
  constexpr int E = D / 32;  // channels of a lane
  constexpr float kLess = 0x1p-24f;
  const int lane = threadIdx.x & 31, g = h / (a.Hq / a.Hkv);
  const long long row = (((long long)s * a.n + i) * a.Hq + h) * D + lane * E;
  const long long kv0 = ((long long)s * a.n * a.Hkv + g) * D + lane * E, step = (long long)a.Hkv * D;
  T* out = static_cast<T*>(a.out) + row;
  const T* k = static_cast<const T*>(a.k) + kv0;
  const T* v = static_cast<const T*>(a.v) + kv0;
  // tokens [0, sinks) and [first, i]
  const int first = max(0, i - a.window + 1), sinks = min(a.n_sink, first);
  const int count = sinks + i + 1 - first;
  auto token = [&](int x) { return x < sinks ? x : x - sinks + first; };

  __syncwarp();  // (lanes of the warp wrote `out`)
  constexpr int kBatch = 8;  // tokens whose loads are in flight together
  auto load = [&](float (&y)[kBatch][E], const T* from, int x0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int e = 0; e < E; ++e) y[b][e] = to_f(from[token(min(x0 + b, count - 1)) * step + e]);
  };

  bool bad[E], some = true;
#pragma unroll
  for (int e = 0; e < E; ++e) bad[e] = !(fabsf(to_f(out[e])) < INFINITY);
  for (int x0 = 0; some && x0 < count; x0 += kBatch) {
    float y[kBatch][E];
    load(y, v, x0);
    some = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) bad[e] &= fabsf(y[b][e]) < INFINITY;
      some |= bad[e];
    }
    some = __any_sync(0xffffffffu, some);
  }
  if (!some) return;

  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(static_cast<const T*>(a.q)[row + e]);
    o[e] = 0.f;
  }
  for (int x0 = 0; x0 < count; x0 += kBatch) {
    float y[kBatch][E], t[kBatch];
    load(y, k, x0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      t[b] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) t[b] = fmaf(qv[e], y[b][e], t[b]);
    }
    load(y, v, x0);
#pragma unroll
    for (int off = 16; off; off >>= 1)
#pragma unroll
      for (int b = 0; b < kBatch; ++b) t[b] += __shfl_xor_sync(0xffffffffu, t[b], off);
    float nm = m;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      t[b] = x0 + b < count ? t[b] * a.scale_log2 : -INFINITY;
      nm = fmaxf(nm, t[b]);
    }
    const float ref = nm == -INFINITY ? 0.f : nm, f = exp2f(m - ref);
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float p = exp2f(t[b] - ref);
      l += p;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x0 + b < count) o[e] = fmaf(p * kLess, y[b][e], o[e]);
    }
    m = nm;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f<T>(o[e] / l * (1.f / kLess));
  if (lane == 0 && a.lse) a.lse[((long long)s * a.Hq + h) * a.n + i] = (m + log2f(l)) * kLn2;
}

}  // namespace skv
