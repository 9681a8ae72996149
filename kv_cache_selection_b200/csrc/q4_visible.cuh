// The 32-token blocks of a 4-bit cache that a call's rows see.
#pragma once

#include "common.cuh"
#include "q4_cache.cuh"

namespace skv {

// Blocks of a stream that any row sees: [0, sinks) and [window, n).
struct Visible {
  int L, sinks, window, n;
  __device__ __forceinline__ int count() const { return sinks + n - window; }
  __device__ __forceinline__ int block(int v) const { return v < sinks ? v : v - sinks + window; }
};
__device__ __forceinline__ Visible visible_of(const WindowArgs& a, int s) {
  Visible x;
  x.L = q4_length(a, s);
  x.n = (x.L + kQ4Tokens - 1) / kQ4Tokens;
  x.sinks = 0;
  x.window = 0;
  if (a.window) {
    x.sinks = (min(a.n_sink, x.L) + kQ4Tokens - 1) / kQ4Tokens;
    const long long lo = (long long)x.L - a.window + 1;  // first token of row 0's window
    x.window = lo >= x.L ? x.n : lo > 0 ? (int)(lo / kQ4Tokens) : 0;
    x.window = max(x.window, x.sinks);
  }
  return x;
}

}  // namespace skv
