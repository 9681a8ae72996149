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

// A tile of query rows takes the cache tokens that all of its rows see: those below
// n_sink and those from `tile_from` (the window of the tile's last text token) on.  Its
// other rows also see tokens before that, from `row_from` on; the kernels join
// those row by row with the text tokens, since what a tile keeps for all of its
// rows (references and exponents of keys and values) must not depend on a token
// that the mask hides from one of them.
__device__ __forceinline__ int row_from(const WindowArgs& a, int L, int i) {
  if (!a.window) return 0;
  const long long from = (long long)L + i - a.window + 1;
  return from <= 0 ? 0 : from >= L ? L : (int)from;
}
__device__ __forceinline__ int tile_from(const WindowArgs& a, int L, int i_last) { return row_from(a, L, i_last); }
// The last text token of row tile `tile` (R rows, G a text token).
__device__ __forceinline__ int tile_last(int tile, int rows, int R, int G) { return (min((tile + 1) * rows, R) - 1) / G; }

}  // namespace skv
