// Causal attention with a sliding window and visible first tokens on the CUDA
// cores, float32 arithmetic, over an optional 4-bit cache followed by the
// call's own tokens.
//
// Query i of stream s stands at position L_s + i (L_s cached tokens).  It sees
// position j <= L_s + i when there is no window, when j > L_s + i - window or
// when j < n_sink; cached positions 0..L_s-1 come from the cache (values
// m + c s, see q4_cache.cuh), the rest from k, v.
#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"

namespace skv {
namespace {

constexpr int kRowsPerWarp = 4;
constexpr int kWarps = 4;
constexpr int kRows = kRowsPerWarp * kWarps;  // query rows of one head per block
constexpr int kTile = kQ4Tokens;              // keys per step

template <int D>
__device__ __forceinline__ void load_block(float (*ks)[D + 1], float (*vs)[D + 1], const uint8_t* blk) {
  using B = Q4Block<D>;
  for (int e = threadIdx.x; e < kTile * D; e += blockDim.x) {
    const int t = e / D, d = e % D;
    const int g = d / kQ4Group, r = d % kQ4Group;
    const uint32_t sk = reinterpret_cast<const uint32_t*>(blk + B::kKs)[t * B::kGroups + g];
    const uint32_t sv = reinterpret_cast<const uint32_t*>(blk + B::kVs)[t * B::kGroups + g];
    const uint32_t xk = *reinterpret_cast<const uint32_t*>(blk + t * B::kRow + (r / 16) * (D / 8) + (g * 2 + (r % 16) / 8) * 4);
    const uint32_t xv = *reinterpret_cast<const uint32_t*>(blk + B::kV + q4_v_word(d, (t & 7) >> 1));
    ks[t][d] = fmaf((float)q4_nibble(xk, r % 8), q4_scale(sk), q4_min(sk));
    vs[t][d] = fmaf((float)q4_nibble(xv, q4_v_nibble(t)), q4_scale(sv), q4_min(sv));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(128) window_simt_kernel(WindowArgs a) {
  __shared__ float Qs[kRows][D + 1];
  __shared__ float Ks[kTile][D + 1];
  __shared__ float Vs[kTile][D + 1];
  const int s = blockIdx.z, h = blockIdx.y, row0 = blockIdx.x * kRows;
  const int g = h / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(a.q) + ((long long)s * a.n * a.Hq + h) * D;
  const T* k = static_cast<const T*>(a.k) + ((long long)s * a.n * a.Hkv + g) * D;
  const T* v = static_cast<const T*>(a.v) + ((long long)s * a.n * a.Hkv + g) * D;
  const long long q_row = (long long)a.Hq * D, k_row = (long long)a.Hkv * D;
  const int L = a.cache ? q4_length(a, s) : 0;
  for (int e = threadIdx.x; e < kRows * D; e += blockDim.x)
    Qs[e / D][e % D] = row0 + e / D < a.n ? to_f(q[(row0 + e / D) * q_row + e % D]) : 0.f;
  float m_i[kRowsPerWarp], l_i[kRowsPerWarp], o[kRowsPerWarp][D / 32];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    m_i[r] = -INFINITY;
    l_i[r] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[r][c] = 0.f;
  }
  // Positions below n_sink, then from the first row's window to the last row:
  // cached tiles start at multiples of kTile, own tiles at L + multiples.
  const long long last = (long long)L + min(a.n, row0 + kRows);                  // end of the visible positions
  const long long first = a.window ? max(0ll, (long long)L + row0 - a.window + 1) : 0;
  const int n_tc = (L + kTile - 1) / kTile;
  const int n_t = n_tc + (int)((last - L + kTile - 1) / kTile);
  for (int tile = 0; tile < n_t; ++tile) {
    const bool cached = tile < n_tc;
    const long long j0 = cached ? (long long)tile * kTile : L + (long long)(tile - n_tc) * kTile;
    const int n_valid = (int)min((long long)kTile, (cached ? (long long)L : last) - j0);
    if (j0 + n_valid <= first && j0 >= a.n_sink) {
      // no row sees the tile: go to the one that holds `first`
      const int next = first < L ? (int)(first / kTile) : n_tc + (int)((first - L) / kTile);
      tile = max(tile, next - 1);
      continue;
    }
    __syncthreads();
    if (cached) {
      load_block<D>(Ks, Vs, static_cast<const uint8_t*>(a.cache) +
                                (((long long)s * a.Hkv + g) * a.cap_blk + tile) * Q4Block<D>::kBytes);
    } else {
      for (int e = threadIdx.x; e < kTile * D; e += blockDim.x) {
        const int t = e / D;
        const bool in = t < n_valid;
        Ks[t][e % D] = in ? to_f(k[(j0 - L + t) * k_row + e % D]) : 0.f;
        Vs[t][e % D] = in ? to_f(v[(j0 - L + t) * k_row + e % D]) : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const int lr = warp * kRowsPerWarp + r, row = row0 + lr;
      if (row >= a.n) continue;  // warp-uniform
      const long long j = j0 + lane, at = (long long)L + row;
      const bool vis = lane < n_valid && j <= at && (!a.window || j > at - a.window || j < a.n_sink);
      float sc = 0.f;
#pragma unroll 8
      for (int c = 0; c < D; ++c) sc += Qs[lr][c] * Ks[lane][c];
      sc = vis ? sc * a.scale_log2 : -INFINITY;
      float top = sc;
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const unsigned seen = __ballot_sync(0xffffffffu, vis);
      if (!seen) continue;  // nothing of the tile is visible to the row (warp-uniform)
      const float m_new = fmaxf(m_i[r], top);
      const float ref = m_new == -INFINITY ? 0.f : m_new;  // every visible logit -inf so far
      const float p = vis ? exp2f(sc - ref) : 0.f;
      const float alpha = exp2f(m_i[r] - ref);
      float psum = p;
#pragma unroll
      for (int off = 16; off; off >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
      l_i[r] = l_i[r] * alpha + psum;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[r][c] *= alpha;
      for (int kk = 0; kk < kTile; ++kk) {
        if (!(seen >> kk & 1u)) continue;  // a NaN in a masked place stays out
        const float pk = __shfl_sync(0xffffffffu, p, kk);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[r][c] += pk * Vs[kk][lane + 32 * c];
      }
      m_i[r] = m_new;
    }
  }
  T* out = static_cast<T*>(a.out) + ((long long)s * a.n * a.Hq + h) * D;
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const int row = row0 + warp * kRowsPerWarp + r;
    if (row >= a.n) continue;
    const float inv = 1.f / l_i[r];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) out[row * q_row + lane + 32 * c] = from_f<T>(o[r][c] * inv);
    if (a.lse && lane == 0) a.lse[((long long)s * a.Hq + h) * a.n + row] = (m_i[r] + log2f(l_i[r])) * kLn2;
  }
}

}  // namespace

cudaError_t launch_window_simt(const WindowArgs& a, int dtype, int d, cudaStream_t st) {
  const dim3 grid((a.n + kRows - 1) / kRows, a.Hq, a.S);
  if (dtype == kDtypeBF16)
    return d == 128 ? launch_kernel(window_simt_kernel<__nv_bfloat16, 128>, grid, dim3(128), 0, st, false, a)
                    : launch_kernel(window_simt_kernel<__nv_bfloat16, 64>, grid, dim3(128), 0, st, false, a);
  return d == 128 ? launch_kernel(window_simt_kernel<float, 128>, grid, dim3(128), 0, st, false, a)
                  : launch_kernel(window_simt_kernel<float, 64>, grid, dim3(128), 0, st, false, a);
}

}  // namespace skv
