// Causal attention with a sliding window and visible first tokens in float32 on
// the CUDA cores: token i sees j <= i with j > i - window or j < n_sink.
//
// A block takes 64 query rows of one head; its two groups of four warps walk
// every other of the 64-key tiles that any row sees (sink tiles, then from row
// 0's window to the diagonal) and join their sums at the end.  Both
// products are register tiles fed from shared memory in 16-byte loads: 8 rows x
// 4 keys a thread for S = Q K^T (Q, K transposed), 8 rows x D/16 channels for
// O += P V, in paired fma instructions, so that one load feeds eight or more
// fmas and the float32 pipe is the bound, not shared memory.
//
// The running maximum starts at -inf; a weight whose key is hidden is stored as
// -0.  Times a finite value that adds nothing; in a tile whose values hold a NaN
// or an infinity the product skips it by its sign bit, so hidden values never
// take part and the other sums keep their bits.
#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace skv {
namespace {

constexpr int kRows = 64, kKeys = 64, kGroup = 128, kThreads = 2 * kGroup;

template <int D>
struct Smem {
  float q[D][kRows];          // transposed
  struct Group {
    float k[D][kKeys];        // transposed
    float v[kKeys][D];
    float p[kKeys][kRows];    // transposed
  } g[2];
};

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) window_simt_kernel(WindowArgs a, int n_tiles) {
  constexpr int C = D / 16;  // channels of O per thread
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D>& all = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int grp = threadIdx.x / kGroup;
  typename Smem<D>::Group& sh = all.g[grp];
  // unit -> (stream, row tile, head): the heads that share keys run side by side
  long long u = blockIdx.x;
  const int h = (int)(u % a.Hq);
  u /= a.Hq;
  const int tile = n_tiles - 1 - (int)(u % n_tiles), s = (int)(u / n_tiles);
  const int g = h / (a.Hq / a.Hkv), i0 = tile * kRows;
  const int tid = threadIdx.x % kGroup, tr = tid >> 4, tc_ = tid & 15;  // rows 8 tr.., keys 4 tc.., channels 4 tc.. (and + 64)
  const long long q_row = (long long)a.Hq * D, k_row = (long long)a.Hkv * D;
  const float* q = static_cast<const float*>(a.q) + ((long long)s * a.n + i0) * q_row + (long long)h * D;
  const float* k = static_cast<const float*>(a.k) + (long long)s * a.n * k_row + (long long)g * D;
  const float* v = static_cast<const float*>(a.v) + (long long)s * a.n * k_row + (long long)g * D;

  // rows of a 64-row tile in, transposed: lane = row, so that the four stores of
  // a 16-byte load meet 32 different banks
  auto load_t = [&](float (*dst)[64], const float* src, long long stride, int n_valid, int first, int step) {
    const int r = tid & 63;
#pragma unroll 4
    for (int c = first; c < D / 4; c += step) {
      const float4 x = r < n_valid ? __ldg(reinterpret_cast<const float4*>(src + r * stride) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      dst[4 * c][r] = x.x;
      dst[4 * c + 1][r] = x.y;
      dst[4 * c + 2][r] = x.z;
      dst[4 * c + 3][r] = x.w;
    }
  };
  load_t(all.q, q, q_row, min(kRows, a.n - i0), threadIdx.x >> 6, kThreads / 64);
  __syncthreads();

  float2 o[4][C];            // row pairs (8 tr + 2 r, + 1)
  float m[8], l[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) o[r][c] = make_float2(0.f, 0.f);

  const int fw = max(0, i0 - a.window + 1) / kKeys;                 // first window tile
  const int ns = min((a.n_sink + kKeys - 1) / kKeys, fw);           // sink tiles before it
  const int nk = ns + tile + 1 - fw;
  for (int j = grp; j < nk; j += 2) {
    const int base = (j < ns ? j : j - ns + fw) * kKeys, n_valid = min(kKeys, a.n - base);
    tc::named_bar_sync(1 + grp, kGroup);  // the previous tile has been read
    load_t(sh.k, k + (long long)base * k_row, k_row, n_valid, tid >> 6, kGroup / 64);
    float odd = 0.f;  // NaN if a value is a NaN or an infinity
#pragma unroll 4
    for (int e = tid; e < kKeys * D / 4; e += kGroup) {
      const int r = e / (D / 4), c = e % (D / 4);
      const float4 x = r < n_valid ? __ldg(reinterpret_cast<const float4*>(v + (base + r) * k_row) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      odd += (x.x - x.x) + (x.y - x.y) + (x.z - x.z) + (x.w - x.w);
      *reinterpret_cast<float4*>(&sh.v[r][4 * c]) = x;
    }
    const bool careful = tc::named_bar_red_or(1 + grp, kGroup, odd != 0.f);
    // S = Q K^T
    float2 acc[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][c] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < D; ++d) {
      const float4 q0 = *reinterpret_cast<const float4*>(&all.q[d][tr * 8]), q1 = *reinterpret_cast<const float4*>(&all.q[d][tr * 8 + 4]);
      const float4 kk = *reinterpret_cast<const float4*>(&sh.k[d][tc_ * 4]);
      const float2 qp[4] = {make_float2(q0.x, q0.y), make_float2(q0.z, q0.w), make_float2(q1.x, q1.y), make_float2(q1.z, q1.w)};
      const float kv[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r][c] = tc::ffma2(qp[r], make_float2(kv[c], kv[c]), acc[r][c]);
    }
    // softmax of 8 rows x 4 keys; a row is spread over 16 lanes
    const bool masked = base + kKeys > i0 + 1 || (base <= i0 + kRows - 1 - a.window && base + kKeys > a.n_sink);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int i = i0 + tr * 8 + r;
      float t[4], top = -INFINITY;
      uint32_t hidden = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        t[c] = ((r & 1) ? acc[r >> 1][c].y : acc[r >> 1][c].x) * a.scale_log2;
        if (masked) {
          const int key = base + tc_ * 4 + c;
          if (key > i || (key <= i - a.window && key >= a.n_sink)) {
            t[c] = -INFINITY;
            hidden |= 1u << c;
          }
        }
        top = fmaxf(top, t[c]);
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float nm = fmaxf(m[r], top), ref = nm == -INFINITY ? 0.f : nm;
      if (nm != m[r]) {
        const float f = exp2f(m[r] - ref);
        l[r] *= f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (r & 1) o[r >> 1][c].y *= f;
          else o[r >> 1][c].x *= f;
        }
        m[r] = nm;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = exp2f(t[c] - ref);
        const bool hide = hidden >> c & 1;
        l[r] += hide ? 0.f : p;
        const float w = hide ? -0.f : p;
        if (r & 1) acc[r >> 1][c].y = w;
        else acc[r >> 1][c].x = w;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float* dst = &sh.p[tc_ * 4 + c][tr * 8];
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0][c].x, acc[0][c].y, acc[1][c].x, acc[1][c].y);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[2][c].x, acc[2][c].y, acc[3][c].x, acc[3][c].y);
    }
    // P of eight rows is written and read by one half warp
    __syncwarp();
    // O += P V
    if (!careful) {
#pragma unroll 4
      for (int key = 0; key < kKeys; ++key) {
        const float4 p0 = *reinterpret_cast<const float4*>(&sh.p[key][tr * 8]), p1 = *reinterpret_cast<const float4*>(&sh.p[key][tr * 8 + 4]);
        const float2 pp[4] = {make_float2(p0.x, p0.y), make_float2(p0.z, p0.w), make_float2(p1.x, p1.y), make_float2(p1.z, p1.w)};
#pragma unroll
        for (int c4 = 0; c4 < C / 4; ++c4) {
          const float4 vv = *reinterpret_cast<const float4*>(&sh.v[key][c4 * 64 + tc_ * 4]);
          const float vs[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r][c4 * 4 + c] = tc::ffma2(pp[r], make_float2(vs[c], vs[c]), o[r][c4 * 4 + c]);
        }
      }
    } else {
#pragma unroll 1
      for (int key = 0; key < kKeys; ++key) {
        float pr[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) pr[r] = sh.p[key][tr * 8 + r];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float x = sh.v[key][(c >> 2) * 64 + tc_ * 4 + (c & 3)];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (__float_as_uint(pr[2 * r]) != 0x80000000u) o[r][c].x = fmaf(pr[2 * r], x, o[r][c].x);
            if (__float_as_uint(pr[2 * r + 1]) != 0x80000000u) o[r][c].y = fmaf(pr[2 * r + 1], x, o[r][c].y);
          }
        }
      }
    }
  }
  // the second group's maximum, sum and O through shared memory (over its own
  // tiles), joined by the first
  float* xo = &all.g[1].k[0][0];   // [64 rows][D]
  float* xm = &all.g[1].p[0][0];   // [64 rows][2]
  tc::named_bar_sync(1 + grp, kGroup);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int off = 8; off; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
    if (grp == 0) continue;
    if (tc_ == 0) {
      xm[(tr * 8 + r) * 2] = m[r];
      xm[(tr * 8 + r) * 2 + 1] = l[r];
    }
#pragma unroll
    for (int c4 = 0; c4 < C / 4; ++c4) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = (r & 1) ? o[r >> 1][c4 * 4 + c].y : o[r >> 1][c4 * 4 + c].x;
      *reinterpret_cast<float4*>(xo + (tr * 8 + r) * D + c4 * 64 + tc_ * 4) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int i = i0 + tr * 8 + r;
    if (i >= a.n) continue;
    const float m2 = xm[(tr * 8 + r) * 2], l2 = xm[(tr * 8 + r) * 2 + 1];
    const float nm = fmaxf(m[r], m2), ref = nm == -INFINITY ? 0.f : nm;
    const float f1 = exp2f(m[r] - ref), f2 = exp2f(m2 - ref);
    const float ls = l[r] * f1 + l2 * f2, inv = 1.f / ls;
    float* out = static_cast<float*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D;
#pragma unroll
    for (int c4 = 0; c4 < C / 4; ++c4) {
      const float4 y = *reinterpret_cast<const float4*>(xo + (tr * 8 + r) * D + c4 * 64 + tc_ * 4);
      const float ys[4] = {y.x, y.y, y.z, y.w};
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[c] = (((r & 1) ? o[r >> 1][c4 * 4 + c].y : o[r >> 1][c4 * 4 + c].x) * f1 + ys[c] * f2) * inv;
      *reinterpret_cast<float4*>(out + c4 * 64 + tc_ * 4) = make_float4(x[0], x[1], x[2], x[3]);
    }
    if (a.lse && tc_ == 0) a.lse[((long long)s * a.Hq + h) * a.n + i] = (nm + log2f(ls)) * kLn2;
  }
}

template <int D>
cudaError_t launch(const WindowArgs& a, cudaStream_t st) {
  cudaError_t e = ensure_dynamic_smem(window_simt_kernel<D>, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  const int n_tiles = (a.n + kRows - 1) / kRows;
  return launch_kernel(window_simt_kernel<D>, dim3((unsigned)((long long)a.S * n_tiles * a.Hq)), dim3(kThreads),
                       sizeof(Smem<D>), st, false, a, n_tiles);
}

}  // namespace

cudaError_t launch_window_simt(const WindowArgs& a, int d, cudaStream_t st) {
  return d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace skv
