// Causal attention with a sliding window and visible first tokens in float32:
// token i sees j <= i with j > i - window or j < n_sink.
//
// Both products run on the tensor cores in tf32 (11-bit significands) at close to
// float32's precision: with x = hi + lo, hi = x rounded to tf32 and lo the rest,
//   x y ~ lo_x hi_y + hi_x lo_y + hi_x hi_y,
// off by 2^-21 of |x y| at most, with signs that do not add up.  mma.sync's tf32
// rate bounds the kernel: 146 TFLOP/s, 49 of the result (4 x 3000 tokens, 16
// heads, d = 64).  The same tiles on the CUDA cores (paired fma) reached 34; three
// bfloat16 parts and six products at the 16-bit rate 42, split by every warp or
// once a block (chains of six dependent products, and registers for two warps a
// scheduler).  Sums are float32; the tensor
// cores cut theirs instead of rounding, so each 16 channels of S and each key
// tile of P V are summed on their own and added on the CUDA cores: 3.0e-7 off in
// all (1500 tokens, d = 128) where one long sum was 1.2e-6 off.
//
// A block takes 64 query rows of one head, a warp 16 of them, and walks the key
// tiles that any row sees (sink tiles, then from row 0's window to the diagonal),
// the next tile's copies in flight.  Tensor-core shape
// m16n8k8; the depth's order is free, so a lane takes four consecutive channels of
// a key (K) or of a value (V) in one 16-byte load, and the fragment of P is the one
// S was left in, with its keys as the depth.
//
// The running maximum starts at -inf; a weight whose key is hidden is -0, which
// adds nothing to a sum.  Where a tile holds a key or value that is not finite (or
// too close to the largest float32 to be rounded) that number is 0 in the product,
// and the rows that see it add it afterwards: hidden values never take part, and
// the other sums keep their bits.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "window_row.cuh"

namespace skv {
namespace {

constexpr int kRows = 64, kThreads = 128, kBlocks = 2;
constexpr float kBig = 0x1.ffep127f;  // from here on rounding to tf32 could overflow

template <int D>
struct Tile {
  static constexpr int kKeys = 4096 / D;   // 64 (D = 64) or 32: two stages of either are 76 or 71 KB
  static constexpr int kKStride = D + 16;  // floats; 16 mod 32: eight lanes of a 16-byte load, all banks
  static constexpr int kVStride = D + 4;   // 2 x 4 mod 32: the same for value pairs
  static constexpr int kV = kKeys * kKStride;
  static constexpr int kFloats = kV + kKeys * kVStride;
  static constexpr int kQ = 2 * kFloats;   // behind the two stages: Q, rows as K's
  static constexpr int kBytes = (kQ + kRows * kKStride) * 4;
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// c += a b, the least products first (part 0: hi, part 1: lo)
__device__ __forceinline__ void mma_parts(float (&c)[4], const uint32_t (&a)[2][4], const uint32_t (&b)[2][2]) {
  mma_tf32(c, a[1], b[0]);
  mma_tf32(c, a[0], b[1]);
  mma_tf32(c, a[0], b[0]);
}

// x as hi + lo (the tensor cores read the upper 19 bits of lo).  kAny: x (of a query)
// may be a NaN, an infinity (hi is, lo is 0; every logit of the row is one of the two
// then) or above kBig (hi is cut, not rounded).
template <bool kAny>
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  const uint32_t b = __float_as_uint(x);
  hi = (b + 0x1000u) & 0xffffe000u;
  if (kAny && !(fabsf(x) < kBig)) hi = x != x ? 0x7fffe000u : b & 0xffffe000u;
  const float r = x - __uint_as_float(hi);
  lo = __float_as_uint(kAny && r != r ? 0.f : r);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocks) window_f32_kernel(const __grid_constant__ WindowArgs a, int n_tiles) {
  using L = Tile<D>;
  constexpr int KT = L::kKeys, NT = KT / 8, KP = D / 16, VQ = D / 32;
  extern __shared__ __align__(16) float smem[];
  // channels of this lane's rows (bits 8 c + 4 b + i) that met a value not finite
  __shared__ uint32_t seen[2][kThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  // unit -> (stream, row tile, head): the heads that share keys run side by side
  long long u = blockIdx.x;
  const int h = (int)(u % a.Hq);
  u /= a.Hq;
  const int tile = n_tiles - 1 - (int)(u % n_tiles), s = (int)(u / n_tiles);
  const int g = h / (a.Hq / a.Hkv), i0 = tile * kRows;
  const int r0 = i0 + warp * 16 + gid;  // this lane's rows: r0, r0 + 8
  const long long q_row = (long long)a.Hq * D, k_row = (long long)a.Hkv * D;
  const float* q = static_cast<const float*>(a.q) + (long long)s * a.n * q_row + (long long)h * D;
  const float* k = static_cast<const float*>(a.k) + (long long)s * a.n * k_row + (long long)g * D;
  const float* v = static_cast<const float*>(a.v) + (long long)s * a.n * k_row + (long long)g * D;

  const int fw = max(0, i0 - a.window + 1) / KT;                        // first window tile
  const int ns = min((int)(((long long)a.n_sink + KT - 1) / KT), fw);   // sink tiles before it
  const int nk = ns + min(i0 + kRows - 1, a.n - 1) / KT + 1 - fw;
  auto base_of = [&](int j) { return (j < ns ? j : j - ns + fw) * KT; };
  // thread -> 16-byte pieces threadIdx.x, + 128, ... of the tile's K, then of its V
  auto load = [&](int j) {
    const int base = base_of(j);
    float* buf = smem + (j & 1) * L::kFloats;
#pragma unroll
    for (int e = threadIdx.x; e < KT * D / 4; e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const bool there = base + r < a.n;
      const long long at = there ? (base + r) * k_row + c : 0;
      copy16(buf + r * L::kKStride + c, k + at, there);
      copy16(buf + L::kV + r * L::kVStride + c, v + at, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 4
  for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const bool there = i0 + r < a.n;
    copy16(smem + L::kQ + r * L::kKStride + c, q + (there ? (i0 + r) * q_row + c : 0), there);
  }
  load(0);
  const float* qt = smem + L::kQ + (warp * 16 + gid) * L::kKStride + tig * 4;
  // O: channels 32 c + 8 tig + i (elements 0, 2: rows r0, r0 + 8) and + 4 (elements 1, 3)
  float o[VQ][4][4], m[2], l[2];
#pragma unroll
  for (int c = 0; c < VQ; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][i][e] = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    m[e] = -INFINITY;
    l[e] = 0.f;
    seen[e][threadIdx.x] = 0u;
  }

  for (int j = 0; j < nk; ++j) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    const int base = base_of(j);
    const float* kt = smem + (j & 1) * L::kFloats;
    const float* vt = kt + L::kV;
    // this thread's own pieces: anything that the products cannot take as it is?
    bool odd = false;
#pragma unroll
    for (int e = threadIdx.x; e < KT * D / 4; e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const float4 x = *reinterpret_cast<const float4*>(kt + r * L::kKStride + c);
      const float4 y = *reinterpret_cast<const float4*>(vt + r * L::kVStride + c);
      odd |= !(fabsf(x.x) < kBig) || !(fabsf(x.y) < kBig) || !(fabsf(x.z) < kBig) || !(fabsf(x.w) < kBig);
      odd |= !(fabsf(y.x) < kBig) || !(fabsf(y.y) < kBig) || !(fabsf(y.z) < kBig) || !(fabsf(y.w) < kBig);
    }
    const bool careful = __syncthreads_or(odd);  // (the tile is there, the one before has been read)
    bool big = false;  // a key that is infinite, or too large to be rounded
    if (careful) {
#pragma unroll
      for (int e = threadIdx.x; e < KT * D / 4; e += kThreads) {
        const float4 x = *reinterpret_cast<const float4*>(kt + e / (D / 4) * L::kKStride + e % (D / 4) * 4);
        big |= fabsf(x.x) >= kBig || fabsf(x.y) >= kBig || fabsf(x.z) >= kBig || fabsf(x.w) >= kBig;
      }
      big = __syncthreads_or(big);
    }
    if (j + 1 < nk) load(j + 1);
    // a warp whose rows see nothing of the tile leaves it out
    const int w0 = i0 + warp * 16;
    if (base > w0 + 15 || (base + KT - 1 <= w0 - a.window && base >= a.n_sink)) continue;

    // ---- S = Q K^T
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] = 0.f;
    auto scores = [&](auto any) {
      constexpr bool kAny = decltype(any)::value;
#pragma unroll 1
      for (int p = 0; p < KP; ++p) {
        uint32_t qa[2][4], qb[2][4];  // two steps of depth 8: channels 4 tig + {0, 1}, {2, 3}
        const float4 x0 = *reinterpret_cast<const float4*>(qt + p * 16);
        const float4 x1 = *reinterpret_cast<const float4*>(qt + 8 * L::kKStride + p * 16);
        split<true>(x0.x, qa[0][0], qa[1][0]);
        split<true>(x1.x, qa[0][1], qa[1][1]);
        split<true>(x0.y, qa[0][2], qa[1][2]);
        split<true>(x1.y, qa[0][3], qa[1][3]);
        split<true>(x0.z, qb[0][0], qb[1][0]);
        split<true>(x1.z, qb[0][1], qb[1][1]);
        split<true>(x0.w, qb[0][2], qb[1][2]);
        split<true>(x1.w, qb[0][3], qb[1][3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float4 y4 = *reinterpret_cast<const float4*>(kt + (t * 8 + gid) * L::kKStride + p * 16 + tig * 4);
          float y[4] = {y4.x, y4.y, y4.z, y4.w};
          if (kAny) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (fabsf(y[i]) >= kBig) y[i] = 0.f;  // (a NaN stays: the logit is one)
          }
          uint32_t ya[2][2], yb[2][2];
          split<false>(y[0], ya[0][0], ya[1][0]);
          split<false>(y[1], ya[0][1], ya[1][1]);
          split<false>(y[2], yb[0][0], yb[1][0]);
          split<false>(y[3], yb[0][1], yb[1][1]);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_parts(acc, qa, ya);
          mma_parts(acc, qb, yb);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][e] += acc[e];
        }
      }
    };
    if (careful) {
      scores(std::true_type());
      // what was 0 in the products, times q as it is: in parts an infinite key would
      // meet q's low part, which is 0 or of the other sign as often as not
#pragma unroll 1
      for (int x = 0; big && x < 2 * NT; ++x) {  // this lane's keys
        const float* row = kt + ((x >> 1) * 8 + tig * 2 + (x & 1)) * L::kKStride;
        const float* q0 = smem + L::kQ + (warp * 16 + gid) * L::kKStride;
        float add[2] = {0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
          const float y = row[c];
          if (!(fabsf(y) >= kBig)) continue;
          add[0] = fmaf(q0[c], y, add[0]);
          add[1] = fmaf(q0[8 * L::kKStride + c], y, add[1]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if (x == 2 * t + b) {
              sc[t][b] += add[0];
              sc[t][2 + b] += add[1];
            }
      }
    } else {
      scores(std::false_type());
    }

    // ---- softmax: element e of tile t is row r0 + 8 (e/2), key 8 t + 2 tig + e%2
    const bool masked = base + KT > w0 + 1 || (base <= w0 + 15 - a.window && base + KT > a.n_sink);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[t][e] *= a.scale_log2;
        top[e >> 1] = fmaxf(top[e >> 1], sc[t][e]);
      }
    uint32_t hidden[2] = {0u, 0u};  // bits 2 t + e%2
    if (masked) {
      top[0] = top[1] = -INFINITY;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = base + t * 8 + tig * 2 + (e & 1), i = r0 + 8 * (e >> 1);
          if (key > i || (key <= i - a.window && key >= a.n_sink)) {
            sc[t][e] = -INFINITY;
            hidden[e >> 1] |= 1u << (2 * t + (e & 1));
          }
          top[e >> 1] = fmaxf(top[e >> 1], sc[t][e]);
        }
    }
    float ref[2], f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      const float nm = fmaxf(m[e], top[e]);
      ref[e] = nm == -INFINITY ? 0.f : nm;
      f[e] = exp2f(m[e] - ref[e]);
      m[e] = nm;
      l[e] *= f[e];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2f(sc[t][e] - ref[e >> 1]);
        const bool hide = hidden[e >> 1] >> (2 * t + (e & 1)) & 1;
        l[e >> 1] += hide ? 0.f : p;
        sc[t][e] = hide ? -0.f : p;
      }

    // ---- O += P V: depth step t = keys 8 t + 2 tig, + 1; 32 channels at a time
    auto values = [&](auto any) {
      constexpr bool kAny = decltype(any)::value;
#pragma unroll
      for (int c = 0; c < VQ; ++c) {
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t pp[2][4];  // (a NaN stays one, in hi or in lo)
          split<false>(sc[t][0], pp[0][0], pp[1][0]);
          split<false>(sc[t][2], pp[0][1], pp[1][1]);
          split<false>(sc[t][1], pp[0][2], pp[1][2]);
          split<false>(sc[t][3], pp[0][3], pp[1][3]);
          const float* at = vt + (t * 8 + tig * 2) * L::kVStride + c * 32 + gid * 4;
          const float4 y0 = *reinterpret_cast<const float4*>(at), y1 = *reinterpret_cast<const float4*>(at + L::kVStride);
          float ya[4] = {y0.x, y0.y, y0.z, y0.w}, yb[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kAny) {
              if (!(fabsf(ya[i]) < kBig)) ya[i] = 0.f;
              if (!(fabsf(yb[i]) < kBig)) yb[i] = 0.f;
            }
            uint32_t yp[2][2];
            split<false>(ya[i], yp[0][0], yp[1][0]);
            split<false>(yb[i], yp[0][1], yp[1][1]);
            mma_parts(acc[i], pp, yp);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][i][e] = fmaf(o[c][i][e], f[e >> 1], acc[i][e]);
      }
    };
    if (!careful) {
      values(std::false_type());
    } else {
      values(std::true_type());
      // what was 0 in the products, for the rows that see it
      uint32_t met[2] = {0u, 0u};
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          const float p0 = __shfl_sync(0xffffffffu, x & 1 ? sc[t][1] : sc[t][0], gid * 4 + (x >> 1));
          const float p1 = __shfl_sync(0xffffffffu, x & 1 ? sc[t][3] : sc[t][2], gid * 4 + (x >> 1));
          const float* row = vt + (t * 8 + x) * L::kVStride + tig * 8;
#pragma unroll
          for (int c = 0; c < VQ; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float y = row[c * 32 + b * 4 + i];
                if (fabsf(y) < kBig) continue;
                const uint32_t bit = fabsf(y) < INFINITY ? 0u : 1u << (c * 8 + b * 4 + i);
                if (__float_as_uint(p0) != 0x80000000u) {
                  o[c][i][b] = fmaf(p0, y, o[c][i][b]);
                  met[0] |= bit;
                }
                if (__float_as_uint(p1) != 0x80000000u) {
                  o[c][i][2 + b] = fmaf(p1, y, o[c][i][2 + b]);
                  met[1] |= bit;
                }
              }
        }
      seen[0][threadIdx.x] |= met[0];
      seen[1][threadIdx.x] |= met[1];
    }
  }
  uint32_t bad[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = r0 + 8 * e;
    float ls = l[e];
    ls += __shfl_xor_sync(0xffffffffu, ls, 1);
    ls += __shfl_xor_sync(0xffffffffu, ls, 2);
    if (i >= a.n) continue;
    const float inv = 1.f / ls;
    float* out = static_cast<float*>(a.out) + ((long long)s * a.n + i) * q_row + (long long)h * D + tig * 8;
#pragma unroll
    for (int c = 0; c < VQ; ++c)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float4 y = make_float4(o[c][0][2 * e + b] * inv, o[c][1][2 * e + b] * inv, o[c][2][2 * e + b] * inv, o[c][3][2 * e + b] * inv);
        const uint32_t odd = (fabsf(y.x) < INFINITY ? 0u : 1u) | (fabsf(y.y) < INFINITY ? 0u : 2u) |
                             (fabsf(y.z) < INFINITY ? 0u : 4u) | (fabsf(y.w) < INFINITY ? 0u : 8u);
        bad[e] |= odd << (c * 8 + b * 4);
        *reinterpret_cast<float4*>(out + c * 32 + b * 4) = y;
      }
    bad[e] = ls == ls ? bad[e] & ~seen[e][threadIdx.x] : 0u;
    if (a.lse && tig == 0) a.lse[((long long)s * a.Hq + h) * a.n + i] = (m[e] + log2f(ls)) * kLn2;
  }
  // rows that are not finite where their sum of weights and all values they saw are:
  // sums of values next to the largest float that overflowed
#pragma unroll 1
  for (int e = 0; e < 2; ++e)
    for (unsigned again = __ballot_sync(0xffffffffu, (e ? bad[1] : bad[0]) != 0u); again;) {
      const int row = (__ffs(again) - 1) >> 2;
      again &= ~(0xfu << (4 * row));
      window_row_again<float, D>(a, s, h, i0 + warp * 16 + row + 8 * e);
    }
}

template <int D>
cudaError_t launch(const WindowArgs& a, cudaStream_t st) {
  const int smem = Tile<D>::kBytes;
  const cudaError_t e = ensure_dynamic_smem(window_f32_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  const int n_tiles = (a.n + kRows - 1) / kRows;
  return launch_kernel(window_f32_kernel<D>, dim3((unsigned)((long long)a.S * n_tiles * a.Hq)), dim3(kThreads), smem, st,
                       false, a, n_tiles);
}

}  // namespace

cudaError_t launch_window_f32(const WindowArgs& a, int d, cudaStream_t st) {
  return d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace skv
