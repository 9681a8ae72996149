// Writing the 4-bit cache and reading it back (format: q4_cache.cuh).
//
// Both kernels give a block of threads one 32-token block of one (stream, KV
// head).  A V word holds codes of eight tokens, so a block that is only partly
// covered by an append is read, merged and written by the one thread block that
// owns it; no two thread blocks of a call share a word.
#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;

// Token range [p0, p1) that the call covers in stream s, clipped to the cache.
struct Span {
  long long start;  // cache token of the call's token 0
  int p0, p1;
};
__device__ __forceinline__ Span span_of(const Q4IoArgs& a, int s) {
  Span sp;
  sp.start = a.starts ? (long long)__ldg(a.starts + s) : (long long)a.start;
  const long long lo = sp.start > 0 ? sp.start : 0;
  const long long hi = sp.start + a.n < a.capacity ? sp.start + a.n : a.capacity;
  sp.p0 = (int)(lo < a.capacity ? lo : a.capacity);
  sp.p1 = (int)(hi > sp.p0 ? hi : sp.p0);
  return sp;
}

// Codes of one token row held by a warp, E channels per lane; kLanes lanes
// share a group.  Returns the packed (s, m) of the lane's group.
template <int E, int kLanes>
__device__ __forceinline__ uint32_t quantise(const float (&x)[E], int (&c)[E]) {
  float lo = x[0], hi = x[0];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    bad |= !(fabsf(x[e]) < INFINITY);
  }
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    bad |= __shfl_xor_sync(0xffffffffu, (int)bad, off) != 0;
  }
  // round down / up to bfloat16 on the bit pattern
  uint32_t mb = __float_as_uint(lo);
  if ((mb & 0xffffu) && (mb >> 31)) mb += 0x10000u;
  mb &= 0xffff0000u;
  const float m = __uint_as_float(mb);
  const float s32 = __double2float_ru(((double)hi - (double)m) / 15.0);
  const uint32_t sb = (__float_as_uint(s32) + 0xffffu) & 0xffff0000u;
  const float s = __uint_as_float(sb);
  bad |= !(fabsf(m) < INFINITY);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    c[e] = 0;
    if (!bad && s > 0.f) c[e] = min(15, max(0, (int)rint(((double)x[e] - (double)m) / (double)s)));
  }
  return bad ? 0x7fc07fc0u : (sb >> 16) | mb;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(Q4IoArgs a) {
  using B = Q4Block<D>;
  constexpr int E = D / 32, kLanes = kQ4Group / E;
  __shared__ uint8_t codes[2][kQ4Tokens][D];
  __shared__ uint32_t scales[2][kQ4Tokens][B::kGroups];
  const int sg = blockIdx.x / a.n_blk, s = sg / a.Hkv, g = sg % a.Hkv;
  const Span sp = span_of(a, s);
  const int b = sp.p0 / kQ4Tokens + blockIdx.x % a.n_blk;
  if ((long long)b * kQ4Tokens >= sp.p1 || sp.p0 >= sp.p1) return;
  const int t_lo = max(sp.p0 - b * kQ4Tokens, 0), t_hi = min(sp.p1 - b * kQ4Tokens, kQ4Tokens);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < 2 * kQ4Tokens; r += kThreads / 32) {
    const int kv = r >> 5, t = r & 31;
    if (t < t_lo || t >= t_hi) continue;
    const long long tok = (long long)b * kQ4Tokens + t - sp.start;
    const T* src = static_cast<const T*>(kv ? a.v : a.k) + (((long long)s * a.n + tok) * a.Hkv + g) * D + lane * E;
    float x[E];
    int c[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = to_f(src[e]);
    const uint32_t sm = quantise<E, kLanes>(x, c);
#pragma unroll
    for (int e = 0; e < E; ++e) codes[kv][t][lane * E + e] = (uint8_t)c[e];
    if (lane % kLanes == 0) scales[kv][t][lane / kLanes] = sm;
  }
  __syncthreads();
  uint8_t* blk = static_cast<uint8_t*>(a.cache) + ((long long)sg * a.cap_blk + b) * B::kBytes;
  // K words: whole rows of the covered tokens
  for (int w = threadIdx.x; w < kQ4Tokens * (D / 8); w += kThreads) {
    const int t = w / (D / 8), tig = (w % (D / 8)) / (D / 32), ww = w % (D / 32);
    if (t < t_lo || t >= t_hi) continue;
    const uint8_t* c = &codes[0][t][(ww >> 1) * 64 + tig * 16 + (ww & 1) * 8];
    *reinterpret_cast<uint32_t*>(blk + t * B::kRow + tig * (D / 8) + ww * 4) =
        q4_pack(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
  }
  // V words: eight tokens each; the others' codes are kept
  for (int w = threadIdx.x; w < D * 4; w += kThreads) {
    const int d = w >> 2, tig = w & 3;
    uint32_t p[4], keep[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int t = (f >> 1) * 16 + (f & 1) * 8 + 2 * tig;
      const bool in0 = t >= t_lo && t < t_hi, in1 = t + 1 >= t_lo && t + 1 < t_hi;
      p[f] = (in0 ? codes[1][t][d] : 0u) | (in1 ? codes[1][t + 1][d] << 16 : 0u);
      keep[f] = (in0 ? 0u : 15u) | (in1 ? 0u : 15u << 16);
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(blk + B::kV + q4_v_word(d, tig));
    const uint32_t mask = q4_pack(keep[0], keep[1], keep[2], keep[3]);
    uint32_t word = q4_pack(p[0], p[1], p[2], p[3]);
    if (mask) word |= *dst & mask;
    *dst = word;
  }
  for (int w = threadIdx.x; w < 2 * kQ4Tokens * B::kGroups; w += kThreads) {
    const int kv = w / (kQ4Tokens * B::kGroups), e = w % (kQ4Tokens * B::kGroups), t = e / B::kGroups;
    if (t < t_lo || t >= t_hi) continue;
    reinterpret_cast<uint32_t*>(blk + (kv ? B::kVs : B::kKs))[e] = scales[kv][t][e % B::kGroups];
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(Q4IoArgs a) {
  using B = Q4Block<D>;
  const int sg = blockIdx.x / a.n_blk, s = sg / a.Hkv, g = sg % a.Hkv;
  const Span sp = span_of(a, s);
  const int b = sp.p0 / kQ4Tokens + blockIdx.x % a.n_blk;
  if ((long long)b * kQ4Tokens >= sp.p1 || sp.p0 >= sp.p1) return;
  const int t_lo = max(sp.p0 - b * kQ4Tokens, 0), t_hi = min(sp.p1 - b * kQ4Tokens, kQ4Tokens);
  const uint8_t* blk = static_cast<const uint8_t*>(a.cache) + ((long long)sg * a.cap_blk + b) * B::kBytes;
  // a thread takes eight channels of one token
  for (int w = threadIdx.x; w < 2 * kQ4Tokens * (D / 8); w += kThreads) {
    const int kv = w / (kQ4Tokens * (D / 8)), t = w / (D / 8) % kQ4Tokens, c8 = w % (D / 8);
    if (t < t_lo || t >= t_hi) continue;
    const uint32_t sm = __ldg(reinterpret_cast<const uint32_t*>(blk + (kv ? B::kVs : B::kKs)) + t * B::kGroups + c8 / 8);
    int c[8];
    if (!kv) {
      const int tig = (c8 % 8) / 2, ww = (c8 / 8) * 2 + c8 % 2;
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(blk + t * B::kRow + tig * (D / 8) + ww * 4));
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = q4_code(x, e);
    } else {
      const int i = (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1), tig = (t & 7) >> 1;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        c[e] = q4_code(__ldg(reinterpret_cast<const uint32_t*>(blk + B::kV + q4_v_word(c8 * 8 + e, tig))), i);
    }
    const long long tok = (long long)b * kQ4Tokens + t - sp.start;
    T* dst = static_cast<T*>(kv ? a.v_out : a.k_out) + (((long long)s * a.n + tok) * a.Hkv + g) * D + c8 * 8;
    const float sc = q4_scale(sm), m = q4_min(sm);
#pragma unroll
    for (int e = 0; e < 8; ++e) dst[e] = from_f<T>(fmaf((float)c[e], sc, m));
  }
}

}  // namespace

cudaError_t launch_q4_append(Q4IoArgs a, int dtype, int d, cudaStream_t st, bool pdl) {
  a.cap_blk = (a.capacity + kQ4Tokens - 1) / kQ4Tokens;
  a.n_blk = min(a.cap_blk, (a.n + kQ4Tokens - 1) / kQ4Tokens + 1);
  const dim3 grid((unsigned)((long long)a.S * a.Hkv * a.n_blk));
  if (dtype == kDtypeBF16)
    return d == 128 ? launch_kernel(q4_append_kernel<__nv_bfloat16, 128>, grid, dim3(kThreads), 0, st, pdl, a)
                    : launch_kernel(q4_append_kernel<__nv_bfloat16, 64>, grid, dim3(kThreads), 0, st, pdl, a);
  return d == 128 ? launch_kernel(q4_append_kernel<float, 128>, grid, dim3(kThreads), 0, st, pdl, a)
                  : launch_kernel(q4_append_kernel<float, 64>, grid, dim3(kThreads), 0, st, pdl, a);
}

cudaError_t launch_q4_read(Q4IoArgs a, int dtype, int d, cudaStream_t st) {
  a.cap_blk = (a.capacity + kQ4Tokens - 1) / kQ4Tokens;
  a.n_blk = min(a.cap_blk, (a.n + kQ4Tokens - 1) / kQ4Tokens + 1);
  const dim3 grid((unsigned)((long long)a.S * a.Hkv * a.n_blk));
  if (dtype == kDtypeBF16)
    return d == 128 ? launch_kernel(q4_read_kernel<__nv_bfloat16, 128>, grid, dim3(kThreads), 0, st, false, a)
                    : launch_kernel(q4_read_kernel<__nv_bfloat16, 64>, grid, dim3(kThreads), 0, st, false, a);
  return d == 128 ? launch_kernel(q4_read_kernel<float, 128>, grid, dim3(kThreads), 0, st, false, a)
                  : launch_kernel(q4_read_kernel<float, 64>, grid, dim3(kThreads), 0, st, false, a);
}

}  // namespace skv
