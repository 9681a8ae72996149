// Writing the 4-bit cache and reading it back (format: q4_cache.cuh).
//
// Both kernels give a block of threads one 32-token block of one (stream, KV
// head).  A V word holds codes of eight tokens, so a block that is only partly
// covered by an append is read, merged and written by the one thread block that
// owns it; no two thread blocks of a call share a word.
#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"
#include "tc_common.cuh"

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

// The scale of a group: (hi - m) / 15 rounded up to bfloat16.  The float32
// quotient is off by at most 3 x 2^-24; where that could change the rounding
// (the quotient on or next to a bfloat16 value, or far from 1) float64 decides.
__device__ __forceinline__ float round_scale(float hi, float m) {
  const float q = (hi - m) * (1.f / 15.f);
  const uint32_t below = __float_as_uint(q * (1.f - 0x1p-21f)) + 0xffffu, above = __float_as_uint(q * (1.f + 0x1p-21f)) + 0xffffu;
  uint32_t bits = above;
  if (((below ^ above) & 0xffff0000u) || !(q >= 0x1p-100f && q <= 0x1p100f))
    bits = __float_as_uint(__double2float_ru(((double)hi - (double)m) / 15.0)) + 0xffffu;
  return __uint_as_float(bits & 0xffff0000u);
}

// Codes of one token row held by a warp, E channels per lane; kLanes lanes
// share a group.  Returns the packed (s, m) of the lane's group.
//   y = (x - m) * (1/s) in float32 is off by at most 15 x 3 x 2^-24 < 2^-18;
//   where that could change the nearest integer float64 decides, so the codes
//   are those of the exact quotient.
template <int E, int kLanes>
__device__ __forceinline__ uint32_t quantise(const float (&x)[E], uint32_t (&c)[E]) {
  float lo = x[0], hi = x[0], big = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    big += x[e] - x[e];  // 0, or NaN where x is a NaN or an infinity
  }
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const unsigned group = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  const bool odd = (__ballot_sync(0xffffffffu, big != 0.f) & group) != 0;
  // round down to bfloat16 on the bit pattern
  uint32_t mb = __float_as_uint(lo);
  if ((mb & 0xffffu) && (mb >> 31)) mb += 0x10000u;
  mb &= 0xffff0000u;
  const float m = __uint_as_float(mb);
  const bool bad = odd || !(fabsf(m) < INFINITY);
  const float s = round_scale(hi, m);
  const float r = s > 0.f ? 1.f / s : 0.f;
  bool near = s > 0.f && !(s >= 0x1p-100f && s <= 0x1p100f);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float y = (x[e] - m) * r;
    const float t = y + 12582912.f;  // 1.5 x 2^23: the nearest integer in the low bits, ties to even
    c[e] = __float_as_uint(t) & 15u;
    near |= fabsf(fabsf(y - (t - 12582912.f)) - 0.5f) < 0x1p-18f;
  }
  if (near && !bad) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      c[e] = (uint32_t)min(15, max(0, (int)rint(((double)x[e] - (double)m) / (double)s)));
  }
  return bad ? 0x7fc07fc0u : (__float_as_uint(s) >> 16) | mb;
}

template <int E>
__device__ __forceinline__ void load_channels(const __nv_bfloat16* src, float (&x)[E]) {
  if (E == 4) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(src));
    x[0] = __uint_as_float(r.x << 16), x[1] = __uint_as_float(r.x & 0xffff0000u);
    x[E - 2] = __uint_as_float(r.y << 16), x[E - 1] = __uint_as_float(r.y & 0xffff0000u);
  } else {
    const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(src));
    x[0] = __uint_as_float(r << 16), x[1] = __uint_as_float(r & 0xffff0000u);
  }
}
template <int E>
__device__ __forceinline__ void load_channels(const float* src, float (&x)[E]) {
  if (E == 4) {
    const float4 r = __ldg(reinterpret_cast<const float4*>(src));
    x[0] = r.x, x[1] = r.y, x[E - 2] = r.z, x[E - 1] = r.w;
  } else {
    const float2 r = __ldg(reinterpret_cast<const float2*>(src));
    x[0] = r.x, x[1] = r.y;
  }
}

// Append.  A warp quantises one token's key or value at a time (coalesced
// loads, four rows in flight); the codes meet in shared memory as bytes, are
// packed there into the block's final image and leave as 16-byte stores.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(Q4IoArgs a) {
  using B = Q4Block<D>;
  constexpr int E = D / 32, kLanes = kQ4Group / E;
  constexpr int kPitch = D + 4;  // code row in bytes, padded by a bank
  __shared__ __align__(16) uint8_t codes[2 * kQ4Tokens * kPitch];
  __shared__ __align__(16) uint8_t image[B::kBytes];
  pdl_wait();
  pdl_trigger();
  const int sg = blockIdx.x / a.n_blk, s = sg / a.Hkv, g = sg % a.Hkv;
  const Span sp = span_of(a, s);
  const int b = sp.p0 / kQ4Tokens + blockIdx.x % a.n_blk;
  if ((long long)b * kQ4Tokens >= sp.p1 || sp.p0 >= sp.p1) return;
  const int t_lo = max(sp.p0 - b * kQ4Tokens, 0), t_hi = min(sp.p1 - b * kQ4Tokens, kQ4Tokens);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // rows 0..31 keys, 32..63 values; a warp takes rows warp, warp + 8, ...
  constexpr int kAtOnce = 4;
  for (int r0 = warp; r0 < 2 * kQ4Tokens; r0 += kAtOnce * (kThreads / 32)) {
    float x[kAtOnce][E];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = r0 + i * (kThreads / 32), kv = r >> 5, t = r & 31;
      if (t >= t_lo && t < t_hi) {
        const long long tok = (long long)b * kQ4Tokens + t - sp.start;
        load_channels(static_cast<const T*>(kv ? a.v : a.k) + (((long long)s * a.n + tok) * a.Hkv + g) * D + lane * E, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = r0 + i * (kThreads / 32), kv = r >> 5, t = r & 31;
      uint32_t c[E];
      const uint32_t sm = quantise<E, kLanes>(x[i], c);
      if (E == 4) *reinterpret_cast<uint32_t*>(codes + r * kPitch + lane * 4) = c[0] | c[1] << 8 | c[E - 2] << 16 | c[E - 1] << 24;
      else *reinterpret_cast<uint16_t*>(codes + r * kPitch + lane * 2) = (uint16_t)(c[0] | c[1] << 8);
      if (lane % kLanes == 0)
        reinterpret_cast<uint32_t*>(image + (kv ? B::kVs : B::kKs))[t * B::kGroups + lane / kLanes] = sm;
    }
  }
  __syncthreads();
  // K words: eight channels of a token
  for (int w = threadIdx.x; w < kQ4Tokens * (D / 8); w += kThreads) {
    const int t = w / (D / 8), c8 = w % (D / 8);
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + t * kPitch + c8 * 8);
    const uint32_t x = c[0], y = c[1];
    *reinterpret_cast<uint32_t*>(image + t * B::kRow + ((c8 % 8) / 2) * (D / 8) + ((c8 / 8) * 2 + c8 % 2) * 4) =
        q4_pack((x & 0xffu) | (x & 0xff00u) << 8, (x >> 16 & 0xffu) | (x >> 24) << 16, (y & 0xffu) | (y & 0xff00u) << 8,
                (y >> 16 & 0xffu) | (y >> 24) << 16);
  }
  // V words: eight tokens of a channel; a thread takes four channels
  for (int w = threadIdx.x; w < D; w += kThreads) {
    const int d4 = w % (D / 4), tig = w / (D / 4);
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = (i >> 2) * 16 + ((i >> 1) & 1) * 8 + 2 * tig + (i & 1);
      x[i] = *reinterpret_cast<const uint32_t*>(codes + (kQ4Tokens + t) * kPitch + d4 * 4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t p[4];
#pragma unroll
      for (int f = 0; f < 4; ++f)  // byte e of two tokens into the halves
        p[f] = (x[2 * f] >> (8 * e) & 0xffu) | (x[2 * f + 1] >> (8 * e) & 0xffu) << 16;
      *reinterpret_cast<uint32_t*>(image + B::kV + q4_v_word(d4 * 4 + e, tig)) = q4_pack(p[0], p[1], p[2], p[3]);
    }
  }
  __syncthreads();
  uint8_t* blk = static_cast<uint8_t*>(a.cache) + ((long long)sg * a.cap_blk + b) * B::kBytes;
  if (t_lo == 0 && t_hi == kQ4Tokens) {
    for (int w = threadIdx.x; w < B::kBytes / 16; w += kThreads)
      reinterpret_cast<uint4*>(blk)[w] = reinterpret_cast<const uint4*>(image)[w];
    return;
  }
  // a partly covered block: K rows and scales of its tokens, V words merged
  for (int w = threadIdx.x; w < B::kV / 4; w += kThreads)
    if (w / (B::kRow / 4) >= t_lo && w / (B::kRow / 4) < t_hi)
      reinterpret_cast<uint32_t*>(blk)[w] = reinterpret_cast<const uint32_t*>(image)[w];
  for (int w = threadIdx.x; w < 2 * kQ4Tokens * B::kGroups; w += kThreads) {
    const int t = w / B::kGroups % kQ4Tokens;
    if (t >= t_lo && t < t_hi)
      reinterpret_cast<uint32_t*>(blk + B::kKs)[w] = reinterpret_cast<const uint32_t*>(image + B::kKs)[w];
  }
  for (int w = threadIdx.x; w < B::kV / 16; w += kThreads) {
    uint32_t keep[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int t = (f >> 1) * 16 + (f & 1) * 8 + 2 * (w & 3);
      keep[f] = (t >= t_lo && t < t_hi ? 0u : 15u) | (t + 1 >= t_lo && t + 1 < t_hi ? 0u : 15u << 16);
    }
    const uint32_t mask = q4_pack(keep[0], keep[1], keep[2], keep[3]);
    if (mask == 0xffffffffu) continue;
    uint4* dst = reinterpret_cast<uint4*>(blk + B::kV) + w;
    const uint4 o = *dst, n = reinterpret_cast<const uint4*>(image + B::kV)[w];
    *dst = make_uint4((o.x & mask) | (n.x & ~mask), (o.y & mask) | (n.y & ~mask), (o.z & mask) | (n.z & ~mask),
                      (o.w & mask) | (n.w & ~mask));
  }
}

// Eight values m + c s of a word's codes picked by the caller: code bits 6..9 of
// a half as the top mantissa bits of 16 + c.
__device__ __forceinline__ float low_value(uint32_t field, float s, float m) {
  return fmaf(__uint_as_float((field << 13 & 0x00780000u) | 0x41800000u) - 16.f, s, m);
}
__device__ __forceinline__ float high_value(uint32_t field, float s, float m) {
  return fmaf(__uint_as_float((field >> 3 & 0x00780000u) | 0x41800000u) - 16.f, s, m);
}
__device__ __forceinline__ uint32_t field_of(uint32_t x, int f) {
  return f == 0 ? q4_field<0>(x) : f == 1 ? q4_field<1>(x) : f == 2 ? q4_field<2>(x) : q4_field<3>(x);
}
__device__ __forceinline__ void store_channels(__nv_bfloat16* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(tc::pack_bf16x2(x[0], x[1]), tc::pack_bf16x2(x[2], x[3]),
                                              tc::pack_bf16x2(x[4], x[5]), tc::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store_channels(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Read back: the block comes into shared memory in 16-byte loads; half of the D
// threads take eight tokens x eight channels of V each (a word holds eight
// tokens), the other half as much of K.
template <typename T, int D>
__global__ void __launch_bounds__(D) q4_read_kernel(Q4IoArgs a) {
  using B = Q4Block<D>;
  __shared__ __align__(16) uint8_t image[B::kBytes];
  const int sg = blockIdx.x / a.n_blk, s = sg / a.Hkv, g = sg % a.Hkv;
  const Span sp = span_of(a, s);
  const int b = sp.p0 / kQ4Tokens + blockIdx.x % a.n_blk;
  if ((long long)b * kQ4Tokens >= sp.p1 || sp.p0 >= sp.p1) return;
  const int t_lo = max(sp.p0 - b * kQ4Tokens, 0), t_hi = min(sp.p1 - b * kQ4Tokens, kQ4Tokens);
  const uint4* blk = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.cache) +
                                                    ((long long)sg * a.cap_blk + b) * B::kBytes);
#pragma unroll
  for (int w = 0; w < (B::kBytes / 16 + D - 1) / D; ++w)
    if (w * D + threadIdx.x < B::kBytes / 16) reinterpret_cast<uint4*>(image)[w * D + threadIdx.x] = __ldg(blk + w * D + threadIdx.x);
  __syncthreads();
  const long long row0 = ((long long)s * a.n + (long long)b * kQ4Tokens - sp.start) * a.Hkv + g;
  if (threadIdx.x < D / 2) {
    const int tig = threadIdx.x & 3, c8 = threadIdx.x >> 2;
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = *reinterpret_cast<const uint32_t*>(image + B::kV + q4_v_word(c8 * 8 + e, tig));
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int t = (f >> 1) * 16 + (f & 1) * 8 + 2 * tig + hi;
        if (t < t_lo || t >= t_hi) continue;
        const uint32_t sm = reinterpret_cast<const uint32_t*>(image + B::kVs)[t * B::kGroups + c8 / 8];
        const float sc = q4_scale(sm), m = q4_min(sm);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = hi ? high_value(field_of(x[e], f), sc, m) : low_value(field_of(x[e], f), sc, m);
        store_channels(static_cast<T*>(a.v_out) + (row0 + (long long)t * a.Hkv) * D + c8 * 8, v);
      }
  } else {
    const int i = threadIdx.x - D / 2, c8 = i % (D / 8);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int t = i / (D / 8) + n * 4;
      if (t < t_lo || t >= t_hi) continue;
      const uint32_t x = *reinterpret_cast<const uint32_t*>(image + t * B::kRow + ((c8 % 8) / 2) * (D / 8) + ((c8 / 8) * 2 + c8 % 2) * 4);
      const uint32_t sm = reinterpret_cast<const uint32_t*>(image + B::kKs)[t * B::kGroups + c8 / 8];
      const float sc = q4_scale(sm), m = q4_min(sm);
      float v[8];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        v[2 * f] = low_value(field_of(x, f), sc, m);
        v[2 * f + 1] = high_value(field_of(x, f), sc, m);
      }
      store_channels(static_cast<T*>(a.k_out) + (row0 + (long long)t * a.Hkv) * D + c8 * 8, v);
    }
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
    return d == 128 ? launch_kernel(q4_read_kernel<__nv_bfloat16, 128>, grid, dim3(d), 0, st, false, a)
                    : launch_kernel(q4_read_kernel<__nv_bfloat16, 64>, grid, dim3(d), 0, st, false, a);
  return d == 128 ? launch_kernel(q4_read_kernel<float, 128>, grid, dim3(d), 0, st, false, a)
                  : launch_kernel(q4_read_kernel<float, 64>, grid, dim3(d), 0, st, false, a);
}

}  // namespace skv
