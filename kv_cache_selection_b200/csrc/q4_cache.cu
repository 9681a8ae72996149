// Writing the 4-bit cache and reading it back (format: q4_cache.cuh).
//
// Both kernels give a block of threads one 32-token block of one (stream, KV
// head).  A V word holds codes of eight tokens, so a block that is only partly
// covered by an append is read, merged and written by the one thread block that
// owns it; no two thread blocks of a call share a word.
//
// Measured (B200, graph replays, 131072 tokens of 4 heads, d = 128, inputs beyond
// L2): append in bf16 94 us (268 MB in, 75 MB out: 3.7 TB/s), bound by instructions
// (82 % of the issue slots; the group ranges, exact ties and the packing), in float32
// 110 us (537 MB in: 5.6 TB/s); read in bf16 58 us (5.9 TB/s), in float32 139 us (4.4
// TB/s), bound by memory writes.  Sizes that no longer fill the SMs are bound by
// latency: a 256-token frame is appended and read back in 6.5 us, two launches of four
// dependent passes and one.
#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"
#include "tc_common.cuh"

namespace skv {
namespace {

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

// min and max that give NaN where an operand is one
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// a - b as d + e exactly (e: what the rounding of d lost)
__device__ __forceinline__ float exact_difference(float a, float b, float& e) {
  const float d = __fsub_rn(a, b), z = __fsub_rn(d, a);
  e = __fsub_rn(__fsub_rn(a, __fsub_rn(d, z)), __fadd_rn(b, z));
  return d;
}

// The scale of a group: (hi - m) / 15 rounded up to bfloat16.  The bfloat16
// value nearest to the float32 quotient is the result or its lower neighbour;
// the sign of 15 s - (hi - m), exact in one fma, tells which (where the
// difference itself was rounded and the fma gives 0, the rest decides).
__device__ __forceinline__ float round_scale(float hi, float m) {
  float rest;
  const float d = exact_difference(hi, m, rest), q = d * (1.f / 15.f);
  if (!(q >= 0x1p-100f && q <= 0x1p100f))  // far from 1 (or 0, or NaN): float64
    return __uint_as_float((__float_as_uint(__double2float_ru(((double)hi - (double)m) / 15.0)) + 0xffffu) & 0xffff0000u);
  uint32_t bits = (__float_as_uint(q) + 0x8000u) & 0xffff0000u;
  const float off = fmaf(__uint_as_float(bits), 15.f, -d);
  if (off < 0.f || (off == 0.f && rest > 0.f)) bits += 0x10000u;
  return __uint_as_float(bits);
}

// What to add to c, at most 1 away from it, for the integer nearest to
// (x - m) / s, ties to even: the remainder x - m - c s is exact in float32 (it is
// at most s and a multiple of the last place of x - m), so its place against
// s / 2 is, too.
__device__ __forceinline__ int settle(float x, float m, float s, int c) {
  float rest;
  const float d = exact_difference(x, m, rest);
  const float e = fmaf(-(float)c, s, d), half = 0.5f * s;
  const bool odd = c & 1;
  if (e > half || (e == half && (rest > 0.f || (rest == 0.f && odd)))) return 1;
  if (e < -half || (e == -half && (rest < 0.f || (rest == 0.f && odd)))) return -1;
  return 0;
}
// x[e]
__device__ __forceinline__ float pick(const float (&x)[8], int e) {
  const bool b0 = e & 1, b1 = e & 2, b2 = e & 4;
  const float p = b0 ? x[1] : x[0], q = b0 ? x[3] : x[2], r = b0 ? x[5] : x[4], t = b0 ? x[7] : x[6];
  const float u = b1 ? q : p, v = b1 ? t : r;
  return b2 ? v : u;
}

// Smallest and largest of the four lanes that hold a group, NaN if any is one.
__device__ __forceinline__ void group_range(float& lo, float& hi) {
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Sixteen channels as loaded, as float32 (eight of them), and the range of their group.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  uint4 r[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r[0] = __ldg(reinterpret_cast<const uint4*>(p));
    r[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { r[0] = r[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(int half, float (&x)[8]) const {
    const uint32_t w[4] = {r[half].x, r[half].y, r[half].z, r[half].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // (smallest, -largest) as one bf16 pair: one shuffle a step for both
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    const uint32_t mn = min2_nan(min2_nan(min2_nan(r[0].x, r[0].y), min2_nan(r[0].z, r[0].w)),
                                 min2_nan(min2_nan(r[1].x, r[1].y), min2_nan(r[1].z, r[1].w)));
    const uint32_t mx = max2_nan(max2_nan(max2_nan(r[0].x, r[0].y), max2_nan(r[0].z, r[0].w)),
                                 max2_nan(max2_nan(r[1].x, r[1].y), max2_nan(r[1].z, r[1].w)));
    uint32_t p = min2_nan(__byte_perm(mn, mx, 0x5410) ^ 0x80000000u, __byte_perm(mn, mx, 0x7632) ^ 0x80000000u);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) p = min2_nan(p, __shfl_xor_sync(0xffffffffu, p, off));
    lo = __uint_as_float(p << 16);
    hi = __uint_as_float((p & 0xffff0000u) ^ 0x80000000u);
  }
};
template <>
struct Raw16<float> {
  float4 r[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(int half, float (&x)[8]) const {
    const float4 a = r[2 * half], b = r[2 * half + 1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    lo = hi = r[0].x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo = min_nan(lo, min_nan(min_nan(r[i].x, r[i].y), min_nan(r[i].z, r[i].w)));
      hi = max_nan(hi, max_nan(max_nan(r[i].x, r[i].y), max_nan(r[i].z, r[i].w)));
    }
    group_range(lo, hi);
  }
};

// Smallest value and scale of a group.
struct Scale {
  float m, s, r;     // r: about 1 / s, 0 where s is not above 0
  bool bad, small;   // not finite; s too far from 1 for r
  __device__ __forceinline__ uint32_t packed() const {
    return bad ? 0x7fc07fc0u : (__float_as_uint(s) >> 16) | __float_as_uint(m);
  }
};
__device__ __forceinline__ Scale scale_of(float lo, float hi) {
  Scale g;
  uint32_t mb = __float_as_uint(lo);  // rounded down to bfloat16 on the bit pattern
  if ((mb & 0xffffu) && (mb >> 31)) mb += 0x10000u;
  g.m = __uint_as_float(mb & 0xffff0000u);
  g.bad = !(fabsf(hi) < INFINITY && fabsf(g.m) < INFINITY);
  g.s = round_scale(hi, g.m);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.r) : "f"(g.s));
  if (!(g.s > 0.f)) g.r = 0.f;
  g.small = g.s > 0.f && !(g.s >= 0x1p-100f && g.s <= 0x1p100f);
  return g;
}

// Codes of eight channels as nibbles (channel e at bits 4e).  y = (x - m) * (1/s)
// in float32 is off by less than 2^-17 (a quotient of at most 15, five half steps
// of relative 2^-24); only where that could change the nearest integer is the
// code settled exactly.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], const Scale& g) {
  const float m = g.m, s = g.s, r = g.r;
  const float2 r2 = make_float2(r, r), nm2 = make_float2(-m, -m), magic = make_float2(12582912.f, 12582912.f);
  const float2 unmagic = make_float2(-12582912.f, -12582912.f);
  float far = 0.f;  // distance from the nearest integer
  float c[8], y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 d = tc::fadd2(make_float2(x[2 * i], x[2 * i + 1]), nm2);
    const float2 t = tc::ffma2(d, r2, magic);  // 1.5 x 2^23 + the nearest integer
    const float2 f = tc::fadd2(t, unmagic);
    const float2 e = tc::ffma2(d, r2, make_float2(-f.x, -f.y));
    c[2 * i] = f.x;
    c[2 * i + 1] = f.y;
    y[2 * i] = e.x;
    y[2 * i + 1] = e.y;
    far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
  }
  // four codes as one float32 integer below 2^16, exactly
  float2 w = make_float2(c[3], c[7]);
#pragma unroll
  for (int e = 2; e >= 0; --e) w = tc::ffma2(w, make_float2(16.f, 16.f), make_float2(c[e], c[e + 4]));
  w = tc::fadd2(w, make_float2(8388608.f, 8388608.f));
  uint32_t word = __byte_perm(__float_as_uint(w.x), __float_as_uint(w.y), 0x5410);
  if ((far > 0.5f - 0x1p-17f || g.small) && !g.bad) {
    if (g.small) {
      word = 0;
#pragma unroll 1
      for (int e = 0; e < 8; ++e)
        word |= (uint32_t)min(15, max(0, (int)rint(((double)pick(x, e) - (double)m) / (double)s))) << (4 * e);
    } else {
      uint32_t todo = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) todo |= fabsf(y[k]) > 0.5f - 0x1p-17f ? 1u << k : 0u;
      while (todo) {  // rarely more than one
        const int e = __ffs(todo) - 1;
        todo &= todo - 1;
        word += (uint32_t)settle(pick(x, e), m, s, (int)(word >> (4 * e) & 15u)) << (4 * e);
      }
    }
  }
  return word;
}

// 8 x 8 nibbles transposed: nibble e of row n -> nibble n of row e
__device__ __forceinline__ void transpose_nibbles(uint32_t (&a)[8]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint32_t x = a[n], y = a[n + 4];
    a[n] = __byte_perm(x, y, 0x5410);
    a[n + 4] = __byte_perm(x, y, 0x7632);
  }
#pragma unroll
  for (int h = 0; h < 8; h += 4)
#pragma unroll
    for (int n = h; n < h + 2; ++n) {
      const uint32_t x = a[n], y = a[n + 2];
      a[n] = __byte_perm(x, y, 0x6240);
      a[n + 2] = __byte_perm(x, y, 0x7351);
    }
#pragma unroll
  for (int n = 0; n < 8; n += 2) {
    const uint32_t x = a[n], y = a[n + 1];
    a[n] = (x & 0x0f0f0f0fu) | (y & 0x0f0f0f0fu) << 4;
    a[n + 1] = (x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
  }
}

// Append.  A lane quantises sixteen channels of a token's key or value, D/16
// lanes a token, with the next token's loads in flight (with eight channels a
// lane the group's range and scale, which each of its lanes computes, cost as
// much as the codes: 130 us where this takes 99).  Eight channels of a key are one word of the block; values
// go through shared memory as nibbles, where a thread transposes eight tokens x
// eight channels into V's words.  The block's image leaves as 16-byte stores.
constexpr int kAppendThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) q4_append_kernel(Q4IoArgs a) {
  using B = Q4Block<D>;
  constexpr int kUnits = D / 8;                            // eight-channel units of a token
  constexpr int kRowLanes = D / 16;                        // lanes of a token
  constexpr int kRowsAtOnce = kAppendThreads / kRowLanes;  // tokens per pass of the block
  constexpr int kPasses = 2 * kQ4Tokens / kRowsAtOnce;
  static_assert(kPasses % 2 == 0, "a pass is all keys or all values");
  __shared__ __align__(16) uint8_t image[B::kBytes];
  __shared__ uint32_t vn[kQ4Tokens][kUnits + 1];      // nibbles of the values
  pdl_wait();
  pdl_trigger();
  const int sg = blockIdx.x / a.n_blk, s = sg / a.Hkv, g = sg % a.Hkv;
  const Span sp = span_of(a, s);
  const int b = sp.p0 / kQ4Tokens + blockIdx.x % a.n_blk;
  if ((long long)b * kQ4Tokens >= sp.p1 || sp.p0 >= sp.p1) return;
  const int t_lo = max(sp.p0 - b * kQ4Tokens, 0), t_hi = min(sp.p1 - b * kQ4Tokens, kQ4Tokens);
  const int c16 = threadIdx.x % kRowLanes, r_of = threadIdx.x / kRowLanes;
  // rows 0..31 keys, 32..63 values; this thread's token of pass p is
  // (p % (kPasses / 2)) * kRowsAtOnce + r_of
  const long long first = (((long long)s * a.n + (long long)b * kQ4Tokens - sp.start + r_of) * a.Hkv + g) * D + c16 * 16;
  const T* k_row = static_cast<const T*>(a.k) + first;
  const T* v_row = static_cast<const T*>(a.v) + first;
  const long long pass_stride = (long long)kRowsAtOnce * a.Hkv * D;
  // the two words of a lane's sixteen key channels are neighbours
  uint8_t* k_word = image + r_of * B::kRow + (c16 % 4) * (D / 8) + (c16 / 4) * 8;
  Raw16<T> next;
  auto fetch = [&](int p) {
    const int pp = p % (kPasses / 2), t = pp * kRowsAtOnce + r_of;
    if (t >= t_lo && t < t_hi) next.load((p >= kPasses / 2 ? v_row : k_row) + pp * pass_stride);
    else next.zero();
  };
  fetch(0);
#pragma unroll 1
  for (int p = 0; p < kPasses; ++p) {
    const bool is_v = p >= kPasses / 2;
    const int t0 = p % (kPasses / 2) * kRowsAtOnce;
    const Raw16<T> now = next;
    if (p + 1 < kPasses) fetch(p + 1);
    float lo, hi, x[8];
    now.range(lo, hi);
    const Scale sc = scale_of(lo, hi);
    now.get(0, x);
    const uint32_t w0 = quantise8(x, sc);
    now.get(1, x);
    const uint32_t w1 = quantise8(x, sc);
    if (is_v) {
      vn[t0 + r_of][2 * c16] = w0;
      vn[t0 + r_of][2 * c16 + 1] = w1;
    } else {
      *reinterpret_cast<uint2*>(k_word + t0 * B::kRow) = make_uint2(q4_rotate(w0), q4_rotate(w1));
    }
    if (c16 % 4 == 0)
      reinterpret_cast<uint32_t*>(image + (is_v ? B::kVs : B::kKs))[(t0 + r_of) * B::kGroups + c16 / 4] = sc.packed();
  }
  __syncthreads();
  if (threadIdx.x < kUnits * 4) {
    const int j = threadIdx.x % kUnits, tig = threadIdx.x / kUnits;
    uint32_t w[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int f = q4_field_of(n);  // field f: tokens 16 (f/2) + 8 (f%2) + 2 tig and the next
      w[n] = vn[(f >> 1) * 16 + (f & 1) * 8 + 2 * tig + q4_half_of(n)][j];
    }
    transpose_nibbles(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) *reinterpret_cast<uint32_t*>(image + B::kV + q4_v_word(j * 8 + e, tig)) = q4_rotate(w[e]);
  }
  __syncthreads();
  uint8_t* blk = static_cast<uint8_t*>(a.cache) + ((long long)sg * a.cap_blk + b) * B::kBytes;
  if (t_lo == 0 && t_hi == kQ4Tokens) {
    for (int w = threadIdx.x; w < B::kBytes / 16; w += kAppendThreads)
      reinterpret_cast<uint4*>(blk)[w] = reinterpret_cast<const uint4*>(image)[w];
    return;
  }
  // a partly covered block: K rows and scales of its tokens, V words merged
  for (int w = threadIdx.x; w < B::kV / 4; w += kAppendThreads)
    if (w / (B::kRow / 4) >= t_lo && w / (B::kRow / 4) < t_hi)
      reinterpret_cast<uint32_t*>(blk)[w] = reinterpret_cast<const uint32_t*>(image)[w];
  for (int w = threadIdx.x; w < 2 * kQ4Tokens * B::kGroups; w += kAppendThreads) {
    const int t = w / B::kGroups % kQ4Tokens;
    if (t >= t_lo && t < t_hi)
      reinterpret_cast<uint32_t*>(blk + B::kKs)[w] = reinterpret_cast<const uint32_t*>(image + B::kKs)[w];
  }
  for (int w = threadIdx.x; w < B::kV / 16; w += kAppendThreads) {
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
        for (int e = 0; e < 8; ++e) v[e] = hi ? high_value(q4_field(x[e], f), sc, m) : low_value(q4_field(x[e], f), sc, m);
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
        v[q4_k_channel(f, 0)] = low_value(q4_field(x, f), sc, m);
        v[q4_k_channel(f, 1)] = high_value(q4_field(x, f), sc, m);
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
    return d == 128 ? launch_kernel(q4_append_kernel<__nv_bfloat16, 128>, grid, dim3(kAppendThreads), 0, st, pdl, a)
                    : launch_kernel(q4_append_kernel<__nv_bfloat16, 64>, grid, dim3(kAppendThreads), 0, st, pdl, a);
  return d == 128 ? launch_kernel(q4_append_kernel<float, 128>, grid, dim3(kAppendThreads), 0, st, pdl, a)
                  : launch_kernel(q4_append_kernel<float, 64>, grid, dim3(kAppendThreads), 0, st, pdl, a);
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
