// Layout and arithmetic of the 4-bit key/value cache.
//
// Quantisation, per token, KV head and group of 64 consecutive channels (keys
// and values alike):
//   m = the group's smallest value, rounded down to bfloat16,
//   s = (largest - m) / 15, rounded up to bfloat16,
//   c = the integer nearest to (x - m) / s, ties to even (0 where s = 0),
// so c is in 0..15 and x ~ m + c s with an error of at most s / 2.  Rounding m
// down and s up keeps the whole group inside [m, m + 15 s]; bfloat16 keeps the
// range of the inputs, at 4 + 32 / 64 = 4.5 bits a value.  c * s is exact in
// float32 (4 x 8 bits), so m + c s is one rounding.  A group that holds a NaN
// or an infinity (or whose m leaves bfloat16's range) stores s = m = NaN and
// reads back as NaN.
//
// The cache is [S][Hkv][ceil(capacity / 32)] blocks of 32 tokens, a block one
// contiguous run of bytes:
//   K codes  [32 tokens][D/2 bytes]      16 D bytes
//   V codes  [D/32 chunks][32 lanes][16]  16 D bytes
//   K scales [32 tokens][D/64]            4 bytes each: s in the low half, m in the high
//   V scales [32 tokens][D/64]
// The code words are laid out as the fragments of an m16n8k16 tensor-core
// product with 16 tokens (K) or 16 channels (V) as its rows, lane = 4 gid + tig:
//   K: token row, tig's 4 (D=128) or 2 (D=64) words; word w holds channels
//      64 (w/2) + 16 tig + 8 (w%2) + 0..7;
//   V: word (channel d, tig) holds the tokens {2 tig, 2 tig + 1, 8 + 2 tig,
//      9 + 2 tig} and the same + 16; d = 8 j + gid sits in chunk j/4, lane
//      4 gid + tig, word j%4.
// Inside a word the eight codes are four pairs (field f: one code in the low
// half, one in the high), placed so that an and-or turns a pair into two fp16
// numbers: fields 0 and 2 of the word itself, 3 and 1 of the word rotated left
// by eight bits; 16 + c for 0 and 3 (code at mantissa bits 6..9), 256 + c for 2
// and 1 (bits 2..5).  As nibbles, rotated left by two bits, a word is
//   n      0    1    2    3    4    5    6    7
//   field  2 l  0 l  1 h  3 h  2 h  0 h  1 l  3 l      (l, h: low, high half)
// K: nibble n is channel n of the word's eight.  V: field f holds the tokens
// 16 (f/2) + 8 (f%2) + 2 tig (low) and the next (high).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace skv {

constexpr int kQ4Tokens = 32;  // tokens per block
constexpr int kQ4Group = 64;   // channels per scale

template <int D>
struct Q4Block {
  static constexpr int kGroups = D / kQ4Group;
  static constexpr int kRow = D / 2;                      // K code bytes of a token
  static constexpr int kV = kQ4Tokens * kRow;             // V codes
  static constexpr int kKs = 2 * kV;                      // K scales
  static constexpr int kVs = kKs + kQ4Tokens * kGroups * 4;
  static constexpr int kBytes = kVs + kQ4Tokens * kGroups * 4;  // 4608 (D=128), 2304 (D=64)
};

__host__ __device__ constexpr int q4_block_bytes(int d) { return 32 * d + 256 * (d / kQ4Group); }

// pairs (low code | high code << 16) of fields 0..3 -> word
__host__ __device__ __forceinline__ uint32_t q4_pack(uint32_t p0, uint32_t p1, uint32_t p2, uint32_t p3) {
  const uint32_t r = (p3 << 6) | (p1 << 2);
  return (p0 << 6) | (p2 << 2) | ((r >> 8) | (r << 24));
}
// Field f of a word as fp16 numbers kQ4Bias<f> + c.
__device__ __forceinline__ uint32_t q4_turn(uint32_t x) { return __funnelshift_l(x, x, 8); }
template <int F>
struct Q4Bias {
  static constexpr float value = F == 0 || F == 3 ? 16.f : 256.f;
};
// x: the word (fields 0, 2) or the word turned (fields 1, 3)
template <int F>
__device__ __forceinline__ uint32_t q4_raw(uint32_t x) {
  return F == 0 || F == 3 ? (x & 0x03C003C0u) | 0x4C004C00u : (x & 0x003C003Cu) | 0x5C005C00u;
}
// Field f of a word, each code at bits 6..9 of its half.
__device__ __forceinline__ uint32_t q4_field(uint32_t x, int f) {
  if (f & 1) x = q4_turn(x);
  if (f == 1 || f == 2) x <<= 4;
  return x & 0x03C003C0u;
}
// Field and half of nibble n, and the K channel of (field, half).
__host__ __device__ __forceinline__ constexpr int q4_field_of(int n) { return 0x31023102 >> (4 * n) & 3; }
__host__ __device__ __forceinline__ constexpr int q4_half_of(int n) { return 0x3C >> n & 1; }
__host__ __device__ __forceinline__ constexpr int q4_k_channel(int f, int half) {
  return (half ? 0x3425 : 0x7061) >> (4 * f) & 7;
}
// Eight nibbles -> word.
__device__ __forceinline__ uint32_t q4_rotate(uint32_t nibbles) { return __funnelshift_l(nibbles, nibbles, 2); }

__device__ __forceinline__ float q4_scale(uint32_t sm) { return __uint_as_float(sm << 16); }
__device__ __forceinline__ float q4_min(uint32_t sm) { return __uint_as_float(sm & 0xffff0000u); }

// Byte offset of the V word of (channel d, tig) within a block.
__device__ __forceinline__ int q4_v_word(int d, int tig) {
  const int j = d >> 3;
  return (j >> 2) * 512 + ((d & 7) * 4 + tig) * 16 + (j & 3) * 4;
}

// E consecutive channels from ch0 (a multiple of E, E divides 8) of token t of a block.
template <int D, int E>
__device__ __forceinline__ void q4_token(const uint8_t* blk, int t, int ch0, float (&k)[E], float (&v)[E]) {
  using B = Q4Block<D>;
  auto word = [&](int at) { return __ldg(reinterpret_cast<const uint32_t*>(blk + at)); };
  const int c8 = ch0 >> 3, gg = ch0 / kQ4Group;
  const uint32_t ks = word(B::kKs + (t * B::kGroups + gg) * 4), vs = word(B::kVs + (t * B::kGroups + gg) * 4);
  const uint32_t kw = word(t * B::kRow + ((c8 & 7) >> 1) * (D / 8) + ((c8 >> 3) * 2 + (c8 & 1)) * 4);
  const int tig = (t & 7) >> 1, n = q4_k_channel((t >> 4) * 2 + (t >> 3 & 1), t & 1);  // the token's nibble in V's words
  auto value = [](uint32_t w, int nibble, uint32_t sm) {
    return fmaf((float)(__funnelshift_r(w, w, 2) >> (4 * nibble) & 15u), q4_scale(sm), q4_min(sm));
  };
#pragma unroll
  for (int e = 0; e < E; ++e) {
    k[e] = value(kw, (ch0 & 7) + e, ks);
    v[e] = value(word(B::kV + q4_v_word(ch0 + e, tig)), n, vs);
  }
}

}  // namespace skv
