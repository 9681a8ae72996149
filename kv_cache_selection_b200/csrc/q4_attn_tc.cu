// Attention of many text tokens over the 4-bit cache on the 5th-generation
// tensor cores: for more query rows (heads of a KV head x text tokens) than the
// streaming kernel of q4_attn.cu takes in one pass, a 128-row tile shares every
// dequantised key tile.
//
// A thread block owns one 128-row tile of one (stream, KV head) and a range of
// 128-token key tiles.  Per key tile
//   raw blocks -> shared memory          one warp, bulk copies into a ring
//   K, V -> fp16 in shared memory        a warpgroup each
//   S = Q K^T, O += P V                  one warp; tcgen05, fp16 in, float32 accumulate
//   P = 2^(S c - m)                      two warpgroups, thread = 64 columns of a row
// with S double-buffered in tensor memory.  The two halves of a row share its
// lazy maximum: one barrier a tile tells whether either wants to raise it.
//
// Keys and values are scaled by powers of two that bring the largest magnitude in
// the block's range of tokens (read off the scales beforehand) into [2^12, 2^13),
// so fp16 serves the cache's range: full precision down to 2^-26 of the largest.
//   K: (c - 8) s has 11 bits and is exact in fp16 (down to that); the groups' m + 8 s times the
//     sums of q enter as one more product of depth 16, both sides in two fp16
//     parts.  So S is as exact as its float32 sums.
//   V: (c - 8) s + (m + 8 s) in one fp16 fma, 2^-11 of a value.
// Queries are scaled per row as in q4_attn.cu.  P is rounded to fp16.
//
// Order inside a tile: the code word (channel d, tig) of V holds eight tokens;
// as one 16-byte chunk of a row of V^T they are the slots 8 tig + 2 f + half of
// their 32-token block, so K's rows (S's columns) take the same order; a K word
// is a chunk of its row with the channels in field order, Q alike.  No value
// moves between threads.
//
// Measured (B200, graph replays, bf16, d = 128, 4 KV heads, 16 text tokens of G = 7
// over 131072 tokens): 60.0 us (30.1 GFLOP: 18.2 us of the tensor cores).  15 % is the
// exponents' pass over the scales and the first copies (17000 of 115000 cycles); then
// a key tile takes 2800 cycles, of which the softmax 2500 (its halves are in step, so
// that its exponentials, 1024 cycles, meet nobody else's).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"
#include "q4_visible.cuh"
#include "tc_common.cuh"

namespace skv {
namespace {
using namespace tc;

constexpr int kThreads = 640;
constexpr int kRaw = 3;          // raw tiles in flight
constexpr float kRaise = 8.0f;   // log2 headroom of the lazy row maximum
constexpr int kPShift = 6;       // P is held as P 2^6 (below 2^14)

__device__ int g_err;  // first error of the pipeline waits of all calls on a device

template <int D>
struct Smem {
  using B = Q4Block<D>;
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtom = 128 * 128;               // 128 rows x 64 fp16
  static constexpr int kTile = kAtoms * kAtom;          // Q or K tile
  static constexpr int kVAtom = D * 128;                // D rows x 64 slots
  static constexpr int kQ = 0;
  static constexpr int kK = kTile;                      // two K tiles
  static constexpr int kV = kK + 2 * kTile;             // two V^T tiles
  static constexpr int kRawTile = 4 * B::kBytes;
  static constexpr int kKx = kV + 2 * 2 * kVAtom;       // two tiles of 128 rows x 16 fp16, no swizzle
  static constexpr int kRawAt = kKx + 2 * 4096;
  static constexpr int kTabBytes = 16 * B::kGroups * 32;  // V scales: [4 blk][4 tig][groups][4 f] (s pair, mid pair)
  static constexpr int kTab = kRawAt + kRaw * kRawTile;
  static constexpr int kHalfMax = kTab + kTabBytes;  // [2][128] float32
  static constexpr int kTop = kHalfMax + 1024;           // largest magnitudes of K, V (float32 bits)
  static constexpr int kBar = kTop + 16;
  // read before the second K tile is written: row scales [128], group sums of q [128][groups]
  static constexpr int kRow = kK + kTile;
  static constexpr int kQs = kRow + 512;
  // raw_full[kRaw], raw_empty[kRaw], k_full[2], k_empty[2], v_full[2], v_empty[2], s[2], p[2], qx, pv, o,
  // done
  static constexpr int kNumBars = 2 * kRaw + 12 + 4;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4;
  static constexpr int kAlloc = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;  // one block per SM
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(kTab % 16 == 0 && kBar % 8 == 0, "alignment");
};

// generic-proxy writes to shared memory become visible to the tensor core
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Instruction descriptor, kind::f16: fp16 A and B (K-major), float32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory matrix descriptor without swizzle: core matrices of 8 rows x 16
// bytes, `lbo` between neighbours along the depth, `sbo` along the rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint32_t bits2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return bits2(__floats2half2_rn(lo, hi)); }
// field F of a word (or of the word turned: q4_raw) as c - 8, (c - 8) s and
// (c - 8) s + mid, in fp16
template <int F>
__device__ __forceinline__ __half2 centred(uint32_t x) {
  return __hsub2(half2_of(q4_raw<F>(x)), __float2half2_rn(Q4Bias<F>::value + 8.f));
}
template <int F>
__device__ __forceinline__ uint32_t dequant(uint32_t x, uint32_t s) {
  return bits2(__hmul2(centred<F>(x), half2_of(s)));
}
template <int F>
__device__ __forceinline__ uint32_t dequant(uint32_t x, uint32_t s, uint32_t mid) {
  return bits2(__hfma2(centred<F>(x), half2_of(s), half2_of(mid)));
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// Do the rows of the tile see token `at` of the visible block number v?
__device__ __forceinline__ bool seen_token(const WindowArgs& a, const Visible& vis, int from, int v, int at) {
  const int tok = v < vis.count() ? vis.block(v) * kQ4Tokens + at : 0x7fffffff;
  return tok < vis.L && (tok >= from || tok < a.n_sink);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q4_attn_tc_kernel(Q4AttnArgs p) {
  using L = Smem<D>;
  using B = Q4Block<D>;
  constexpr int NG = B::kGroups;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler has to see shared memory)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const WindowArgs& a = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // unit -> (stream, KV head, row tile, split)
  int u = blockIdx.x;
  const int sp = u % p.W;
  u /= p.W;
  const int rb = u % p.n_rb;
  const int sg = u / p.n_rb;
  const int g = sg % a.Hkv, s = sg / a.Hkv;
  const int G = a.Hq / a.Hkv, R = G * a.n, row0 = rb * 128;
  const Visible vis = visible_of(a, s);
  const int from = tile_from(a, vis.L, tile_last(rb, 128, R, G));
  const int tiles = (vis.count() + 3) / 4;
  const int t_begin = (int)((long long)tiles * sp / p.W), n = (int)((long long)tiles * (sp + 1) / p.W) - t_begin;

  auto bar = [&](int i) { return sb + L::kBar + 8u * i; };
  auto raw_full = [&](int i) { return bar(i); };
  auto raw_empty = [&](int i) { return bar(kRaw + i); };
  auto k_full = [&](int i) { return bar(2 * kRaw + i); };
  auto k_empty = [&](int i) { return bar(2 * kRaw + 2 + i); };
  auto v_full = [&](int i) { return bar(2 * kRaw + 4 + i); };
  auto v_empty = [&](int i) { return bar(2 * kRaw + 6 + i); };
  auto s_full = [&](int i) { return bar(2 * kRaw + 8 + i); };
  auto p_full = [&](int i) { return bar(2 * kRaw + 10 + i); };
  const uint32_t qx_full = bar(2 * kRaw + 12), pv_done = bar(2 * kRaw + 13), o_done = bar(2 * kRaw + 14),
                 all_done = bar(2 * kRaw + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmem);
  uint32_t* tops = reinterpret_cast<uint32_t*>(smem + L::kTop);
  float* half_max = reinterpret_cast<float*>(smem + L::kHalfMax);
  int* err = &g_err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 4);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 4);
      mbar_init(v_empty(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 8);
    }
    mbar_init(qx_full, 8);
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(all_done, 1);
    *abort_flag = 0;
    tops[0] = tops[1] = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  const uint8_t* base = static_cast<const uint8_t*>(a.cache) + (long long)sg * a.cap_blk * B::kBytes;
  auto load_raw = [&](int j) {
    const int v0 = (t_begin + j) * 4, nb = min(4, vis.count() - v0), sl = j % kRaw;
    mbar_arrive_expect_tx(raw_full(sl), nb * B::kBytes);
    for (int b = 0; b < nb; ++b)
      bulk_load(sb + L::kRawAt + sl * L::kRawTile + b * B::kBytes, base + (long long)vis.block(v0 + b) * B::kBytes,
                B::kBytes, raw_full(sl));
  };
  if (threadIdx.x == 0)
    for (int j = 0; j < min(n, kRaw); ++j) load_raw(j);
  // the largest |m + 8 s| + 8 s of the visible tokens' groups, K and V: an upper
  // bound of every value (a maximum, so the order of the atomics does not matter)
  if (warp > 0 && (warp < 12 || warp >= 16)) {
    float top[2] = {0.f, 0.f};
    const int end = min((t_begin + n) * 4, vis.count()) * kQ4Tokens;
    const int mine = warp < 12 ? threadIdx.x - 32 : threadIdx.x - 160;  // 480 threads
    using Words = typename std::conditional<NG == 2, uint2, uint32_t>::type;
#pragma unroll 8
    for (int x = t_begin * 4 * kQ4Tokens + mine; x < end; x += 480) {
      const bool seen = seen_token(a, vis, from, x / kQ4Tokens, x % kQ4Tokens);
      const uint8_t* blk = base + (long long)vis.block(x / kQ4Tokens) * B::kBytes + (x % kQ4Tokens) * (NG * 4);
      const Words kw = __ldg(reinterpret_cast<const Words*>(blk + B::kKs)), vw = __ldg(reinterpret_cast<const Words*>(blk + B::kVs));
#pragma unroll
      for (int w = 0; w < 2 * NG; ++w) {
        const uint32_t sm = reinterpret_cast<const uint32_t*>(w < NG ? &kw : &vw)[w % NG];
        const float sc = q4_scale(sm), y = fmaf(sc, 8.f, fabsf(fmaf(sc, 8.f, q4_min(sm))));
        if (seen) top[w / NG] = fmaxf(top[w / NG], y);
      }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int off = 16; off; off >>= 1) top[kv] = fmaxf(top[kv], __shfl_xor_sync(0xffffffffu, top[kv], off));
      if (lane == 0) atomicMax(tops + kv, __float_as_uint(top[kv]));
    }
  }
  if (warp >= 12 && warp < 16) {
    // Q: thread = row, scaled by a power of two, channels of a chunk in field order
    const int tid = threadIdx.x - 384, row = row0 + tid, rr = min(row, R - 1);
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                    (((long long)s * a.n + rr / G) * a.Hq + g * G + rr % G) * D);
    // read twice, eight chunks at a time (all of them in registers would spill)
    float top = 0.f;
#pragma unroll 8
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = __ldg(q + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(&x)[e];
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
      }
    }
    int ex = (int)(__float_as_uint(top) >> 23);
    ex = ex == 0 && top == 0.f ? 137 : ex == 255 ? 137 : max(ex, 12);
    const float up = row < R ? __uint_as_float((uint32_t)(264 - ex) << 23) : 0.f;
    reinterpret_cast<float*>(smem + L::kRow)[tid] = __uint_as_float((uint32_t)(ex - 10) << 23) * a.scale_log2;
#pragma unroll 1
    for (int gg = 0; gg < NG; ++gg) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 x = __ldg(q + gg * 8 + c);
        float y[8], t = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(&x)[e];
          y[2 * e] = __uint_as_float(w << 16) * up;
          y[2 * e + 1] = __uint_as_float(w & 0xffff0000u) * up;
          t += y[2 * e] + y[2 * e + 1];
        }
        sum += t;
        uint4 o;
#pragma unroll
        for (int f = 0; f < 4; ++f)
          reinterpret_cast<uint32_t*>(&o)[f] = pack_half2(y[q4_k_channel(f, 0)], y[q4_k_channel(f, 1)]);
        *reinterpret_cast<uint4*>(smem + L::kQ + gg * L::kAtom + tid * 128 + ((c ^ (tid & 7)) << 4)) = o;
      }
      reinterpret_cast<float*>(smem + L::kQs)[tid * NG + gg] = sum;
    }
    for (int b = 0; b < 2; ++b)  // the unused half of the depth-16 rows
      *reinterpret_cast<uint4*>(smem + L::kKx + b * 4096 + 2048 + tid * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  __syncthreads();
  // exponents that bring it into [2^12, 2^13) (116 where the bound itself overflows;
  // the values, below 2^128, are below 2^12 then), as far down as exp2i reaches
  const int eK = max((int)(tops[0] >> 23) - 127 - 12, -126), eV = max((int)(tops[1] >> 23) - 127 - 12, kPShift - 126);
  auto col_s = [](int x) { return (uint32_t)(x * 128); };
  constexpr uint32_t kColO = 256, kColQx = 384;

  if (warp < 4) {
    if (warp == 0) {
      // ---------------------------------------------------------- loader
      if (lane == 0) {
        int issued = min(n, kRaw);
        for (int j = issued; j < n; ++j) {
          if (!mbar_wait(raw_empty(j % kRaw), ((j / kRaw) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
          load_raw(j);
          issued = j + 1;
        }
        for (int j = max(0, issued - kRaw); j < issued; ++j) drain_wait(raw_full(j % kRaw), (j / kRaw) & 1, err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer
      if (n > 0) {
        constexpr uint32_t id_s = idesc_f16(128, 128), id_o = idesc_f16(128, D);
        const uint64_t dq = sdesc_sw128(sb + L::kQ, 16, 1024), dk = sdesc_sw128(sb + L::kK, 16, 1024);
        const uint64_t dv = sdesc_sw128(sb + L::kV, 16, 1024), dx = sdesc_plain(sb + L::kKx, 2048, 128);
        auto issue_s = [&](int j) {
          const uint64_t k0 = dk + (uint64_t)((j & 1) * (L::kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * L::kAtom + (kk & 3) * 32) >> 4);
            mma_ss_e(tmem + col_s(j & 1), dq + off, k0 + off, id_s, kk > 0 ? 1u : 0u);
          }
          mma_ts_e(tmem + col_s(j & 1), tmem + kColQx, dx + (uint64_t)((j & 1) * (4096 >> 4)), id_s, 1u);
          commit_e(s_full(j & 1));
          commit_e(k_empty(j & 1));
        };
        bool ok = warp_spin_wait(qx_full, 0, err, kErrWaitLoad, abort_flag) &&
                  warp_spin_wait(k_full(0), 0, err, kErrWaitLoad, abort_flag);
        if (ok) {
          fence_after_sync();
          issue_s(0);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (j + 1 < n) {  // S(j+1) overwrites P(j-1), which P V(j-1), issued before, has read
            if (!(ok = warp_spin_wait(k_full((j + 1) & 1), ((j + 1) >> 1) & 1, err, kErrWaitLoad, abort_flag))) break;
            fence_after_sync();
            issue_s(j + 1);
          }
          if (!(ok = warp_spin_wait(v_full(j & 1), (j >> 1) & 1, err, kErrWaitLoad, abort_flag))) break;
          if (!(ok = warp_spin_wait(p_full(j & 1), (j >> 1) & 1, err, kErrWaitP, abort_flag))) break;
          fence_after_sync();
          const uint64_t v0 = dv + (uint64_t)((j & 1) * (2 * L::kVAtom >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_e(tmem + kColO, tmem + col_s(j & 1) + (kk >> 2) * 64 + (kk & 3) * 8, v0 + (uint64_t)(((kk >> 2) * L::kVAtom + (kk & 3) * 32) >> 4),
                   id_o, (j > 0 || kk > 0) ? 1u : 0u);
          commit_e(pv_done);
          commit_e(v_empty(j & 1));
          if (j == n - 1) commit_e(o_done);
        }
        commit_e(all_done);
        if (lane == 0) drain_wait(all_done, 0, err);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    const int half = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane, row = row0 + r;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16), t_o = t_lane + kColO + half * (D / 2);
    const bool real = row < R;
    float m_used = -INFINITY, l = 0.f, c = 0.f;
    bool ok = n > 0;
    if (ok) {
      // (finite: the largest queries and keys need not meet in a channel; and above 0,
      // for hidden columns of -inf: where it is raised, logits are below 2^-90)
      c = fminf(fmaxf(reinterpret_cast<const float*>(smem + L::kRow)[r] * exp2i(eK), 0x1p-126f), 0x1.fffffep127f);
      if (half == 0) {
        // the row's sums of q for the product of depth 16: per group hi hi lo lo,
        // against m + 8 s as hi lo hi lo (a factor of 4 moved over: fp16's range)
        uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          const float q = reinterpret_cast<const float*>(smem + L::kQs)[r * NG + gg] * 0.25f;
          const float hi = __half2float(__float2half_rn(q));
          x[2 * gg] = pack_half2(hi, hi);
          x[2 * gg + 1] = pack_half2(q - hi, q - hi);
        }
        tmem_st8(t_lane + kColQx, x);
        tmem_st_wait();
        fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qx_full);
    }
    for (int j = 0; j < n; ++j) {
      if (ok) ok = warp_wait_all(s_full(j & 1), (j >> 1) & 1, err, kErrWaitAcc, abort_flag);
      fence_after_sync();
      const uint32_t t_s = t_lane + col_s(j & 1) + half * 64;
      const int v0 = (t_begin + j) * 4;
      const bool full = v0 + 4 <= vis.count() && vis.block(v0 + 3) * kQ4Tokens + kQ4Tokens <= vis.L &&
                        (vis.block(v0) * kQ4Tokens >= from || vis.block(v0 + 3) * kQ4Tokens + kQ4Tokens <= a.n_sink);
      if (!full) {  // hidden columns of S become -inf in tensor memory
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          uint32_t seen = 0;  // slots of the block that the rows see
#pragma unroll 1
          for (int q = 0; q < 32; ++q)
            if (seen_token(a, vis, from, v0 + half * 2 + b, ((q & 7) >> 2) * 16 + ((q >> 1) & 1) * 8 + (q >> 3) * 2 + (q & 1)))
              seen |= 1u << q;
          uint32_t sv[32];
          tmem_ld32(t_s + b * 32, sv);
          tmem_ld_wait_dep(sv);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (!(seen >> q & 1)) sv[q] = __float_as_uint(-INFINITY);
          tmem_st32(t_s + b * 32, sv);
        }
        tmem_st_wait();
      }
      // S is read twice, 32 columns at a time (for the maximum, for the weights),
      // in loops that stay rolled: six roles share the instruction caches
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t sv[32];
        tmem_ld32(t_s + b * 32, sv);
        tmem_ld_wait_dep(sv);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
          for (int jj = 0; jj < 8; jj += 2)
            m4[q4] = max3f(m4[q4], __uint_as_float(sv[8 * q4 + jj]), __uint_as_float(sv[8 * q4 + jj + 1]));
      }
      const float mx = reference_of(fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]) * c);
      // both halves learn whether one of them asks for a raise, or gave up
      if (named_bar_red_or(3, 256, !ok || mx > m_used + kRaise)) {
        half_max[half * 128 + r] = mx;
        if (named_bar_red_or(3, 256, !ok)) break;
        const float m_new = fmaxf(m_used, fmaxf(mx, half_max[(half ^ 1) * 128 + r]));
        const bool raise = m_new > m_used + kRaise;
        const float f = raise ? ex2_approx(m_used - m_new) : 1.f;
        l *= f;
        if (raise) m_used = m_new;
        if (j > 0) {
          // O must hold every earlier tile's P V
          if (!(ok = warp_wait_all(pv_done, (j - 1) & 1, err, kErrWaitAcc, abort_flag))) continue;
          fence_after_sync();
          for (int c0 = 0; c0 < D / 64; ++c0) {
            uint32_t v[32];
            tmem_ld32(t_o + c0 * 32, v);
            tmem_ld_wait_dep(v);
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) v[jj] = __float_as_uint(__uint_as_float(v[jj]) * f);
            tmem_st32(t_o + c0 * 32, v);
          }
          tmem_st_wait();
        }
      }
      const float ref = m_used == -INFINITY ? 0.f : m_used;
      const float bias = (float)kPShift - ref;
      const float2 c2 = make_float2(c, c), b2 = make_float2(bias, bias);
      float2 ls = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int c0 = 0; c0 < 2; ++c0) {
        uint32_t pk[16], sv[32];
        tmem_ld32(t_s + c0 * 32, sv);
        tmem_ld_wait_dep(sv);
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
          const float2 t = ffma2(make_float2(__uint_as_float(sv[2 * jj]), __uint_as_float(sv[2 * jj + 1])), c2, b2);
          const float2 pp = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          ls = fadd2(ls, pp);
          pk[jj] = pack_half2(pp.x, pp.y);
        }
        tmem_st16(t_s + c0 * 16, pk);  // over this half's own columns of S
      }
      tmem_st_wait();
      l += ls.x + ls.y;
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(j & 1));
    }
    if (ok) ok = warp_wait_all(o_done, 0, err, kErrWaitAcc, abort_flag);
    ok = ok && !*abort_flag;
    // l of the row's two halves
    half_max[half * 128 + r] = l;
    named_bar_sync(3, 256);
    l += half_max[(half ^ 1) * 128 + r];
    const long long at = ((long long)blockIdx.x * 128 + r);
    float* po = p.part_o + at * D + half * (D / 2);
    if (ok) {
      fence_after_sync();
      const float back = exp2i(eV - kPShift);
#pragma unroll
      for (int c0 = 0; c0 < D / 64; ++c0) {
        uint32_t v[32];
        tmem_ld32(t_o + c0 * 32, v);
        tmem_ld_wait_dep(v);
        if (real) {
          float4* dst = reinterpret_cast<float4*>(po + c0 * 32);
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            dst[q4] = make_float4(__uint_as_float(v[4 * q4]) * back, __uint_as_float(v[4 * q4 + 1]) * back,
                                  __uint_as_float(v[4 * q4 + 2]) * back, __uint_as_float(v[4 * q4 + 3]) * back);
        }
      }
    } else if (real) {  // no tiles (or an abandoned call): nothing to add
      for (int d = 0; d < D / 2; d += 4) *reinterpret_cast<float4*>(po + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // An infinite maximum has the merge take the row again.  Beside keys of 2^12 small
    // ones are held to 2^-22 (8 times a scale's 2^-25), which 128 channels of q below
    // 2^11 make 2^-4 of S, so a logit is off by up to c 2^-4: 2^-11, with c below 2^-7
    // (largest logits of some 10^5; usual ones have 2^-17).
    if (real && half == 0)
      *reinterpret_cast<float2*>(p.part_ml + at * 2) =
          !ok ? make_float2(-INFINITY, 0.f) : c >= 0x1p-7f ? make_float2(INFINITY, 0.f) : make_float2(m_used, l * exp2i(-kPShift));
  } else if (warp < 16) {
    // ------------------------------------------------------- dequantise K
    const int w4 = warp & 3, tid = w4 * 32 + lane;
    // this thread's row of a tile is slot `lane` of block w4
    const int f_of = (lane & 7) >> 1, tig_of = lane >> 3, half_of = lane & 1;
    const int tok_of = (f_of >> 1) * 16 + (f_of & 1) * 8 + tig_of * 2 + half_of;
    // the lanes of eight slots read different 16-byte chunks (tig = x ^ it), so
    // that neither loads nor stores meet a bank twice: x = 0 2 3 1 for f = 0..3
    const int x_of = ((f_of ^ (f_of >> 1)) & 1) << 1 | f_of >> 1;
    const float norm = exp2i(-eK);
    for (int j = 0; j < n; ++j) {
      const int sl = j % kRaw, b2 = j & 1;
      // the row scales and sums of q lie in the second K tile until they are read
      if (j == 1 && !warp_wait_all(qx_full, 0, err, kErrWaitLoad, abort_flag)) break;
      if (!warp_wait_all(raw_full(sl), (j / kRaw) & 1, err, kErrWaitLoad, abort_flag)) break;
      if (!warp_wait_all(k_empty(b2), ((j >> 1) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
      const uint8_t* raw = smem + L::kRawAt + sl * L::kRawTile + w4 * B::kBytes;
      const bool seen = seen_token(a, vis, from, (t_begin + j) * 4 + w4, tok_of);
      uint32_t s2[NG], x[4] = {0, 0, 0, 0};
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        const uint32_t sm = reinterpret_cast<const uint32_t*>(raw + B::kKs)[tok_of * NG + gg];
        const float sc = seen ? q4_scale(sm) * norm : 0.f;
        const float y = seen ? fmaf(q4_scale(sm), 8.f, q4_min(sm)) * norm * 4.f : 0.f;
        const float hi = __half2float(__float2half_rn(y));
        s2[gg] = pack_half2(sc, sc);
        x[2 * gg] = x[2 * gg + 1] = pack_half2(hi, y - hi);
      }
      *reinterpret_cast<uint4*>(smem + L::kKx + b2 * 4096 + tid * 16) = make_uint4(x[0], x[1], x[2], x[3]);
      const uint8_t* kr = raw + tok_of * B::kRow;
      uint8_t* dst = smem + L::kK + b2 * L::kTile + tid * 128;
#pragma unroll 1
      for (int it = 0; it < 4; ++it) {
        const int tig = x_of ^ it;
        uint32_t w[D / 32];
        if (D == 128) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(kr + tig * 16);
        else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(kr + tig * 8);
#pragma unroll
        for (int ww = 0; ww < D / 32; ++ww) {
          const int gg = ww >> 1;
          const uint32_t turned = q4_turn(w[ww]);
          *reinterpret_cast<uint4*>(dst + gg * L::kAtom + (((tig * 2 + (ww & 1)) ^ (tid & 7)) << 4)) =
              make_uint4(dequant<0>(w[ww], s2[gg]), dequant<1>(turned, s2[gg]), dequant<2>(w[ww], s2[gg]),
                         dequant<3>(turned, s2[gg]));
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_full(b2));
        mbar_arrive(raw_empty(sl));
      }
    }
  } else {
    // ------------------------------------------------------- dequantise V
    // A thread prepares the scales of one slot (block w4, slot lane), then takes
    // the words of one tig of its warp's block: channels 8 j + sub.
    const int w4 = warp & 3;
    const int f_of = (lane & 7) >> 1, tig_of = lane >> 3, half_of = lane & 1;
    const int tok_of = (f_of >> 1) * 16 + (f_of & 1) * 8 + tig_of * 2 + half_of;
    // lanes of eight stores: four tigs, two channels 4 apart: eight different chunks
    const int tig = lane & 3, sub = (lane >> 2 & 1) * 4 + (lane >> 3);
    const float norm = exp2i(-eV);
    for (int j = 0; j < n; ++j) {
      const int sl = j % kRaw, b2 = j & 1;
      if (!warp_wait_all(raw_full(sl), (j / kRaw) & 1, err, kErrWaitLoad, abort_flag)) break;
      if (!warp_wait_all(v_empty(b2), ((j >> 1) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
      const uint8_t* raw = smem + L::kRawAt + sl * L::kRawTile + w4 * B::kBytes;
      uint8_t* tab = smem + L::kTab + w4 * (4 * NG * 32);  // [tig][group][f] (s pair, m + 8 s pair) of the warp's block
      const bool seen = seen_token(a, vis, from, (t_begin + j) * 4 + w4, tok_of);
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        const uint32_t sm = reinterpret_cast<const uint32_t*>(raw + B::kVs)[tok_of * NG + gg];
        float sc = q4_scale(sm), mid = fmaf(sc, 8.f, q4_min(sm));
        if (!seen) sc = mid = 0.f;
        __half* x = reinterpret_cast<__half*>(tab) + ((tig_of * NG + gg) * 4 + f_of) * 4 + half_of;
        x[0] = __float2half_rn(sc * norm);
        x[2] = __float2half_rn(mid * norm);
      }
      __syncwarp();
      uint8_t* dst = smem + L::kV + b2 * 2 * L::kVAtom + (w4 >> 1) * L::kVAtom + sub * 128 + ((((w4 & 1) * 4 + tig) ^ sub) << 4);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(raw + B::kV + c * 512 + (sub * 4 + tig) * 16);
        const uint4* x = reinterpret_cast<const uint4*>(tab + (tig * NG + c / 2) * 32);
        const uint4 t0 = x[0], t1 = x[1];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t turned = q4_turn(ws[e]);
          *reinterpret_cast<uint4*>(dst + (c * 4 + e) * 1024) =
              make_uint4(dequant<0>(ws[e], t0.x, t0.y), dequant<1>(turned, t0.z, t0.w), dequant<2>(ws[e], t1.x, t1.y),
                         dequant<3>(turned, t1.z, t1.w));
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(v_full(b2));
        mbar_arrive(raw_empty(sl));
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_q4_attn_tc(const Q4AttnArgs& p, int d, cudaStream_t st) {
  const dim3 grid((unsigned)((long long)p.w.S * p.w.Hkv * p.n_rb * p.W));
  cudaError_t e;
  if (d == 128) {
    if ((e = ensure_dynamic_smem(q4_attn_tc_kernel<128>, Smem<128>::kAlloc)) != cudaSuccess) return e;
    return launch_kernel(q4_attn_tc_kernel<128>, grid, dim3(kThreads), Smem<128>::kAlloc, st, false, p);
  }
  if ((e = ensure_dynamic_smem(q4_attn_tc_kernel<64>, Smem<64>::kAlloc)) != cudaSuccess) return e;
  return launch_kernel(q4_attn_tc_kernel<64>, grid, dim3(kThreads), Smem<64>::kAlloc, st, false, p);
}

cudaError_t q4_attn_tc_status(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
  return e;
}

}  // namespace skv
