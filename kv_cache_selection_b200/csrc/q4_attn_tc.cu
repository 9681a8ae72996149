// Attention of many text tokens over the 4-bit cache on the 5th-generation
// tensor cores: for more query rows (heads of a KV head x text tokens) than the
// streaming kernel of q4_attn.cu takes in one pass, a 128-row tile shares every
// dequantised key tile.
//
// A thread block owns one 128-row tile of one (stream, KV head) and a range of
// 128-token key tiles.  Per key tile
//   raw blocks -> shared memory          one warp, bulk copies into a ring
//   K, V -> fp16 in shared memory        a warpgroup each
//   S = Q K^T, O += P V                  tcgen05, fp16 in, float32 accumulate
//   P = 2^(S c - m)                      softmax warpgroup, thread = row
// with S double-buffered in tensor memory.
//
// With numbers scaled by a power of two per tile (its largest magnitude into
// [1, 2)) fp16 serves the cache's whole range; the tile's exponent returns in
// S's scale (K) and in P's (V, relative to the largest V tile so far).
//   K: (c - 8) s has 11 bits and is exact in fp16; the groups' m + 8 s times the
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
#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"
#include "q4_visible.cuh"
#include "tc_common.cuh"

namespace skv {
namespace {
using namespace tc;

constexpr int kThreads = 512;
// registers: launched at 128 a thread; loader and MMA issuer 64, softmax 208,
// the two dequantising warpgroups 112: 64 + 208 + 2 x 112 <= 4 x 128
constexpr int kRegsLow = 64, kRegsSoftmax = 208, kRegsDequant = 112;
static_assert(kRegsLow + kRegsSoftmax + 2 * kRegsDequant <= 4 * 128, "register split exceeds the launch");
constexpr int kRaw = 3;          // raw tiles in flight
constexpr float kRaise = 8.0f;   // log2 headroom of the lazy row maximum
constexpr int kPShift = 6;       // P is held as P 2^6 (below 2^14)
constexpr int kTileTokens = 128;

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
  static constexpr int kQs = kRawAt + kRaw * kRawTile;   // group sums of q [128][groups]
  static constexpr int kTab = kQs + 128 * B::kGroups * 4;  // V scales: [4 blk][4 tig][groups][4 f] (s pair, mid pair)
  static constexpr int kRow = kTab + 16 * B::kGroups * 32;  // row scales [128]
  static constexpr int kExp = kRow + 512;                // exponents K[4], V[4]; maxima [2][2][4]
  static constexpr int kPoison = kExp + 32 + 64;         // [4 tiles][groups][4 words]
  static constexpr int kBar = kPoison + 4 * B::kGroups * 16;
  // raw_full[kRaw], raw_empty[kRaw], k_full[2], k_empty[2], v_full[2], v_empty[2], s[2], p[2], q, pv, o, done, qx
  static constexpr int kNumBars = 2 * kRaw + 12 + 5;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4;
  static constexpr int kAlloc = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;  // one block per SM
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(kTab % 16 == 0 && kBar % 8 == 0, "alignment");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
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
// field F of a word as (c - 8) s, and as (c - 8) s + mid, in fp16
template <int F>
__device__ __forceinline__ uint32_t dequant(uint32_t w, uint32_t s) {
  const uint32_t r = q4_field<F>(w) | 0x4C004C00u;  // 16 + c
  return bits2(__hmul2(__hsub2(half2_of(r), __half2half2(__ushort_as_half(0x4E00))), half2_of(s)));
}
template <int F>
__device__ __forceinline__ uint32_t dequant(uint32_t w, uint32_t s, uint32_t mid) {
  const uint32_t r = q4_field<F>(w) | 0x4C004C00u;  // 16 + c
  return bits2(__hfma2(__hsub2(half2_of(r), __half2half2(__ushort_as_half(0x4E00))), half2_of(s), half2_of(mid)));
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q4_attn_tc_kernel(Q4AttnArgs p) {
  using L = Smem<D>;
  using B = Q4Block<D>;
  constexpr int NG = B::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
  const int i_first = row0 / G, i_last = (min(row0 + 128, R) - 1) / G;
  const Visible vis = visible_of(a, s);
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
  const uint32_t q_full = bar(2 * kRaw + 12), pv_done = bar(2 * kRaw + 13), o_done = bar(2 * kRaw + 14), all_done = bar(2 * kRaw + 15),
                 qx_full = bar(2 * kRaw + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmem);
  int* exp_k = reinterpret_cast<int*>(smem + L::kExp);
  int* exp_v = exp_k + 4;
  float* maxima = reinterpret_cast<float*>(exp_k + 8);  // [K, V][2][4 warps]
  uint32_t* poison = reinterpret_cast<uint32_t*>(smem + L::kPoison);
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
      mbar_init(p_full(i), 4);
    }
    mbar_init(q_full, 4);
    mbar_init(qx_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(all_done, 1);
    *abort_flag = 0;
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
  auto col_s = [](int x) { return (uint32_t)(x * 128); };
  constexpr uint32_t kColO = 256, kColQx = 384;

  if (warp < 4) {
    regs_dec<kRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------- loader
      if (lane == 0) {
        const uint8_t* base = static_cast<const uint8_t*>(a.cache) + (long long)sg * a.cap_blk * B::kBytes;
        int issued = 0;
        for (int j = 0; j < n; ++j) {
          const int sl = j % kRaw;
          if (!mbar_wait(raw_empty(sl), ((j / kRaw) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
          const int v0 = (t_begin + j) * 4, nb = min(4, vis.count() - v0);
          mbar_arrive_expect_tx(raw_full(sl), nb * B::kBytes);
          for (int b = 0; b < nb; ++b)
            bulk_load(sb + L::kRawAt + sl * L::kRawTile + b * B::kBytes, base + (long long)vis.block(v0 + b) * B::kBytes,
                      B::kBytes, raw_full(sl));
          issued = j + 1;
        }
        for (int j = max(0, issued - kRaw); j < issued; ++j) drain_wait(raw_full(j % kRaw), (j / kRaw) & 1, err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer
      if (lane == 0 && n > 0) {
        constexpr uint32_t id_s = idesc_f16(128, 128), id_o = idesc_f16(128, D);
        const uint64_t dq = sdesc_sw128(sb + L::kQ, 16, 1024), dk = sdesc_sw128(sb + L::kK, 16, 1024);
        const uint64_t dv = sdesc_sw128(sb + L::kV, 16, 1024), dx = sdesc_plain(sb + L::kKx, 2048, 128);
        auto issue_s = [&](int j) {
          const uint64_t k0 = dk + (uint64_t)((j & 1) * (L::kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * L::kAtom + (kk & 3) * 32) >> 4);
            mma_ss(tmem + col_s(j & 1), dq + off, k0 + off, id_s, kk > 0 ? 1u : 0u);
          }
          mma_ts(tmem + col_s(j & 1), tmem + kColQx, dx + (uint64_t)((j & 1) * (4096 >> 4)), id_s, 1u);
          mma_commit(s_full(j & 1));
          mma_commit(k_empty(j & 1));
        };
        bool ok = mbar_wait(q_full, 0, err, kErrWaitLoad, abort_flag) &&
                  mbar_wait(qx_full, 0, err, kErrWaitLoad, abort_flag) &&
                  mbar_wait(k_full(0), 0, err, kErrWaitLoad, abort_flag);
        if (ok) {
          fence_after_sync();
          issue_s(0);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (j + 1 < n) {  // S(j+1) overwrites P(j-1), which P V(j-1), issued before, has read
            if (!(ok = mbar_wait(k_full((j + 1) & 1), ((j + 1) >> 1) & 1, err, kErrWaitLoad, abort_flag))) break;
            fence_after_sync();
            issue_s(j + 1);
          }
          if (!(ok = mbar_wait(v_full(j & 1), (j >> 1) & 1, err, kErrWaitLoad, abort_flag))) break;
          if (!(ok = mbar_wait(p_full(j & 1), (j >> 1) & 1, err, kErrWaitP, abort_flag))) break;
          fence_after_sync();
          const uint64_t v0 = dv + (uint64_t)((j & 1) * (2 * L::kVAtom >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + kColO, tmem + col_s(j & 1) + kk * 8, v0 + (uint64_t)(((kk >> 2) * L::kVAtom + (kk & 3) * 32) >> 4),
                   id_o, (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(pv_done);
          mma_commit(v_empty(j & 1));
          if (j == n - 1) mma_commit(o_done);
        }
        mma_commit(all_done);
        drain_wait(all_done, 0, err);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int quarter = warp & 3, r = quarter * 32 + lane, row = row0 + r;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16), t_o = t_lane + kColO;
    const bool real = row < R;
    const int i = min(row, R - 1) / G;
    float m_used = -INFINITY, l = 0.f, c_row = 0.f;
    int E = -1000;  // exponent that O is relative to
    uint32_t nan_groups = 0;
    bool ok = n > 0 && warp_wait(q_full, 0, err, kErrWaitLoad, abort_flag);
    if (ok) {
      c_row = reinterpret_cast<const float*>(smem + L::kRow)[r];
      // the row's sums of q for the product of depth 16: per group hi hi lo lo,
      // against m + 8 s as hi lo hi lo (2^8 moved from one to the other: fp16's range)
      uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        const float q = reinterpret_cast<const float*>(smem + L::kQs)[r * NG + gg] * 0x1p-8f;
        const float hi = __half2float(__float2half_rn(q));
        x[2 * gg] = pack_half2(hi, hi);
        x[2 * gg + 1] = pack_half2(q - hi, q - hi);
      }
      tmem_st8(t_lane + kColQx, x);
      tmem_st_wait();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(qx_full);
    }
    for (int j = 0; ok && j < n; ++j) {
      if (!(ok = warp_spin_wait(s_full(j & 1), (j >> 1) & 1, err, kErrWaitAcc, abort_flag))) break;
      // V's exponent and poison words come with v_full
      if (!(ok = warp_wait(v_full(j & 1), (j >> 1) & 1, err, kErrWaitLoad, abort_flag))) break;
      fence_after_sync();
      const uint32_t t_s = t_lane + col_s(j & 1);
      const float c = c_row * exp2i(exp_k[j & 3]);
      const int eV = exp_v[j & 3];
      uint32_t sv[128];
      tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
      tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
      tmem_ld_wait();
      const int v0 = (t_begin + j) * 4;
      bool full = v0 + 4 <= vis.count() && vis.block(v0 + 3) * kQ4Tokens + kQ4Tokens <= vis.L;
      if (a.window)
        full = full && ((long long)vis.block(v0) * kQ4Tokens > (long long)vis.L + i_last - a.window ||
                        vis.block(v0 + 3) * kQ4Tokens + kQ4Tokens <= a.n_sink);
      if (!full) {
        const long long from = a.window ? (long long)vis.L + i - a.window + 1 : 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          // the block's tokens that the row sees, as a mask over its slots
          uint32_t seen = 0;
          const bool there = v0 + b < vis.count();
          const int t0 = there ? vis.block(v0 + b) * kQ4Tokens : 0;
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const int tok = t0 + ((q & 7) >> 2) * 16 + ((q >> 1) & 1) * 8 + (q >> 3) * 2 + (q & 1);
            const bool see = there && tok < vis.L && (tok >= from || tok < a.n_sink);
            if (see) seen |= 1u << q;
            else sv[b * 32 + q] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int gg = 0; gg < NG; ++gg)
            if (seen & poison[((j & 3) * NG + gg) * 4 + b]) nan_groups |= 1u << gg;
        }
      }
      float m8[8];
#pragma unroll
      for (int q8 = 0; q8 < 8; ++q8) {
        m8[q8] = __uint_as_float(sv[16 * q8]);
#pragma unroll
        for (int jj = 1; jj < 15; jj += 2)
          m8[q8] = max3f(m8[q8], __uint_as_float(sv[16 * q8 + jj]), __uint_as_float(sv[16 * q8 + jj + 1]));
        m8[q8] = fmaxf(m8[q8], __uint_as_float(sv[16 * q8 + 15]));
      }
      const float mx = fmaxf(fmaxf(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5])), fmaxf(m8[6], m8[7]));
      const float m_new = fmaxf(m_used, mx * c);
      const bool raise = m_new > m_used + kRaise;
      if (__any_sync(0xffffffffu, raise) || eV > E) {
        const float f = raise ? ex2_approx(m_used - m_new) : 1.f;
        l *= f;
        if (j > 0) {
          // O must hold every earlier tile's P V
          if (!(ok = warp_wait(pv_done, (j - 1) & 1, err, kErrWaitAcc, abort_flag))) break;
          fence_after_sync();
          const float fo = eV > E ? f * exp2i(max(E - eV, -126)) : f;
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t v[32];
            tmem_ld32(t_o + c0 * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) v[jj] = __float_as_uint(__uint_as_float(v[jj]) * fo);
            tmem_st32(t_o + c0 * 32, v);
          }
          tmem_st_wait();
        }
        if (raise) m_used = m_new;
        E = max(E, eV);
      }
      const float ref = m_used == -INFINITY ? 0.f : m_used;
      const int shift = max(eV - E + kPShift, -40);  // beyond: 2^-40 of the largest value, l stays exact
      const float bias = (float)shift - ref;
      const float2 c2 = make_float2(c, c), b2 = make_float2(bias, bias);
      float2 ls = make_float2(0.f, 0.f);
#pragma unroll
      for (int c0 = 0; c0 < 4; ++c0) {
        uint32_t pk[16];
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
          const float2 t = ffma2(make_float2(__uint_as_float(sv[c0 * 32 + 2 * jj]), __uint_as_float(sv[c0 * 32 + 2 * jj + 1])),
                                 c2, b2);
          const float2 pp = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          ls = fadd2(ls, pp);
          pk[jj] = pack_half2(pp.x, pp.y);
        }
        tmem_st16(t_s + c0 * 16, pk);
      }
      tmem_st_wait();
      l = fmaf(ls.x + ls.y, exp2i(-shift), l);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(j & 1));
    }
    if (ok) ok = warp_wait(o_done, 0, err, kErrWaitAcc, abort_flag);
    ok = ok && !*abort_flag;
    const long long at = ((long long)blockIdx.x * 128 + r);
    if (ok) {
      fence_after_sync();
      const float back = exp2i(min(max(E - kPShift, -126), 127));
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t v[32];
        tmem_ld32(t_o + c0 * 32, v);
        tmem_ld_wait();
        const float add = (nan_groups >> (c0 / 2) & 1) ? NAN : 0.f;
        if (real) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + c0 * 32);
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            dst[q4] = make_float4(fmaf(__uint_as_float(v[4 * q4]), back, add), fmaf(__uint_as_float(v[4 * q4 + 1]), back, add),
                                  fmaf(__uint_as_float(v[4 * q4 + 2]), back, add), fmaf(__uint_as_float(v[4 * q4 + 3]), back, add));
        }
      }
    } else if (real) {  // no tiles (or an abandoned call): nothing to add
      for (int d = 0; d < D; d += 4) *reinterpret_cast<float4*>(p.part_o + at * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (real) *reinterpret_cast<float2*>(p.part_ml + at * 2) = ok ? make_float2(m_used, l) : make_float2(-INFINITY, 0.f);
  } else {
    // --------------------------------------------- dequantise: K or V
    regs_dec<kRegsDequant>();
    const bool is_v = warp >= 12;
    const int w4 = warp & 3, tid = w4 * 32 + lane;
    if (!is_v) {
      // Q: thread = row, scaled by a power of two, channels of a chunk in field order
      const int row = row0 + tid;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                               (((long long)s * a.n + min(row, R - 1) / G) * a.Hq + g * G + min(row, R - 1) % G) * D;
      float top = 0.f;
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(xs[e] << 16)), fabsf(__uint_as_float(xs[e] & 0xffff0000u))));
      }
      int ex = (int)(__float_as_uint(top) >> 23);
      ex = ex == 0 && top == 0.f ? 137 : ex == 255 ? 137 : max(ex, 12);
      const float up = __uint_as_float((uint32_t)(264 - ex) << 23), down = __uint_as_float((uint32_t)(ex - 10) << 23);
      reinterpret_cast<float*>(smem + L::kRow)[tid] = down * a.scale_log2;
      float sum[NG];
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) sum[gg] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + c);
        const float y[8] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                            __uint_as_float(x.y & 0xffff0000u), __uint_as_float(x.z << 16),
                            __uint_as_float(x.z & 0xffff0000u), __uint_as_float(x.w << 16),
                            __uint_as_float(x.w & 0xffff0000u)};
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (row < R)
          o = make_uint4(pack_half2(y[q4_k_channel(0, 0)] * up, y[q4_k_channel(0, 1)] * up),
                         pack_half2(y[q4_k_channel(1, 0)] * up, y[q4_k_channel(1, 1)] * up),
                         pack_half2(y[q4_k_channel(2, 0)] * up, y[q4_k_channel(2, 1)] * up),
                         pack_half2(y[q4_k_channel(3, 0)] * up, y[q4_k_channel(3, 1)] * up));
        *reinterpret_cast<uint4*>(smem + L::kQ + (c >> 3) * L::kAtom + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) = o;
        sum[c >> 3] += (((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]))) * up;
      }
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) reinterpret_cast<float*>(smem + L::kQs)[tid * NG + gg] = row < R ? sum[gg] : 0.f;
      for (int b = 0; b < 2; ++b)  // the unused half of the depth-16 rows
        *reinterpret_cast<uint4*>(smem + L::kKx + b * 4096 + 2048 + tid * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    // this thread's slot of a tile: block w4, slot lane
    const int f_of = (lane & 7) >> 1, tig_of = lane >> 3, half_of = lane & 1;
    const int tok_of = (f_of >> 1) * 16 + (f_of & 1) * 8 + tig_of * 2 + half_of;  // its token in the block
    float* wmax = maxima + (is_v ? 8 : 0);
    const int bar_id = is_v ? 2 : 1;
    for (int j = 0; j < n; ++j) {
      const int sl = j % kRaw, b2 = j & 1;
      bool ok = warp_wait(raw_full(sl), (j / kRaw) & 1, err, kErrWaitLoad, abort_flag);
      if (ok) ok = warp_wait(is_v ? v_empty(b2) : k_empty(b2), ((j >> 1) & 1) ^ 1, err, kErrWaitEmpty, abort_flag);
      const uint8_t* raw = smem + L::kRawAt + sl * L::kRawTile;
      // scales of this thread's token; 0 where no row of the tile sees it
      const int vb = (t_begin + j) * 4 + w4;
      const int tok = vb < vis.count() ? vis.block(vb) * kQ4Tokens + tok_of : 0x7fffffff;
      const bool keep = !a.window || tok < a.n_sink;
      const bool some = ok && tok < vis.L && (keep || (long long)tok > (long long)vis.L + i_first - a.window);
      const bool every = keep || (long long)tok > (long long)vis.L + i_last - a.window;
      float sc[NG], mid[NG], top = 0.f;
      uint32_t bad = 0;
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        sc[gg] = mid[gg] = 0.f;
        if (some) {
          const uint32_t sm = reinterpret_cast<const uint32_t*>(raw + w4 * B::kBytes + (is_v ? B::kVs : B::kKs))[tok_of * NG + gg];
          sc[gg] = q4_scale(sm);
          mid[gg] = fmaf(sc[gg], 8.f, q4_min(sm));
          if (is_v && !every && sc[gg] != sc[gg]) {  // rows that see it become NaN in the softmax
            sc[gg] = mid[gg] = 0.f;
            bad |= 1u << gg;
          }
          top = fmaxf(top, fmaf(sc[gg], 8.f, fabsf(mid[gg])));
        }
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (lane == 0) wmax[b2 * 4 + w4] = top;
      if (is_v) {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          const uint32_t word = __ballot_sync(0xffffffffu, bad >> gg & 1);
          if (lane == 0) poison[((j & 3) * NG + gg) * 4 + w4] = word;
        }
      }
      if (named_bar_red_or(bar_id, 128, !ok)) break;  // a warp gave up: all leave
      top = fmaxf(fmaxf(wmax[b2 * 4], wmax[b2 * 4 + 1]), fmaxf(wmax[b2 * 4 + 2], wmax[b2 * 4 + 3]));
      // the tile's largest magnitude into [1, 2)
      const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 120);
      const float norm = exp2i(-e);
      if (tid == 0) (is_v ? exp_v : exp_k)[j & 3] = e;
      if (!is_v) {
        uint32_t s2[NG], x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          s2[gg] = pack_half2(sc[gg] * norm, sc[gg] * norm);
          const float y = mid[gg] * norm * 0x1p8f, hi = __half2float(__float2half_rn(y));
          x[2 * gg] = x[2 * gg + 1] = pack_half2(hi, y - hi);
        }
        *reinterpret_cast<uint4*>(smem + L::kKx + b2 * 4096 + tid * 16) = make_uint4(x[0], x[1], x[2], x[3]);
        // row = slot; the four lanes of a slot pair of eight read different
        // 16-byte chunks (tig = x ^ i), so loads and stores meet no bank twice
        const int x_of = ((f_of ^ (f_of >> 1)) & 1) << 1 | f_of >> 1;  // 0 2 3 1 for f = 0..3
        const uint8_t* kr = raw + w4 * B::kBytes + tok_of * B::kRow;
        uint8_t* dst = smem + L::kK + b2 * L::kTile + tid * 128;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int tig = x_of ^ it;
          uint32_t w[D / 32];
          if (D == 128) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(kr + tig * 16);
          else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(kr + tig * 8);
#pragma unroll
          for (int ww = 0; ww < D / 32; ++ww) {
            const int gg = ww >> 1;
            const uint4 o = make_uint4(dequant<0>(w[ww], s2[gg]), dequant<1>(w[ww], s2[gg]), dequant<2>(w[ww], s2[gg]),
                                       dequant<3>(w[ww], s2[gg]));
            *reinterpret_cast<uint4*>(dst + gg * L::kAtom + (((tig * 2 + (ww & 1)) ^ (tid & 7)) << 4)) = o;
          }
        }
      } else {
        // scales by (block, tig, group, field): a word's eight tokens
        __half* tab = reinterpret_cast<__half*>(smem + L::kTab);
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          __half* t = tab + (((w4 * 4 + tig_of) * NG + gg) * 4 + f_of) * 4 + half_of;
          t[0] = __float2half_rn(sc[gg] * norm);
          t[2] = __float2half_rn(mid[gg] * norm);
        }
        named_bar_sync(bar_id, 128);
        const int d = tid % D, x_of = (d >> 1) & 3;
        uint8_t* dst = smem + L::kV + b2 * 2 * L::kVAtom + d * 128;
#pragma unroll
        for (int bb = 0; bb < 4 * D / 128; ++bb) {
          const int b = (tid / D) * 2 + bb;  // D = 64: two threads share a channel
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int tig = x_of ^ it;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(raw + b * B::kBytes + B::kV + q4_v_word(d, tig));
            const uint4* t = reinterpret_cast<const uint4*>(tab + ((b * 4 + tig) * NG + d / kQ4Group) * 16);
            const uint4 t0 = t[0], t1 = t[1];
            const uint4 o = make_uint4(dequant<0>(w, t0.x, t0.y), dequant<1>(w, t0.z, t0.w), dequant<2>(w, t1.x, t1.y),
                                       dequant<3>(w, t1.z, t1.w));
            *reinterpret_cast<uint4*>(dst + (b >> 1) * L::kVAtom + ((((b & 1) * 4 + tig) ^ (d & 7)) << 4)) = o;
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(is_v ? v_full(b2) : k_full(b2));
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
