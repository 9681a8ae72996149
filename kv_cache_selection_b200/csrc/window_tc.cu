// Causal attention with a sliding window and visible first tokens on the
// 5th-generation tensor cores (bf16 in, float32 accumulate): token i sees
// j <= i with j > i - window or j < n_sink.
//
// A thread block takes two 128-row query tiles A, B (256 consecutive rows of
// one head) and walks the 128-key tiles that any of its rows sees: the sink
// tiles, then those from row 0's window to the diagonal.  Per key tile and
// query tile S = Q K^T goes to tensor memory, a softmax warpgroup (thread =
// row) turns it into P in place, and O += P V reads P from tensor memory.
//
// The running maximum is lazy (raised when a logit exceeds it by more than
// 2^8); it starts at -inf, so a row whose first tiles are hidden takes its
// maximum from the first tile it sees.  Weights are rounded to bf16 for the
// product with V (2^-8 of a weight, the precision of V itself); their sum is
// float32.
//
// A hidden value enters P V with weight 0, and 0 x NaN is NaN: a row that ends
// with a non-finite output is computed again from its visible tokens alone, on
// the CUDA cores (slow, and only where the inputs hold a NaN or an infinity or
// the result overflows).
//
// Warps (384 threads): 0 TMA producer, 1 tensor-memory owner and MMA issuer,
// 4..7 softmax of tile A, 8..11 of tile B.
#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace skv {
namespace {
using namespace tc;

constexpr int kSlots = 4;  // K/V ring slots of one 128-key tile
constexpr int kThreads = 384;
// launched at 168 registers a thread; warpgroup 0 drops to 72, the softmax
// warpgroups rise to 216: 128 x 72 + 256 x 216 = 384 x 168
constexpr int kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split exceeds the launch");
constexpr float kRaise = 8.0f;

// first error of the pipeline waits of all calls on a device
__device__ int g_err;

template <int D>
struct Smem {
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = 128 * 128;
  static constexpr int kTile = kAtoms * kAtomBytes;  // 128 rows x D bf16
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTile;
  static constexpr int kBar = kKV + kSlots * kTile;
  // q[2], kv_full[kSlots], kv_empty[kSlots], s_full[2], p_full[2], o_done[2], done
  static constexpr int kNumBars = 2 + 2 * kSlots + 7;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4;
  // at least 116 KB: a second block (it would need all tensor memory too) never shares the SM
  static constexpr int kAlloc = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;
};

// One row again, from its visible tokens alone; a warp, lane = D/32 channels.
template <int D>
__device__ __noinline__ void row_again(const WindowArgs& a, int s, int h, int i) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, g = h / (a.Hq / a.Hkv);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (((long long)s * a.n + i) * a.Hq + h) * D + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(q[e]);
    o[e] = 0.f;
  }
  const int first = max(0, i - a.window + 1);
  for (int j = 0; j <= i; ++j) {
    if (j >= a.n_sink && j < first) j = first;
    const long long at = (((long long)s * a.n + j) * a.Hkv + g) * D + lane * E;
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) t = fmaf(qv[e], to_f(static_cast<const __nv_bfloat16*>(a.k)[at + e]), t);
#pragma unroll
    for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    t *= a.scale_log2;
    const float nm = fmaxf(m, t);
    const float ref = nm == -INFINITY ? 0.f : nm;
    const float f = ex2_approx(m - ref), p = ex2_approx(t - ref);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * to_f(static_cast<const __nv_bfloat16*>(a.v)[at + e]);
    m = nm;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f<__nv_bfloat16>(o[e] / l);
  if (a.lse && lane == 0) a.lse[((long long)s * a.Hq + h) * a.n + i] = (m + __log2f(l)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, WindowArgs a, int n_pairs) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // unit -> (stream, pair, KV group, head of the group): the heads that share a
  // K/V range run next to one another
  const int G = a.Hq / a.Hkv;
  long long u = blockIdx.x;
  const int h = (int)(u % a.Hq);
  u /= a.Hq;
  const int pair = n_pairs - 1 - (int)(u % n_pairs);
  const int s = (int)(u / n_pairs);
  const int g = h / G;
  const int iA = pair * 256, iB = iA + 128;
  // key tiles: the sinks' [0, ns), then [fw, diagonal]
  const int fw = max(0, iA - a.window + 1) / 128;
  const int ns = min((a.n_sink + 127) / 128, fw);
  const int nA = ns + 2 * pair + 1 - fw;
  const int nB = iB < a.n ? nA + 1 : 0;
  const int n_load = max(nA, nB);
  auto key_tile = [&](int j) { return j < ns ? j : j - ns + fw; };

  auto bar_q = [&](int x) { return sb + L::kBar + 8u * x; };
  auto bar_full = [&](int sl) { return sb + L::kBar + 8u * (2 + sl); };
  auto bar_empty = [&](int sl) { return sb + L::kBar + 8u * (2 + kSlots + sl); };
  auto bar_s = [&](int x) { return sb + L::kBar + 8u * (2 + 2 * kSlots + x); };
  auto bar_p = [&](int x) { return sb + L::kBar + 8u * (4 + 2 * kSlots + x); };
  auto bar_o = [&](int x) { return sb + L::kBar + 8u * (6 + 2 * kSlots + x); };
  const uint32_t bar_done = sb + L::kBar + 8u * (8 + 2 * kSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmem);
  int* err = &g_err;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar_q(x), 1);
      mbar_init(bar_s(x), 1);
      mbar_init(bar_p(x), 4);
      mbar_init(bar_o(x), 1);
    }
    for (int sl = 0; sl < kSlots; ++sl) {
      mbar_init(bar_full(sl), 1);
      mbar_init(bar_empty(sl), 1);
    }
    mbar_init(bar_done, 1);
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
  // columns: S/P of A at 0, of B at 128, O of A at 256, O of B at 384
  auto col_s = [](int x) { return (uint32_t)(x * 128); };
  auto col_o = [](int x) { return (uint32_t)(256 + x * 128); };

  if (warp < 4) regs_dec<kRegsLow>();
  if (warp == 0) {
    if (lane == 0) {
      // order Q_A, K_0, Q_B, V_0, K_1, ...: S_A(0) needs only the first two
      auto load_q = [&](int x) {
        mbar_arrive_expect_tx(bar_q(x), L::kTile);
        for (int at = 0; at < L::kAtoms; ++at)
          tma_load_4d(sb + L::kQ + x * L::kTile + at * L::kAtomBytes, &tm_q, bar_q(x), at * 64, h, iA + x * 128, s);
      };
      load_q(0);
      bool qb = false;
      int issued = 0;
      for (int idx = 0; idx < 2 * n_load; ++idx) {
        const int sl = idx % kSlots;
        if (!mbar_wait(bar_empty(sl), ((idx / kSlots) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
        const int r0 = key_tile(idx >> 1) * 128;
        mbar_arrive_expect_tx(bar_full(sl), L::kTile);
        const uint32_t dst = sb + L::kKV + sl * L::kTile;
        for (int at = 0; at < L::kAtoms; ++at)
          tma_load_4d(dst + at * L::kAtomBytes, (idx & 1) ? &tm_v : &tm_k, bar_full(sl), at * 64, g, r0, s);
        issued = idx + 1;
        if (idx == 0 && nB > 0) {
          load_q(1);
          qb = true;
        }
      }
      drain_wait(bar_q(0), 0, err);
      if (qb) drain_wait(bar_q(1), 0, err);
      for (int idx = max(0, issued - kSlots); idx < issued; ++idx) drain_wait(bar_full(idx % kSlots), (idx / kSlots) & 1, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t id_o = idesc_bf16(128, D, false, true);
      const uint64_t dq0 = sdesc_sw128(sb + L::kQ, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sb + L::kKV, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sb + L::kKV, L::kAtomBytes, 1024);
      auto slot16 = [&](int idx) { return (uint64_t)((idx % kSlots) * (L::kTile >> 4)); };
      auto wait_slot = [&](int idx) {
        return mbar_wait(bar_full(idx % kSlots), (idx / kSlots) & 1, err, kErrWaitLoad, abort_flag);
      };
      auto issue_s = [&](int x, int j) {  // S_x = Q_x K_j^T
        const uint64_t dq = dq0 + (uint64_t)((x * L::kTile) >> 4), dk = dk0 + slot16(2 * j);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * L::kAtomBytes + (kk & 3) * 32) >> 4);
          mma_ss(tmem + col_s(x), dq + off, dk + off, id_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar_s(x));
      };
      auto issue_pv = [&](int x, int j, int n) {  // O_x += P_x V_j
        const uint64_t dv = dv0 + slot16(2 * j + 1);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + col_o(x), tmem + col_s(x) + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id_o,
                 (j > 0 || kk > 0) ? 1u : 0u);
        if (j == n - 1) mma_commit(bar_o(x));
      };
      bool ok = wait_slot(0) && mbar_wait(bar_q(0), 0, err, kErrWaitLoad, abort_flag);
      if (ok) {
        fence_after_sync();
        issue_s(0, 0);
        if (nB > 0 && (ok = mbar_wait(bar_q(1), 0, err, kErrWaitLoad, abort_flag))) {
          fence_after_sync();
          issue_s(1, 0);
        }
        if (ok) mma_commit(bar_empty(0));
      }
      for (int j = 0; ok && j < n_load; ++j) {
        if (!(ok = wait_slot(2 * j + 1))) break;  // V_j
        const bool next_k = j + 1 < n_load;
        if (j < nA) {
          if (!(ok = mbar_wait(bar_p(0), j & 1, err, kErrWaitP, abort_flag))) break;
          fence_after_sync();
          issue_pv(0, j, nA);
        }
        if (next_k && !(ok = wait_slot(2 * (j + 1)))) break;  // K_{j+1}
        if (j + 1 < nA) issue_s(0, j + 1);
        if (j < nB) {
          if (!(ok = mbar_wait(bar_p(1), j & 1, err, kErrWaitP, abort_flag))) break;
          fence_after_sync();
          issue_pv(1, j, nB);
        }
        mma_commit(bar_empty((2 * j + 1) % kSlots));
        if (j + 1 < nB) issue_s(1, j + 1);
        if (next_k) mma_commit(bar_empty((2 * (j + 1)) % kSlots));
      }
      mma_commit(bar_done);
      drain_wait(bar_done, 0, err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    regs_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2, nX = x == 0 ? nA : nB;
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const int i = iA + x * 128 + r;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_o = t_lane + col_o(x), t_s = t_lane + col_s(x);
    const float c = a.scale_log2;
    float m_used = -INFINITY, l = 0.f;
    bool ok = nX > 0;
    for (int j = 0; ok && j < nX; ++j) {
      if (!(ok = warp_spin_wait(bar_s(x), j & 1, err, kErrWaitAcc, abort_flag))) break;
      fence_after_sync();
      uint32_t sv[128];
      tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
      tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
      tmem_ld_wait();
      // visible columns of this row: below `end`, and from `lo` on or below `sink`
      const int base = key_tile(j) * 128;
      const int end = i + 1 - base, lo = i - a.window + 1 - base, sink = a.n_sink - base;
      if (__any_sync(0xffffffffu, end < 128 || (lo > 0 && sink < 128))) {
#pragma unroll
        for (int jj = 0; jj < 128; ++jj)
          if (jj >= end || (jj < lo && jj >= sink)) sv[jj] = __float_as_uint(-INFINITY);
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
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? ex2_approx(m_used - m_new) : 1.f;
        if (j > 0) {  // O holds P V of every earlier tile: S_j was issued after them
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t v[32];
            tmem_ld32(t_o + c0 * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) v[jj] = __float_as_uint(__uint_as_float(v[jj]) * f);
            tmem_st32(t_o + c0 * 32, v);
          }
          tmem_st_wait();
        }
        l *= f;
        if (raise) m_used = m_new;
      }
      const float ref = m_used == -INFINITY ? 0.f : m_used;  // nothing visible yet: every weight is 0
      const float2 c2 = make_float2(c, c), nm2 = make_float2(-ref, -ref);
      float2 ls = make_float2(0.f, 0.f);
#pragma unroll
      for (int c0 = 0; c0 < 4; ++c0) {
        uint32_t pk[16];
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
          const float2 t = ffma2(make_float2(__uint_as_float(sv[c0 * 32 + 2 * jj]), __uint_as_float(sv[c0 * 32 + 2 * jj + 1])),
                                 c2, nm2);
          const float2 pp = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          ls = fadd2(ls, pp);
          pk[jj] = pack_bf16x2(pp.x, pp.y);
        }
        tmem_st16(t_s + c0 * 16, pk);
      }
      tmem_st_wait();
      l += ls.x + ls.y;
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p(x));
    }
    if (ok) ok = warp_wait(bar_o(x), 0, err, kErrWaitAcc, abort_flag);
    if (ok && !*abort_flag) {
      fence_after_sync();
      const float inv = 1.f / l;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D;
      bool bad = !(fabsf(inv) < INFINITY);
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t v[32];
        tmem_ld32(t_o + c0 * 32, v);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int jj = 0; jj < 16; ++jj) {
          const float y0 = __uint_as_float(v[2 * jj]) * inv, y1 = __uint_as_float(v[2 * jj + 1]) * inv;
          bad |= !(fabsf(y0) < INFINITY) || !(fabsf(y1) < INFINITY);
          pk[jj] = pack_bf16x2(y0, y1);
        }
        if (i < a.n) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c0 * 32);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) dst[q4] = make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
        }
      }
      if (i < a.n && a.lse) a.lse[((long long)s * a.Hq + h) * a.n + i] = (m_used + __log2f(l)) * kLn2;
      unsigned again = __ballot_sync(0xffffffffu, bad && i < a.n);
      __syncwarp();
      while (again) {
        const int b = __ffs(again) - 1;
        again &= again - 1;
        row_again<D>(a, s, h, iA + x * 128 + quarter * 32 + b);
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

template <int D>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const WindowArgs& a,
                   cudaStream_t st) {
  const int smem = Smem<D>::kAlloc;
  cudaError_t e = ensure_dynamic_smem(window_tc_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  const int n_pairs = (a.n + 255) / 256;
  return launch_kernel(window_tc_kernel<D>, dim3((unsigned)((long long)a.S * n_pairs * a.Hq)), dim3(kThreads), smem, st,
                       false, tq, tk, tv, a, n_pairs);
}

}  // namespace

cudaError_t launch_window_tc(const WindowArgs& a, int d, cudaStream_t st) {
  const uint64_t D = d, Hq = a.Hq, Hkv = a.Hkv, N = a.n, S = a.S;
  const uint64_t dq[4] = {D, Hq, N, S}, sq[3] = {D * 2, Hq * D * 2, N * Hq * D * 2};
  const uint64_t dk[4] = {D, Hkv, N, S}, sk[3] = {D * 2, Hkv * D * 2, N * Hkv * D * 2};
  const uint32_t box[4] = {64, 1, 128, 1};
  CUtensorMap tq, tk, tv;
  if (encode_tmap_bf16_4d(&tq, a.q, dq, sq, box) || encode_tmap_bf16_4d(&tk, a.k, dk, sk, box) ||
      encode_tmap_bf16_4d(&tv, a.v, dk, sk, box))
    return cudaErrorInvalidValue;
  return d == 128 ? launch<128>(tq, tk, tv, a, st) : launch<64>(tq, tk, tv, a, st);
}

cudaError_t window_tc_status(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
  return e;
}

}  // namespace skv
