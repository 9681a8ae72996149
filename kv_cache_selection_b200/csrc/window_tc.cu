// Causal attention with a sliding window and visible first tokens on the
// 5th-generation tensor cores (bf16 in, float32 accumulate): token i sees
// j <= i with j > i - window or j < n_sink.
//
// A thread block takes two 128-row query tiles A, B (256 consecutive rows of
// one head) and walks the 128-key tiles that any of its rows sees: the sink
// tiles, then those from row 0's window to the diagonal.  Per key tile and
// query tile S = Q K^T goes to tensor memory, a softmax warpgroup (thread =
// row) turns it into P in place, and O += P V reads P from tensor memory, each
// half of its keys as soon as it is there.
//
// The S tiles form one sequence q = 0, 1, ... (A and B in turn; A alone where B
// has no rows) over kS buffers in tensor memory: S(q + kS) is issued right after
// P V(q).  With d = 64 there is room for three, so that the softmax of a tile
// never waits for the products of the one before; with d = 128 for two.
//
// The running maximum is lazy (raised when a logit exceeds it by more than
// 2^8); it starts at -inf, so a row whose first tiles are hidden takes its
// maximum from the first tile it sees.  Weights are rounded to bf16 for the
// product with V (2^-8 of a weight, the precision of V itself); their sum is
// float32.
//
// A hidden value enters P V with weight 0, and 0 x NaN is NaN, and sums of values next
// to the largest float overflow: a row that ends with an output that is not finite,
// though its sum of weights is, goes through window_row_again (slow, and only
// where the inputs hold a NaN, an infinity or values that large, or where logits
// beyond 2^27 leave no weight to hold).
//
// Measured (B200): 65536 tokens, 28 heads, d = 128, window 4096: 3365 us, 1112
// TFLOP/s; 4 x 4001 tokens, 14 heads, d = 64, window 1024: 125 us, 413 TFLOP/s.  At
// d = 128 a pair of key tiles takes 3650 cycles for 2048 of products and 2048 of
// exponentials: the bound is the chain S -> softmax (2180 cycles, half of them
// exponentials) -> P V -> next S of each query tile, with two in flight.  At d = 64
// (products of N = 64 cost as much as of N = 128) it is the scheduler that two
// softmax warps share with the MMA warp.
//
// Warps (384 threads): 0 TMA producer, 1 tensor-memory owner and MMA issuer,
// 4..7 softmax of tile A, 8..11 of tile B.  The MMA warp shares its scheduler with a
// warp of each softmax, so its waits suspend instead of polling.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "window_row.cuh"

namespace skv {
namespace {
using namespace tc;

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
  static constexpr int kS = D == 64 ? 3 : 2;      // S buffers
  static constexpr int kSlots = D == 64 ? 8 : 4;  // K/V ring slots of one 128-key tile
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = 128 * 128;
  static constexpr int kTile = kAtoms * kAtomBytes;  // 128 rows x D bf16
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTile;
  static constexpr int kBar = kKV + kSlots * kTile;
  // q[2], kv_full[kSlots], kv_empty[kSlots], s_full[kS], p_full[kS][2 halves], pv_done[2][even, odd tiles], done
  static constexpr int kNumBars = 2 + 2 * kSlots + 3 * kS + 5;
  static constexpr int kTmem = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmem + 4;
  static constexpr int kBytes = kAbort + 4;
  // at least 116 KB: a second block (it would need all tensor memory too) never shares the SM
  static constexpr int kAlloc = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;
};

// Ties loaded registers to a wait before it, so that no use moves above that.
__device__ __forceinline__ void after_wait(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowArgs a, int n_pairs) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // unit -> (pair, stream, head): the heads that share a K/V range run next to
  // one another, the units with the fewest keys last
  const int G = a.Hq / a.Hkv;
  int u = blockIdx.x;
  const int h = u % a.Hq;
  u /= a.Hq;
  const int s = u % a.S, pair = n_pairs - 1 - u / a.S;
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
  constexpr int kS = L::kS, kSlots = L::kSlots;
  auto bar_full = [&](int sl) { return sb + L::kBar + 8u * (2 + sl); };
  auto bar_empty = [&](int sl) { return sb + L::kBar + 8u * (2 + kSlots + sl); };
  auto bar_s = [&](int b) { return sb + L::kBar + 8u * (2 + 2 * kSlots + b); };
  auto bar_p = [&](int b, int half) { return sb + L::kBar + 8u * (2 + 2 * kSlots + kS + 2 * b + half); };
  // P V of key tile j: phase j / 2 of its own parity's barrier.  Who sees S of
  // tile j knows that P V of tile j - 3 is done, so j - 1 (the neighbour of j - 3
  // on that barrier) can be waited for at any time
  auto bar_pv = [&](int x, int j) { return sb + L::kBar + 8u * (2 + 2 * kSlots + 3 * kS + 2 * x + (j & 1)); };
  const uint32_t bar_done = sb + L::kBar + 8u * (6 + 2 * kSlots + 3 * kS);
  // K runs `lead` tiles ahead of V: the ring holds K_0 .. K_lead, V_0, K_lead+1, V_1, ...
  const int lead = (kS - 1) / (nB > 0 ? 2 : 1);
  auto pos_k = [&](int j) { return j <= lead ? j : 2 * j - lead; };
  auto pos_v = [&](int j) { return min(n_load, lead + j + 1) + j; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmem);
  int* err = &g_err;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar_q(x), 1);
      mbar_init(bar_pv(x, 0), 1);
      mbar_init(bar_pv(x, 1), 1);
    }
    for (int b = 0; b < kS; ++b) {
      mbar_init(bar_s(b), 1);
      mbar_init(bar_p(b, 0), 4);
      mbar_init(bar_p(b, 1), 4);
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
  // columns: kS buffers of S/P, then O of A, O of B
  auto col_s = [](int b) { return (uint32_t)(b * 128); };
  auto col_o = [](int x) { return (uint32_t)(kS * 128 + x * D); };

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
      int jk = 0, jv = 0;  // tiles of K and V so far
      for (int idx = 0; idx < 2 * n_load; ++idx) {
        const int sl = idx % kSlots;
        const bool is_v = jk == n_load || (jk > lead + jv);
        const int j = is_v ? jv++ : jk++;
        if (!mbar_wait(bar_empty(sl), ((idx / kSlots) & 1) ^ 1, err, kErrWaitEmpty, abort_flag)) break;
        const int r0 = key_tile(j) * 128;
        mbar_arrive_expect_tx(bar_full(sl), L::kTile);
        const uint32_t dst = sb + L::kKV + sl * L::kTile;
        for (int at = 0; at < L::kAtoms; ++at)
          tma_load_4d(dst + at * L::kAtomBytes, is_v ? &tm_v : &tm_k, bar_full(sl), at * 64, g, r0, s);
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
    {
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t id_o = idesc_bf16(128, D, false, true);
      const uint64_t dq0 = sdesc_sw128(sb + L::kQ, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sb + L::kKV, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sb + L::kKV, L::kAtomBytes, 1024);
      auto slot16 = [&](int pos) { return (uint64_t)((pos % kSlots) * (L::kTile >> 4)); };
      auto wait_slot = [&](int pos) {
        return warp_wait_all(bar_full(pos % kSlots), (pos / kSlots) & 1, err, kErrWaitLoad, abort_flag);
      };
      auto slot_ready = [&](int pos) { return mbar_test_wait(bar_full(pos % kSlots), (pos / kSlots) & 1); };
      // S = Q_x K_j^T into buffer b; last: no other tile of queries reads K_j
      auto issue_s = [&](int x, int j, int b, bool last) {
        uint64_t dq = dq0 + (uint64_t)((x * L::kTile) >> 4), dk = dk0 + slot16(pos_k(j));
        const uint32_t t_s = tmem + col_s(b);
        asm volatile("" : "+l"(dq), "+l"(dk));  // the sums below stay here: hoisted, they would not fit the registers
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * L::kAtomBytes + (kk & 3) * 32) >> 4);
          mma_ss_e(t_s, dq + off, dk + off, id_s, kk > 0 ? 1u : 0u);
        }
        commit_e(bar_s(b));
        if (last) commit_e(bar_empty(pos_k(j) % kSlots));
      };
      int b = 0;          // buffer and turn of the tile at hand
      uint32_t turn = 0;
      // One S tile of the sequence: O_x += P V_j, then S of (x2, j2), kS places on,
      // into the same buffer.  The time from P to that S is on the path that bounds
      // the kernel: what a half step waits for is asked for at once, and one vote
      // settles it when everything is there already.
      auto step = [&](auto x_, int j, bool first_v, bool last_v, bool more, int x2, int j2, bool first_k, bool last_k) {
        constexpr int x = decltype(x_)::value;
        const int pv = pos_v(j);
        bool there = mbar_test_wait(bar_p(b, 0), turn);
        if (first_v) there = there & slot_ready(pv);
        uint64_t dv = dv0 + slot16(pv);
        const uint32_t o = tmem + col_o(x), p = tmem + col_s(b);
        asm volatile("" : "+l"(dv));
        if (!__any_sync(0xffffffffu, there) &&
            !((!first_v || wait_slot(pv)) && warp_wait_all(bar_p(b, 0), turn, err, kErrWaitP, abort_flag)))
          return false;
        fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_e(o, p + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id_o, (j > 0 || kk > 0) ? 1u : 0u);
        there = mbar_test_wait(bar_p(b, 1), turn);
        if (more && first_k) there = there & slot_ready(pos_k(j2));
        if (!__any_sync(0xffffffffu, there) && !((!more || !first_k || wait_slot(pos_k(j2))) &&
                                                 warp_wait_all(bar_p(b, 1), turn, err, kErrWaitP, abort_flag)))
          return false;
        fence_after_sync();
#pragma unroll
        for (int kk = 4; kk < 8; ++kk) mma_ts_e(o, p + kk * 8, dv + (uint64_t)((kk * 2048) >> 4), id_o, 1u);
        commit_e(bar_pv(x, j));  // before S's commit: who sees that S may count on this one
        if (more) issue_s(x2, j2, b, last_k);
        if (last_v) commit_e(bar_empty(pv % kSlots));
        if (++b == kS) {
          b = 0;
          turn ^= 1;
        }
        return true;
      };
      using A = std::integral_constant<int, 0>;
      using Bt = std::integral_constant<int, 1>;
      const int nq = nA + nB;
      bool ok = true;
      if (nB > 0) {  // A_0 B_0 A_1 B_1 ... B_nA
        for (int q = 0; ok && q < min(kS, nq); ++q) {
          const int x = q >= 2 * nA || (q & 1) ? 1 : 0, j = min(q >> 1, nA);
          if (!(ok = wait_slot(pos_k(j)) && warp_wait_all(bar_q(x), 0, err, kErrWaitLoad, abort_flag))) break;
          fence_after_sync();
          issue_s(x, j, q, x == 1);
        }
        for (int j = 0; ok && j < nA; ++j) {
          if (kS == 2) {
            if (!(ok = step(A(), j, true, false, true, j + 1 < nA ? 0 : 1, j + 1, true, j + 1 == nA))) break;
            ok = step(Bt(), j, false, true, j + 1 < nA, 1, j + 1, false, true);
          } else {
            if (!(ok = step(A(), j, true, false, j + 1 < nA, 1, j + 1, false, true))) break;
            ok = step(Bt(), j, false, true, j + 2 <= nA, j + 2 < nA ? 0 : 1, j + 2, true, j + 2 == nA);
          }
        }
        if (ok) ok = step(Bt(), nA, true, true, false, 1, 0, false, false);
      } else {  // A alone
        for (int j = 0; ok && j < min(kS, nA); ++j) {
          if (!(ok = wait_slot(pos_k(j)) && warp_wait_all(bar_q(0), 0, err, kErrWaitLoad, abort_flag))) break;
          fence_after_sync();
          issue_s(0, j, j, true);
        }
        for (int j = 0; ok && j < nA; ++j) ok = step(A(), j, true, true, j + kS < nA, 0, j + kS, true, true);
      }
      commit_e(bar_done);
      if (lane == 0) drain_wait(bar_done, 0, err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    regs_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2, nX = x == 0 ? nA : nB;
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const int i = iA + x * 128 + r;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_o = t_lane + col_o(x);
    const float c = a.scale_log2;
    float m_used = -INFINITY, l = 0.f;
    bool ok = nX > 0;
    for (int j = 0; ok && j < nX; ++j) {
      // place of this S tile in the sequence
      const int q = nB == 0 ? j : x == 0 ? 2 * j : min(2 * j + 1, 2 * nA), b = q % kS;
      const uint32_t t_s = t_lane + col_s(b);
      if (!(ok = warp_spin_wait(bar_s(b), (q / kS) & 1, err, kErrWaitAcc, abort_flag))) break;
      fence_after_sync();
      // A row sees columns below `end`, and from `lo` on or below `sink`.  Hidden
      // ones become -inf in tensor memory before S is read: a separate rolled
      // loop, so that the masks cost the main path no registers.  Per 32 columns
      // the warp's rows (32 consecutive) tell whether there is anything to hide.
      const int base = key_tile(j) * 128;
      const int end0 = i - lane + 1 - base, lo0 = end0 - a.window, sink = a.n_sink - base;  // of lane 0
      if (end0 < 128 || (lo0 + 31 > 0 && sink < 128)) {
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          if (end0 >= c0 + 32 && (lo0 + 31 <= c0 || sink >= c0 + 32)) continue;
          // visible columns of the 32 as a mask (shifts of 64 bits: counts 0..32)
          auto below = [&](int x) { return (uint32_t)((1ull << min(max(x - c0, 0), 32)) - 1); };
          const uint32_t see = below(end0 + lane) & (~below(lo0 + lane) | below(sink));
          uint32_t v[32];
          tmem_ld32(t_s + c0, v);
          tmem_ld_wait_dep(v);
#pragma unroll
          for (int jj = 0; jj < 32; ++jj)
            if (!(see >> jj & 1)) v[jj] = __float_as_uint(-INFINITY);
          tmem_st32(t_s + c0, v);
        }
        tmem_st_wait();
      }
      uint32_t sv[128];
      tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
      tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
      tmem_ld_wait_dep(*reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
      after_wait(*reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
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
      const float m_new = fmaxf(m_used, reference_of(mx * c));
      const bool raise = m_new > m_used + kRaise;
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? ex2_approx(m_used - m_new) : 1.f;
        if (j > 0) {
          // O must hold P V of every earlier tile
          if (!(ok = warp_wait(bar_pv(x, j - 1), ((j - 1) >> 1) & 1, err, kErrWaitAcc, abort_flag))) break;
          fence_after_sync();
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t v[32];
            tmem_ld32(t_o + c0 * 32, v);
            tmem_ld_wait_dep(v);
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
        if (c0 & 1) {  // the weights of 64 keys
          tmem_st_wait();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p(b, c0 >> 1));
        }
      }
      l += ls.x + ls.y;
    }
    if (ok) ok = warp_wait(bar_pv(x, nX - 1), ((nX - 1) >> 1) & 1, err, kErrWaitAcc, abort_flag);
    if (ok && !*abort_flag) {
      fence_after_sync();
      const float inv = 1.f / l;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D;
      bool bad = false;
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t v[32];
        tmem_ld32(t_o + c0 * 32, v);
        tmem_ld_wait_dep(v);
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
      // (a NaN in the sum of weights: a visible logit was one, so the row is NaN)
      unsigned again = __ballot_sync(0xffffffffu, bad && l == l && i < a.n);
      __syncwarp();
      while (again) {
        const int b = __ffs(again) - 1;
        again &= again - 1;
        window_row_again<__nv_bfloat16, D>(a, s, h, iA + x * 128 + quarter * 32 + b);
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
