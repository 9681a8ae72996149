// Attention of a few text tokens over the 4-bit cache (format: q4_cache.cuh),
// streamed once, codes fed to the tensor cores without being dequantised.
//
// With codes c, scales s and smallest values m per (token j, group g):
//   q . k_j  = sum_g [ s_jg (q_g . c_jg) + m_jg sum(q_g) ],
//   O        = sum_j p_j v_j = sum_j (p_j s_jg) (c_jg - 8) + sum_j p_j (m_jg + 8 s_jg).
// The codes are exact fp16 numbers, so both sums are fp16 products with float32
// accumulation, and the scales meet float32 numbers only.  In bf16 calls a pair
// of codes is one and of the word as it stands: in a half's low ten bits a code
// is a subnormal number, c 2^-18 or c 2^-22, which the tensor cores take exactly;
// Q (or P s) is 16 times larger where it meets the latter.  What the rounding of
// P s to fp16 would do to a code of 15 is halved by centring: 8 sum(P s), of the
// rounded P s, comes from one more product with a constant and is taken off at
// the end.  Against codes c - 8 made by subtractions (float32 calls keep those:
// sums of half the size) 71 -> 59 us for 4 streams of up to 131072 tokens, G = 7,
// D = 128.  The rows are the G query heads of a KV
// head times the text tokens, eight to a tile.
//   Q: scaled by a power of two per row (largest element in [2^10, 2^11)); bf16
//     values are then exact in fp16, float32 ones are split into two fp16 parts
//     (NS = 2), 22 bits.  S is summed in units of 2^18, which keep it in range
//     whatever the keys.
//   P s: in fp16 relative to the largest V scale met so far (a power of two
//     R_g per group, lazily raised as the row maximum is): 2^-11 off at most,
//     an eighth of what the bf16 result rounds by; float32 again takes two parts.
//   P: relative to a row maximum that moves only when a logit exceeds it by
//     more than 2^6, so that most blocks need one vote and no shuffle.
// The tensor cores cut their float32 sums instead of rounding them, which a long
// sum adds up: in float32 calls eight channels of S and each block's P V are summed
// on their own, least parts first, and added on the CUDA cores (6.8e-7 off over
// 32768 tokens, d = 128, where running sums were 4.6e-6 off; as fast).  A bf16 result
// does not see it.
// Tensor-core shape m16n8k16 with tokens (K) or channels (V) as the 16 rows and
// query rows as the 8 columns: the fragments come from shared memory as stored,
// S^T turns into P^T's fragment by an 8x8 transpose, and nothing but 4-bit codes
// is staged.  A tcgen05 product would need the tile dequantised into shared
// memory first, 4x the bytes per value, for rows that fill 8 of its 128.
//
// The visible 32-token blocks of all (stream, KV head) are numbered in order
// and dealt evenly to the W workers (thread blocks), so ragged streams balance;
// a worker writes one partial (max, sum, O) per (stream, KV head) it meets, and
// q4_merge_kernel joins them in worker order with what a row sees on its own: the
// text tokens and, with a window, the cache tokens that later rows of its tile do not
// see (q4_visible.cuh).  Where it is cheaper (q4_alone) each (stream, KV head) has a
// thread block of its own, which writes the results itself.
//
// Measured (B200, graph replays, bf16, d = 128, G = 7, one text token, caches beyond
// L2): 4 ragged streams of up to 131072 tokens, 4 KV heads, 53.7 us (4.6 TB/s of
// the cache; 245 MB would take 37.4 at the copy rate), 131072 tokens of one stream
// 24.6 us (75 MB: 11.5).  About 8 us of each are the first copies' latency and the
// merge; the loop streams at some 5 TB/s, the tensor-core and integer pipes each
// half busy and 12 warps an SM too few to hide the latencies between them (measured
// apart, at 56.5 us: with 8 warps 61.5, with 16, three stages each, 57.5).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "q4_cache.cuh"
#include "q4_visible.cuh"
#include "tc_common.cuh"

namespace skv {
namespace {

// Warps of a worker: as many as their registers allow without spills.
template <int NT, int NS>
constexpr int warps_of() {
  return NT * NS == 1 ? 12 : 8;
}
// What bounds their registers: 168 a thread, but 128 where they fit (d = 64), which
// leaves room for a block of the merge to come in beside a worker that still runs (one
// token over 16384, d = 64: 9.1 us, with 132 registers 10.3).
template <int D, int NT, int NS>
constexpr int most_threads() {
  return D == 64 && NT * NS == 1 ? 512 : warps_of<NT, NS>() * 32;
}
constexpr int kStages = 4;      // blocks in flight per warp
constexpr float kRaise = 6.f;   // log2 headroom of the lazy row maximum
constexpr float kMinR = 0x1p-118f;  // least V reference (kPScale / R stays finite)
constexpr float kPScale = 512.f;    // P s <= 2^6 * 512 < 65504

// Sums of weights times values can overflow where their quotient, a mean of the
// values, does not (values above 2^128 over the tokens' number): a row whose result is
// not finite is taken again with values in units of 1 / kLess.
constexpr float kLess = 0x1p-40f;

constexpr int kOwnText = 32;  // most text tokens of a call whose thread blocks join them one by one

__device__ int g_err;  // first error of the ring's waits of all calls on a device

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {  // c = A B
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// The four fields of a word as fp16 pairs: c - 8, or, as they stand in the word,
// the subnormal numbers c 2^-18 (fields 0, 3) and c 2^-22 (fields 1, 2).
template <bool kCentred>
__device__ __forceinline__ void codes_of(uint32_t x, uint32_t (&f)[4]) {
  const uint32_t y = q4_turn(x);
  if (!kCentred) {
    f[0] = x & 0x03C003C0u;
    f[1] = y & 0x003C003Cu;
    f[2] = x & 0x003C003Cu;
    f[3] = y & 0x03C003C0u;
    return;
  }
  f[0] = q4_raw<0>(x);
  f[1] = q4_raw<1>(y);
  f[2] = q4_raw<2>(x);
  f[3] = q4_raw<3>(y);
  const __half2 near = __float2half2_rn(24.f), far = __float2half2_rn(264.f);
  f[0] = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&f[0]), near));
  f[1] = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&f[1]), far));
  f[2] = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&f[2]), far));
  f[3] = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&f[3]), near));
}

// A token's scale words.
template <int NG>
__device__ __forceinline__ void scales_of(const uint8_t* scales, int tok, uint32_t (&sm)[NG]) {
  if (NG == 2) *reinterpret_cast<uint2*>(sm) = *reinterpret_cast<const uint2*>(scales + tok * 8);
  else sm[0] = *reinterpret_cast<const uint32_t*>(scales + tok * 4);
}

__device__ __forceinline__ void load_channels(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_channels(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The numbering of the visible blocks of all (stream, KV head) and their deal to
// the workers: q blocks each, the first r one more (32-bit arithmetic: the host
// checks that a cache has less than 2^31 blocks).
struct Deal {
  int total, W, q, r;
  __device__ __forceinline__ int first(int w) const { return w * q + min(w, r); }
  __device__ __forceinline__ int owner(int x) const {
    const int head = r * (q + 1);
    return x < head ? x / (q + 1) : r + (x - head) / q;
  }
};
// Visible blocks of a KV head in the streams before `end` (a whole warp calls it:
// lengths on the device are summed by its lanes).
template <bool kRagged>
__device__ __forceinline__ int blocks_before(const WindowArgs& a, int end) {
  if (!kRagged) return end * visible_of(a, 0).count();
  int sum = 0;
  for (int s = threadIdx.x & 31; s < end; s += 32) sum += visible_of(a, s).count();
  return __reduce_add_sync(0xffffffffu, sum);
}
// The stream of block number x (below the total), and the number of its first block.
template <bool kRagged>
__device__ __forceinline__ int stream_of(const WindowArgs& a, int x, int& first) {
  if (!kRagged) {
    const int each = visible_of(a, 0).count() * a.Hkv, s = x / each;
    first = s * each;
    return s;
  }
  const int lane = threadIdx.x & 31;
  first = 0;
  for (int s0 = 0;; s0 += 32) {
    const int mine = s0 + lane < a.S ? visible_of(a, s0 + lane).count() * a.Hkv : 0;
    int upto = mine;  // of streams s0 .. s0 + lane
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, first + upto > x);
    if (past || s0 + 32 >= a.S) {  // (always found for x below the total)
      const int at = past ? __ffs(past) - 1 : 31;
      first += __shfl_sync(0xffffffffu, upto - mine, at);
      return min(s0 + at, a.S - 1);
    }
    first += __shfl_sync(0xffffffffu, upto, 31);
  }
}
template <bool kRagged>
__device__ __forceinline__ Deal deal_of(const WindowArgs& a, int W) {
  Deal d;
  d.total = blocks_before<kRagged>(a, a.S) * a.Hkv;
  d.W = min(W, d.total);  // every worker that counts owns a block
  d.q = d.W ? d.total / d.W : 0;
  d.r = d.total - d.q * d.W;
  return d;
}

// A row's running maximum (log2), sum and accumulator, in a warp: E channels a lane.
template <int E>
struct RowSum {
  float m = -INFINITY, l = 0.f, acc[E];
  __device__ __forceinline__ RowSum() {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
  }
  __device__ __forceinline__ void join(float m2, float l2, const float (&v)[E], float unit = 1.f) {  // acc += unit v (weights relative to 2^m2)
    const float nm = fmaxf(m, m2);
    const float ref = nm == -INFINITY ? 0.f : nm;
    const float f1 = tc::ex2_approx(m - ref), f2 = tc::ex2_approx(m2 - ref);
    l = l * f1 + l2 * f2;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f1 + v[e] * (f2 * unit);
    m = nm;
  }
};
// What the row (text token i, head h) sees beside the cache tokens of its whole tile:
// cache tokens behind its own window's edge and before that of the tile's last
// text token, and the text tokens; of both the ones first, first + step, ...
// kAll: all that it sees, with values in units of 1 / kLess.
template <typename T, int D, bool kAll = false>
__device__ __forceinline__ void join_own(const WindowArgs& a, int L, int s, int h, int g, int i, int i_last, int first,
                                         int step, RowSum<D / 32>& sum) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(a.q) + (((long long)s * a.n + i) * a.Hq + h) * D + lane * E;
  float qv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = to_f(q[e]) * a.scale_log2;
  // four tokens' loads and sums over the lanes at once, then one by one
  auto run = [&](int j, int end, auto load) {
    auto some = [&](auto count) {
      constexpr int N = decltype(count)::value;
      float t[N], k[N][E], v[N][E];
#pragma unroll
      for (int b = 0; b < N; ++b) {
        load(j + b * step, k[b], v[b]);
        t[b] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) t[b] = fmaf(qv[e], k[b][e], t[b]);
      }
#pragma unroll
      for (int off = 16; off; off >>= 1)
#pragma unroll
        for (int b = 0; b < N; ++b) t[b] += __shfl_xor_sync(0xffffffffu, t[b], off);
#pragma unroll
      for (int b = 0; b < N; ++b) {
        if (t[b] != t[b]) sum.l = t[b];  // a NaN logit makes the row NaN
        sum.join(t[b], 1.f, v[b], kAll ? kLess : 1.f);
      }
      j += N * step;
    };
    while (j < end - 3 * step) some(std::integral_constant<int, 4>());
    while (j < end) some(std::integral_constant<int, 1>());
  };
  if (a.window || kAll) {
    const int end = kAll ? L : tile_from(a, L, i_last), sinks = a.window ? min(a.n_sink, end) : 0;
    const uint8_t* cache = static_cast<const uint8_t*>(a.cache) + ((long long)s * a.Hkv + g) * a.cap_blk * Q4Block<D>::kBytes;
    auto cached = [&](int j, float (&k)[E], float (&v)[E]) {
      q4_token<D, E>(cache + (long long)(j / kQ4Tokens) * Q4Block<D>::kBytes, j % kQ4Tokens, lane * E, k, v);
    };
    if (kAll) run(first, sinks, cached);
    run(max(row_from(a, L, i), sinks) + first, end, cached);
  }
  auto text = [&](int j, float (&k)[E], float (&v)[E]) {
    const long long at = (((long long)s * a.n + j) * a.Hkv + g) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = to_f(static_cast<const T*>(a.k)[at + e]);
      v[e] = to_f(static_cast<const T*>(a.v)[at + e]);
    }
  };
  // text tokens: the first ones below n_sink, and those of the window
  const int sinks = a.window ? (int)min(max((long long)a.n_sink - L, 0ll), i + 1ll) : 0;
  const int from = a.window ? max(sinks, i - a.window + 1) : 0;
  run(first, sinks, text);
  run(from + first, i + 1, text);
}

// Row maxima (log2) from which on the weights may be too small to hold (reference_of).
constexpr float kHuge = 0x1p22f;
constexpr uint32_t kAllGroups = 7u;  // whatever their values

// One row again by kWarps warps (all of a block's, or one), token by token, where its
// result is not finite in the groups of channels `groups`, or its logits are huge:
// slow, and only where sums overflow or inputs hold a NaN, an infinity or keys and
// queries far beyond the usual.  A visible NaN scale explains its group's result,
// which stands then.  acc, ml: shared memory for the warps' sums.
template <typename T, int D, int kWarps>
__device__ __noinline__ void row_again(const WindowArgs& a, int L, int s, int h, int g, int i, uint32_t groups,
                                       float (*acc)[D], float (*ml)[2]) {
  using B = Q4Block<D>;
  constexpr int E = D / 32, kScan = 8;
  const int lane = threadIdx.x & 31, warp = kWarps == 1 ? 0 : threadIdx.x >> 5;
  const uint8_t* cache = static_cast<const uint8_t*>(a.cache) + ((long long)s * a.Hkv + g) * a.cap_blk * B::kBytes;
  const int from = row_from(a, L, i), sinks = min(a.n_sink, from), count = sinks + L - from;
  uint32_t nan = 0;
  for (int x0 = warp * 32 + lane; x0 < count; x0 += kWarps * 32 * kScan) {
    uint32_t sm[kScan][B::kGroups];
#pragma unroll
    for (int b = 0; b < kScan; ++b) {
      const int x = min(x0 + b * kWarps * 32, count - 1), j = x < sinks ? x : x - sinks + from;
      const uint8_t* at = cache + (long long)(j / kQ4Tokens) * B::kBytes + B::kVs + j % kQ4Tokens * (B::kGroups * 4);
#pragma unroll
      for (int gg = 0; gg < B::kGroups; ++gg) sm[b][gg] = __ldg(reinterpret_cast<const uint32_t*>(at) + gg);
    }
#pragma unroll
    for (int b = 0; b < kScan; ++b)
#pragma unroll
      for (int gg = 0; gg < B::kGroups; ++gg)
        if (q4_scale(sm[b][gg]) != q4_scale(sm[b][gg])) nan |= 1u << gg;
  }
  if (kWarps == 1) {
    nan = __reduce_or_sync(0xffffffffu, nan);
  } else {
    const int first = __syncthreads_or(nan & 1u), second = __syncthreads_or(nan & 2u);
    nan = (first ? 1u : 0u) | (second ? 2u : 0u);
  }
  if ((groups & ~nan) == 0) return;
  RowSum<E> sum;
  join_own<T, D, true>(a, L, s, h, g, i, i, warp, kWarps, sum);
  T* out = static_cast<T*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D;
  float* lse = a.lse ? a.lse + ((long long)s * a.Hq + h) * a.n + i : nullptr;
  if (kWarps == 1) {
    if (lane == 0 && lse) *lse = (sum.m + log2f(sum.l)) * kLn2;
#pragma unroll
    for (int e = 0; e < E; ++e) out[lane * E + e] = from_f<T>(sum.acc[e] / sum.l * (1.f / kLess));
    return;
  }
  ml[warp][0] = sum.m;
  ml[warp][1] = sum.l;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = sum.acc[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  RowSum<1> all;
  for (int w = 0; w < kWarps; ++w) {
    const float v[1] = {acc[w][threadIdx.x]};
    all.join(ml[w][0], ml[w][1], v);
  }
  out[threadIdx.x] = from_f<T>(all.acc[0] / all.l * (1.f / kLess));
  if (threadIdx.x == 0 && lse) *lse = (all.m + log2f(all.l)) * kLn2;
}

// How a call is shared out: over the workers (one length, or lengths on the device),
// or a thread block alone for each (stream, KV head).
enum Share { kEven, kRagged, kOwn };

template <typename T, int D, int NT, int NS, Share kShare>
__global__ void __launch_bounds__(most_threads<D, NT, NS>(), 1) q4_attn_kernel(const __grid_constant__ Q4AttnArgs p) {
  using B = Q4Block<D>;
  constexpr int kWarps = warps_of<NT, NS>();
  constexpr int NG = B::kGroups;
  constexpr int KW = D / 32;          // K words per (token row, tig)
  constexpr int MT = D / 16;          // 16-channel tiles of O
  constexpr int kRows = 8 * NT;
  constexpr int kStride = D + 4;      // padded row of the partials in shared memory
  constexpr bool kAlone = kShare == kOwn;
  constexpr bool kCentred = NS == 2;  // codes as c - 8, else as subnormals
  // with Q (P s) 16 times larger where the code is c 2^-22
  constexpr float kCodeNear = 0x1p-18f, kCodeFar = 0x1p-22f, kUnit = 0x1p-18f;
  extern __shared__ __align__(16) uint8_t smem[];
  const WindowArgs& a = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int G = a.Hq / a.Hkv, R = G * a.n;
  const int row0 = blockIdx.y * kRows;
  uint8_t* ring = smem + warp * (kStages * B::kBytes);
  const uint32_t ring_u32 = tc::smem_u32(ring);
  // a warp's ring is its own: barriers and abort flag need no block-wide barrier
  __shared__ __align__(8) uint64_t s_bars[kWarps * kStages];
  __shared__ int s_abort[kWarps];
  volatile int* abort_flag = s_abort + warp;
  const uint32_t bars = tc::smem_u32(s_bars + warp * kStages);
  if (lane == 0) {
    *abort_flag = 0;
#pragma unroll
    for (int i = 0; i < kStages; ++i) tc::mbar_init(bars + 8u * i, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  int done = 0;     // blocks this warp has taken from its ring
  bool ok = true;

  pdl_wait();
  pdl_trigger();
  int x = 0, x_end = 1, s = kAlone ? blockIdx.x / a.Hkv : 0, s_base = 0;
  if (!kAlone) {
    const Deal deal = deal_of<kShare == kRagged>(a, p.W);
    if ((int)blockIdx.x >= deal.W) return;
    x = deal.first(blockIdx.x);
    x_end = deal.first(blockIdx.x + 1);
    s = stream_of<kShare == kRagged>(a, x, s_base);
  }
  Visible vis = visible_of(a, s);
  const int i_last = tile_last(blockIdx.y, kRows, R, G);

  while (x < x_end) {
    int g = blockIdx.x % a.Hkv, v0 = 0, v1 = vis.count();
    if (!kAlone) {
      while (x >= s_base + a.Hkv * vis.count()) {
        s_base += a.Hkv * vis.count();
        vis = visible_of(a, ++s);
      }
      g = (x - s_base) / vis.count();
      v0 = (x - s_base) - g * vis.count();
      v1 = min(vis.count(), v0 + (x_end - x));
    }
    const uint8_t* base = static_cast<const uint8_t*>(a.cache) + ((long long)s * a.Hkv + g) * a.cap_blk * B::kBytes;

    // Q's loads go out before the ring's, which would be ahead of them in every
    // queue of the memory system
    float qv[NT][KW][8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + gid;
      const T* q = static_cast<const T*>(a.q) + (((long long)s * a.n + r / G) * a.Hq + g * G + r % G) * D;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        if (r < R) {
          load_channels(q + (w >> 1) * 64 + tig * 16 + (w & 1) * 8, qv[nt][w]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) qv[nt][w][e] = 0.f;
        }
      }
    }
    // the warp's blocks v0 + warp, + kWarps, ...: its n-th (of the kernel) goes to
    // stage n % kStages
    auto issue = [&](int v, int n) {
      const uint32_t bar = bars + 8u * (n % kStages);
      tc::mbar_arrive_expect_tx(bar, B::kBytes);
      tc::bulk_load(ring_u32 + (n % kStages) * B::kBytes, base + (long long)vis.block(v) * B::kBytes, B::kBytes, bar);
    };
    int issued = done;
    if (lane == 0)
      for (int v = v0 + warp; v < v1 && issued < done + kStages; v += kWarps) issue(v, issued++);
    issued = done + min(kStages, max(0, (v1 - v0 - warp + kWarps - 1) / kWarps));

    // ---- Q fragments, per-row scale and group sums
    uint32_t qf[NT][NS][MT][2];
    float qsum[NT][NG][2], rs[NT][2];
    uint32_t huge_rows = 0;  // bit 2 nt + e
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(qv[nt][w][e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest element into [2^10, 2^11); 1 for a zero row or one with an infinity
      int ex = (int)(__float_as_uint(top) >> 23);
      // (the least exponent keeps 2^(264 - ex), or 16 times it, finite)
      ex = ex == 0 && top == 0.f ? 137 : ex == 255 ? 137 : max(ex, kCentred ? 12 : 16);
      const float up = __uint_as_float((uint32_t)(264 - ex) << 23);  // 2^(10 - (ex - 127))
      // S is summed in units of 2^18, which leave it below the largest key (q is below
      // 2^11, 128 channels); the row factor 2^(ex - 137) takes that up, or, where q is
      // so large that it could overflow, S itself afterwards
      const bool huge = ex >= 200;
      const float down = __uint_as_float((uint32_t)(huge ? ex - 10 : ex + 8) << 23);
      float sum[NG];
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) sum[gg] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const float by = !kCentred && (f == 1 || f == 2) ? 16.f * up : up;
          const float x0 = qv[nt][w][q4_k_channel(f, 0)] * by, x1 = qv[nt][w][q4_k_channel(f, 1)] * by;
          const __half2 hi = __floats2half2_rn(x0, x1);
          const float2 h = __half22float2(hi);
          qf[nt][0][2 * w + (f >> 1)][f & 1] = half2_bits(hi);
          if (kCentred) {
            qf[nt][NS - 1][2 * w + (f >> 1)][f & 1] = half2_bits(__floats2half2_rn(x0 - h.x, x1 - h.y));
            sum[w >> 1] += (x0 + x1) * kUnit;
          } else {
            sum[w >> 1] += (h.x + h.y) * (f == 1 || f == 2 ? kCodeFar : kCodeNear);
          }
        }
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 1);
        sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 2);
      }
      // this lane's columns of S^T are rows 2 tig and 2 tig + 1 of the tile
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = (2 * tig + e) * 4;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) qsum[nt][gg][e] = __shfl_sync(0xffffffffu, sum[gg], from);
        rs[nt][e] = __shfl_sync(0xffffffffu, down, from) * a.scale_log2;
        if (__shfl_sync(0xffffffffu, huge, from)) huge_rows |= 1u << (2 * nt + e);
      }
    }

    // o8: eight times the sum of P s as rounded, in O's fragment (all channels alike)
    constexpr int NC = kCentred ? 0 : NG;
    float o8[NT][NC + 1][4];
    // m: row maximum in log2 units; mr: m, or 0 for -inf; above: the logit (before rs) that raises it
    float o[NT][MT][4], corr[NT][NG][2], l[NT][2], m[NT][2], mr[NT][2], above[NT][2], vR[NG], vs[NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
#pragma unroll
      for (int gg = 0; gg < NC; ++gg)
#pragma unroll
        for (int e = 0; e < 4; ++e) o8[nt][gg][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] = 0.f;
        m[nt][e] = above[nt][e] = -INFINITY;
        mr[nt][e] = 0.f;
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) corr[nt][gg][e] = 0.f;
      }
    }
#pragma unroll
    for (int gg = 0; gg < NG; ++gg) {
      vR[gg] = kMinR;
      vs[gg] = kPScale / kMinR;
    }

    const int from = tile_from(a, vis.L, i_last);
    const bool any_huge = __any_sync(0xffffffffu, huge_rows != 0);
    for (int v = v0 + warp; ok && v < v1; v += kWarps, ++done) {
      const int stage = done % kStages;
      const uint32_t bar = bars + 8u * stage, parity = (done / kStages) & 1;
      if (!(ok = tc::warp_wait_all(bar, parity, &g_err, tc::kErrWaitLoad, abort_flag))) break;
      const uint8_t* blk = ring + stage * B::kBytes;
      const int t0 = vis.block(v) * kQ4Tokens;
      const bool plain = !any_huge && t0 + kQ4Tokens <= vis.L && (t0 >= from || t0 + kQ4Tokens <= a.n_sink);
      // ---- S^T = K Q^T, 16 tokens at a time; t rs = logits in log2 units
      float t[NT][2][4];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        uint32_t ka[KW], kb[KW];
        const uint8_t* kr = blk + (kt * 16 + gid) * B::kRow + tig * (D / 8);
        if (D == 128) {
          *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(kr);
          *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(kr + 8 * B::kRow);
        } else {
          *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(kr);
          *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(kr + 8 * B::kRow);
        }
        float acc[NT][NG][4];
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t fa[4], fb[4];
          codes_of<kCentred>(ka[w], fa);
          codes_of<kCentred>(kb[w], fb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float (&c)[4] = acc[nt][w >> 1];
            if (kCentred) {
              float part[4];
              mma16816_first(part, fa[0], fb[0], fa[1], fb[1], qf[nt][NS - 1][2 * w][0], qf[nt][NS - 1][2 * w][1]);
              mma16816(part, fa[2], fb[2], fa[3], fb[3], qf[nt][NS - 1][2 * w + 1][0], qf[nt][NS - 1][2 * w + 1][1]);
              mma16816(part, fa[0], fb[0], fa[1], fb[1], qf[nt][0][2 * w][0], qf[nt][0][2 * w][1]);
              mma16816(part, fa[2], fb[2], fa[3], fb[3], qf[nt][0][2 * w + 1][0], qf[nt][0][2 * w + 1][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) c[e] = (w & 1) == 0 ? part[e] : c[e] + part[e];
            } else {
              if ((w & 1) == 0)
                mma16816_first(c, fa[0], fb[0], fa[1], fb[1], qf[nt][0][2 * w][0], qf[nt][0][2 * w][1]);
              else
                mma16816(c, fa[0], fb[0], fa[1], fb[1], qf[nt][0][2 * w][0], qf[nt][0][2 * w][1]);
              mma16816(c, fa[2], fb[2], fa[3], fb[3], qf[nt][0][2 * w + 1][0], qf[nt][0][2 * w + 1][1]);
            }
          }
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t sms[NG];
          scales_of(blk + B::kKs, kt * 16 + hh * 8 + gid, sms);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const uint32_t sm = sms[gg];
            const float sc = q4_scale(sm), mid = kCentred ? fmaf(sc, 8.f, q4_min(sm)) : q4_min(sm);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float sum = gg == 0 ? mid * qsum[nt][0][e] : fmaf(mid, qsum[nt][gg][e], t[nt][kt][hh * 2 + e]);
                t[nt][kt][hh * 2 + e] = fmaf(sc, kCentred ? acc[nt][gg][hh * 2 + e] * kUnit : acc[nt][gg][hh * 2 + e], sum);
              }
          }
        }
      }
      // ---- V scales of this lane's tokens (t0 + 16 kt + 8 hh + gid)
      float sv[2][2][NG], mv[2][2][NG];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t sms[NG];
          scales_of(blk + B::kVs, kt * 16 + hh * 8 + gid, sms);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            const uint32_t sm = sms[gg];
            sv[kt][hh][gg] = q4_scale(sm);
            mv[kt][hh][gg] = fmaf(sv[kt][hh][gg], 8.f, q4_min(sm));
          }
        }
      // ---- masks: hidden tokens get a logit of -inf and a V scale of 0 (and the rows of
      // large queries their 2^18, here rather than in a branch of its own: 1 us of 53)
      if (!plain) {
        if (any_huge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (huge_rows >> (2 * nt + (c & 1)) & 1) t[nt][c >> 2][c & 3] *= 1.f / kUnit;
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int tok = t0 + kt * 16 + hh * 8 + gid;
            if (tok < vis.L && (tok >= from || tok < a.n_sink)) continue;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) sv[kt][hh][gg] = mv[kt][hh][gg] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) t[nt][kt][hh * 2] = t[nt][kt][hh * 2 + 1] = -INFINITY;
          }
      }
      // ---- lazy row maximum and V reference
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            raise |= t[nt][c >> 1][(c & 1) * 2 + e] > above[nt][e];
          }
        }
#pragma unroll
      for (int gg = 0; gg < NG; ++gg)
        raise |= fmaxf(fmaxf(sv[0][0][gg], sv[0][1][gg]), fmaxf(sv[1][0][gg], sv[1][1][gg])) > vR[gg];
      if (__any_sync(0xffffffffu, raise)) {
        float fo[NT][2], fv[NG];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(t[nt][0][e], t[nt][0][2 + e]), fmaxf(t[nt][1][e], t[nt][1][2 + e]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float nm = fmaxf(m[nt][e], tc::reference_of(top * rs[nt][e]));
            fo[nt][e] = nm == m[nt][e] ? 1.f : tc::ex2_approx(m[nt][e] - nm);
            m[nt][e] = nm;
            mr[nt][e] = nm == -INFINITY ? 0.f : nm;
            above[nt][e] = (fmaf(fabsf(nm), -0x1p-21f, nm) + kRaise) / rs[nt][e];
            l[nt][e] *= fo[nt][e];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) corr[nt][gg][e] *= fo[nt][e];
          }
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          float top = fmaxf(fmaxf(sv[0][0][gg], sv[0][1][gg]), fmaxf(sv[1][0][gg], sv[1][1][gg]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          const float up = __uint_as_float((__float_as_uint(top) + 0x7fffffu) & 0x7f800000u);  // next power of two
          const float nr = fmaxf(vR[gg], up);
          fv[gg] = vR[gg] / nr;
          vR[gg] = nr;
          vs[gg] = kPScale / nr;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][mt][e] *= fo[nt][e & 1] * fv[mt / 4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gg = 0; gg < NC; ++gg)
#pragma unroll
            for (int e = 0; e < 4; ++e) o8[nt][gg][e] *= fo[nt][e & 1] * fv[gg];
      }
      // ---- P, its sums, and P s as fp16 fragments
      uint32_t pf[NT][NS][NG][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float p0 = tc::ex2_approx(fmaf(t[nt][kt][hh * 2], rs[nt][0], -mr[nt][0]));
            const float p1 = tc::ex2_approx(fmaf(t[nt][kt][hh * 2 + 1], rs[nt][1], -mr[nt][1]));
            l[nt][0] += p0;
            l[nt][1] += p1;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
              // tokens of fields 0 and 3 (kt == hh): 16 times less
              const float s0 = sv[kt][hh][gg] * (!kCentred && kt == hh ? vs[gg] * (kCodeFar / kCodeNear) : vs[gg]);
              const float x0 = p0 * s0, x1 = p1 * s0;
              corr[nt][gg][0] = fmaf(p0, mv[kt][hh][gg], corr[nt][gg][0]);
              corr[nt][gg][1] = fmaf(p1, mv[kt][hh][gg], corr[nt][gg][1]);
              const __half2 hi = __floats2half2_rn(x0, x1);
              pf[nt][0][gg][kt][hh] = transpose8x8(half2_bits(hi));
              if (NS == 2) {
                const float2 h = __half22float2(hi);
                pf[nt][NS - 1][gg][kt][hh] = transpose8x8(half2_bits(__floats2half2_rn(x0 - h.x, x1 - h.y)));
              }
            }
          }
      }
      // ---- the weights' own sums, then O^T += V^T P^T, 32 channels at a time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gg = 0; gg < NC; ++gg) {
          constexpr uint32_t near8 = 0x02000200u, far8 = 0x00200020u;  // code 8
          mma16816(o8[nt][gg], near8, near8, far8, far8, pf[nt][0][gg][0][0], pf[nt][0][gg][0][1]);
          mma16816(o8[nt][gg], far8, far8, near8, near8, pf[nt][0][gg][1][0], pf[nt][0][gg][1][1]);
        }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(blk + B::kV + c * 512 + lane * 16);
        const int gg = c / 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t x0 = half ? w.z : w.x, x1 = half ? w.w : w.y;
          uint32_t fa[4], fb[4];
          codes_of<kCentred>(x0, fa);
          codes_of<kCentred>(x1, fb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (kCentred) {
              float acc[4];
              mma16816_first(acc, fa[0], fb[0], fa[1], fb[1], pf[nt][NS - 1][gg][0][0], pf[nt][NS - 1][gg][0][1]);
              mma16816(acc, fa[2], fb[2], fa[3], fb[3], pf[nt][NS - 1][gg][1][0], pf[nt][NS - 1][gg][1][1]);
              mma16816(acc, fa[0], fb[0], fa[1], fb[1], pf[nt][0][gg][0][0], pf[nt][0][gg][0][1]);
              mma16816(acc, fa[2], fb[2], fa[3], fb[3], pf[nt][0][gg][1][0], pf[nt][0][gg][1][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][2 * c + half][e] += acc[e];
            } else {
              mma16816(o[nt][2 * c + half], fa[0], fb[0], fa[1], fb[1], pf[nt][0][gg][0][0], pf[nt][0][gg][0][1]);
              mma16816(o[nt][2 * c + half], fa[2], fb[2], fa[3], fb[3], pf[nt][0][gg][1][0], pf[nt][0][gg][1][1]);
            }
          }
        }
      }
      __syncwarp();
      if (v + kStages * kWarps < v1) {
        if (lane == 0) issue(v + kStages * kWarps, done + kStages);
        ++issued;
      }
    }
    if (!ok) {  // a copy did not arrive in time: wait for what is in flight before the ring is reused
      if (lane == 0)
        for (int n = max(done, issued - kStages); n < issued; ++n) tc::drain_wait(bars + 8u * (n % kStages), (n / kStages) & 1, &g_err);
      __syncwarp();
    }
    done = issued;

    // ---- the warps' results into shared memory (over the drained ring)
    __syncthreads();
    float* wo = reinterpret_cast<float*>(smem);                        // [kWarps][kRows][kStride]
    float* wml = wo + kWarps * kRows * kStride;                        // [kWarps][kRows][2]
    float* row_ml = wml + kWarps * kRows * 2;                          // [kRows][2]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) corr[nt][gg][e] += __shfl_xor_sync(0xffffffffu, corr[nt][gg][e], off);
        }
        if (gid == 0) {
          float* ml = wml + ((warp * kRows) + nt * 8 + 2 * tig + e) * 2;
          ml[0] = m[nt][e];
          ml[1] = l[nt][e];
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          wo[(warp * kRows + nt * 8 + 2 * tig + (e & 1)) * kStride + mt * 16 + (e >> 1) * 8 + gid] =
              fmaf((kCentred ? o[nt][mt][e] : o[nt][mt][e] - o8[nt][kCentred ? 0 : mt / 4][e]) * (1.f / (kPScale * (kCentred ? 1.f : kCodeFar))), vR[mt / 4], corr[nt][mt / 4][e & 1]);
    }
    __syncthreads();
    const long long part = (long long)blockIdx.y * (p.W + a.S * a.Hkv) + blockIdx.x + s * a.Hkv + g;
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kWarps * 32) {
      const int r = e / (D / 4), c = e % (D / 4);
      if (row0 + r >= R) break;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wml[(w * kRows + r) * 2]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = tc::ex2_approx(wml[(w * kRows + r) * 2] - ref);
        ls += f * wml[(w * kRows + r) * 2 + 1];
        const float4 x4 = *reinterpret_cast<const float4*>(wo + (w * kRows + r) * kStride + c * 4);
        acc.x += f * x4.x;
        acc.y += f * x4.y;
        acc.z += f * x4.z;
        acc.w += f * x4.w;
      }
      // alone: over the first warp's row, which no other thread reads here
      *reinterpret_cast<float4*>(kAlone ? wo + r * kStride + c * 4 : p.part_o + (part * kRows + r) * D + c * 4) = acc;
      if (c == 0) *reinterpret_cast<float2*>(kAlone ? row_ml + r * 2 : p.part_ml + (part * kRows + r) * 2) = make_float2(mx, ls);
    }
    if (kAlone) {  // a warp per row: its sum, then its own tokens
      __syncthreads();
      constexpr int E = D / 32;
      for (int r = warp; r < min(kRows, R - row0); r += kWarps) {
        const int i = (row0 + r) / G, h = g * G + (row0 + r) % G;
        RowSum<E> sum;
        sum.m = row_ml[r * 2];
        sum.l = row_ml[r * 2 + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) sum.acc[e] = wo[r * kStride + lane * E + e];
        join_own<T, D>(a, vis.L, s, h, g, i, i_last, 0, 1, sum);
        T* out = static_cast<T*>(a.out) + (((long long)s * a.n + i) * a.Hq + h) * D + lane * E;
        bool large = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          large |= !(fabsf(sum.acc[e]) < INFINITY);
          out[e] = from_f<T>(sum.acc[e] / sum.l);
        }
        const unsigned again = __ballot_sync(0xffffffffu, large && sum.l == sum.l);
        if (lane == 0 && a.lse) a.lse[((long long)s * a.Hq + h) * a.n + i] = (sum.m + log2f(sum.l)) * kLn2;
        uint32_t groups = NG == 1 ? (again ? 1u : 0u) : (again & 0xffffu ? 1u : 0u) | (again >> 16 ? 2u : 0u);
        if (fabsf(sum.m) >= kHuge) groups = kAllGroups;
        if (groups) row_again<T, D, 1>(a, vis.L, s, h, g, i, groups, nullptr, nullptr);
      }
      return;
    }
    // the next segment's copies come over what was written here
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    x += v1 - v0;
  }
}

// One block per (stream, query head, text token): the workers' partials of its
// KV head and the row's own tokens (join_own), dealt to eight warps, each with its
// own running maximum; then the eight are joined in order.
constexpr int kMergeWarps = 8;
template <typename T, int D, bool kRaggedLengths>
__global__ void __launch_bounds__(kMergeWarps * 32) q4_merge_kernel(const __grid_constant__ Q4AttnArgs p) {
  constexpr int E = D / 32;  // channels per lane
  __shared__ float s_acc[kMergeWarps][D];
  __shared__ float s_ml[kMergeWarps][2];
  const WindowArgs& a = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const long long rw = blockIdx.x;
  const int i = (int)(rw % a.n), h = (int)(rw / a.n % a.Hq), s = (int)(rw / a.n / a.Hq);
  const int g = h / G, row = i * G + h % G;
  RowSum<E> sum;
  // the row's own tokens (inputs of the call: read before the wait)
  const Visible vis = visible_of(a, s);
  join_own<T, D>(a, vis.L, s, h, g, i, tile_last(row / p.rows, p.rows, G * a.n, G), warp, kMergeWarps, sum);
  // where the partials are
  int w0 = 0, w1 = -1, r = 0;
  long long part0 = 0;
  const int sg = s * a.Hkv + g;
  if (p.rows == 128) {  // the tensor-core kernel: W partials per (stream, KV head, row tile)
    part0 = ((long long)sg * p.n_rb + row / 128) * p.W;
    r = row % 128;
    w1 = p.W - 1;
  } else if (vis.count() > 0) {
    const Deal deal = deal_of<kRaggedLengths>(a, p.W);
    const int base = blocks_before<kRaggedLengths>(a, s) * a.Hkv + g * vis.count();
    w0 = deal.owner(base);
    w1 = deal.owner(base + vis.count() - 1);
    part0 = (long long)(row / p.rows) * (p.W + a.S * a.Hkv) + sg;
    r = row % p.rows;
  }
  pdl_wait();
  {
    constexpr int kBatch = 8;
    for (int w = w0 + warp; w <= w1; w += kMergeWarps * kBatch) {
      float2 ml[kBatch];
      float v[kBatch][E];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int u = w + b * kMergeWarps;
        if (u <= w1) {
          const long long at = (part0 + u) * p.rows + r;
          ml[b] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
          const float* src = p.part_o + at * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) v[b][e] = src[e];
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (w + b * kMergeWarps <= w1) sum.join(ml[b].x, ml[b].y, v[b]);
    }
  }
  if (lane == 0) {
    s_ml[warp][0] = sum.m;
    s_ml[warp][1] = sum.l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = sum.acc[e];
  __syncthreads();
  float mx = -INFINITY;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, s_ml[w][0]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  bool large = false;
  for (int d = threadIdx.x; d < D; d += kMergeWarps * 32) {
    float o = 0.f, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      const float f = tc::ex2_approx(s_ml[w][0] - ref);
      ls += f * s_ml[w][1];
      o += f * s_acc[w][d];
    }
    static_cast<T*>(a.out)[(((long long)s * a.n + i) * a.Hq + h) * D + d] = from_f<T>(o / ls);
    if (d == 0 && a.lse) a.lse[((long long)s * a.Hq + h) * a.n + i] = (mx + log2f(ls)) * kLn2;
    large = !(fabsf(o) < INFINITY) && ls == ls;
  }
  if (__syncthreads_or(large || fabsf(mx) >= kHuge)) {
    const int first = __syncthreads_or(large && warp < 2), second = __syncthreads_or(large && warp >= 2);
    row_again<T, D, kMergeWarps>(a, vis.L, s, h, g, i, fabsf(mx) >= kHuge ? kAllGroups : (first ? 1u : 0u) | (second ? 2u : 0u),
                                 s_acc, s_ml);
  }
}

template <typename T, int D>
cudaError_t launch_merge(const Q4AttnArgs& p, cudaStream_t st) {
  const long long rows = (long long)p.w.S * p.w.Hq * p.w.n;
  return launch_kernel(p.w.lengths ? q4_merge_kernel<T, D, true> : q4_merge_kernel<T, D, false>, dim3((unsigned)rows),
                       dim3(kMergeWarps * 32), 0, st, true, p);
}

template <typename T, int D, int NT, int NS, Share kShare>
cudaError_t launch_as(const Q4AttnArgs& p, unsigned workers, cudaStream_t st) {
  using B = Q4Block<D>;
  constexpr int kWarps = warps_of<NT, NS>();
  constexpr int ring = kWarps * kStages * B::kBytes;
  constexpr int merge = (kWarps * (D + 4 + 2) + 2) * 8 * NT * 4;
  constexpr int smem = ring > merge ? ring : merge;
  const cudaError_t e = ensure_dynamic_smem(q4_attn_kernel<T, D, NT, NS, kShare>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(q4_attn_kernel<T, D, NT, NS, kShare>, dim3(workers, p.n_rb), dim3(kWarps * 32), smem, st, false, p);
}
template <typename T, int D, int NT, int NS>
cudaError_t launch(const Q4AttnArgs& p, cudaStream_t st) {
  if (p.W == 0) return launch_as<T, D, NT, NS, kOwn>(p, p.w.S * p.w.Hkv, st);
  const cudaError_t e = p.w.lengths ? launch_as<T, D, NT, NS, kRagged>(p, p.W, st) : launch_as<T, D, NT, NS, kEven>(p, p.W, st);
  return e != cudaSuccess ? e : launch_merge<T, D>(p, st);
}

// Blocks that can be visible in a stream, by what the host knows.
long long most_blocks(const WindowArgs& a) {
  const long long len = a.lengths ? a.capacity : a.length, all = (len + 31) / 32;
  if (!a.window) return all;
  return std::min(all, (std::min<long long>(a.n_sink, len) + 31) / 32 + (a.window + 31ll) / 32 + 1);
}

}  // namespace

Q4Plan q4_plan(int S, int Hq, int Hkv, int n, int dtype, int d, int n_sm) {
  Q4Plan pl{};
  const long long R = (long long)(Hq / Hkv) * n;
  // Measured in bf16 over 131072 tokens (4 KV heads, d = 128) and 32768 (2, d = 64),
  // us: 12 rows as 8-row tiles 36.6, 10.3, as one of 16 rows 33.0, 11.2; 32 rows as
  // 16-row tiles 53.2, 12.4, as one of 128 rows on tcgen05 52.0, 16.4 (whatever the
  // rows, up to 128); more 16-row tiles each add some 20 us to the former.  float32
  // takes two parts of everything, which fit the registers for eight rows only.
  pl.rows = dtype == kDtypeF32 || R <= 8 ? 8 : R <= 32 ? 16 : 128;
  pl.n_rb = (int)((R + pl.rows - 1) / pl.rows);
  const long long sg = (long long)S * Hkv;
  size_t parts;
  if (pl.rows == 128) {
    pl.W = (int)std::max(1ll, n_sm / (sg * pl.n_rb));
    parts = (size_t)sg * pl.n_rb * pl.W * 128;
  } else {
    pl.W = std::max(1, n_sm / pl.n_rb);
    parts = (size_t)pl.n_rb * (pl.W + sg) * pl.rows;
  }
  pl.o_bytes = parts * d * 4;
  pl.bytes = pl.o_bytes + parts * 8;
  return pl;
}

// One thread block per (stream, KV head, row tile) that takes all of its blocks,
// joins the text tokens and writes the results (no partials, no second launch), or
// the blocks dealt evenly to W workers and merged?  In units of what a block costs a
// worker (some 0.11 us), with b blocks each for P pairs: ceil(P / W) rounds of 49 + b
// against 68 once and 60 + b a pair, over W (lengths known to the device alone: P / W
// + 1/4 rounds).  Measured (d = 128, G = 7, us, own
// against dealt): 4 pairs of 1, 10, 32 blocks 5.7 : 6.8, 6.6 : 7.2, 8.8 : 7.9; 152
// pairs of 64, 256 24 : 24, 69 : 52; 256 pairs 25 : 36, 72 : 78; 300 pairs 36 : 42,
// 102 : 91; 400 pairs 43 : 57, 106 : 116; 1024 pairs of up to 32, ragged, 55 : 122.
bool q4_alone(const WindowArgs& a, const Q4Plan& pl) {
  if (pl.rows == 128 || a.n > kOwnText) return false;
  const long long b = most_blocks(a), pairs = (long long)a.S * a.Hkv, W = pl.W;
  // rounds x 4 W; of different lengths they overlap
  const long long rounds = a.lengths ? std::max(4 * W, 4 * pairs + W) : (pairs + W - 1) / W * 4 * W;
  return rounds * (49 + b) <= 4 * (68 * W + (60 + b) * pairs);
}

cudaError_t launch_q4_attn(const WindowArgs& a, const Q4Plan& pl, void* workspace, int dtype, int d, cudaStream_t st) {
  Q4AttnArgs p{};
  p.w = a;
  p.W = pl.W;
  p.rows = pl.rows;
  p.n_rb = pl.n_rb;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.o_bytes);
  if (q4_alone(a, pl)) p.W = 0;
  if (dtype == kDtypeF32) return d == 128 ? launch<float, 128, 1, 2>(p, st) : launch<float, 64, 1, 2>(p, st);
  if (pl.rows == 8) return d == 128 ? launch<__nv_bfloat16, 128, 1, 1>(p, st) : launch<__nv_bfloat16, 64, 1, 1>(p, st);
  if (pl.rows == 16) return d == 128 ? launch<__nv_bfloat16, 128, 2, 1>(p, st) : launch<__nv_bfloat16, 64, 2, 1>(p, st);
  // no more splits than 128-token tiles can be visible
  p.W = (int)std::max(1ll, std::min((long long)p.W, (most_blocks(a) + 3) / 4));
  const cudaError_t e = launch_q4_attn_tc(p, d, st);
  if (e != cudaSuccess) return e;
  return d == 128 ? launch_merge<__nv_bfloat16, 128>(p, st) : launch_merge<__nv_bfloat16, 64>(p, st);
}

cudaError_t q4_attn_status(int* code) {
  cudaError_t e = cudaDeviceSynchronize();
  const int zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
  return e;
}

}  // namespace skv
