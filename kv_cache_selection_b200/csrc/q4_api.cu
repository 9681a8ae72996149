// Host side of the calls over a caller-owned 4-bit cache (statekv_q4_*) and of
// sink_window_prefill: argument checks and launches (include/statekv.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "statekv.h"
#include "kernels.h"
#include "q4_cache.cuh"

namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  skv::set_free_error(buf);
  return code;
}

// Shapes shared by every call over a 4-bit cache.
int check_cache_shape(int S, int Hkv, int d, int capacity) {
  if (S < 1 || Hkv < 1 || capacity < 1)
    return fail(STATEKV_ERR_INVALID_ARG, "bad shape: n_streams=%d Hkv=%d capacity=%d", S, Hkv, capacity);
  if (d != 64 && d != 128) return fail(STATEKV_ERR_UNSUPPORTED, "head dim %d not in {64,128}", d);
  if (capacity > (1 << 30)) return fail(STATEKV_ERR_UNSUPPORTED, "capacity %d above 2^30 tokens", capacity);
  const long long blocks = (long long)S * Hkv * ((capacity + 31ll) / 32);
  if (S > 65535 || Hkv > 65535 || blocks > 0x7fffffffll)
    return fail(STATEKV_ERR_UNSUPPORTED, "n_streams=%d x Hkv=%d x capacity=%d is too large", S, Hkv, capacity);
  return STATEKV_OK;
}

int check_dtype(int dtype) {
  if (dtype != STATEKV_BF16 && dtype != STATEKV_F32) return fail(STATEKV_ERR_INVALID_ARG, "bad dtype %d", dtype);
  return STATEKV_OK;
}

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

struct Range {
  const void* p;
  size_t n;
  const char* name;
};
bool overlap(const Range& x, const Range& y) {
  const uintptr_t a0 = (uintptr_t)x.p, b0 = (uintptr_t)y.p;
  return x.p && y.p && x.n > 0 && y.n > 0 && a0 < b0 + y.n && b0 < a0 + x.n;
}
template <int NO, int NI>
int check_disjoint(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (const Range& i : ins)
      if (overlap(outs[o], i)) return fail(STATEKV_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, i.name);
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return fail(STATEKV_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, outs[p].name);
  }
  return STATEKV_OK;
}

size_t cache_bytes(int S, int Hkv, int d, int capacity) {
  return (size_t)S * Hkv * (((size_t)capacity + 31) / 32) * skv::q4_block_bytes(d);
}

int sm_count() {
  static int cached[64];  // a device's SM count does not change
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return n;
  }
  if (cached[dev]) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) cached[dev] = n;
  return n;
}

// Shapes of a decode over a cache.
int check_decode_shape(int S, int Hq, int Hkv, int d, int capacity, int n_text, int dtype) {
  int rc;
  if ((rc = check_cache_shape(S, Hkv, d, capacity)) || (rc = check_dtype(dtype))) return rc;
  if (Hq < 1 || Hq % Hkv) return fail(STATEKV_ERR_INVALID_ARG, "Hq (%d) %% Hkv (%d) != 0", Hq, Hkv);
  if (n_text < 1) return fail(STATEKV_ERR_INVALID_ARG, "n_text=%d must be >= 1", n_text);
  if (Hq > 65535 || n_text > 65535 || (long long)(Hq / Hkv) * n_text > 65535 * 8ll ||
      (long long)S * Hq * n_text > 0x7fffffffll)
    return fail(STATEKV_ERR_UNSUPPORTED, "n_streams=%d x Hq=%d x n_text=%d is too large", S, Hq, n_text);
  return STATEKV_OK;
}

// A range of n tokens from `start` (host value, or per stream from the device).
int check_range(int start, const int32_t* starts, int n, int capacity) {
  if (n < 0) return fail(STATEKV_ERR_INVALID_ARG, "negative token count %d", n);
  if (starts) {
    if (misaligned(starts, 4)) return fail(STATEKV_ERR_INVALID_ARG, "starts must be 4-byte aligned");
    return STATEKV_OK;
  }
  if (start < 0) return fail(STATEKV_ERR_INVALID_ARG, "negative start %d", start);
  if ((long long)start + n > capacity)
    return fail(STATEKV_ERR_CAPACITY, "tokens [%d, %lld) do not fit a cache of %d", start, (long long)start + n, capacity);
  return STATEKV_OK;
}

}  // namespace

extern "C" {

long long statekv_q4_bytes(int n_streams, int Hkv, int d, int capacity) {
  const int rc = check_cache_shape(n_streams, Hkv, d, capacity);
  return rc ? rc : (long long)cache_bytes(n_streams, Hkv, d, capacity);
}

int statekv_q4_append(void* cache, int n_streams, int Hkv, int d, int capacity, const void* k, const void* v, int n,
                      int dtype, int start, const int32_t* starts, void* stream) {
  int rc;
  if ((rc = check_cache_shape(n_streams, Hkv, d, capacity)) || (rc = check_dtype(dtype)) ||
      (rc = check_range(start, starts, n, capacity)))
    return rc;
  if (n == 0) return STATEKV_OK;
  if (!cache || !k || !v) return fail(STATEKV_ERR_INVALID_ARG, "null cache, k or v pointer");
  if (misaligned(cache, 16) || misaligned(k, 16) || misaligned(v, 16))
    return fail(STATEKV_ERR_INVALID_ARG, "cache, k and v must be 16-byte aligned");
  const size_t kb = (size_t)n_streams * n * Hkv * d * (dtype == STATEKV_BF16 ? 2 : 4);
  const Range outs[] = {{cache, cache_bytes(n_streams, Hkv, d, capacity), "cache"}};
  const Range ins[] = {{k, kb, "k"}, {v, kb, "v"}, {starts, (size_t)n_streams * 4, "starts"}};
  if ((rc = check_disjoint(outs, ins))) return rc;
  skv::Q4IoArgs a{};
  a.cache = cache;
  a.k = k;
  a.v = v;
  a.starts = starts;
  a.start = start;
  a.n = n;
  a.S = n_streams;
  a.Hkv = Hkv;
  a.capacity = capacity;
  const cudaError_t e = skv::launch_q4_append(a, dtype, d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(STATEKV_ERR_CUDA, "q4 append launch failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

int statekv_q4_read(const void* cache, int n_streams, int Hkv, int d, int capacity, int start, const int32_t* starts,
                    int n, int dtype, void* k, void* v, void* stream) {
  int rc;
  if ((rc = check_cache_shape(n_streams, Hkv, d, capacity)) || (rc = check_dtype(dtype)) ||
      (rc = check_range(start, starts, n, capacity)))
    return rc;
  if (n == 0) return STATEKV_OK;
  if (!cache || !k || !v) return fail(STATEKV_ERR_INVALID_ARG, "null cache, k or v pointer");
  if (misaligned(cache, 16) || misaligned(k, 16) || misaligned(v, 16))
    return fail(STATEKV_ERR_INVALID_ARG, "cache, k and v must be 16-byte aligned");
  const size_t kb = (size_t)n_streams * n * Hkv * d * (dtype == STATEKV_BF16 ? 2 : 4);
  const Range outs[] = {{k, kb, "k"}, {v, kb, "v"}};
  const Range ins[] = {{cache, cache_bytes(n_streams, Hkv, d, capacity), "cache"},
                       {starts, (size_t)n_streams * 4, "starts"}};
  if ((rc = check_disjoint(outs, ins))) return rc;
  skv::Q4IoArgs a{};
  a.cache = const_cast<void*>(cache);
  a.k_out = k;
  a.v_out = v;
  a.starts = starts;
  a.start = start;
  a.n = n;
  a.S = n_streams;
  a.Hkv = Hkv;
  a.capacity = capacity;
  const cudaError_t e = skv::launch_q4_read(a, dtype, d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(STATEKV_ERR_CUDA, "q4 read launch failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

long long statekv_q4_decode_workspace(int n_streams, int Hq, int Hkv, int d, int n_text, int dtype) {
  const int rc = check_decode_shape(n_streams, Hq, Hkv, d, 1, n_text, dtype);
  return rc ? rc : (long long)skv::q4_plan(n_streams, Hq, Hkv, n_text, dtype, d, sm_count()).bytes;
}

int statekv_q4_decode(const void* cache, int n_streams, int Hq, int Hkv, int d, int capacity, const void* q,
                      const void* k, const void* v, int n_text, int dtype, int length, const int32_t* lengths,
                      int window, int n_sink, void* out, float* lse, void* workspace, long long workspace_bytes,
                      void* stream) {
  int rc;
  if ((rc = check_decode_shape(n_streams, Hq, Hkv, d, capacity, n_text, dtype))) return rc;
  if (window < 0 || n_sink < 0)
    return fail(STATEKV_ERR_INVALID_ARG, "window=%d and n_sink=%d must not be negative", window, n_sink);
  if (!lengths && (length < 0 || length > capacity))
    return fail(STATEKV_ERR_INVALID_ARG, "length=%d outside [0, capacity=%d]", length, capacity);
  if (!cache || !q || !k || !v || !out || !workspace)
    return fail(STATEKV_ERR_INVALID_ARG, "null input, output or workspace pointer");
  if (misaligned(workspace, 16)) return fail(STATEKV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const skv::Q4Plan pl = skv::q4_plan(n_streams, Hq, Hkv, n_text, dtype, d, sm_count());
  if (workspace_bytes < (long long)pl.bytes)
    return fail(STATEKV_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", workspace_bytes, pl.bytes);
  if (misaligned(cache, 16) || misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16))
    return fail(STATEKV_ERR_INVALID_ARG, "cache/q/k/v/out must be 16-byte aligned");
  if (misaligned(lse, 4) || misaligned(lengths, 4))
    return fail(STATEKV_ERR_INVALID_ARG, "lse and lengths must be 4-byte aligned");
  const size_t es = dtype == STATEKV_BF16 ? 2 : 4;
  const size_t qb = (size_t)n_streams * n_text * Hq * d * es, kb = (size_t)n_streams * n_text * Hkv * d * es;
  const Range outs[] = {{out, qb, "out"}, {lse, (size_t)n_streams * Hq * n_text * 4, "lse"},
                        {workspace, pl.bytes, "workspace"}};
  const Range ins[] = {{cache, cache_bytes(n_streams, Hkv, d, capacity), "cache"}, {q, qb, "q"}, {k, kb, "k"},
                       {v, kb, "v"}, {lengths, (size_t)n_streams * 4, "lengths"}};
  if ((rc = check_disjoint(outs, ins))) return rc;
  skv::WindowArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.cache = cache;
  a.lengths = lengths;
  a.length = length;
  a.capacity = capacity;
  a.cap_blk = (capacity + 31) / 32;
  a.n = n_text;
  a.S = n_streams;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.window = window;
  a.n_sink = n_sink;
  a.scale_log2 = skv::kLog2e / sqrtf((float)d);
  const cudaError_t e = skv::launch_q4_attn(a, pl, workspace, dtype, d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(STATEKV_ERR_CUDA, "q4 decode launch failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

int sink_window_prefill_batched(const void* q, const void* k, const void* v, int n_seq, int n_tokens, int Hq, int Hkv,
                                int d, int dtype, int window, int n_sink, void* out, float* lse, void* stream) {
  int rc;
  if (n_seq < 1 || n_tokens < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv)
    return fail(STATEKV_ERR_INVALID_ARG, "bad shape: n_seq=%d n_tokens=%d Hq=%d Hkv=%d", n_seq, n_tokens, Hq, Hkv);
  if ((rc = check_dtype(dtype))) return rc;
  if (d != 64 && d != 128) return fail(STATEKV_ERR_UNSUPPORTED, "head dim %d not in {64,128}", d);
  if (window < 1) return fail(STATEKV_ERR_INVALID_ARG, "window=%d must be >= 1", window);
  if (n_sink < 0) return fail(STATEKV_ERR_INVALID_ARG, "n_sink=%d must not be negative", n_sink);
  if (n_seq > 65535 || Hq > 65535 || n_tokens > (1 << 24))
    return fail(STATEKV_ERR_UNSUPPORTED, "n_seq=%d, Hq=%d or n_tokens=%d too large", n_seq, Hq, n_tokens);
  if ((long long)n_seq * Hq * ((n_tokens + 63ll) / 64) > 0x7fffffffll)
    return fail(STATEKV_ERR_UNSUPPORTED, "n_seq=%d x Hq=%d x n_tokens=%d is too large", n_seq, Hq, n_tokens);
  if (n_tokens == 0) return STATEKV_OK;
  if (!q || !k || !v || !out) return fail(STATEKV_ERR_INVALID_ARG, "null pointer");
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16))
    return fail(STATEKV_ERR_INVALID_ARG, "q/k/v/out must be 16-byte aligned");
  if (misaligned(lse, 4)) return fail(STATEKV_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const size_t es = dtype == STATEKV_BF16 ? 2 : 4;
  const size_t qb = (size_t)n_seq * n_tokens * Hq * d * es, kb = (size_t)n_seq * n_tokens * Hkv * d * es;
  const Range outs[] = {{out, qb, "out"}, {lse, (size_t)n_seq * Hq * n_tokens * 4, "lse"}};
  const Range ins[] = {{q, qb, "q"}, {k, kb, "k"}, {v, kb, "v"}};
  if ((rc = check_disjoint(outs, ins))) return rc;
  skv::WindowArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.n = n_tokens;
  a.S = n_seq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  // more than all tokens is all tokens (the kernels round both up to tiles)
  a.window = std::min(window, n_tokens);
  a.n_sink = std::min(n_sink, n_tokens);
  a.scale_log2 = skv::kLog2e / sqrtf((float)d);
  const cudaError_t e = dtype == STATEKV_BF16 ? skv::launch_window_tc(a, d, static_cast<cudaStream_t>(stream))
                                              : skv::launch_window_f32(a, d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(STATEKV_ERR_CUDA, "sink_window_prefill launch failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

int sink_window_prefill(const void* q, const void* k, const void* v, int n_tokens, int Hq, int Hkv, int d, int dtype,
                        int window, int n_sink, void* out, float* lse, void* stream) {
  return sink_window_prefill_batched(q, k, v, 1, n_tokens, Hq, Hkv, d, dtype, window, n_sink, out, lse, stream);
}

int statekv_q4_status(int* code) {
  if (!code) return fail(STATEKV_ERR_INVALID_ARG, "null argument");
  int tc = 0;
  cudaError_t e = skv::q4_attn_status(code);
  if (e == cudaSuccess) e = skv::q4_attn_tc_status(&tc);
  if (*code == 0) *code = tc;
  if (e != cudaSuccess) return fail(STATEKV_ERR_CUDA, "status read failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

int sink_window_status(int* code) {
  if (!code) return fail(STATEKV_ERR_INVALID_ARG, "null argument");
  const cudaError_t e = skv::window_tc_status(code);
  if (e != cudaSuccess) return fail(STATEKV_ERR_CUDA, "status read failed: %s", cudaGetErrorString(e));
  return STATEKV_OK;
}

}  // extern "C"
