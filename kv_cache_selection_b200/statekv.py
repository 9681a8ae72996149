"""Python binding of libstatekv (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module checks
tensor shapes, dtypes and devices, passes raw device pointers and the current
CUDA stream through the C ABI (include/statekv.h) and wraps borrowed device
buffers as torch tensors without copying.  There is no fallback: if the
library is missing, importing this module raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("STATEKV_LIB", os.path.join(_PKG, "lib", "libstatekv.so"))

BF16, F32 = 0, 1
MASKS = {"frame_causal": 0, "frame_bidir": 1}
SELECTS = {"global": 0, "per_kv_head": 1, "recency": 2}
DETAILED = {"native": 0, "q4": 1}
N_STAGES = 8
STAGES = ["attention", "attention_combine", "score", "select", "gather", "decode", "decode_combine",
          "attention_chained"]
ERRORS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED", -3: "CAPACITY", -4: "OOM", -5: "CUDA"}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libstatekv.so not found at {LIB_PATH}; build it with "
        "`python -m kv_cache_selection_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i = ctypes.c_int
_pp = ctypes.POINTER(ctypes.c_void_p)
_ip = ctypes.POINTER(ctypes.c_int)

_SIGS = {
    "statekv_create": (_i, [_pp, _i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "statekv_create_batched": (_i, [_pp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "statekv_reserve_layers": (_i, [_vp, _i]),
    "statekv_prefill_frame": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "statekv_prefill_frame_host": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "statekv_get_compressed": (_i, [_vp, _i, _pp, _pp, _pp, _pp, _ip]),
    "statekv_get_detailed": (_i, [_vp, _i, _pp, _pp, _pp, _ip]),
    "statekv_set_detailed_format": (_i, [_vp, _i]),
    "statekv_get_detailed_q4": (_i, [_vp, _i, _pp, _ip, _pp, _ip]),
    "statekv_get_step_stats": (_i, [_vp, _pp, _pp, _ip]),
    "statekv_frames": (_i, [_vp, _i]),
    "statekv_profile_enable": (_i, [_vp, _i]),
    "statekv_profile_read": (_i, [_vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong)]),
    "statekv_kernel_launches": (ctypes.c_longlong, [_vp]),
    "statekv_device_status": (_i, [_vp, _ip]),
    "statekv_set_wait_limit": (_i, [_vp, ctypes.c_longlong]),
    "statekv_destroy": (_i, [_vp]),
    "statekv_last_error": (ctypes.c_char_p, [_vp]),
    "statekv_step_noalloc": (_i, [_i] * 8 + [_vp] * 7 + [_i] + [_vp] * 8 + [_i, _i, _vp]),
    "statekv_decode": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]),
    "full_causal_prefill": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "full_causal_prefill_batched": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "statekv_q4_bytes": (ctypes.c_longlong, [_i, _i, _i, _i]),
    "statekv_q4_append": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "statekv_q4_read": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _i, _i, _vp, _vp, _vp]),
    "statekv_q4_decode": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _vp, _vp, _vp,
                               ctypes.c_longlong, _vp]),
    "statekv_q4_decode_workspace": (ctypes.c_longlong, [_i, _i, _i, _i, _i, _i]),
    "sink_window_prefill": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "statekv_q4_status": (_i, [_ip]),
    "sink_window_status": (_i, [_ip]),
    "sink_window_prefill_batched": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class StateKVError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


def _check(rc, handle=None):
    if rc != 0:
        msg = lib.statekv_last_error(handle)
        raise StateKVError(rc, msg.decode() if msg else "")


_CODES = {torch.bfloat16: BF16, torch.float32: F32}


def _dtype_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is not None:
        return code
    if dtype in ("bf16", torch.bfloat16, BF16):
        return BF16
    if dtype in ("f32", torch.float32, F32):
        return F32
    raise ValueError(f"unsupported dtype {dtype!r}")


def _torch_dtype(code: int):
    return torch.bfloat16 if code == BF16 else torch.float32


# the current device and whether its current stream is capturing, without the
# wrappers' own checks (CUDA is up: the callers hold tensors on it)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
# the current stream's handle without building a torch.cuda.Stream object
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, device_index=None) -> int:
    if stream is None:
        if _raw_current_stream is not None and device_index is not None:
            return _raw_current_stream(device_index)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class _DevView:
    """Exposes a borrowed device buffer through __cuda_array_interface__."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {
            "shape": tuple(int(s) for s in shape), "typestr": typestr,
            "data": (int(ptr), False), "version": 3, "strides": None,
        }


def borrow(ptr: int, shape, dtype: torch.dtype) -> torch.Tensor:
    """Zero-copy torch view of library-owned device memory."""
    if dtype == torch.bfloat16:
        t = torch.as_tensor(_DevView(ptr, shape, "<i2"), device="cuda")
        return t.view(torch.bfloat16)
    typestr = {torch.float32: "<f4", torch.int32: "<i4", torch.uint8: "|u1"}[dtype]
    return torch.as_tensor(_DevView(ptr, shape, typestr), device="cuda")


def _need(t: torch.Tensor, shape, dtype, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class StateKV:
    """One StateKV cache builder (one or n_streams video streams, any layers).

    detailed="q4" holds the detailed state D in 4 bits a value (Q4Cache):
    get_detailed and decode then deal with what that keeps of the keys and values.
    """

    def __init__(self, Hq, Hkv, d, T, B, max_frames, dtype="bf16", mask="frame_causal",
                 select="global", n_streams=1, detailed="native"):
        if detailed not in DETAILED:
            raise ValueError(f"detailed must be one of {sorted(DETAILED)}, not {detailed!r}")
        self.Hq, self.Hkv, self.d, self.T, self.B = Hq, Hkv, d, T, B
        self.max_frames, self.S = max_frames, n_streams
        self.dtype_code = _dtype_code(dtype)
        self.dtype = _torch_dtype(self.dtype_code)
        self.mask, self.select, self.detailed = mask, select, detailed
        lead = () if n_streams == 1 else (n_streams,)
        self._step_shapes = (lead + (T, Hq, d), lead + (T, Hkv, d), lead + (T,))  # q/out, k/v, pos
        h = ctypes.c_void_p()
        rc = lib.statekv_create_batched(ctypes.byref(h), n_streams, Hq, Hkv, d, T, B, max_frames,
                                        self.dtype_code, MASKS[mask], SELECTS[select])
        _check(rc)
        self._h = h
        if detailed != "native":
            _check(lib.statekv_set_detailed_format(h, DETAILED[detailed]), h)

    @property
    def handle(self):
        return self._h

    def _lead(self):
        return () if self.S == 1 else (self.S,)

    def reserve_layers(self, n_layers: int):
        _check(lib.statekv_reserve_layers(self._h, n_layers), self._h)

    def prefill_frame(self, layer, q, k, v, pos, out=None, stream=None):
        """One cache-builder step; returns out [.., T, Hq, d]."""
        sq, skv, sp = self._step_shapes
        _need(q, sq, self.dtype, "q")
        _need(k, skv, self.dtype, "k")
        _need(v, skv, self.dtype, "v")
        _need(pos, sp, torch.int32, "pos")
        if out is None:
            out = torch.empty_like(q)
        _need(out, sq, self.dtype, "out")
        rc = lib.statekv_prefill_frame(self._h, layer, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       pos.data_ptr(), out.data_ptr(), _stream_ptr(stream, q.get_device()))
        _check(rc, self._h)
        return out

    def profile(self, on=True):
        """Per-stage device timing: False/0 off, True/1 one event pair per
        kernel, 2 the attention and its split merge under one event pair
        (stage "attention_chained")."""
        _check(lib.statekv_profile_enable(self._h, int(on)), self._h)

    def profile_read(self):
        """{stage: (total_ms, launches)} since the last read (synchronises)."""
        ms = (ctypes.c_double * N_STAGES)()
        cnt = (ctypes.c_longlong * N_STAGES)()
        _check(lib.statekv_profile_read(self._h, ms, cnt), self._h)
        return {name: (ms[i], cnt[i]) for i, name in enumerate(STAGES) if name}

    def device_status(self) -> int:
        """0, or the first error code a kernel recorded (synchronises)."""
        code = ctypes.c_int()
        _check(lib.statekv_device_status(self._h, ctypes.byref(code)), self._h)
        return code.value

    def set_wait_limit(self, ns: int):
        """Pipeline-wait limit of the tensor-core kernels (<= 0: the default)."""
        _check(lib.statekv_set_wait_limit(self._h, int(ns)), self._h)

    def kernel_launches(self) -> int:
        return lib.statekv_kernel_launches(self._h)

    def prefill_frame_host(self, layer, q, k, v, pos, out, stream=None):
        """Same step from host tensors (pinned for asynchronous copies); `out`
        (host) is filled once `stream` reaches the end of the call."""
        L = self._lead()
        for t, shape, dt, name in ((q, L + (self.T, self.Hq, self.d), self.dtype, "q"),
                                   (k, L + (self.T, self.Hkv, self.d), self.dtype, "k"),
                                   (v, L + (self.T, self.Hkv, self.d), self.dtype, "v"),
                                   (pos, L + (self.T,), torch.int32, "pos"),
                                   (out, L + (self.T, self.Hq, self.d), self.dtype, "out")):
            if t.device.type != "cpu" or tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous host tensor {shape} {dt}")
        rc = lib.statekv_prefill_frame_host(self._h, layer, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            pos.data_ptr(), out.data_ptr(), _stream_ptr(stream))
        _check(rc, self._h)
        return out

    def decode(self, layer, q, k, v, out=None, lse=None, with_lse=True, stream=None):
        """Attention of n text tokens over the layer's detailed state D and
        causally over themselves: q [.., n, Hq, d], k/v [.., n, Hkv, d].
        Returns (out, lse [.., Hq, n] or None)."""
        L = self._lead()
        n = q.shape[-3]
        _need(q, L + (n, self.Hq, self.d), self.dtype, "q")
        _need(k, L + (n, self.Hkv, self.d), self.dtype, "k")
        _need(v, L + (n, self.Hkv, self.d), self.dtype, "v")
        if out is None:
            out = torch.empty_like(q)
        _need(out, L + (n, self.Hq, self.d), self.dtype, "out")
        if lse is None and with_lse:
            lse = torch.empty(L + (self.Hq, n), dtype=torch.float32, device=q.device)
        if lse is not None:
            _need(lse, L + (self.Hq, n), torch.float32, "lse")
        rc = lib.statekv_decode(self._h, layer, q.data_ptr(), k.data_ptr(), v.data_ptr(), n, out.data_ptr(),
                                lse.data_ptr() if lse is not None else None, _stream_ptr(stream))
        _check(rc, self._h)
        return out, lse

    def frames(self, layer) -> int:
        return lib.statekv_frames(self._h, layer)

    def get_compressed(self, layer):
        """Borrowed views of C: k, v [S][Hkv][B][d], pos, score [S][Hkv][B], len."""
        k, v, p, s = (ctypes.c_void_p() for _ in range(4))
        n = ctypes.c_int()
        _check(lib.statekv_get_compressed(self._h, layer, ctypes.byref(k), ctypes.byref(v),
                                          ctypes.byref(p), ctypes.byref(s), ctypes.byref(n)),
               self._h)
        S, H, B, d = self.S, self.Hkv, max(self.B, 0), self.d
        return dict(
            k=borrow(k.value, (S, H, B, d), self.dtype), v=borrow(v.value, (S, H, B, d), self.dtype),
            pos=borrow(p.value, (S, H, B), torch.int32), score=borrow(s.value, (S, H, B), torch.float32),
            len=n.value)

    def get_detailed(self, layer):
        """Borrowed views of D: k, v [S][Hkv][max_frames*T][d], pos [S][max_frames*T], len;
        with detailed="q4" a Q4Cache `cache` over it instead of k and v."""
        if self.detailed == "q4":
            return self._detailed_q4(layer)
        k, v, p = (ctypes.c_void_p() for _ in range(3))
        n = ctypes.c_int()
        _check(lib.statekv_get_detailed(self._h, layer, ctypes.byref(k), ctypes.byref(v),
                                        ctypes.byref(p), ctypes.byref(n)), self._h)
        S, H, N, d = self.S, self.Hkv, self.max_frames * self.T, self.d
        return dict(k=borrow(k.value, (S, H, N, d), self.dtype), v=borrow(v.value, (S, H, N, d), self.dtype),
                    pos=borrow(p.value, (S, N), torch.int32), len=n.value)

    def _detailed_q4(self, layer):
        c, p = ctypes.c_void_p(), ctypes.c_void_p()
        cap, n = ctypes.c_int(), ctypes.c_int()
        _check(lib.statekv_get_detailed_q4(self._h, layer, ctypes.byref(c), ctypes.byref(cap), ctypes.byref(p),
                                           ctypes.byref(n)), self._h)
        data = borrow(c.value, (lib.statekv_q4_bytes(self.S, self.Hkv, self.d, cap.value),), torch.uint8)
        return dict(cache=Q4Cache(self.Hkv, self.d, cap.value, self.S, data=data),
                    pos=borrow(p.value, (self.S, cap.value), torch.int32), len=n.value)

    def step_stats(self):
        """Borrowed views of the last step's lse [S][Hq][T] and pool scores [S][Hkv][B+T]."""
        l, s = ctypes.c_void_p(), ctypes.c_void_p()
        n = ctypes.c_int()
        _check(lib.statekv_get_step_stats(self._h, ctypes.byref(l), ctypes.byref(s), ctypes.byref(n)),
               self._h)
        return dict(lse=borrow(l.value, (self.S, self.Hq, self.T), torch.float32),
                    pool_score=borrow(s.value, (self.S, self.Hkv, self.B + self.T), torch.float32),
                    pool_len=n.value)

    def close(self):
        if getattr(self, "_h", None):
            lib.statekv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def full_causal_prefill(q, k, v, out=None, lse=None, with_lse=True, stream=None):
    """Full causal attention over q [(S,) N, Hq, d], k/v [(S,) N, Hkv, d]."""
    batched = q.dim() == 4
    S = q.shape[0] if batched else 1
    N, Hq, d = q.shape[-3:]
    Hkv = k.shape[-2]
    code = _dtype_code(q.dtype)
    lead = (S,) if batched else ()
    _need(q, lead + (N, Hq, d), q.dtype, "q")
    _need(k, lead + (N, Hkv, d), q.dtype, "k")
    _need(v, lead + (N, Hkv, d), q.dtype, "v")
    if out is None:
        out = torch.empty_like(q)
    _need(out, lead + (N, Hq, d), q.dtype, "out")
    if lse is None and with_lse:
        lse = torch.empty(lead + (Hq, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, lead + (Hq, N), torch.float32, "lse")
    rc = lib.full_causal_prefill_batched(q.data_ptr(), k.data_ptr(), v.data_ptr(), S, N, Hq, Hkv, d,
                                         code, out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                         _stream_ptr(stream))
    _check(rc)
    return out, lse


def _int32(x, name):
    """x, if the library's 32-bit arguments hold it (ctypes would cut it off)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}={x} does not fit 32 bits")
    return x


def _on(dev):
    """Makes a tensor's device the current one; returns the device to go back
    to, or -1 where it already was."""
    now = _current_device()
    if now == dev:
        return -1
    torch.cuda.set_device(dev)
    return now


def _back(dev):
    if dev >= 0:
        torch.cuda.set_device(dev)


@functools.lru_cache(maxsize=None)
def _float32_on(device):
    """A float32 tensor on the device, to make others like it."""
    return torch.empty((), dtype=torch.float32, device=device)


def _empty(like, shape, stream):
    """A new tensor of like's type and device for work on `stream` (allocated
    for that stream, so that its memory is not still in use by work queued
    elsewhere)."""
    if stream is None:
        return like.new_empty(shape)
    st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream_ptr(stream), device=like.device)
    with torch.cuda.stream(st):
        return like.new_empty(shape)


class Q4Cache:
    """Keys and values of n_streams sequences in 4.5 bits a value (one layer).

    A group of 64 channels of a token's key or value keeps codes 0..15, a scale
    and a smallest value (include/statekv.h has the rounding).  The buffer is a
    torch tensor, `data` (a new one, which waits for the current stream, unless one
    is given); every call runs on `stream`, or on the current stream.  Leading [S] dimensions of q, k and v may be left out
    when n_streams is 1.
    """

    def __init__(self, Hkv, d, capacity, n_streams=1, device=None, data=None):
        for x, name in ((Hkv, "Hkv"), (d, "d"), (capacity, "capacity"), (n_streams, "n_streams")):
            _int32(x, name)
        n = lib.statekv_q4_bytes(n_streams, Hkv, d, capacity)
        if n < 0:
            _check(int(n))
        self.Hkv, self.d, self.capacity, self.S = Hkv, d, capacity, n_streams
        if data is None:
            data = torch.zeros(n, dtype=torch.uint8, device="cuda" if device is None else device)
            if data.is_cuda and not torch.cuda.is_current_stream_capturing():
                # calls may come on any stream: none may run ahead of the fill, or of
                # work that still uses the memory (a captured fill is its graph's)
                torch.cuda.current_stream(data.device).synchronize()
        else:
            _need(data, (n,), torch.uint8, "data")
        self.data = data
        self._dev = self.data.get_device()
        self._ptr = self.data.data_ptr()
        self._proto = {t: torch.empty((), dtype=t, device=self.data.device) for t in (torch.bfloat16, torch.float32)}
        # workspaces of decodes on the current stream, by stream and size: one
        # call at a time uses them (the lock), in the stream's order
        self._ws, self._ws_bytes, self._lock = {}, {}, threading.Lock()

    def _need(self, t, heads, name, dtype, n=None):
        """Checks a [(S,) n, heads, d] tensor on the cache's device; returns its n."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        shape = t.shape
        if n is None:
            n = shape[-3] if len(shape) >= 3 else 0
        if not (t.is_cuda and t.dtype is dtype and (shape == (self.S, n, heads, self.d) or (self.S == 1 and shape == (n, heads, self.d)))
                and t.is_contiguous() and t.get_device() == self._dev):
            lead = (self.S,) if t.dim() == 4 or self.S != 1 else ()
            _need(t, lead + (n, heads, self.d), dtype, name)
            raise ValueError(f"{name} is on {t.device}, the cache on {self.data.device}")
        return n

    def _need_like(self, t, shape, dtype, name):
        _need(t, shape, dtype, name)
        if t.get_device() != self._dev:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.data.device}")

    def _at(self, at, name):
        """(host value, device pointer) of a token number or an int32 [S] tensor."""
        if isinstance(at, torch.Tensor):
            self._need_like(at, (self.S,), torch.int32, name)
            return 0, at.data_ptr()
        at = int(at)
        return (_int32(at, name) if at >> 31 else at), None

    def append(self, k, v, start, stream=None):
        """Quantise k, v [(S,) n, Hkv, d] into cache tokens start .. start+n-1
        (start: a number, or int32 [S] on the device for a start per stream,
        where tokens outside the cache are dropped)."""
        host, dev = self._at(start, "start")
        dt = k.dtype
        code = _dtype_code(dt)
        n = self._need(k, self.Hkv, "k", dt)
        self._need(v, self.Hkv, "v", dt, n)
        back = _on(self._dev)
        try:
            rc = lib.statekv_q4_append(self._ptr, self.S, self.Hkv, self.d, self.capacity, k.data_ptr(), v.data_ptr(),
                                       n, code, host, dev, _stream_ptr(stream, self._dev))
        finally:
            _back(back)
        _check(rc)

    def read(self, start, n, dtype="bf16", k=None, v=None, stream=None):
        """Keys and values [S][n][Hkv][d] of cache tokens start .. start+n-1
        (start as in append; rows of tokens outside the cache are left as they
        were, and are unset in tensors that this call creates)."""
        code = _dtype_code(dtype)
        dt = _torch_dtype(code)
        shape = (self.S, n, self.Hkv, self.d)
        host, dev = self._at(start, "start")
        if _int32(n, "n") < 0:
            raise ValueError(f"negative token count {n}")
        if k is None:
            k = _empty(self._proto[dt], shape, stream)
        else:
            self._need_like(k, shape, dt, "k")
        if v is None:
            v = torch.empty_like(k) if stream is None else _empty(k, shape, stream)
        else:
            self._need_like(v, shape, dt, "v")
        back = _on(self._dev)
        try:
            rc = lib.statekv_q4_read(self._ptr, self.S, self.Hkv, self.d, self.capacity, host, dev, n, code,
                                     k.data_ptr(), v.data_ptr(), _stream_ptr(stream, self._dev))
        finally:
            _back(back)
        _check(rc)
        return k, v

    def decode(self, q, k, v, length, window=0, n_sink=0, out=None, lse=None, with_lse=True, stream=None):
        """Attention of n text tokens over the first `length` cache tokens (a
        number, or int32 [S] on the device) and causally over themselves:
        q [(S,) n, Hq, d], k/v [(S,) n, Hkv, d]; with window > 0 a token at
        position p sees positions above p - window and those below n_sink.
        Returns (out, lse [(S,) Hq, n] or None)."""
        host, dev = self._at(length, "length")
        if (window | n_sink) >> 31:  # (negative ones are the library's to refuse)
            _int32(window, "window"), _int32(n_sink, "n_sink")
        dt = q.dtype
        code = _dtype_code(dt)
        shape = q.shape
        Hq = shape[-2]
        n = self._need(q, Hq, "q", dt)
        self._need(k, self.Hkv, "k", dt, n)
        self._need(v, self.Hkv, "v", dt, n)
        if out is None:
            out = torch.empty_like(q) if stream is None else _empty(q, shape, stream)
        else:
            self._need_like(out, shape, dt, "out")
        if with_lse or lse is not None:
            ls = (self.S, Hq, n) if len(shape) == 4 else (Hq, n)
            if lse is None:
                proto = self._proto[torch.float32]
                lse = proto.new_empty(ls) if stream is None else _empty(proto, ls, stream)
            else:
                self._need_like(lse, ls, torch.float32, "lse")
        back = _on(self._dev)
        try:
            need = self._ws_bytes.get((Hq, n, code))
            if need is None:
                need = lib.statekv_q4_decode_workspace(self.S, Hq, self.Hkv, self.d, n, code)
                if need < 0:
                    _check(int(need))
                self._ws_bytes[(Hq, n, code)] = need
            st = _stream_ptr(stream, self._dev)
            args = (self._ptr, self.S, Hq, self.Hkv, self.d, self.capacity, q.data_ptr(), k.data_ptr(), v.data_ptr(), n,
                    code, host, dev, window, n_sink, out.data_ptr(), lse.data_ptr() if lse is not None else None)
            if stream is not None or _capturing():
                # a workspace of the call's own: the stream may be anybody's, and
                # a captured graph keeps its memory to itself
                ws = _empty(self._proto[torch.bfloat16], (need // 2,), stream)
                rc = lib.statekv_q4_decode(*args, ws.data_ptr(), need, st)
            else:
                with self._lock:
                    ws = self._ws.get(st)
                    if ws is None or ws[0] < need:
                        t = _empty(self._proto[torch.bfloat16], (need // 2,), None)
                        ws = self._ws[st] = (need, t.data_ptr(), t)
                    rc = lib.statekv_q4_decode(*args, ws[1], ws[0], st)
        finally:
            _back(back)
        _check(rc)
        return out, lse


def q4_status() -> int:
    """0, or the first error code that Q4Cache.decode's kernels recorded on the
    current device since the last call (synchronises)."""
    code = ctypes.c_int()
    _check(lib.statekv_q4_status(ctypes.byref(code)))
    return code.value


def sink_window_prefill(q, k, v, window, n_sink=0, out=None, lse=None, with_lse=True, stream=None):
    """Causal attention with a sliding window and n_sink first tokens that stay
    visible, over q [(S,) N, Hq, d], k/v [(S,) N, Hkv, d]: token i sees j <= i
    with j > i - window or j < n_sink.  Returns (out, lse [(S,) Hq, N] or None)."""
    if (window | n_sink) >> 31:  # (negative ones are the library's to refuse)
        _int32(window, "window"), _int32(n_sink, "n_sink")
    shape, kshape, dt = q.shape, k.shape, q.dtype
    if len(shape) != 3 and len(shape) != 4:
        raise ValueError(f"q must be [(S,) N, Hq, d], not {tuple(shape)}")
    lead = (shape[0],) if len(shape) == 4 else ()
    S = shape[0] if lead else 1
    N, Hq, d = shape[-3:]
    Hkv = kshape[-2]
    code = _dtype_code(dt)
    dev = q.get_device()
    if not (q.is_cuda and q.is_contiguous() and kshape == lead + (N, Hkv, d) and v.shape == kshape and k.dtype is dt
            and v.dtype is dt and k.is_contiguous() and v.is_contiguous() and k.get_device() == dev == v.get_device()):
        _need(q, lead + (N, Hq, d), dt, "q")
        for t, name in ((k, "k"), (v, "v")):
            _need(t, lead + (N, Hkv, d), dt, name)
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    mine = out is None, lse is None
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(q, shape, stream)
    if lse is None and with_lse:
        proto = q if dt is torch.float32 else _float32_on(q.device)
        lse = proto.new_empty(lead + (Hq, N)) if stream is None else _empty(proto, lead + (Hq, N), stream)
    if mine != (True, True):
        for t, own, want, wdt, name in ((out, mine[0], lead + (N, Hq, d), dt, "out"),
                                        (lse, mine[1], lead + (Hq, N), torch.float32, "lse")):
            if own:
                continue
            _need(t, want, wdt, name)
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    back = _on(dev)
    try:
        rc = lib.sink_window_prefill_batched(q.data_ptr(), k.data_ptr(), v.data_ptr(), S, N, Hq, Hkv, d, code, window,
                                             n_sink, out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                             _stream_ptr(stream, dev))
    finally:
        _back(back)
    _check(rc)
    return out, lse


def sink_window_status() -> int:
    """0, or the first error code that sink_window_prefill's kernels recorded on
    the current device since the last call (synchronises)."""
    code = ctypes.c_int()
    _check(lib.sink_window_status(ctypes.byref(code)))
    return code.value
