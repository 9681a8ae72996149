"""The 4-bit cache and sink-window prefill without a GPU: pins of the oracle's
definitions, and the refusals that the library's host checks make before any
device call (the pointers are never dereferenced)."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import statekv_oracle as O


# ------------------------------------------------------------------ oracle pins
def test_bf16_grid_brackets_the_value():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(2000) * 10.0 ** g.integers(-30, 30, 2000), [0.0, 1.0, -1.0, 2.0 ** -133, -3.5]])
    lo, hi = O.bf16_grid(x, up=False), O.bf16_grid(x, up=True)
    assert (lo <= x).all() and (hi >= x).all()
    for r in (lo, hi):   # every result is a bfloat16 value
        assert (torch.tensor(r).float().bfloat16().double().numpy() == r).all()
    exact = torch.tensor(x).float().bfloat16().double().numpy() == x
    assert (lo[exact] == hi[exact]).all()
    near = torch.tensor(x).bfloat16().double().numpy()
    assert ((near == lo) | (near == hi)).all()


def test_q4_handworked_group():
    """0, 1/4, ..., 15/4 and repeats: m = 0, s = 1/4, every value held exactly;
    a value midway between two codes goes to the even one."""
    x = np.tile(np.arange(16) / 4.0, 4)
    assert (O.q4_held(x) == x).all()
    x[1], x[2], x[3] = 0.125, 0.375, 0.625      # 0.5, 1.5, 2.5 steps
    c, s, m = O.q4_codes(x)
    assert s[0] == 0.25 and m[0] == 0.0
    assert list(c[0, 1:4]) == [0.0, 2.0, 2.0]


def test_q4_error_is_at_most_half_a_step():
    g = np.random.default_rng(1)
    x = g.standard_normal((50, 128)) * np.exp(g.standard_normal((50, 1)) * 5) + g.standard_normal((50, 1)) * 100
    c, s, m = O.q4_codes(x)
    assert c.min() >= 0 and c.max() <= 15
    err = np.abs(O.q4_held(x) - x).reshape(50, 2, 64)
    assert (err <= s[..., None] / 2 * (1 + 1e-12)).all()
    # exact rational check of one group
    xs, sm, mm = [Fraction(float(t)) for t in x[3, :64]], Fraction(float(s[3, 0])), Fraction(float(m[3, 0]))
    assert mm <= min(xs) and mm + 15 * sm >= max(xs)
    assert [int(t) for t in c[3, 0]] == [round((t - mm) / sm) for t in xs]


def test_q4_flat_and_poisoned_groups():
    x = np.full((2, 128), 0.75)
    assert (O.q4_held(x) == x).all()
    x[0, 70] = np.nan
    x[1, 3] = np.inf
    h = O.q4_held(x)
    assert (h[0, :64] == 0.75).all() and np.isnan(h[0, 64:]).all()
    assert np.isnan(h[1, :64]).all() and (h[1, 64:] == 0.75).all()


@pytest.mark.parametrize("L", [0, 5])
def test_window_attention_wide_window_is_causal(L):
    g = np.random.default_rng(2)
    n, Hq, Hkv, d = 7, 4, 2, 64
    q, k, v = g.standard_normal((L + n, Hq, d)), g.standard_normal((L + n, Hkv, d)), g.standard_normal((L + n, Hkv, d))
    ref, ref_lse = O.causal_attention(q, k, v)
    for window in (0, L + n):
        out, lse, _, _ = O.window_attention(q[L:], k[L:], v[L:], k[:L], v[:L], window=window)
        np.testing.assert_allclose(out, ref[L:], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse, ref_lse[:, L:], rtol=1e-12)


def test_window_attention_by_hand():
    """Equal keys: the output is the mean of the visible values."""
    n, d = 6, 64
    q, k = np.zeros((n, 1, d)), np.zeros((n, 1, d))
    v = np.broadcast_to(np.arange(n, dtype=float)[:, None, None], (n, 1, d))
    out, lse, _, _ = O.window_attention(q, k, v, window=2, n_sink=1)
    want = [0, 0.5, 1.0, (0 + 2 + 3) / 3, (0 + 3 + 4) / 3, (0 + 4 + 5) / 3]
    np.testing.assert_allclose(out[:, 0, 0], want)
    np.testing.assert_allclose(np.exp(lse[0]), [1, 2, 3, 3, 3, 3])


# -------------------------------------------------------------------- refusals
P = 1 << 20   # fake 16-byte aligned addresses, 1 GiB apart


def _p(i, off=0):
    return ctypes.c_void_p(P + i * (1 << 30) + off)


def _lib():
    from kv_cache_selection_b200 import statekv as S
    return S


def _msg():
    return _lib().lib.statekv_last_error(None)


def test_q4_bytes():
    f = _lib().lib.statekv_q4_bytes
    assert f(1, 4, 128, 131072) == 131072 * 4 * 2 * (64 + 8)          # 4.5 bits a value
    assert f(3, 2, 64, 1) == 3 * 2 * 32 * 2 * (32 + 4)               # whole blocks of 32 tokens
    assert f(1, 2, 64, 33) == 2 * f(1, 2, 64, 32)
    assert f(1, 1, 64, 1 << 30) == (1 << 30) * 72                    # beyond 32 bits
    for bad, code in (((0, 1, 64, 8), -1), ((1, 0, 64, 8), -1), ((1, 1, 64, 0), -1), ((1, 1, 96, 8), -2),
                      ((1, 1, 64, (1 << 30) + 1), -2), ((65536, 1, 64, 8), -2), ((64, 64, 64, 1 << 30), -2)):
        assert f(*bad) == code, bad


@pytest.mark.parametrize("call", ["append", "read"])
def test_q4_range_refusals(call):
    S = _lib()

    def f(cache=_p(0), Sn=1, Hkv=2, d=64, cap=100, k=_p(1), v=_p(2), n=10, dtype=0, start=0, starts=None):
        if call == "append":
            return S.lib.statekv_q4_append(cache, Sn, Hkv, d, cap, k, v, n, dtype, start, starts, None)
        return S.lib.statekv_q4_read(cache, Sn, Hkv, d, cap, start, starts, n, dtype, k, v, None)

    assert f(n=0) == 0                                   # nothing to do
    assert f(n=0, cache=None, k=None, v=None) == 0
    assert f(n=-1) == -1
    assert f(start=-1) == -1
    assert f(start=91) == -3 and b"fit" in _msg()
    assert f(start=(1 << 31) - 1, n=(1 << 31) - 1) == -3  # no wrap-around
    assert f(d=32) == -2
    assert f(dtype=2) == -1
    assert f(Sn=0) == -1
    assert f(cap=0) == -1
    for name in ("cache", "k", "v"):
        assert f(**{name: None}) == -1
        assert f(**{name: _p(5, 8)}) == -1 and b"16-byte" in _msg()
    assert f(starts=_p(6, 2)) == -1 and b"4-byte" in _msg()
    assert f(k=_p(0, 64)) == -1 and b"overlaps" in _msg()
    assert f(v=_p(0, 4096)) == -1
    if call == "read":
        assert f(k=_p(1), v=_p(1, 16)) == -1


def test_q4_decode_refusals():
    S = _lib()

    def f(cache=_p(0), Sn=1, Hq=4, Hkv=2, d=64, cap=100, q=_p(1), k=_p(2), v=_p(3), n=3, dtype=0, length=50,
          lengths=None, window=0, n_sink=0, out=_p(4), lse=_p(5), ws=_p(8), wb=1 << 28):
        return S.lib.statekv_q4_decode(cache, Sn, Hq, Hkv, d, cap, q, k, v, n, dtype, length, lengths, window, n_sink,
                                       out, lse, ws, wb, None)

    assert f(Hq=3) == -1
    assert f(Hq=0) == -1
    assert f(d=256) == -2
    assert f(n=0) == -1
    assert f(n=65536) == -2
    need = S.lib.statekv_q4_decode_workspace(1, 4, 2, 64, 3, 0)
    assert need > 0 and S.lib.statekv_q4_decode_workspace(1, 4, 3, 64, 3, 0) == -1
    assert f(wb=need - 1) == -1 and b"workspace" in _msg()
    assert f(ws=_p(4)) == -1 and f(ws=_p(0)) == -1
    assert f(dtype=5) == -1
    assert f(length=101) == -1 and f(length=-1) == -1
    assert f(window=-1) == -1 and f(n_sink=-1) == -1
    for name in ("cache", "q", "k", "v", "out", "ws"):
        assert f(**{name: None}) == -1
        assert f(**{name: _p(7, 4)}) == -1
    assert f(lse=_p(5, 2)) == -1 and f(lengths=_p(6, 1)) == -1
    assert f(out=_p(1)) == -1 and b"out overlaps q" in _msg()
    assert f(out=_p(0, 1024)) == -1
    assert f(lse=_p(4, 16)) == -1
    assert f(lengths=_p(5), lse=_p(5)) == -1


def test_sink_window_prefill_refusals():
    S = _lib()

    def f(q=_p(0), k=_p(1), v=_p(2), n_seq=2, n=5, Hq=4, Hkv=2, d=64, dtype=0, window=3, n_sink=1, out=_p(3), lse=_p(4)):
        return S.lib.sink_window_prefill_batched(q, k, v, n_seq, n, Hq, Hkv, d, dtype, window, n_sink, out, lse, None)

    assert f(n=0) == 0
    assert f(n=-1) == -1 and f(n_seq=0) == -1 and f(Hq=3) == -1
    assert f(d=80) == -2 and f(dtype=9) == -1
    assert f(window=0) == -1 and b"window" in _msg()
    assert f(n_sink=-1) == -1
    assert f(n=(1 << 24) + 1) == -2
    for name in ("q", "k", "v", "out"):
        assert f(**{name: None}) == -1
        assert f(**{name: _p(7, 2)}) == -1
    assert f(lse=_p(4, 1)) == -1
    assert f(out=_p(2)) == -1 and f(lse=_p(0)) == -1
    assert S.lib.sink_window_prefill(None, None, None, 4, 2, 1, 64, 0, 3, 0, None, None, None) == -1


def test_binding_refusals():
    """The binding's own checks, on tensors that are not on a CUDA device."""
    S = _lib()
    with pytest.raises(S.StateKVError):
        S.Q4Cache(1, 80, 10, device="cpu")
    c = S.Q4Cache(2, 64, 40, n_streams=2, device="cpu")
    assert c.data.numel() == S.lib.statekv_q4_bytes(2, 2, 64, 40)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: c.append(k, k, 0), lambda: c.decode(k, k, k, 4), lambda: c.read(0, 3, k=k, v=k),
                 lambda: S.sink_window_prefill(k, k, k, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="dtype"):
        c.append(k.half(), k.half(), 0)


def test_handle_refusals():
    """A handle's 4-bit detailed state: what is refused without a device."""
    S = _lib()
    assert S.lib.statekv_set_detailed_format(None, 1) == -1
    assert S.lib.statekv_get_detailed_q4(None, 0, None, None, None, None) == -1
    with pytest.raises(ValueError, match="detailed"):
        S.StateKV(4, 2, 64, 16, 32, 4, detailed="q8")
