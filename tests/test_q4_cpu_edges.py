"""Refusals of the 4-bit cache's and the windowed attention's binding that need no
GPU: numbers that the library's 32-bit arguments do not hold, tensors of too many
or too few dimensions."""

import pytest
import torch


def _lib():
    from kv_cache_selection_b200 import statekv as S
    return S


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, -2 ** 32 + 1])
def test_numbers_beyond_32_bits_are_refused(x):
    """Cut off to 32 bits they would name another token, length or window."""
    S = _lib()
    c = S.Q4Cache(2, 64, 40, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    calls = {
        "start": [lambda: c.append(k, k, x), lambda: c.read(x, 3)],
        "n": [lambda: c.read(0, x)],
        "length": [lambda: c.decode(k, k, k, x)],
        "window": [lambda: c.decode(k, k, k, 4, window=x), lambda: S.sink_window_prefill(k, k, k, x)],
        "n_sink": [lambda: c.decode(k, k, k, 4, window=3, n_sink=x), lambda: S.sink_window_prefill(k, k, k, 4, n_sink=x)],
        "Hkv": [lambda: S.Q4Cache(x, 64, 40, device="cpu")],
        "d": [lambda: S.Q4Cache(2, x, 40, device="cpu")],
        "capacity": [lambda: S.Q4Cache(2, 64, x, device="cpu")],
        "n_streams": [lambda: S.Q4Cache(2, 64, 40, n_streams=x, device="cpu")],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"{name}=.*32 bits"):
                f()


@pytest.mark.parametrize("shape", [(2, 1, 5, 4, 64), (4, 64), (64,)])
def test_sink_window_prefill_refuses_other_dimensions(shape):
    """Of a q with two leading dimensions only the first sequence was computed."""
    S = _lib()
    q, k = torch.zeros(shape), torch.zeros(5, 2, 64)
    with pytest.raises(ValueError, match="q must be"):
        S.sink_window_prefill(q, k, k, 4)
