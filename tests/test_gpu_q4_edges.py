"""The 4-bit cache's decode and sink_window_prefill at the edges of what a call
may hold: the largest windows and sink counts, infinite keys, values that only
some rows see, values and keys next to the largest float, NaN inputs, many
streams.  Inputs, limits and the oracle are those of test_gpu_q4.py; for decodes
`mass` is taken of what the kernels round, the parts of a held value
v = (c - 8) s + mid, mid = m + 8 s:
  * up to 32 rows: P s is rounded, 2^-11 (or 2^-22) of P |(c - 8) s|, which is
    at most P (|v| + |mid|);
  * more rows in bf16: P, the value and mid are rounded, 2^-11 of P |v|, P |v| and
    P |mid|;
so mass = sum_j p_j (2 |v_j| + |mid_j|) bounds both."""

import numpy as np
import pytest
import torch

from oracle import statekv_oracle as O
from tests.test_gpu_q4 import DT, Want, _skv, check_attention, cuda, exact_tensor, reference, same, tokens

pytestmark = pytest.mark.gpu

P_DECODE = {"bf16": 2.0 ** -11, "f32": 0.0}
P_PREFILL = {"bf16": 2.0 ** -8, "f32": 0.0}
INT_MAX = 2 ** 31 - 1


def part_of(want, rows):
    w = Want((want[0][rows], want[1][:, rows], want[2][rows], want[3][:, rows]))
    w.keys = want.keys
    return w


def decode_reference(q, k, v, pk, pv, window, n_sink):
    """reference() over the tokens that a cache holds for pk, pv [L][Hkv][d]."""
    if pk.shape[0] == 0:
        return reference(q, k, v, None, None, window, n_sink)
    w = reference(q, k, v, O.q4_held(pk), O.q4_held(pv), window, n_sink)
    _, s, m = O.q4_codes(pv)
    mid = np.repeat(np.abs(m + 8 * s), 64, -1).reshape(pv.shape)
    mid_mass = O.window_attention(q, k, torch.zeros(v.shape), O.q4_held(pk), mid, window, n_sink)[2]
    full = Want((w[0], w[1], 2 * w[2] + mid_mass, w[3]))
    full.keys = w.keys
    return full


# ------------------------------------------------------- the largest arguments
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,n_sink", [(INT_MAX, 0), (1, INT_MAX), (50, INT_MAX - 126), (INT_MAX, INT_MAX)])
def test_sink_window_prefill_of_the_largest_windows(window, n_sink, d, dtype):
    """2^31 - 1 as "all tokens", in the window and in the first tokens."""
    n, Hq, Hkv = 391, 2, 1
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    q, _ = tokens(2, 1, n, Hq, d, dtype, loud=False)
    out = torch.full((1, n, Hq, d), float("nan"), dtype=DT[dtype], device="cuda")
    lse = torch.full((1, Hq, n), float("nan"), device="cuda")
    _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=n_sink, out=out, lse=lse)
    check_attention(out[0], lse[0], reference(q[0], k[0], v[0], None, None, 0, 0), dtype, P_PREFILL[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("window,n_sink", [(INT_MAX, 0), (1, INT_MAX), (50, INT_MAX - 30), (INT_MAX, INT_MAX)])
def test_decode_of_the_largest_windows(window, n_sink, n, dtype):
    S, Hq, Hkv, d, L = 1, 8, 2, 64, 333
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    c = _skv().Q4Cache(Hkv, d, L + 5)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L, window=window, n_sink=n_sink)
    check_attention(out[0], lse[0], decode_reference(q[0], k[0], v[0], pk[0], pv[0], 0, 0), dtype,
                    P_DECODE[dtype])


# --------------------------------------------------------------- infinite keys
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sink_window_prefill_of_infinite_keys(sign, d, dtype):
    """An infinite channel of a key that rows see.  Head 0's queries give it a
    logit of -inf: it weighs nothing, the row is what the other keys make it.
    Head 1's give +inf, head 2's 0 x inf: NaN by definition."""
    n, Hq, Hkv, window, at = 260, 3, 1, 70, 100
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    q, _ = tokens(2, 1, n, Hq, d, dtype, loud=False)
    q[..., 0, 7] = -sign * (q[..., 0, 7].abs() + 0.1)
    q[..., 1, 7] = sign * (q[..., 1, 7].abs() + 0.1)
    q[..., 2, 7] = 0.0
    clean = reference(q[0], k[0], v[0], None, None, window, 2)
    k[0, at, 0, 7] = sign * float("inf")
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)
    far = k.clone()
    far[0, at, 0, 7] = sign * 1e30           # head 0: a logit below -1e28, a weight of 0 as well
    w = reference(q[0], far[0], v[0], None, None, window, 2)
    sees = slice(at, at + window)
    want = Want((w[0][:, :1], w[1][:1], w[2][:, :1], clean[3][:1]))   # (limits of the finite logits)
    want.keys = n
    check_attention(out[0, :, :1], lse[0, :1], want, dtype, P_PREFILL[dtype])
    assert torch.isnan(out[0, sees, 1:]).all() and torch.isnan(lse[0, 1:, sees]).all()
    for rows in (slice(0, at), slice(at + window, n)):
        check_attention(out[0, rows], lse[0][:, rows], part_of(clean, rows), dtype, P_PREFILL[dtype])


@cuda
@pytest.mark.parametrize("where", ["q", "k", "v", "v[0]"])
def test_sink_window_prefill_of_nan_inputs_costs_no_more(where):
    """Inputs full of NaNs (or one NaN value in every 100th token) take the time of
    finite ones and no multiple of it: ten times as much is allowed where rows that
    are recomputed one by one take some hundred times as much."""
    n, Hq, Hkv, d, window = 4096, 4, 1, 64, 1024
    k, v = tokens(1, 1, n, Hkv, d, "bf16")
    q, _ = tokens(2, 1, n, Hq, d, "bf16", loud=False)
    ins = {"q": q.cuda(), "k": k.cuda(), "v": v.cuda()}

    def ms():
        call = lambda: _skv().sink_window_prefill(ins["q"], ins["k"], ins["v"], window, n_sink=4)
        out, _ = call()
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(), call(), b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, out

    clean, _ = ms()
    if where == "v[0]":
        ins["v"][:, ::100, :, 0] = float("nan")
    else:
        ins[where][:] = float("nan")
    odd, out = ms()
    rows = out[0, 100:, :, :1] if where == "v[0]" else out
    assert torch.isnan(rows).all()
    if where == "v[0]":
        assert torch.isfinite(out[..., 1:]).all()
    assert odd <= 10 * clean, f"{odd:.3f} ms against {clean:.3f}"


@cuda
@pytest.mark.parametrize("where", ["q", "k", "v", "one"])
def test_sink_window_prefill_of_nan_inputs_costs_no_more_in_float32(where):
    """The same in float32, and for a single NaN in one channel."""
    n, Hq, Hkv, d, window = 4096, 4, 1, 64, 1024
    k, v = tokens(1, 1, n, Hkv, d, "f32")
    q, _ = tokens(2, 1, n, Hq, d, "f32", loud=False)
    ins = {"q": q.cuda(), "k": k.cuda(), "v": v.cuda()}

    def ms():
        call = lambda: _skv().sink_window_prefill(ins["q"], ins["k"], ins["v"], window, n_sink=4)
        out, _ = call()
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(), call(), b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, out

    clean, _ = ms()
    if where == "one":
        ins["v"][0, 2000, 0, 7] = float("nan")
    else:
        ins[where][:] = float("nan")
    odd, out = ms()
    assert torch.isnan(out[0, 2000:2000 + window, :, 7] if where == "one" else out).all()
    if where == "one":
        assert torch.isnan(out).sum() == window * Hq
    assert odd <= 10 * clean, f"{odd:.3f} ms against {clean:.3f}"


@cuda
@pytest.mark.parametrize("where", ["k", "v", "one", "text"])
@pytest.mark.parametrize("L,n", [(300, 1), (65536, 1), (65536, 16)])
def test_decode_of_nan_inputs_costs_no_more(L, n, where):
    """The same for a decode over a cache that holds NaNs (everywhere, or in one group of
    64 channels of one token), or whose text keys are NaN."""
    S, Hq, Hkv, d = 1, 7, 1, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda m, H: torch.randn((S, m, H, d), generator=g, device="cuda").bfloat16()
    pk, pv, k, v, q = r(L, Hkv), r(L, Hkv), r(n, Hkv), r(n, Hkv), r(n, Hq)

    def ms():
        c = _skv().Q4Cache(Hkv, d, L)
        c.append(pk, pv, 0)
        call = lambda: c.decode(q, k, v, L)
        out, _ = call()
        best = float("inf")
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(), call(), b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, out

    clean, want = ms()
    if where == "one":
        pv[0, 5, 0, 70] = float("nan")
    else:
        {"k": pk, "v": pv, "text": k}[where][:] = float("nan")
    odd, out = ms()
    assert torch.isnan(out[..., 64:] if where == "one" else out).all()
    if where == "one":
        assert same(out[..., :64], want[..., :64])
    assert odd <= 10 * clean, f"{odd:.3f} ms against {clean:.3f}"


# -------------------------------------------- tokens that only some rows see
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq", [(3, 7), (2, 7), (30, 7), (70, 2)])
@pytest.mark.parametrize("which", ["v", "k", "both"])
@pytest.mark.parametrize("size", [1e6, 1e30])
def test_decode_hidden_finite_values_have_no_influence(size, which, n, Hq, dtype):
    """A large key or value that the window hides from all but the first text
    tokens: their rows see it, the others keep the precision of what they see."""
    S, Hkv, d, L, window = 1, 1, 128, 300, 120
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    at = L - window + 1                      # text token 0 alone sees it
    if which != "k":
        pv[:, at] *= size
    if which != "v":
        pk[:, at] *= size
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L, window=window, n_sink=2)
    want = decode_reference(q[0], k[0], v[0], pk[0], pv[0], window, 2)
    check_attention(out[0, 1:], lse[0][:, 1:], part_of(want, slice(1, n)), dtype, P_DECODE[dtype])
    check_attention(out[0], lse[0], want, dtype, P_DECODE[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,n,window,n_sink", [
    (100, 9, 1, 0), (100, 9, 4, 0), (100, 9, 9, 3), (64, 40, 37, 0), (64, 40, 70, 64), (33, 33, 33, 33),
    (1, 5, 3, 0), (2000, 6, 1500, 1), (2000, 60, 31, 500), (0, 8, 3, 0)])
def test_decode_at_the_edge_of_the_window(L, n, window, n_sink, d, dtype):
    """Every position at which a window's edge can stand among cached tokens, first
    tokens and text tokens, with one, two and seven heads a KV head, over lengths on
    the host and on the device."""
    S, Hkv = 2, 2
    for G in (1, 2, 7):
        pk, pv = tokens(1, S, max(L, 1), Hkv, d, dtype)
        k, v = tokens(2, S, n, Hkv, d, dtype)
        q, _ = tokens(3, S, n, G * Hkv, d, dtype, loud=False)
        c = _skv().Q4Cache(Hkv, d, L + 7, n_streams=S)
        c.data.fill_(255)
        if L:
            c.append(pk.cuda(), pv.cuda(), 0)
        lens = [L, L // 2]
        at = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for where, of in ((L, [L, L]), (at, lens)):
            out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), where, window=window, n_sink=n_sink)
            for s in range(S):
                want = decode_reference(q[s], k[s], v[s], pk[s, :of[s]], pv[s, :of[s]], window, n_sink)
                check_attention(out[s], lse[s], want, dtype, P_DECODE[dtype])


# ---------------------------------------------------------- the largest floats
LARGE = [
    # Hq (of one KV head), n, L: 8 rows, 14 rows, 112, 280
    (7, 1, 300), (7, 1, 1700), (7, 2, 900), (7, 16, 900), (7, 40, 900), (40, 1, 900)]


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n,L", LARGE)
def test_decode_of_large_keys(Hq, n, L, dtype):
    """Keys of up to 2^124 that meet queries as small, and the reverse: logits of
    ordinary size."""
    S, Hkv, d = 1, 1, 128
    for e in (120, -100, -122):
        pk, pv = tokens(1, S, L, Hkv, d, dtype)
        k, v = tokens(2, S, n, Hkv, d, dtype)
        q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
        pk, k, q = pk * 2.0 ** e, k * 2.0 ** e, q * 2.0 ** -e
        c = _skv().Q4Cache(Hkv, d, L)
        c.append(pk.cuda(), pv.cuda(), 0)
        out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
        check_attention(out[0], lse[0], decode_reference(q[0], k[0], v[0], pk[0], pv[0], 0, 0), dtype,
                        P_DECODE[dtype])


def decode_values(size, Hq, n, L, dtype, flat):
    S, Hkv, d = 1, 1, 128
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    if flat:
        pv, v = pv.abs() + 4, torch.full_like(v, 6.0)
    pv, v = pv * size, v * size
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
    check_attention(out[0], lse[0], decode_reference(q[0], k[0], v[0], pk[0], pv[0], 0, 0), dtype, P_DECODE[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n,L", LARGE)
@pytest.mark.parametrize("size", [2.0 ** 116, 2.0 ** -100])
def test_decode_of_large_and_tiny_values(size, Hq, n, L, dtype):
    """Values of one sign or of both beyond what one scale of fp16 numbers would hold."""
    for flat in (False, True):
        decode_values(size, Hq, n, L, dtype, flat)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n,L", LARGE)
def test_decode_of_values_whose_sum_overflows(Hq, n, L, dtype):
    """Values next to the largest float, whose sum over the tokens would not fit: the
    result, their mean, does."""
    for flat in (False, True):
        decode_values(2.0 ** 124, Hq, n, L, dtype, flat)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_decode_of_large_text_values(n, dtype):
    """The text tokens' own values next to the largest float, an ordinary cache."""
    S, Hq, Hkv, d, L = 1, 7, 1, 128, 200
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    k[:] = 0
    v = (v.abs() + 4) * 2.0 ** 124
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    for past in (L, 0):
        out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), past)
        check_attention(out[0], lse[0], decode_reference(q[0], k[0], v[0], pk[0, :past], pv[0, :past], 0, 0), dtype,
                        P_DECODE[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,L", [(1, 300), (1, 1700), (40, 900)])
def test_decode_of_large_and_poisoned_values_in_a_window(n, L, dtype):
    """Values whose sum overflows beside a group of 64 channels that holds a NaN: the
    rows that see it are NaN in that group alone."""
    S, Hq, Hkv, d, window, n_sink = 1, 7, 1, 128, 200, 4
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    pv, v = (pv.abs() + 4) * 2.0 ** 124, (v.abs() + 4) * 2.0 ** 124
    want = decode_reference(q[0], k[0], v[0], pk[0], pv[0], window, n_sink)
    sees = 25                                # rows below it see the token
    at = L - window + sees
    pv[0, at, 0, 70] = float("nan")
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L, window=window, n_sink=n_sink)
    rows = min(n, sees)
    assert torch.isnan(out[0, :rows, :, 64:]).all()
    got = out.clone()
    got[0, :rows, :, 64:] = torch.from_numpy(want[0][:rows, :, 64:]).to(out)
    check_attention(got[0], lse[0], want, dtype, P_DECODE[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [5, 30])
@pytest.mark.parametrize("e", [40, 100, 118])
def test_decode_of_tiny_queries_that_see_no_cached_token(e, window, dtype):
    """More than 32 rows whose tile sees nothing of the cache, queries of 2^-e and text
    keys of 2^e."""
    S, Hq, Hkv, d, L, n = 1, 8, 1, 64, 33, 50
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    pk, k, q = pk * 2.0 ** e, k * 2.0 ** e, q * 2.0 ** -e
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    for past in (L, 0):
        out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), past, window=window)
        check_attention(out[0], lse[0], decode_reference(q[0], k[0], v[0], pk[0, :past], pv[0, :past], window, 0), dtype,
                        P_DECODE[dtype])


def huge_rows(out, lse, q, k, v, keys, values, at, signs, dtype, p_step):
    """Rows over keys that include a huge one, all channels alike, at `at`: heads of
    sign 1 take its value, heads of sign -1 what the other tokens make (0: not
    checked).  The value is off by its own rounding and by that of the weight times
    its scale, 2^-11 or in float32 2^-22 of P |(c - 8) s|, at most P (|v| + |mid|) and so
    3 max |v| with P = 1; 128-row calls round v and mid instead, the same bound."""
    n, Hq, d = q.shape
    step, other = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype], np.arange(len(keys)) != at
    weight = max(p_step, 2.0 ** -22)
    got, glse, qd = O.to_f64(out.cpu()), O.to_f64(lse.cpu()), O.to_f64(q)
    for h, sign in enumerate(signs):
        if sign > 0:
            want = np.broadcast_to(values[at, 0], (n, d))
            logit = qd[:, h] @ keys[at, 0] / np.sqrt(d)
            assert (np.abs(got[:, h] - want) <= step * np.abs(want) + weight * 3 * np.abs(values[at, 0]).max()).all()
            assert (np.abs(glse[h] - logit) <= 2.0 ** -19 * np.abs(logit)).all()
        elif sign < 0:
            w = reference(q[:, h:h + 1], k, v, keys[other], values[other], 0, 0)
            part = Want((w[0], w[1], 2 * w[2] + np.abs(values).max(), w[3]))
            part.keys = w.keys
            check_attention(out[:, h:h + 1], lse[h:h + 1], part, dtype, p_step)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,n,L", LARGE)
@pytest.mark.parametrize("size", [1e5, 1e7, 1e10, 1e20])
def test_decode_of_huge_logits(size, Hq, n, L, dtype):
    """A key so large that its logits are beyond float32's integers."""
    S, Hkv, d, at = 1, 1, 128, 37
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    signs = [1 if h % 2 else -1 for h in range(Hq)]
    q = torch.randn(S, n, Hq, d, generator=torch.Generator().manual_seed(3)) + 2 * torch.tensor(signs)[:, None]
    q = q.to(DT[dtype])
    pk[:, at] = size
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
    huge_rows(out[0], lse[0], q[0], k[0], v[0], O.q4_held(pk[0]), O.q4_held(pv[0]), at, signs, dtype,
              P_DECODE[dtype])


@cuda
@pytest.mark.parametrize("size", [1e3, 3e4, 1e6, 1e10, 1e20])
def test_decode_of_many_rows_beside_a_huge_key(size):
    """Rows that a huge visible key weighs nothing for keep the logits of the others:
    queries away from it, 280 rows."""
    S, Hq, Hkv, d, n, L, at = 1, 7, 1, 128, 40, 900, 37
    pk, pv = tokens(1, S, L, Hkv, d, "bf16")
    k, v = tokens(2, S, n, Hkv, d, "bf16")
    q = (torch.randn(S, n, Hq, d, generator=torch.Generator().manual_seed(3)) - 2).bfloat16()
    pk[:, at] = size
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
    other = torch.arange(L) != at
    want = decode_reference(q[0], k[0], v[0], pk[0, other], pv[0, other], 0, 0)
    e = 2.0 ** -11                           # what statekv.h allows a logit
    wide = Want((want[0], want[1], want[2] * (1 + 2 * e / P_DECODE["bf16"]), want[3]))
    wide.keys = want.keys
    check_attention(out[0], None, wide, "bf16", P_DECODE["bf16"])
    assert (np.abs(O.to_f64(lse[0].cpu()) - want[1]) <= e + 2.0 ** -19 * want[3] + 2.0 ** -20 + 2.0 ** -23 * np.abs(want[1])).all()


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e5, 1e7, 1e10, 1e20])
def test_sink_window_prefill_of_huge_logits(size, d, dtype):
    n, Hq, Hkv, at = 300, 4, 1, 1
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    signs = [1 if h % 2 else -1 for h in range(Hq)]
    q = torch.randn(1, n, Hq, d, generator=torch.Generator().manual_seed(3)) + 2 * torch.tensor(signs)[:, None]
    q = q.to(DT[dtype])
    k[:, at] = size
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), n)
    past = 2                                 # the rows from here on see it
    huge_rows(out[0, past:], lse[0][:, past:], q[0, past:], k[0, past:], v[0, past:], O.to_f64(k[0, :past]), O.to_f64(v[0, :past]),
              at, signs, dtype, P_PREFILL[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 120, 2.0 ** 124, 2.0 ** -100])
def test_sink_window_prefill_of_large_values(size, d, dtype):
    n, Hq, Hkv, window = 500, 3, 1, 200
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    q, _ = tokens(2, 1, n, Hq, d, dtype, loud=False)
    v = (v.abs() + 4) * size
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)
    check_attention(out[0], lse[0], reference(q[0], k[0], v[0], None, None, window, 2), dtype, P_PREFILL[dtype])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 40])
def test_decode_of_values_with_very_wide_ranges(n, dtype):
    """Values whose scale differs by up to 2^48 between tokens, against the bounds that
    statekv.h states: what fp16 cannot hold of a weight times a scale is off by 2^-29
    of the largest (2^-33 in float32) times 8, a token; beyond 32 rows 2^-30 of the
    largest weight, a token, and 2^-36 of the largest value."""
    S, Hq, Hkv, d, L = 1, 7, 1, 128, 300
    g = torch.Generator().manual_seed(8)
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    pv = pv * torch.exp2(torch.randint(-24, 25, (1, L, 1, 1), generator=g).float()).to(DT[dtype])
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    c = _skv().Q4Cache(Hkv, d, L)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
    want = decode_reference(q[0], k[0], v[0], pk[0], pv[0], 0, 0)
    logits = np.einsum("nhd,jd->nhj", O.to_f64(q[0]), O.q4_held(pk[0])[:, 0]) / np.sqrt(d)
    weight = np.exp(logits.max(-1) - want[1].T)[..., None]          # the largest cached one, normalised
    scale, top = O.q4_codes(pv[0])[1].max(), np.abs(O.q4_held(pv[0])).max()
    floor = L * 8 * (2.0 ** -33 if dtype == "f32" else 2.0 ** -29) * weight * scale
    if dtype == "bf16" and Hq * n > 32:
        floor = L * 2.0 ** -30 * weight * top + 2.0 ** -36 * top
    # check_attention's limits, and the floor
    step, e = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype], 2.0 ** -19 * want[3].T[..., None]
    lim = step * np.abs(want[0]) + want[2] * (P_DECODE[dtype] + 2 * e + (64 + want.keys / 16) * 2.0 ** -23) + floor
    err = np.abs(O.to_f64(out[0].cpu()) - want[0])
    fine = bool((err <= lim).all())
    assert fine, f"out: worst {np.max(err / lim):.3g} of its limit"


# ---------------------------------------------------------------- many streams
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (9500, 40)])
def test_decode_of_many_long_streams_is_shared_out(window, n_sink, dtype):
    """70 streams of up to 12000 tokens, most of them short or empty, in a cache so
    long that their blocks are dealt to the workers (which write partials into the
    workspace): more streams than a warp has lanes."""
    S, Hq, Hkv, d, cap, n = 70, 4, 2, 64, 12000, 1
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 400, (S,), generator=g, dtype=torch.int32)
    lens[::3] = 0
    lens[[5, 31, 32, 40, 64]] = torch.tensor([12000, 7777, 8191, 11500, 9601], dtype=torch.int32)
    lens[-2:] = 0
    pk, pv = tokens(1, 1, cap, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    of = [(torch.roll(pk, 37 * s, 1), torch.roll(pv, 37 * s, 1)) for s in range(S)]  # every stream holds other tokens
    c = _skv().Q4Cache(Hkv, d, cap, n_streams=S)
    c.append(torch.cat([x[0] for x in of]).cuda(), torch.cat([x[1] for x in of]).cuda(), 0)
    ins = [t.cuda() for t in (q, k, v, lens)]
    out, lse = c.decode(*ins, window=window, n_sink=n_sink)
    for _, _, ws in c._ws.values():
        ws.view(torch.uint8).fill_(255)
    again, _ = c.decode(*ins, window=window, n_sink=n_sink)
    assert same(out, again) and _skv().q4_status() == 0
    assert any((ws.view(torch.uint8) != 255).any().item() for _, _, ws in c._ws.values())
    for s in range(S):
        L = int(lens[s])
        want = decode_reference(q[s], k[s], v[s], of[s][0][0, :L], of[s][1][0, :L], window, n_sink)
        check_attention(out[s], lse[s], want, dtype, P_DECODE[dtype])


# ------------------------------------------------------------ streams, arguments
@cuda
def test_a_new_cache_is_ready_for_any_stream():
    """A cache made while the current stream is busy, and appended to at once on
    another: its fill does not come after the tokens."""
    Hkv, d, n = 2, 64, 500
    k, v = tokens(1, 1, n, Hkv, d, "bf16")
    ins = [k.cuda(), v.cuda()]
    side = torch.cuda.Stream()
    for cycles in (0, 40_000_000):           # the kernels are loaded, then some 20 ms
        torch.cuda.synchronize()
        torch.cuda._sleep(cycles)
        c = _skv().Q4Cache(Hkv, d, n)
        c.append(*ins, 0, stream=side)
    torch.cuda.synchronize()
    for t, x in zip(c.read(0, n, dtype="f32"), (k, v)):
        assert same(t.cpu(), exact_tensor(O.q4_held(x), "f32"))


@cuda
@pytest.mark.parametrize("detailed", ["native", "q4"])
def test_a_new_handle_is_ready_for_any_stream(detailed):
    """The same for a handle whose first step, on another stream, allocates its layer:
    positions (and native keys) that the step appended stay."""
    Hq, Hkv, d, T, B = 4, 2, 64, 128, 64
    k, v = tokens(1, 1, T, Hkv, d, "bf16")
    q, _ = tokens(2, 1, T, Hq, d, "bf16", loud=False)
    pos = torch.arange(1, T + 1, dtype=torch.int32)
    ins = [t.cuda() for t in (q[0], k[0], v[0], pos)]
    side = torch.cuda.Stream()
    for cycles in (0, 40_000_000):
        torch.cuda.synchronize()
        h = _skv().StateKV(Hq, Hkv, d, T, B, 2, detailed=detailed)
        torch.cuda._sleep(cycles)
        with torch.cuda.stream(side):
            h.prefill_frame(0, *ins)
        torch.cuda.synchronize()
        D, C = h.get_detailed(0), h.get_compressed(0)
        assert D["len"] == T and C["len"] == B
        assert same(D["pos"][0, :T].cpu(), pos)
        assert (C["pos"][..., :B] > 0).all()
        if detailed == "native":
            assert same(D["k"][0, :, :T].cpu(), k[0].transpose(0, 1).contiguous())
        h.close()


# ------------------------------------------------------------ writing and reading
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bits", "powers", "mixed", "subnormal", "offset", "two"])
def test_append_of_any_numbers(kind, dtype):
    """Random bit patterns, magnitudes from the least subnormal number up, groups of one
    small range far from 0, groups of two values: the held values are the oracle's."""
    g = np.random.default_rng(7)
    n, H, d = 300, 2, 128
    shape = (1, n, H, d)
    x = {"bits": lambda: g.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32).view(np.float32).copy(),
         "powers": lambda: g.standard_normal(shape) * np.exp2(g.integers(-149, 120, (1, n, H, 1))),
         "mixed": lambda: g.standard_normal(shape) * np.exp2(g.integers(-20, 20, shape)),
         "subnormal": lambda: g.standard_normal(shape) * 2.0 ** -140,
         "offset": lambda: 1e30 + 1e24 * g.standard_normal(shape),
         "two": lambda: np.where(g.random(shape) < 0.5, 1, -1) * np.exp2(g.integers(-140, 127, (1, n, H, 1)))}[kind]()
    with np.errstate(over="ignore"):
        t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DT[dtype])
    t = torch.where(t.float() < -3.38e38, torch.zeros_like(t), t)    # (below the least bfloat16: NaN)
    c = _skv().Q4Cache(H, d, n)
    c.append(t.cuda(), (-t).clamp(min=-3.38e38).cuda(), 0)
    for got, src in zip(c.read(0, n, dtype="f32"), (t, (-t).clamp(min=-3.38e38))):
        want = exact_tensor(O.q4_held(src.float()), "f32")
        got = got.cpu()
        fine = bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())
        assert fine, kind
