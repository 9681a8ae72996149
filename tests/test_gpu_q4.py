"""GPU parity of the 4-bit cache (append, read, decode) and of
sink_window_prefill against the float64 oracle.

Tolerances (t = the output type's half step, 2^-8 bf16, 2^-24 f32, relative):
  * read back: exact.  m + c s has one float32 rounding (c s is exact), then one
    to bf16; the codes themselves are decided exactly.
  * attention, per element: t |out| for the last rounding, plus, times
    mass = sum_j p_j |v_j|:
      - weights rounded before they meet the values: 2^-8 (bf16 prefill), 2^-11
        (bf16 over the cache), nothing in float32;
      - 2 e for logits that are off by e (it enters weight and sum):
        e = 2^-19 span, 32 half steps of float32 on sums of the size
        span = max_j sum_d |q_d k_jd| / sqrt(d);
      - (64 + keys / 16) 2^-23 for summing in chunks of 16 keys;
  * lse: e + 2^-20 + 2^-23 |lse|.
"""

import numpy as np
import pytest
import torch

from oracle import statekv_oracle as O

pytestmark = pytest.mark.gpu
cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _skv():
    from kv_cache_selection_b200 import statekv
    return statekv


def tokens(seed, S, n, H, d, dtype, loud=True):
    """k, v (or q, v) [S][n][H][d] on the CPU: normal, two loud channels, every
    7th token along one direction."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((S, n, H, d), generator=g)
    if loud:
        k[..., 3] *= 4
        k[..., d // 2 + 3] *= 4
    u = torch.randn(d, generator=g)
    k[:, ::7] += 4 * u / u.norm()
    v = torch.randn((S, n, H, d), generator=g)
    return k.to(DT[dtype]), v.to(DT[dtype])


def same(a, b):
    """torch.equal as a plain truth value (a failing assert prints no tensors)."""
    return bool(a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b))


def exact_tensor(x, dtype):
    """float64 values -> one float32 rounding -> the type."""
    return torch.from_numpy(np.asarray(x)).float().to(DT[dtype])


def check_attention(out, lse, want, dtype, p_step):
    w_out, w_lse, mass, span = want
    t = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    e = 2.0 ** -19 * span                                  # [Hq][n]
    lim = t * np.abs(w_out) + mass * (p_step + 2 * e.T[..., None] + (64 + want.keys / 16) * 2.0 ** -23)
    err = np.abs(O.to_f64(out.cpu()) - w_out)
    fine = bool(np.isfinite(err).all() and (err <= lim).all())
    assert fine, f"out: worst {np.max(err / lim):.3g} of its limit"
    if lse is not None:
        err = np.abs(O.to_f64(lse.cpu()) - w_lse)
        lim = e + 2.0 ** -20 + 2.0 ** -23 * np.abs(w_lse)
        fine = bool((err <= lim).all())
        assert fine, f"lse: worst {np.max(err / lim):.3g} of its limit"


class Want(tuple):
    keys = 0


def reference(q, k, v, past_k, past_v, window, n_sink):
    w = Want(O.window_attention(q, k, v, past_k, past_v, window, n_sink))
    w.keys = k.shape[0] + (0 if past_k is None else past_k.shape[0])
    return w


# ----------------------------------------------------------------- write, read
CASES = [
    # S, Hkv, d, capacity, start, n
    (1, 1, 64, 1, 0, 1),
    (1, 1, 128, 32, 0, 32),
    (2, 2, 64, 100, 3, 1),          # one token inside a block
    (1, 4, 128, 300, 31, 2),        # across a block border
    (3, 2, 128, 97, 0, 97),         # odd capacity, to its end
    (1, 3, 64, 1000, 517, 256),
    (2, 1, 128, 65, 64, 1),         # the last token of a block-and-a-bit
]


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,Hkv,d,cap,start,n", CASES)
def test_append_and_read_back(S, Hkv, d, cap, start, n, dtype):
    c = _skv().Q4Cache(Hkv, d, cap, n_streams=S)
    c.data.fill_(255)                                     # whatever was there
    old_k, old_v = tokens(1, S, cap, Hkv, d, dtype)
    c.append(old_k.cuda(), old_v.cuda(), 0)
    k, v = tokens(2, S, n, Hkv, d, dtype, loud=False)
    c.append(k.cuda(), v.cuda(), start)
    for t, new, old in zip(c.read(0, cap, dtype=dtype), (k, v), (old_k, old_v)):
        full = torch.cat([old[:, :start], new, old[:, start + n:]], 1)
        assert same(t.cpu(), exact_tensor(O.q4_held(full), dtype))
    other = "f32" if dtype == "bf16" else "bf16"
    for t, new in zip(c.read(start, n, dtype=other), (k, v)):
        assert same(t.cpu(), exact_tensor(O.q4_held(new), other))


@cuda
def test_append_values_next_to_borders():
    """Values midway between two codes, a float32 step to either side of it, and
    scales that sit on or next to a bfloat16 value."""
    g = np.random.default_rng(5)
    x = np.empty((40, 64), dtype=np.float32)
    for r in range(40):
        s = np.float32(O.bf16_grid(np.exp(g.uniform(-20, 20)), up=True))
        m = np.float32(O.bf16_grid(g.standard_normal() * s * 4, up=False))
        x[r] = m + (g.integers(0, 15, 64) + 0.5).astype(np.float32) * s
        x[r, ::3] = np.nextafter(x[r, ::3], np.float32(np.inf))
        x[r, 1::3] = np.nextafter(x[r, 1::3], np.float32(-np.inf))
        x[r, 0], x[r, 1] = m, m + np.float32(15) * s
        if r % 3 == 1:
            x[r, 1] = np.nextafter(x[r, 1], np.float32(np.inf))
        if r % 3 == 2:
            x[r, 0] = np.nextafter(x[r, 0], np.float32(-np.inf))
    k = torch.from_numpy(x).view(1, 40, 1, 64).cuda()
    c = _skv().Q4Cache(1, 64, 40)
    c.append(k, k, 0)
    for t in c.read(0, 40, dtype="f32"):
        assert same(t.cpu(), exact_tensor(O.q4_held(k.cpu()), "f32"))


@cuda
@pytest.mark.parametrize("d", [64, 128])
def test_append_extreme_groups(d):
    """Flat groups, tiny and huge magnitudes, NaN and infinities in one group."""
    k = torch.randn(1, 12, 1, d, generator=torch.Generator().manual_seed(3))
    k[0, 0] = 0.0
    k[0, 1] = -1.5
    k[0, 2] *= 1e-30
    k[0, 3] *= 1e30
    k[0, 4] = 3e38 * torch.sign(k[0, 4])
    k[0, 5, 0, 5] = float("nan")
    k[0, 6, 0, d - 1] = float("inf")
    k[0, 7, 0, 0] = -float("inf")
    k[0, 8] += 1000.0
    k[0, 9, 0, 1:] = 0.0
    k = k.cuda()
    c = _skv().Q4Cache(1, d, 12)
    c.append(k, -k, 0)
    for t, x in zip(c.read(0, 12, dtype="f32"), (k, -k)):
        want = exact_tensor(O.q4_held(x.cpu()), "f32")
        assert same(t.cpu().nan_to_num(nan=7e37), want.nan_to_num(nan=7e37))


@cuda
def test_starts_per_stream_and_rows_outside_the_cache():
    """A start per stream on the device; tokens before 0 or behind the capacity
    are dropped by append and left as they were by read."""
    S, Hkv, d, cap, n = 4, 2, 64, 70, 20
    c = _skv().Q4Cache(Hkv, d, cap, n_streams=S)
    old_k, old_v = tokens(1, S, cap, Hkv, d, "f32")
    c.append(old_k.cuda(), old_v.cuda(), 0)
    k, v = tokens(2, S, n, Hkv, d, "f32")
    starts = [-5, 13, 60, 2 ** 31 - 3]
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    c.append(k.cuda(), v.cuda(), at)
    full = [old_k.clone(), old_v.clone()]
    for s, p in enumerate(starts):
        for i in range(n):
            if 0 <= p + i < cap:
                full[0][s, p + i], full[1][s, p + i] = k[s, i], v[s, i]
    held = [exact_tensor(O.q4_held(f), "f32") for f in full]
    for t, h in zip(c.read(0, cap, dtype="f32"), held):
        assert same(t.cpu(), h)
    mark = [torch.full((S, n, Hkv, d), -77.0, device="cuda") for _ in range(2)]
    got = c.read(at, n, dtype="f32", k=mark[0], v=mark[1])
    for t, h in zip(got, held):
        for s, p in enumerate(starts):
            for i in range(n):
                want = h[s, p + i] if 0 <= p + i < cap else torch.full((Hkv, d), -77.0)
                assert same(t[s, i].cpu(), want)


# ---------------------------------------------------------------------- decode
DECODE = [
    # S, Hq, Hkv, d, length, n, window, n_sink
    (1, 1, 1, 64, 0, 1, 0, 0),            # nothing cached
    (1, 2, 1, 64, 1, 1, 0, 0),
    (1, 14, 2, 64, 128, 1, 0, 0),
    (1, 28, 4, 128, 777, 1, 0, 0),
    (1, 28, 4, 128, 545, 2, 0, 0),        # 14 rows of a KV head
    (2, 28, 4, 128, 333, 3, 0, 0),        # 21 rows
    (1, 14, 2, 64, 1000, 16, 0, 0),
    (1, 6, 6, 128, 300, 19, 0, 0),        # one head per KV head
    (3, 8, 1, 64, 161, 5, 0, 0),
    (1, 10, 2, 128, 600, 40, 0, 0),       # 200 rows
    (1, 4, 2, 64, 500, 1, 1, 0),          # the token alone
    (1, 4, 2, 64, 500, 3, 2, 0),
    (2, 14, 2, 64, 700, 3, 100, 4),
    (1, 28, 4, 128, 700, 5, 33, 70),      # sinks past a block
    (1, 28, 4, 128, 90, 20, 30, 200),     # sinks reach into the text
    (1, 7, 1, 128, 640, 30, 64, 1),
    (1, 7, 1, 128, 640, 30, 10, 0),       # text tokens that see no cached one
    (1, 130, 1, 64, 100, 1, 0, 0),        # 130 query heads on one KV head
    (1, 48, 12, 64, 5000, 17, 0, 0),      # several key tiles per block of the 128-row kernel
    (1, 40, 10, 128, 6007, 20, 0, 0),
    (2, 60, 20, 64, 3001, 9, 2000, 40),
]


def run_decode(S, Hq, Hkv, d, length, n, window, n_sink, dtype, ragged=False, seed=0):
    cap = length + 37
    c = _skv().Q4Cache(Hkv, d, cap, n_streams=S)
    c.data.fill_(255)                     # tokens behind the length: NaN scales, full codes
    pk, pv = tokens(seed + 1, S, max(length, 1), Hkv, d, dtype)
    if length:
        c.append(pk.cuda(), pv.cuda(), 0)
    k, v = tokens(seed + 2, S, n, Hkv, d, dtype)
    q, _ = tokens(seed + 3, S, n, Hq, d, dtype, loud=False)
    lens = [max(0, length - 41 * s) for s in range(S)] if ragged else [length] * S
    at = torch.tensor(lens, dtype=torch.int32, device="cuda") if ragged else length
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), at, window=window, n_sink=n_sink)
    hk, hv = O.q4_held(pk), O.q4_held(pv)
    wants = [reference(q[s], k[s], v[s], hk[s, :lens[s]], hv[s, :lens[s]], window, n_sink) for s in range(S)]
    return c, (q, k, v, at), out, lse, wants


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,Hq,Hkv,d,length,n,window,n_sink", DECODE)
def test_decode_matches_oracle(S, Hq, Hkv, d, length, n, window, n_sink, dtype):
    c, ins, out, lse, wants = run_decode(S, Hq, Hkv, d, length, n, window, n_sink, dtype)
    for s in range(S):
        check_attention(out[s], lse[s], wants[s], dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)
    again, _ = c.decode(ins[0].cuda(), ins[1].cuda(), ins[2].cuda(), ins[3], window=window, n_sink=n_sink)
    assert same(out, again)        # no order of arrival in any sum
    assert _skv().q4_status() == 0


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,window,n_sink", [(1, 0, 0), (4, 60, 5), (25, 0, 0)])
def test_decode_lengths_per_stream(n, window, n_sink, dtype):
    """Streams of lengths 130, 89, 48, 7 (and clipped values) in one call."""
    c, ins, out, lse, wants = run_decode(4, 8, 2, 64, 130, n, window, n_sink, dtype, ragged=True)
    for s in range(4):
        check_attention(out[s], lse[s], wants[s], dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)
    odd = torch.tensor([-4, 10 ** 9, 0, 130], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, c.capacity, 0, 130], dtype=torch.int32, device="cuda")
    pk, pv = tokens(9, 4, c.capacity, 2, 64, dtype)
    c.append(pk.cuda(), pv.cuda(), 0)
    a = c.decode(*(t.cuda() for t in ins[:3]), odd, window=window, n_sink=n_sink)
    b = c.decode(*(t.cuda() for t in ins[:3]), near, window=window, n_sink=n_sink)
    assert same(a[0], b[0]) and same(a[1], b[1])


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 30])
def test_decode_hidden_nan_has_no_influence(n, dtype):
    """NaN keys and values outside the window, and in text tokens a row does not
    see, leave the row's result as it is without them; rows that see one are NaN."""
    S, Hq, Hkv, d, L, window = 1, 14, 2, 64, 200, 50
    pk, pv = tokens(1, S, L, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    nan = float("nan")

    def run(pk, pv, k, v):
        c = _skv().Q4Cache(Hkv, d, L)
        c.append(pk.cuda(), pv.cuda(), 0)
        return c.decode(q.cuda(), k.cuda(), v.cuda(), L, window=window, n_sink=3)[0].cpu()

    clean = run(pk, pv, k, v)
    bk, bv = pk.clone(), pv.clone()
    bk[:, 4:L - window + 1] = nan
    bv[:, 4:L - window + 1] = nan
    bv[:, 100, 0, 2] = float("inf")
    assert same(run(bk, bv, k, v), clean)
    if n > 2:
        bk, bv, tk, tv = pk.clone(), pv.clone(), k.clone(), v.clone()
        hid = L - window + 10                 # the window of row i begins at L + i - window + 1
        bk[:, hid] = nan
        bv[:, hid] = nan
        tv[:, 20] = nan
        tk[:, 22] = nan
        got = run(bk, bv, tk, tv)
        assert same(got[:, 10:20], clean[:, 10:20])
        assert torch.isnan(got[:, :10]).all() and torch.isnan(got[:, 20:]).all()


@cuda
def test_decode_of_keys_with_wide_ranges():
    """Keys and values whose scale differs by orders of magnitude between tokens
    and heads; some tokens flat (s = 0)."""
    S, Hq, Hkv, d, L, n = 1, 14, 2, 128, 300, 2
    for dtype in ("f32", "bf16"):
        pk, pv = tokens(1, S, L, Hkv, d, dtype)
        f = torch.exp2(torch.randint(-12, 13, (1, L, 1, 1), generator=torch.Generator().manual_seed(8)).float())
        pv = (pv.float() * f).to(DT[dtype])
        pk = (pk.float() * torch.minimum(f, torch.ones(()))).to(DT[dtype])
        pk[:, 50], pv[:, 60] = 0.25, -3.0
        k, v = tokens(2, S, n, Hkv, d, dtype)
        q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
        c = _skv().Q4Cache(Hkv, d, L)
        c.append(pk.cuda(), pv.cuda(), 0)
        for nn in (1, n):
            out, lse = c.decode(q[:, :nn].contiguous().cuda(), k[:, :nn].contiguous().cuda(),
                                v[:, :nn].contiguous().cuda(), L)
            want = reference(q[0, :nn], k[0, :nn], v[0, :nn], O.q4_held(pk)[0], O.q4_held(pv)[0], 0, 0)
            check_attention(out[0], lse[0], want, dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)


@cuda
def test_decode_of_large_logits():
    """Logits of several hundred: the running maximum moves, early weights vanish;
    and rows whose logits are all far below zero."""
    S, Hq, Hkv, d, L, n = 1, 7, 1, 128, 400, 1
    for sign in (1.0, -1.0):
        g = torch.Generator().manual_seed(4)
        u = torch.ones(d) * sign
        q = torch.ones(S, n, Hq, d) * 4
        pk = torch.randn(S, L, Hkv, d, generator=g) * 0.2 + u * torch.linspace(1, 8, L)[None, :, None, None]
        pv = torch.randn(S, L, Hkv, d, generator=g)
        k, v = pk[:, :n].clone(), pv[:, :n].clone()
        if sign < 0:
            k = pk[:, -n:].clone()
        c = _skv().Q4Cache(Hkv, d, L)
        c.append(pk.cuda(), pv.cuda(), 0)
        out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), L)
        check_attention(out[0], lse[0], reference(q[0], k[0], v[0], O.q4_held(pk)[0], O.q4_held(pv)[0], 0, 0), "f32", 0.0)


@cuda
def test_decode_captured_in_a_graph_follows_device_lengths():
    """A generation loop captured once: each replay attends, appends its token
    and moves the device length; two graphs replayed in turn do not disturb one
    another."""
    S, Hq, Hkv, d, cap, steps = 2, 14, 2, 64, 96, 5
    dtype = "bf16"
    Q4 = _skv().Q4Cache
    loops = []
    for which in range(2):
        c = Q4(Hkv, d, cap, n_streams=S)
        pk, pv = tokens(10 + which, S, 60, Hkv, d, dtype)
        c.append(pk.cuda(), pv.cuda(), 0)
        lens0 = torch.tensor([60, 33], dtype=torch.int32)
        lens = lens0.cuda()
        q = torch.empty(S, 1, Hq, d, dtype=DT[dtype], device="cuda")
        k = torch.empty(S, 1, Hkv, d, dtype=DT[dtype], device="cuda")
        v = torch.empty_like(k)

        def step(c=c, q=q, k=k, v=v, lens=lens):
            r = c.decode(q, k, v, lens)
            c.append(k, v, lens)
            lens.add_(1)
            return r

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.zero_(), k.zero_(), v.zero_()
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out, lse = step()
        torch.cuda.current_stream().wait_stream(side)
        c.append(pk.cuda(), pv.cuda(), 0)
        lens.copy_(lens0)
        loops.append((graph, c, q, k, v, lens, out, lse, [list(pk), list(pv)], [60, 33]))
    for t in range(steps):
        fed = []
        for which, (graph, c, q, k, v, *_rest) in enumerate(loops):
            nk, nv = tokens(100 + 10 * t + which, S, 1, Hkv, d, dtype)
            nq, _ = tokens(200 + 10 * t + which, S, 1, Hq, d, dtype, loud=False)
            q.copy_(nq), k.copy_(nk), v.copy_(nv)
            fed.append((nq, nk, nv))
            graph.replay()
        torch.cuda.synchronize()
        for (graph, c, q, k, v, lens, out, lse, past, at), (nq, nk, nv) in zip(loops, fed):
            for s in range(S):
                pk, pv = past[0][s][:at[s]], past[1][s][:at[s]]
                check_attention(out[s], lse[s], reference(nq[s], nk[s], nv[s], O.q4_held(pk), O.q4_held(pv), 0, 0),
                                dtype, 2.0 ** -11)
                past[0][s], past[1][s] = torch.cat([pk, nk[s]]), torch.cat([pv, nv[s]])
                at[s] += 1
            assert lens.tolist() == at


@cuda
def test_decode_on_two_streams_at_once():
    """Two decodes of one cache on two streams share nothing but the cache."""
    c, ins, out, _, _ = run_decode(1, 28, 4, 128, 3000, 1, 0, 0, "bf16")
    q, k, v = (t.cuda() for t in ins[:3])
    q2 = torch.roll(q, 1, -2).contiguous()
    want2 = c.decode(q2, k, v, ins[3])[0].clone()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        o1, _ = c.decode(q, k, v, ins[3], stream=a)
        o2, _ = c.decode(q2, k, v, ins[3], stream=b)
        torch.cuda.synchronize()
        assert same(o1, out) and same(o2, want2)


@cuda
def test_decode_optional_outputs_and_leading_dimension():
    c, ins, out, lse, _ = run_decode(1, 4, 2, 64, 50, 2, 0, 0, "f32")
    q, k, v = (t.cuda() for t in ins[:3])
    o, z = c.decode(q[0], k[0], v[0], 50)
    assert o.shape == (2, 4, 64) and z.shape == (4, 2) and same(o, out[0]) and same(z, lse[0])
    mine, none = c.decode(q, k, v, 50, out=torch.empty_like(q), with_lse=False)
    assert none is None and same(mine, out)


@cuda
def test_cuda_refusals():
    S = _skv()
    c = S.Q4Cache(2, 64, 40)
    k = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(S.StateKVError, match="CAPACITY"):
        c.append(k, k, 38)
    with pytest.raises(S.StateKVError, match="CAPACITY"):
        c.read(40, 1)
    with pytest.raises(S.StateKVError, match="length"):
        c.decode(q, k, k, 41)
    for bad in (k.float(), k[:, :2], k.transpose(1, 2), k.cpu(), torch.zeros(1, 3, 1, 64, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            c.append(k, bad, 0)
    with pytest.raises(ValueError, match="contiguous"):
        c.append(torch.zeros(1, 2, 3, 64, device="cuda").transpose(1, 2), k.float(), 0)
    with pytest.raises(ValueError, match="int32|dtype"):
        c.append(k, k, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(S.StateKVError, match="window"):
        S.sink_window_prefill(q, k, k, 0)


# --------------------------------------------------------- sink-window prefill
PREFILL = [
    # S, n, Hq, Hkv, d, window, n_sink
    (1, 1, 1, 1, 64, 1, 0),
    (1, 5, 2, 1, 128, 1, 0),               # every token sees itself alone
    (1, 130, 4, 2, 64, 7, 3),
    (2, 257, 14, 2, 64, 64, 4),
    (1, 300, 28, 4, 128, 128, 16),
    (1, 400, 3, 3, 128, 1000, 0),          # window beyond the sequence: causal
    (1, 500, 4, 1, 64, 129, 200),          # sinks past a tile
    (3, 383, 6, 2, 128, 100, 1),
    (1, 700, 2, 2, 64, 256, 130),
    (1, 641, 2, 1, 128, 127, 640),         # sinks cover everything
]


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,n,Hq,Hkv,d,window,n_sink", PREFILL)
def test_sink_window_prefill_matches_oracle(S, n, Hq, Hkv, d, window, n_sink, dtype):
    k, v = tokens(1, S, n, Hkv, d, dtype)
    q, _ = tokens(2, S, n, Hq, d, dtype, loud=False)
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=n_sink)
    again, _ = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=n_sink)
    assert same(out, again)
    assert _skv().sink_window_status() == 0
    for s in range(S):
        want = reference(q[s], k[s], v[s], None, None, window, n_sink)
        check_attention(out[s], lse[s], want, dtype, 2.0 ** -8 if dtype == "bf16" else 0.0)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sink_window_prefill_wide_window_is_full_causal(dtype):
    n, Hq, Hkv, d = 333, 14, 2, 64
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    q, _ = tokens(2, 1, n, Hq, d, dtype, loud=False)
    out, lse = _skv().sink_window_prefill(q[0].cuda(), k[0].cuda(), v[0].cuda(), n)
    full, full_lse = _skv().full_causal_prefill(q[0].cuda(), k[0].cuda(), v[0].cuda())
    want = reference(q[0], k[0], v[0], None, None, 0, 0)
    for o, z in ((out, lse), (full, full_lse)):
        check_attention(o, z, want, dtype, 2.0 ** -8 if dtype == "bf16" else 0.0)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sink_window_prefill_hidden_nan_has_no_influence(dtype):
    """A token whose key and value are NaN or infinite changes the rows that see
    it and no other: neither earlier ones of its tile nor those whose window has
    passed it.  The bf16 kernel computes a row that shares a tile with such a
    value again with unrounded weights, so there the rows that do not see it are
    held to the limits of any result (unrounded weights are off by less than the
    2^-8 that they allow), the float32 rows to the very bits."""
    n, Hq, Hkv, d, window = 420, 4, 2, 64, 90
    k, v = tokens(1, 1, n, Hkv, d, dtype)
    q, _ = tokens(2, 1, n, Hq, d, dtype, loud=False)

    def run(k, v):
        return _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)[0].cpu()

    clean = run(k, v)
    bad_k, bad_v = k.clone(), v.clone()
    bad_v[:, 200] = float("nan")
    bad_v[:, 203, 0, 5] = float("inf")
    bad_k[:, 210] = float("nan")
    got = run(bad_k, bad_v)
    if dtype == "f32":
        assert same(got[:, :200], clean[:, :200])
        assert same(got[:, 210 + window:], clean[:, 210 + window:])
    want = O.window_attention(q[0], k[0], v[0], None, None, window, 2)
    for rows in (slice(0, 200), slice(210 + window, n)):
        part = Want((want[0][rows], want[1][:, rows], want[2][rows], want[3][:, rows]))
        part.keys = n
        check_attention(got[0, rows], None, part, dtype, 2.0 ** -8 if dtype == "bf16" else 0.0)
    assert torch.isnan(got[:, 200:200 + window]).all()
    assert torch.isnan(got[:, 210:210 + window]).all()
    assert torch.isinf(got[:, 203 + window - 1, 0, 5]).all() or torch.isnan(got[:, 203 + window - 1, 0, 5]).all()


@cuda
def test_sink_window_prefill_of_large_logits():
    """Sink logits hundreds above or below the window's."""
    n, Hq, Hkv, d = 300, 2, 1, 64
    for dtype in ("bf16", "f32"):
        for a, b in ((30.0, 1.0), (-30.0, 1.0), (1.0, -30.0)):
            g = torch.Generator().manual_seed(6)
            k = torch.randn(1, n, Hkv, d, generator=g) * 0.1 + b
            k[:, :4] = a + torch.randn(1, 4, Hkv, d, generator=g) * 0.1
            v = torch.randn(1, n, Hkv, d, generator=g)
            q = torch.ones(1, n, Hq, d)
            q, k, v = (t.to(DT[dtype]) for t in (q, k, v))
            out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), 40, n_sink=4)
            check_attention(out[0], lse[0], reference(q[0], k[0], v[0], None, None, 40, 4), dtype,
                            2.0 ** -8 if dtype == "bf16" else 0.0)


@cuda
def test_prefill_then_generate_over_the_cache():
    """The operators together: a sequence is prefilled with window and sinks, its
    keys and values go into the 4-bit cache, tokens are generated over it (same
    window), each appended after its step, and the cache is read back."""
    S, n, Hq, Hkv, d, window, n_sink, dtype = 2, 150, 14, 2, 64, 48, 4, "bf16"
    skv = _skv()
    k, v = tokens(1, S, n, Hkv, d, dtype)
    q, _ = tokens(2, S, n, Hq, d, dtype, loud=False)
    out, lse = skv.sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=n_sink)
    c = skv.Q4Cache(Hkv, d, n + 3, n_streams=S)
    c.append(k.cuda(), v.cuda(), 0)
    for s in range(S):
        check_attention(out[s], lse[s], reference(q[s], k[s], v[s], None, None, window, n_sink), dtype, 2.0 ** -8)
    for t in range(3):
        nk, nv = tokens(50 + t, S, 1, Hkv, d, dtype)
        nq, _ = tokens(60 + t, S, 1, Hq, d, dtype, loud=False)
        o, z = c.decode(nq.cuda(), nk.cuda(), nv.cuda(), n + t, window=window, n_sink=n_sink)
        for s in range(S):
            check_attention(o[s], z[s], reference(nq[s], nk[s], nv[s], O.q4_held(k[s]), O.q4_held(v[s]), window, n_sink),
                            dtype, 2.0 ** -11)
        c.append(nk.cuda(), nv.cuda(), n + t)
        k, v = torch.cat([k, nk], 1), torch.cat([v, nv], 1)
    for t, x in zip(c.read(0, n + 3), (k, v)):
        assert same(t.cpu(), exact_tensor(O.q4_held(x), dtype))


# ------------------------------------------------- a handle's detailed state D
def handles(S, T, frames, dtype, Hq=6, Hkv=2, d=64, B=40):
    skv = _skv()
    return [skv.StateKV(Hq, Hkv, d, T, B, frames + 1, dtype=dtype, n_streams=S, detailed=x) for x in ("native", "q4")]


def frame(seed, S, T, Hq, Hkv, d, dtype):
    k, v = tokens(seed, S, T, Hkv, d, dtype)
    q, _ = tokens(seed + 500, S, T, Hq, d, dtype, loud=False)
    pos = (torch.arange(T, dtype=torch.int32) + seed * T).expand(S, T).contiguous()
    return [t if S > 1 else t[0] for t in (q, k, v, pos)]


@cuda
@pytest.mark.parametrize("host", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,T", [(1, 37), (2, 64), (1, 1)])
def test_handle_with_detailed_state_in_4_bits(S, T, dtype, host):
    """Frames of 37, 64 and 1 tokens: every result of a step is the native
    handle's, bit for bit; D holds the rounded keys and values; a decode attends
    to them (with the 8-row and, in bf16, the 128-row kernel)."""
    Hq, Hkv, d, frames = 6, 2, 64, 3
    hs = handles(S, T, frames, dtype)
    seen = []
    for n in range(frames):
        ins = frame(n, S, T, Hq, Hkv, d, dtype)
        seen.append(ins)
        outs = []
        for h in hs:
            if host and n != 1:          # the second frame comes from device buffers
                pinned = [t.pin_memory() for t in ins]
                out = torch.empty_like(pinned[0]).pin_memory()
                h.prefill_frame_host(0, *pinned, out)
                torch.cuda.synchronize()
            else:
                out = h.prefill_frame(0, *(t.cuda() for t in ins)).cpu()
            outs.append(out)
        assert same(*outs)
        stats = [h.step_stats() for h in hs]
        assert same(stats[0]["lse"], stats[1]["lse"])
        C = [h.get_compressed(0) for h in hs]
        m = C[0]["len"]
        assert m == C[1]["len"]
        for key in ("k", "v", "pos", "score"):
            assert same(C[0][key][:, :, :m], C[1][key][:, :, :m]), key
    D0, D1 = (h.get_detailed(0) for h in hs)
    N = frames * T
    assert D0["len"] == D1["len"] == N and same(D0["pos"][:, :N], D1["pos"][:, :N])
    k, v = (torch.cat([(f[i] if S > 1 else f[i][None]) for f in seen], 1) for i in (1, 2))
    for got, x in zip(D1["cache"].read(0, N, dtype=dtype), (k, v)):
        assert same(got.cpu(), exact_tensor(O.q4_held(x), dtype))
    for n in (1, 9):
        nk, nv = tokens(70 + n, S, n, Hkv, d, dtype)
        nq, _ = tokens(80 + n, S, n, Hq, d, dtype, loud=False)
        ins = [t.cuda() if S > 1 else t[0].cuda() for t in (nq, nk, nv)]
        out, lse = hs[1].decode(0, *ins)
        again, _ = D1["cache"].decode(*ins, N)
        assert same(out, again)
        part, plse = D1["cache"].decode(*ins, N, window=20, n_sink=3)   # the borrowed cache, with a window
        for o, z, window, n_sink in ((out, lse, 0, 0), (part, plse, 20, 3)):
            for s in range(S):
                want = reference(nq[s], nk[s], nv[s], O.q4_held(k[s]), O.q4_held(v[s]), window, n_sink)
                check_attention(o[s] if S > 1 else o, z[s] if S > 1 else z, want, dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)
    assert hs[1].device_status() == 0 and _skv().q4_status() == 0
    for h in hs:
        h.close()


@cuda
def test_handle_decode_before_any_frame_and_format_refusals():
    skv = _skv()
    native, q4 = handles(1, 16, 2, "bf16")
    for h in (native, q4):
        h.reserve_layers(1)
    q, k, v, _ = (t.cuda() for t in frame(1, 1, 16, 6, 2, 64, "bf16"))
    a, b = (h.decode(0, q[:2].contiguous(), k[:2].contiguous(), v[:2].contiguous()) for h in (native, q4))
    assert q4.get_detailed(0)["len"] == 0
    assert q4.kernel_launches() == 1          # nothing to share out, nothing to merge
    want = reference(q[:2].cpu(), k[:2].cpu(), v[:2].cpu(), None, None, 0, 0)
    check_attention(b[0], b[1], want, "bf16", 2.0 ** -11)
    check_attention(a[0], a[1], want, "bf16", 2.0 ** -8)
    lib = skv.lib
    for h, fmt in ((native, 1), (q4, 0)):
        assert lib.statekv_set_detailed_format(h.handle, fmt) == -2     # a layer is there
        assert lib.statekv_set_detailed_format(h.handle, 7) == -1
    import ctypes
    p = ctypes.c_void_p()
    assert lib.statekv_get_detailed(q4.handle, 0, ctypes.byref(p), None, None, None) == -2
    assert lib.statekv_get_detailed(q4.handle, 0, None, None, ctypes.byref(p), None) == 0 and p.value
    assert lib.statekv_get_detailed_q4(native.handle, 0, ctypes.byref(p), None, None, None) == -2
    assert lib.statekv_get_detailed_q4(q4.handle, 3, None, None, None, None) == -1
    for h in (native, q4):
        h.close()


@cuda
def test_handle_decode_captured_in_a_graph():
    """A captured decode reads the handle's D and scratch; one that needs more
    scratch than there is is refused, and later growth leaves the graph's alone."""
    S, T, Hq, Hkv, d = 1, 50, 6, 2, 64
    skv = _skv()
    h = handles(S, T, 3, "bf16")[1]
    for n in range(3):
        h.prefill_frame(0, *(t.cuda() for t in frame(n, S, T, Hq, Hkv, d, "bf16")))
    q, k, v, _ = (t.cuda() for t in frame(9, S, T, Hq, Hkv, d, "bf16"))
    one = [t[:1].clone() for t in (q, k, v)]
    many = [t.contiguous() for t in (q, k, v)]
    before = h.kernel_launches()
    want = h.decode(0, *one)[0].clone()
    assert h.kernel_launches() == before + 1  # 150 tokens: a block per KV head
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            out, _ = h.decode(0, *one)
            with pytest.raises(skv.StateKVError, match="capture"):
                h.decode(0, *many)
    out.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert same(out, want)
    before = h.kernel_launches()
    h.decode(0, *many)                  # grows the scratch
    assert h.kernel_launches() == before + 2  # 150 rows of a KV head: splits and their merge
    one[0].mul_(2)
    want = h.decode(0, *one)[0].clone()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert same(out, want)
    h.close()


# ------------------------------------------------------------- longer sequences
@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (100, 75)])
def test_decode_of_many_text_tokens(window, n_sink, dtype):
    """150 text tokens (300 rows of a KV head) after 70 cached ones: most of what a
    row sees are text tokens."""
    c, ins, out, lse, wants = run_decode(2, 4, 2, 64, 70, 150, window, n_sink, dtype)
    for s in range(2):
        check_attention(out[s], lse[s], wants[s], dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)


@cuda
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32"), (128, "f32")])
def test_sink_window_prefill_gives_the_same_bits_again(d, dtype):
    """Enough blocks for every order of arrival: ten runs, one result."""
    k, v = tokens(1, 2, 2500, 2, d, dtype)
    q, _ = tokens(2, 2, 2500, 14, d, dtype, loud=False)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    first = _skv().sink_window_prefill(q, k, v, 300, n_sink=4)
    for _ in range(9):
        again = _skv().sink_window_prefill(q, k, v, 300, n_sink=4)
        assert same(first[0], again[0]) and same(first[1], again[1])
    assert _skv().sink_window_status() == 0


@cuda
@pytest.mark.parametrize("d", [64, 128])
def test_sink_window_prefill_f32_of_the_largest_values(d):
    """float32 values that no rounding up survives: 3.4e38 in a value (rows that see
    it are huge in one channel, the others untouched) and in a key that meets tiny
    queries (one dominant logit of 4e7), both inside and outside the window."""
    n, window, top = 300, 70, 3.4028e38
    k, v = tokens(1, 1, n, 1, d, "f32")
    q, _ = tokens(2, 1, n, 2, d, "f32", loud=False)
    clean = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)[0].cpu()
    v[0, 100, 0, 5] = top
    v[0, 131, 0, 9] = -top
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)
    check_attention(out[0], lse[0], reference(q[0], k[0], v[0], None, None, window, 2), "f32", 0.0)
    assert same(out[:, :100].cpu(), clean[:, :100]) and same(out[:, 131 + window:].cpu(), clean[:, 131 + window:])
    k[0, 60, 0, 7] = top
    q[0, 40:90] *= 1e-30
    q[0, 40:90, :, 7] = 1e-30
    out, lse = _skv().sink_window_prefill(q.cuda(), k.cuda(), v.cuda(), window, n_sink=2)
    w = reference(q[0], k[0], v[0], None, None, window, 2)
    rows = slice(0, 90)                    # the rows behind it meet 3.4e38 with queries of size 1
    part = Want((w[0][rows], w[1][:, rows], w[2][rows], w[3][:, rows]))
    part.keys = w.keys
    check_attention(out[0, rows], lse[0][:, rows], part, "f32", 0.0)


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,window,n_sink", [(1, 0, 0), (3, 0, 0), (3, 90, 5)])
def test_decode_is_the_same_on_either_side_of_a_kernel_border(n, window, n_sink, dtype):
    """300 cached tokens (one block per KV head), 799 (shared out and merged) and, in
    a cache whose lengths only the device knows, different ones."""
    S, Hq, Hkv, d = 2, 8, 2, 64
    pk, pv = tokens(1, S, 800, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    ins = [t.cuda() for t in (q, k, v)]
    c = _skv().Q4Cache(Hkv, d, 800, n_streams=S)
    c.append(pk.cuda(), pv.cuda(), 0)
    hk, hv = O.q4_held(pk), O.q4_held(pv)
    lens = torch.tensor([768, 0], dtype=torch.int32, device="cuda")
    for at, of in ((300, [300] * 2), (799, [799] * 2), (lens, [768, 0])):
        out, lse = c.decode(*ins, at, window=window, n_sink=n_sink)
        for s in range(S):
            want = reference(q[s], k[s], v[s], hk[s, :of[s]], hv[s, :of[s]], window, n_sink)
            check_attention(out[s], lse[s], want, dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)


@cuda
@pytest.mark.parametrize("d", [64, 128])
def test_decode_f32_of_a_long_cache_keeps_its_precision(d):
    """Long float32 sums: the weights are off by 2^-22 (the exponential), 2^-22 (two
    fp16 parts) and 2^-21 (the roundings of a logit of size 8) at most, 2^-20
    together, independent of the values they meet, so the result is off by no more
    relative to its norm; twice that leaves room for the sums over the blocks.  A
    bias of the sums would show as a multiple of it."""
    S, Hq, Hkv, L, n = 2, 14, 2, 32768, 1
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((S, L, Hkv, d), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((S, n, Hq, d), generator=g, device="cuda")
    c = _skv().Q4Cache(Hkv, d, L, n_streams=S)
    c.append(k, v, 0)
    tk, tv = (torch.randn((S, n, Hkv, d), generator=g, device="cuda") for _ in range(2))
    out, _ = c.decode(q, tk, tv, L)
    hk, hv = c.read(0, L, dtype="f32")
    K, V = (torch.cat([x, y], 1).double().repeat_interleave(Hq // Hkv, 2) for x, y in ((hk, tk), (hv, tv)))
    w = torch.softmax(torch.einsum("sihd,sjhd->shij", q.double(), K) / d ** 0.5, -1)
    want = torch.einsum("shij,sjhd->sihd", w, V)
    rel = ((out.double() - want).norm() / want.norm()).item()
    assert rel <= 2.0 ** -19, f"{rel:.3g}"


@cuda
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (200, 40)])
def test_decode_of_many_streams_of_different_lengths(window, n_sink, dtype):
    """75 streams, a third of them empty, the last ones too, shared out over the
    workers: every stream meets its own tokens."""
    S, Hq, Hkv, d, cap, n = 75, 4, 2, 64, 900, 1
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, cap + 1, (S,), generator=g, dtype=torch.int32)
    lens[::3] = 0
    lens[-2:] = 0
    pk, pv = tokens(1, S, cap, Hkv, d, dtype)
    k, v = tokens(2, S, n, Hkv, d, dtype)
    q, _ = tokens(3, S, n, Hq, d, dtype, loud=False)
    c = _skv().Q4Cache(Hkv, d, cap, n_streams=S)
    c.append(pk.cuda(), pv.cuda(), 0)
    out, lse = c.decode(q.cuda(), k.cuda(), v.cuda(), lens.cuda(), window=window, n_sink=n_sink)
    hk, hv = O.q4_held(pk), O.q4_held(pv)
    for s in range(S):
        L = int(lens[s])
        want = reference(q[s], k[s], v[s], hk[s, :L], hv[s, :L], window, n_sink)
        check_attention(out[s], lse[s], want, dtype, 2.0 ** -11 if dtype == "bf16" else 0.0)
