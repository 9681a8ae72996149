"""Cases of the 4-bit cache and the sink-window operators, with their plain forms.

Four operators, used one after another by a program that keeps a long video's
keys and values in 4 bits:

  write    k, v of n new tokens are quantised into the cache (then read back,
           so that what the cache holds is compared as values);
  read     a range of cached tokens is read back as keys and values;
  decode   n text tokens attend over the cache, causally over themselves, with
           an optional sliding window and first tokens that stay visible;
  prefill  causal attention of a whole sequence with a sliding window and first
           tokens (sinks) that stay visible.

Quantisation: per token, head and group of 64 consecutive channels, the values
x become codes c in 0..15 with x ~ m + c * s.  m is the group's smallest value
rounded down to bfloat16, s = (largest - m) / 15 rounded up to bfloat16, c the
integer nearest to (x - m) / s (ties to even; 0 where s = 0).  Keys and values
are treated alike.
"""

import math

import torch

own = False

GROUP = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one 256-token video frame of an 8B-class layer joins a half-full cache: a call per frame and layer, latency counts
        dict(name="write_frame_8b", op="write", S=1, Hkv=4, d=128, n=256, cap=131072, start=65536, ragged=False, dtype="bf16"),
        # the detailed state of 512 such frames is turned into a 4-bit cache in one call
        dict(name="write_video_8b", op="write", S=1, Hkv=4, d=128, n=131072, cap=131072, start=0, ragged=False, dtype="bf16"),
        # an odd range of a 1B-class layer's cache, two streams that stand at different tokens, back in float32
        dict(name="read_1b_f32", op="read", S=2, Hkv=2, d=64, n=5001, cap=16384, start=37, ragged=True, dtype="f32"),
        # the whole cache of an 8B-class layer back in bf16
        dict(name="read_video_8b", op="read", S=1, Hkv=4, d=128, n=131072, cap=131072, start=0, ragged=False, dtype="bf16"),
        # one generated token over 64 frames of a 1B-class layer: the smallest decode, latency counts
        dict(name="decode_1b", op="decode", S=1, Hq=14, Hkv=2, d=64, n=1, length=16384, ragged=False, window=0, n_sink=0, dtype="bf16"),
        # one generated token over 512 frames of an 8B-class layer
        dict(name="decode_8b", op="decode", S=1, Hq=28, Hkv=4, d=128, n=1, length=131072, ragged=False, window=0, n_sink=0, dtype="bf16"),
        # a question of 16 tokens over the same cache
        dict(name="decode_8b_question", op="decode", S=1, Hq=28, Hkv=4, d=128, n=16, length=131072, ragged=False, window=0, n_sink=0, dtype="bf16"),
        # one token each for four streams of different lengths
        dict(name="decode_8b_streams", op="decode", S=4, Hq=28, Hkv=4, d=128, n=1, length=131072, ragged=True, window=0, n_sink=0, dtype="bf16"),
        # three text tokens in float32 that see the last 1000 tokens and four sinks
        dict(name="decode_1b_window_f32", op="decode", S=2, Hq=14, Hkv=2, d=64, n=3, length=16381, ragged=True, window=1000, n_sink=4, dtype="f32"),
        # an odd short sequence of a 1B-class layer in float32
        dict(name="prefill_1b_f32", op="prefill", S=1, Hq=14, Hkv=2, d=64, n=1111, window=300, n_sink=4, dtype="f32"),
        # four odd sequences of a 1B-class layer, window of four frames
        dict(name="prefill_1b_batch", op="prefill", S=4, Hq=14, Hkv=2, d=64, n=4001, window=1024, n_sink=8, dtype="bf16"),
        # 256 frames of an 8B-class layer as one sequence, a window as wide as the compressed state (4096) and 16 sinks
        dict(name="prefill_8b", op="prefill", S=1, Hq=28, Hkv=4, d=128, n=65536, window=4096, n_sink=16, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    S = rng.choice([1, 1, 2, 3, 4])
    if op in ("write", "read"):
        n = _log_int(rng, 1, min(131072, 131072 * 4 * 128 // (S * Hkv * d * (2 if dtype == "f32" else 1))))
        cap = n + _log_int(rng, 1, 4096)
        return dict(op=op, S=S, Hkv=Hkv, d=d, n=n, cap=cap, start=rng.randint(0, cap - n), ragged=rng.random() < 0.4, dtype=dtype)
    G = rng.choice([1, 2, 3, 4, 6, 7, 8])
    n_sink = rng.choice([0, 1, 4, 16, 130])
    if op == "decode":
        n = _log_int(rng, 1, 20)
        length = _log_int(rng, 1, min(131072, 4 * 131072 * 4 * 128 // (S * Hkv * d)))
        if dtype == "f32":
            length = min(length, 32768)
        window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        return dict(op=op, S=S, Hq=G * Hkv, Hkv=Hkv, d=d, n=n, length=length, ragged=rng.random() < 0.4, window=window,
                    n_sink=n_sink if window else 0, dtype=dtype)
    window = _log_int(rng, 1, 4096)
    n = _log_int(rng, 1, 3000 if dtype == "f32" else min(65536, 65536 * 28 * 128 // (S * G * Hkv * d)))
    return dict(op=op, S=S, Hq=G * Hkv, Hkv=Hkv, d=d, n=n, window=window, n_sink=n_sink, dtype=dtype)


# -------------------------------------------------------------------- inputs
def _offsets(case, most):
    """Where each stream stands: `most` (the start of a range, a length), or per-stream values up to it."""
    if not case["ragged"]:
        return [most] * case["S"]
    return [most - (most * s) // (2 * case["S"]) - (s % 2 if most > 1 else 0) for s in range(case["S"])]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _tokens(case, g, n):
    """k, v [S][n][Hkv][d]: normal, every 97th token a sink (k along one direction), two loud key channels."""
    shape = (case["S"], n, case["Hkv"], case["d"])
    u = _randn(g, case["d"])
    u /= u.norm()
    k = _randn(g, *shape)
    k[..., 3] *= 4.0
    k[..., case["d"] // 2 + 3] *= 4.0
    k[:, ::97] += 4.0 * u
    v = _randn(g, *shape)
    return k.to(TYPES[case["dtype"]]), v.to(TYPES[case["dtype"]]), u


def _inputs(case, seed):
    """The case's inputs as a dict of tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 12345)
    dt = TYPES[case["dtype"]]
    if case["op"] == "write":
        k, v, _ = _tokens(case, g, case["n"])
        return dict(k=k, v=v, at=_offsets(case, case["start"]))
    if case["op"] == "read":
        k, v, _ = _tokens(case, g, case["cap"])
        return dict(cached_k=k, cached_v=v, at=_offsets(case, case["start"]))
    if case["op"] == "decode":
        ck, cv, u = _tokens(case, g, case["length"])
        k, v, _ = _tokens(case, g, case["n"])
        q = _randn(g, case["S"], case["n"], case["Hq"], case["d"]) + 1.5 * u
        return dict(cached_k=ck, cached_v=cv, k=k, v=v, q=q.to(dt), at=_offsets(case, case["length"]))
    k, v, u = _tokens(case, g, case["n"])
    q = _randn(g, case["S"], case["n"], case["Hq"], case["d"]) + 1.5 * u
    return dict(q=q.to(dt), k=k, v=v)


def prepare(case, seed):
    x = _inputs(case, seed)
    st = dict(case=dict(case))
    st.update({name: x[name] for name in ("q", "k", "v") if name in x})
    if "at" in x:  # one number where the streams stand together, else a tensor on the device
        st["at"] = torch.tensor(x["at"], dtype=torch.int32, device="cuda") if case["ragged"] else x["at"][0]
    if case["op"] == "prefill":
        return st
    cap = case["length"] if case["op"] == "decode" else case["cap"]
    if own:
        from kv_cache_selection_b200.statekv import Q4Cache

        st["cache"] = Q4Cache(case["Hkv"], case["d"], cap, n_streams=case["S"])
        if "cached_k" in x:
            st["cache"].append(x["cached_k"], x["cached_v"], 0)
    elif "cached_k" in x:
        st["cache"] = [_quantise(x["cached_k"]), _quantise(x["cached_v"])]
    else:
        st["cache"] = [[torch.zeros((case["S"], cap, case["Hkv"], case["d"]), dtype=torch.uint8, device="cuda")]
                       + [torch.zeros((case["S"], cap, case["Hkv"], case["d"] // GROUP), device="cuda") for _ in range(2)]
                       for _ in range(2)]
    return st


# ---------------------------------------------------------------- plain forms
def _bf16_down(x):
    """float32 x rounded towards minus infinity to a bfloat16 value (still float32)."""
    b = x.view(torch.int32)
    low = (b & 0xFFFF) != 0
    b = (b & -0x10000) + torch.where((x < 0) & low, 0x10000, 0).to(torch.int32)
    return b.view(torch.float32)


def _quantise(x):
    """[codes uint8 (shape of x), s, m float32 (a value per group)] of x [..., d].  Codes and scales are decided in 64 bits: they sit next to borders."""
    xg = x.float().unflatten(-1, (-1, GROUP))
    m = _bf16_down(xg.amin(-1))
    s64 = (xg.amax(-1).double() - m.double()) / 15.0
    s = s64.float()
    s = torch.where(s.double() < s64, torch.nextafter(s, torch.full_like(s, math.inf)), s)
    s = -_bf16_down(-s)
    c = torch.round((xg.double() - m.double()[..., None]) / s.double()[..., None])
    c = torch.where(s[..., None] > 0, c, torch.zeros_like(c)).clamp(0, 15)
    return [c.to(torch.uint8).flatten(-2), s, m]


def _values(q4):
    """float32 values of [codes, s, m]."""
    c, s, m = q4
    return (m[..., None] + c.unflatten(-1, (-1, GROUP)).float() * s[..., None]).flatten(-2)


def _put(held, streams, rows, new):
    held[0][streams, rows], held[1][streams, rows], held[2][streams, rows] = new


def _rows(st, n):
    """Index [S][n] of the tokens that each stream's range holds."""
    at = st["at"]
    at = at.long()[:, None] if torch.is_tensor(at) else torch.full((st["case"]["S"], 1), at, device="cuda")
    return at + torch.arange(n, device="cuda")


def _attend(q, k, v, visible):
    """out, lse of q [.., n, Hq, d] over k, v [.., L, Hkv, d] in float32; visible broadcasts to [.., Hkv, G, n, L]."""
    n, Hq, d = q.shape[-3:]
    Hkv = k.shape[-2]
    qg = q.float().transpose(-3, -2).unflatten(-3, (Hkv, Hq // Hkv)).flatten(-3, -2)     # [.., Hkv, G*n, d]
    s = qg @ k.float().transpose(-3, -2).transpose(-2, -1)
    s = (s / math.sqrt(d)).unflatten(-2, (Hq // Hkv, n))
    s = s.masked_fill(~visible, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(-3, -2) @ v.float().transpose(-3, -2)).unflatten(-2, (Hq // Hkv, n)) / l
    lse = (top + torch.log(l)).squeeze(-1)
    return o.flatten(-4, -3).transpose(-3, -2), lse.flatten(-3, -2)


def _plain(st):
    c = st["case"]
    dt = TYPES[c["dtype"]]
    S, n = c["S"], c["n"]
    if c["op"] in ("write", "read"):
        rows = _rows(st, n)
        streams = torch.arange(S, device="cuda")[:, None]
        if c["op"] == "write":
            _put(st["cache"][0], streams, rows, _quantise(st["k"]))
            _put(st["cache"][1], streams, rows, _quantise(st["v"]))
        return [_values([part[streams, rows] for part in held]).to(dt) for held in st["cache"]]
    if c["op"] == "decode":
        L = c["length"]
        at = _rows(st, 1)                                                               # [S][1]: cached tokens
        j = torch.arange(L + n, device="cuda")
        i = torch.arange(n, device="cuda")[:, None]
        here = torch.where(j < L, j, at[:, None] + j - L)                               # [S][1][L + n]: positions
        place = at[:, None] + i                                                         # [S][n][1]
        ok = torch.where(j < L, j < at[:, None], j - L <= i)
        if c["window"]:
            ok = ok & ((here > place - c["window"]) | (here < c["n_sink"]))
        k = torch.cat([_values(st["cache"][0]), st["k"].float()], 1)
        v = torch.cat([_values(st["cache"][1]), st["v"].float()], 1)
        o, lse = _attend(st["q"], k, v, ok[:, None, None])
        return o.to(dt), lse
    # prefill: blocks of query rows with the keys that they can see, so that a long sequence fits
    out, lses = [], []
    block = 1024
    for i0 in range(0, n, block):
        i1 = min(n, i0 + block)
        w0 = max(0, i0 - c["window"] + 1)
        j = torch.cat([torch.arange(min(c["n_sink"], w0), device="cuda"), torch.arange(w0, i1, device="cuda")])
        i = torch.arange(i0, i1, device="cuda")[:, None]
        ok = (j <= i) & ((j > i - c["window"]) | (j < c["n_sink"]))
        o, lse = _attend(st["q"][:, i0:i1], st["k"][:, j], st["v"][:, j], ok)
        out.append(o.to(dt))
        lses.append(lse)
    return torch.cat(out, 1), torch.cat(lses, -1)


def run(st):
    if not own:
        return _plain(st)
    c = st["case"]
    if c["op"] == "write":
        st["cache"].append(st["k"], st["v"], st["at"])
        return st["cache"].read(st["at"], c["n"], dtype=c["dtype"])
    if c["op"] == "read":
        return st["cache"].read(st["at"], c["n"], dtype=c["dtype"])
    if c["op"] == "decode":
        return st["cache"].decode(st["q"], st["k"], st["v"], st["at"], window=c["window"], n_sink=c["n_sink"])
    from kv_cache_selection_b200.statekv import sink_window_prefill

    return sink_window_prefill(st["q"], st["k"], st["v"], c["window"], n_sink=c["n_sink"])


# ---------------------------------------------------------------------- work
def _pairs(n, first, window, n_sink):
    """Visible (query, key) pairs of n queries at positions first.. over all earlier tokens and themselves."""
    def causal(i):  # of the queries at positions 0 .. i-1
        return i * (i + 1) // 2

    last = first + n
    if not window:
        return causal(last) - causal(first)
    full = min(max(n_sink + window - 1, first), last)  # from here on a query sees window + n_sink tokens
    return causal(full) - causal(first) + (last - full) * (window + n_sink)


def work(case):
    c, es = case, BYTES[case["dtype"]]
    row = c["Hkv"] * (c["d"] // 2 + 4 * (c["d"] // GROUP))     # cached bytes of a token's keys (or values)
    if c["op"] in ("write", "read"):
        plain = 2 * c["S"] * c["n"] * c["Hkv"] * c["d"] * es
        packed = 2 * c["S"] * c["n"] * row
        return {"bytes": (2 * plain + 2 * packed) if c["op"] == "write" else plain + packed, "flops": 0}
    qo = 2 * c["S"] * c["n"] * c["Hq"] * c["d"] * es + 4 * c["S"] * c["n"] * c["Hq"]
    kv = 2 * c["S"] * c["n"] * c["Hkv"] * c["d"] * es
    if c["op"] == "decode":
        seen, pairs = 0, 0
        for at in _offsets(c, c["length"]):
            seen += at if not c["window"] else min(at, min(c["n_sink"], at) + max(0, min(at, c["window"] - 1)))
            pairs += _pairs(c["n"], at, c["window"], c["n_sink"])
        return {"bytes": qo + kv + 2 * seen * row, "flops": 4 * c["Hq"] * c["d"] * pairs}
    return {"bytes": qo + kv, "flops": 4 * c["S"] * c["Hq"] * c["d"] * _pairs(c["n"], 0, c["window"], c["n_sink"])}


# --------------------------------------------------------------------- exact
def _held_exact(x):
    """What the cache holds of x [..., d], in 64 bits, from the definition: brackets on the bfloat16 grid and a comparison with the two neighbours."""
    y = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)

    def grid(t):  # spacing of bfloat16 values at |t| (8 significant bits, subnormals below 2**-126)
        _, e = torch.frexp(t.abs())
        return torch.ldexp(torch.ones_like(t), torch.where(t == 0, torch.full_like(e, -133), (e - 8).clamp(min=-133)))

    low = y.min(-1, keepdim=True).values
    m = torch.floor(low / grid(low)) * grid(low)
    step = (y.max(-1, keepdim=True).values - m) / 15
    s = torch.ceil(step / grid(step)) * grid(step)
    t = torch.where(s > 0, (y - m) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    down = torch.floor(t)
    up = (t - down > 0.5) | ((t - down == 0.5) & (torch.remainder(down, 2) == 1))
    return (m + (down + up.double()).clamp(0, 15) * s).reshape(x.shape)


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    S, n, d = c["S"], c["n"], c["d"]
    if c["op"] == "write":
        return [_held_exact(x["k"]), _held_exact(x["v"])]
    if c["op"] == "read":
        return [torch.stack([_held_exact(t[s, at:at + n]) for s, at in enumerate(x["at"])]) for t in (x["cached_k"], x["cached_v"])]
    outs, lses = [], []
    for s in range(S):
        first = 0
        k, v = x["k"][s].double(), x["v"][s].double()
        if c["op"] == "decode":
            first = x["at"][s]
            k = torch.cat([_held_exact(x["cached_k"][s, :first]), k])
            v = torch.cat([_held_exact(x["cached_v"][s, :first]), v])
        o = torch.empty((n, c["Hq"], d), dtype=torch.float64, device="cuda")
        z = torch.empty((c["Hq"], n), dtype=torch.float64, device="cuda")
        for i0 in range(0, n, 512):
            i = torch.arange(first + i0, first + min(n, i0 + 512), device="cuda")
            j = torch.arange(0, int(i[-1]) + 1, device="cuda")
            if c["window"]:
                j = j[(j < c["n_sink"]) | (j > int(i[0]) - c["window"])]
            hide = j[None, :] > i[:, None]
            if c["window"]:
                hide |= (j[None, :] <= i[:, None] - c["window"]) & (j[None, :] >= c["n_sink"])
            for h in range(c["Hq"]):
                g = h // (c["Hq"] // c["Hkv"])
                a = torch.einsum("id,jd->ij", x["q"][s, i0:i0 + len(i), h].double(), k[j, g]) * d ** -0.5
                a[hide] = -math.inf
                z[h, i0:i0 + len(i)] = torch.logsumexp(a, 1)
                o[i0:i0 + len(i), h] = torch.softmax(a, 1) @ v[j, g]
        outs.append(o)
        lses.append(z)
    return torch.stack(outs), torch.stack(lses)
