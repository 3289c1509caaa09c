"""Measured cases of the hybrid-layer operators: rotary positions, the gated recurrence, and
softmax attention over a sliding window with sinks.

A hybrid stack puts layers of softmax attention over a sliding window (and a few first tokens
that stay visible) between its linear-attention and gated-recurrence layers; the window's queries
and keys carry rotary positions.  Each case is one pass through one operator as a training step
or a serving loop calls it.  ``own`` false: plain forms in elementary torch operations, 32 bits.
``own`` true: the library's entry points.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's queries and keys of 128 sequences at their own far positions
        dict(name="rotary_decode", op="rotary", backward=False, dtype="bf16", B=128, Hq=32, Hk=8, N=1, d=128, rot=128,
             layout="half", scaling="ramp", factor=16.0, positions=True),
        # a training batch in 32 bits, half of each head rotated, packed documents, a ragged length
        dict(name="rotary_packed_f32", op="rotary", backward=False, dtype="f32", B=8, Hq=12, Hk=12, N=4093, d=64, rot=32,
             layout="interleaved", scaling="none", factor=1.0, positions=True),
        # gradients of a long context's queries and keys, frequencies scaled for its length
        dict(name="rotary_long_bwd", op="rotary", backward=True, dtype="bf16", B=1, Hq=32, Hk=8, N=65536, d=128, rot=128,
             layout="half", scaling="ramp", factor=8.0, positions=False),
        # one decode step of 128 sequences through a layer of 4096 channels
        dict(name="recurrence_step", op="recurrence", form="step", dtype="bf16", B=128, N=1, D=4096, initial=True),
        # an ordinary training batch: few channels, so the sequence itself has to be split
        dict(name="recurrence_fwd", op="recurrence", form="forward", dtype="bf16", B=4, N=2048, D=512, initial=False),
        # 32 bits, ragged in both directions, continued from an earlier segment's state
        dict(name="recurrence_fwd_odd_f32", op="recurrence", form="forward", dtype="f32", B=3, N=1021, D=333, initial=True),
        # gradients of a long segment at full width
        dict(name="recurrence_long_bwd", op="recurrence", form="backward", dtype="bf16", B=1, N=65536, D=4096,
             initial=True),
        # an ordinary training batch
        dict(name="window_fwd", op="window", form="forward", dtype="bf16", B=4, Hq=8, Hk=8, N=2048, d=64, window=512,
             sinks=4, ragged=False),
        # the prefill of one long prompt, heads shared four to one
        dict(name="window_long_fwd", op="window", form="forward", dtype="bf16", B=1, Hq=16, Hk=4, N=65536, d=128,
             window=2048, sinks=16, ragged=False),
        # gradients of a training sequence, heads shared four to one
        dict(name="window_bwd", op="window", form="backward", dtype="bf16", B=1, Hq=16, Hk=4, N=8192, d=128, window=1024,
             sinks=4, ragged=False),
        # gradients in 32 bits of a padded batch, no power of two anywhere
        dict(name="window_ragged_bwd_f32", op="window", form="backward", dtype="f32", B=3, Hq=6, Hk=2, N=509, d=32,
             window=100, sinks=3, ragged=True),
        # one decode step of 128 sequences on full caches
        dict(name="window_decode", op="window", form="decode", dtype="bf16", B=128, Hq=32, Hk=8, N=6000, d=128,
             window=2048, sinks=4, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "recurrence", "window", "window"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "rotary":
        d = rng.choice((32, 64, 128))
        Hk = rng.choice((1, 2, 4, 8))
        scaling = rng.choice(("none", "linear", "ntk", "ramp"))
        B = _log(rng, 1, 128)
        return dict(op=op, backward=rng.random() < 0.5, dtype=dtype, B=B, Hq=Hk * rng.choice((1, 2, 4)), Hk=Hk,
                    N=_log(rng, 1, max(2, 65536 // B)), d=d, rot=rng.choice((d, d // 2, d // 4)),
                    layout=rng.choice(("half", "interleaved")), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0, 32.0)), positions=rng.random() < 0.5)
    if op == "recurrence":
        form = rng.choice(("forward", "forward", "backward", "step"))
        B = _log(rng, 1, 128 if form == "step" else 16)
        top = 65536 if dtype == "bf16" else 32768
        return dict(op=op, form=form, dtype=dtype, B=B, N=1 if form == "step" else _log(rng, 1, top // B),
                    D=_log(rng, 17, 4096), initial=True if form == "step" else rng.random() < 0.5)
    form = rng.choice(("forward", "backward", "decode"))
    Hk = rng.choice((1, 2, 4))
    d = rng.choice((32, 64, 128))
    if form == "decode":
        return dict(op=op, form=form, dtype=dtype, B=_log(rng, 1, 128), Hq=Hk * rng.choice((1, 2, 4, 8)), Hk=Hk,
                    N=_log(rng, 1, 20000), d=d, window=_log(rng, 16, 2048), sinks=rng.choice((0, 1, 4, 16)),
                    ragged=rng.random() < 0.5)
    B = rng.choice((1, 1, 2, 3))
    top = 16384 if dtype == "bf16" else 2048
    N = _log(rng, 1, top // B)
    return dict(op=op, form=form, dtype=dtype, B=B, Hq=Hk * rng.choice((1, 2, 4)), Hk=Hk, N=N, d=d,
                window=_log(rng, 16, 2048), sinks=rng.choice((0, 1, 4, 16)), ragged=rng.random() < 0.3)


# ---------------------------------------------------------------------------------- the inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rotary_options(case):
    return dict(rot=case["rot"], layout=case["layout"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                original=4096, ramp=(1.0, 32.0), amplitude=1.0 if case["scaling"] != "ramp" else 0.1 * math.log(case["factor"]) + 1.0)


def prepare(case, seed):
    dev, t = "cuda", _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen).to(t)

    B, N = case["B"], case["N"]
    if case["op"] == "rotary":
        pos = None
        if case["positions"] and N == 1:  # every sequence at its own position
            pos = torch.randint(0, 65536, (B, 1), device=dev, generator=gen, dtype=torch.int32)
        elif case["positions"]:  # packed documents: positions start again
            length = torch.randint(1, N + 1, (B, 1), device=dev, generator=gen, dtype=torch.int32)
            pos = (torch.arange(N, device=dev, dtype=torch.int32)[None, :] % length).contiguous()
        return dict(case=case, q=normal(B, case["Hq"], N, case["d"]), k=normal(B, case["Hk"], N, case["d"]), positions=pos,
                    offset=0 if pos is not None else 1000, options=_rotary_options(case))
    if case["op"] == "recurrence":
        D = case["D"]
        shape = (B, D) if case["form"] == "step" else (B, N, D)
        alpha = torch.sigmoid(3.0 + 1.5 * torch.randn(shape, device=dev, generator=gen))
        if case["form"] != "step":  # a document boundary now and then closes every gate
            alpha *= (torch.rand((B, N, 1), device=dev, generator=gen) > 0.001).float()
        x = normal(*shape)
        h0 = torch.randn((B, D), device=dev, generator=gen) if case["initial"] else None
        state = dict(case=case, x=x, alpha=alpha, h0=h0)
        if case["form"] == "backward":
            state["h"] = _scan(alpha, x.float(), h0).to(t)
            state["dh"] = normal(*shape)
            state["dhN"] = torch.randn((B, D), device=dev, generator=gen) if case["initial"] else None
            del state["x"]
        return state
    d, Hq, Hk, W, S = case["d"], case["Hq"], case["Hk"], case["window"], case["sinks"]
    state = dict(case=case)
    if case["form"] == "decode":
        state.update(kc=normal(B, Hk, S + W, d), vc=normal(B, Hk, S + W, d), q=normal(B, Hq, d), k=normal(B, Hk, d),
                     v=normal(B, Hk, d))
        low = N // 2 if case["ragged"] else N
        state["pos"] = torch.randint(low, N + 1, (B,), device=dev, generator=gen, dtype=torch.int32)
        return state
    state.update(q=normal(B, Hq, N, d), k=normal(B, Hk, N, d), v=normal(B, Hk, N, d), lens=None)
    if case["ragged"]:
        state["lens"] = torch.randint(0, N + 1, (B,), device=dev, generator=gen, dtype=torch.int32)
    if case["form"] == "backward":
        o, lse = _window_forward(state)
        state.update(o=o, lse=lse, dout=normal(B, Hq, N, d))
    return state


# ---------------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "rotary":
        return _rotary(state, case)
    if case["op"] == "recurrence":
        return {"step": _step, "forward": _forward, "backward": _backward}[case["form"]](state)
    return {"forward": _window_forward, "backward": _window_backward, "decode": _window_decode}[case["form"]](state)


def _run_own(s, case):
    import causal_kernelized_attention_gb300 as la

    if case["op"] == "rotary":
        call = la.la_rotary_backward if case["backward"] else la.la_rotary_forward
        return call(s["q"], s["k"], positions=s["positions"], offset=s["offset"], **s["options"])
    if case["op"] == "recurrence":
        if case["form"] == "step":
            return la.la_recurrence_step(s["h0"], s["x"], s["alpha"]), s["h0"]
        if case["form"] == "forward":
            return la.la_recurrence_forward(s["x"], s["alpha"], h0=s["h0"])
        dx, dalpha, dh0 = la.la_recurrence_backward(s["alpha"], s["h"], s["dh"], h0=s["h0"], dhN=s["dhN"])
        return dx, dalpha, dh0
    W, S = case["window"], case["sinks"]
    if case["form"] == "forward":
        return la.la_window_forward(s["q"], s["k"], s["v"], W, sinks=S, lens=s["lens"])
    if case["form"] == "backward":
        return la.la_window_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], W, sinks=S, lens=s["lens"])
    return la.la_window_decode_step(s["kc"], s["vc"], s["q"], s["k"], s["v"], s["pos"], W, sinks=S), s["kc"], s["vc"]


# ---- rotary positions: pair (a, b) of a head turned by position * frequency
def _frequencies(o):
    i = torch.arange(0, o["rot"], 2, device="cuda", dtype=torch.float64)
    base = o["base"]
    if o["scaling"] == "ntk":
        base = base * o["factor"] ** (o["rot"] / max(o["rot"] - 2, 1))
    f = base ** (-i / o["rot"])
    if o["scaling"] == "linear":
        f = f / o["factor"]
    if o["scaling"] == "ramp":  # fast pairs keep their frequency, slow ones are interpolated
        lo, hi = o["ramp"]
        g = ((o["original"] * f / (2 * math.pi) - lo) / (hi - lo)).clamp(0, 1)
        f = f * (g + (1 - g) / o["factor"])
    return f


def _rotary(s, case):
    o = s["options"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(s["offset"], s["offset"] + case["N"], device="cuda")[None, :]
    angle = pos.double()[:, None, :, None] * _frequencies(o)  # angles of far positions need 64 bits
    cos, sin = (o["amplitude"] * angle.cos()).float(), (o["amplitude"] * angle.sin()).float()
    if case["backward"]:
        sin = -sin
    return _turn(s["q"], cos, sin, o), _turn(s["k"], cos, sin, o)


def _turn(x, cos, sin, o):
    rot = o["rot"]
    y = x.float()
    if o["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin, y[..., rot:]), -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        y = torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), y[..., rot:]), -1)
    return y.to(x.dtype)


# ---- gated recurrence: h_t = alpha_t h_{t-1} + x_t, each channel on its own
def _scan(alpha, x, h0):
    """All h_t in 32 bits by doubling: runs of 1, 2, 4, ... tokens joined pairwise."""
    h, a = x, alpha
    if h0 is not None:
        h = torch.cat((h[:, :1] + a[:, :1] * h0[:, None], h[:, 1:]), 1)
    n = 1
    while n < x.shape[1]:
        h, a = (torch.cat((h[:, :n], h[:, n:] + a[:, n:] * h[:, :-n]), 1),
                torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1))
        n *= 2
    return h


def _step(s):
    h = s["alpha"] * s["h0"] + s["x"].float()
    s["h0"].copy_(h)
    return h.to(s["x"].dtype), s["h0"]


def _forward(s):
    h = _scan(s["alpha"], s["x"].float(), s["h0"])
    return h.to(s["x"].dtype), h[:, -1].contiguous()


def _backward(s):
    a, dh = s["alpha"], s["dh"].float()
    later = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)  # the gate that the next token applies
    g = _scan(later.flip(1), dh.flip(1), s["dhN"]).flip(1)
    first = torch.zeros_like(a[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat((first, s["h"][:, :-1].float()), 1)
    return g.to(s["dh"].dtype), g * before, None if s["h0"] is None else a[:, 0] * g[:, 0]


# ---- softmax attention over a window and sinks
_ROWS = 128  # queries of one block of the band


def _band(s):
    """Blocks of _ROWS queries, each with the keys that its window can reach and the sinks:
    q [B,Hk,blocks,g*_ROWS,d], keys and values [B,Hk,blocks,sinks+span,d], the mask of what is
    visible [B,blocks,_ROWS,sinks+span], and the places of the keys [blocks,sinks+span]."""
    c = s["case"]
    B, Hq, Hk, N, d, W, S = (c[n] for n in ("B", "Hq", "Hk", "N", "d", "window", "sinks"))
    W, S = min(W, N), min(S, N)
    blocks = -(-N // _ROWS)
    back = -(-(W - 1) // _ROWS) * _ROWS
    place = (torch.arange(blocks, device="cuda")[:, None] * _ROWS + torch.arange(-back, _ROWS, device="cuda"))
    place = torch.cat((torch.arange(S, device="cuda").expand(blocks, S), place), 1)
    sink = torch.arange(place.shape[1], device="cuda") < S
    row = torch.arange(blocks * _ROWS, device="cuda").view(blocks, _ROWS, 1)
    j = place[:, None, :]
    seen = (j <= row) & (sink | ((j >= S) & (row - j < W)))
    n = torch.full((B,), N, device="cuda") if s["lens"] is None else s["lens"].clamp(0, N)
    seen = seen[None] & (row[None] < n[:, None, None, None])
    at = place.clamp(0, N - 1)
    q = _blocks(s["q"], Hk, blocks)
    return q, s["k"].float()[:, :, at], s["v"].float()[:, :, at], seen, at


def _blocks(x, Hk, blocks):
    """[B,Hq,N,d] -> [B,Hk,blocks,g*_ROWS,d] in 32 bits, short last blocks filled with zeros."""
    B, Hq, N, d = x.shape
    y = torch.zeros((B, Hq, blocks * _ROWS, d), device="cuda")
    y[:, :, :N] = x
    return y.view(B, Hk, Hq // Hk, blocks, _ROWS, d).transpose(2, 3).reshape(B, Hk, blocks, -1, d)


def _rows(y, Hq, N):
    """[B,Hk,blocks,g*_ROWS,d] -> [B,Hq,N,d]."""
    B, Hk, blocks, _, d = y.shape
    y = y.view(B, Hk, blocks, Hq // Hk, _ROWS, d).transpose(2, 3)
    return y.reshape(B, Hq, blocks * _ROWS, d)[:, :, :N]


def _scores(q, k, seen, g):
    z = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    return z.masked_fill_(~seen[:, None].repeat(1, 1, 1, g, 1), -math.inf)


def _window_forward(s):
    c = s["case"]
    q, k, v, seen, _ = _band(s)
    z = _scores(q, k, seen, c["Hq"] // c["Hk"])
    top = z.amax(-1, keepdim=True)
    safe = top.masked_fill(top == -math.inf, 0.0)
    p = (z - safe).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp_min(1e-30)
    lse = safe + total.log()
    return (_rows(o, c["Hq"], c["N"]).to(s["q"].dtype).contiguous(),
            _rows(lse, c["Hq"], c["N"])[..., 0].contiguous())


def _window_backward(s):
    c = s["case"]
    B, Hq, Hk, N, d = (c[n] for n in ("B", "Hq", "Hk", "N", "d"))
    q, k, v, seen, at = _band(s)
    blocks = q.shape[2]
    z = _scores(q, k, seen, Hq // Hk)
    lse = _blocks(s["lse"].masked_fill(s["lse"] == -math.inf, 0.0)[..., None], Hk, blocks)
    p = (z - lse).exp_()
    del z
    dout = _blocks(s["dout"], Hk, blocks)
    delta = (dout * _blocks(s["o"], Hk, blocks)).sum(-1, keepdim=True)
    dv = p.transpose(-1, -2) @ dout
    ds = p * (dout @ v.transpose(-1, -2) - delta) * (1.0 / math.sqrt(d))
    dq = _rows(ds @ k, Hq, N).to(s["q"].dtype).contiguous()
    dk = ds.transpose(-1, -2) @ q
    return dq, _join(dk, at, N).to(s["k"].dtype), _join(dv, at, N).to(s["v"].dtype)


def _join(y, at, N):
    """Sums the blocks' shares [B,Hk,blocks,span,d] at their keys' places: [B,Hk,N,d]."""
    B, Hk, blocks, span, d = y.shape
    out = torch.zeros((B, Hk, N, d), device="cuda")
    return out.index_add_(2, at.reshape(-1), y.reshape(B, Hk, blocks * span, d))


def _slots(pos, W, S):
    """Where token `pos` is kept, and which slots hold a visible token [B, S + W]."""
    pos = pos.long()[:, None]
    slot = torch.arange(S + W, device="cuda")[None, :]
    token = torch.where(slot < S, slot, pos - (pos - slot) % W)  # the last token of that slot up to pos
    seen = torch.where(slot < S, slot <= pos, token >= S)
    return torch.where(pos < S, pos, S + (pos - S) % W)[:, 0], seen


def _window_decode(s):
    c = s["case"]
    B, Hq, Hk, d, W, S = (c[n] for n in ("B", "Hq", "Hk", "d", "window", "sinks"))
    slot, seen = _slots(s["pos"], W, S)
    every = torch.arange(B, device="cuda")
    s["kc"][every, :, slot] = s["k"]
    s["vc"][every, :, slot] = s["v"]
    q = s["q"].float().view(B, Hk, Hq // Hk, d)
    z = (q @ s["kc"].float().transpose(-1, -2)) * (1.0 / math.sqrt(d))
    z = z.masked_fill(~seen[:, None, None, :], -math.inf)
    p = (z - z.amax(-1, keepdim=True)).exp()
    o = (p @ s["vc"].float()) / p.sum(-1, keepdim=True)
    return o.view(B, Hq, d).to(s["q"].dtype), s["kc"], s["vc"]


# ---------------------------------------------------------------------------------- the work
def _visible(N, W, S):
    """Pairs of a query and a key that it sees, in one sequence of N tokens."""
    W, S = min(W, N), min(S, N)
    band = W * (W + 1) // 2 + (N - W) * W
    # sinks that have left the window: for query p, those below p - W + 1
    out = max(0, N - W)
    full = max(0, out - S)
    return band + (out - full) * (out - full + 1) // 2 + full * S


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, N = case["B"], case["N"]
    if case["op"] == "rotary":
        n = B * (case["Hq"] + case["Hk"]) * N * case["d"]
        return {"bytes": 2 * n * e, "flops": 3 * n * case["rot"] // case["d"]}
    if case["op"] == "recurrence":
        n, first = B * N * case["D"], B * case["D"] * 4 * (1 if case["initial"] else 0)
        if case["form"] == "backward":  # alpha, h, dh in; dx, dalpha out
            return {"bytes": n * (4 + 3 * e + 4) + 3 * first, "flops": 3 * n}
        return {"bytes": n * (4 + 2 * e) + first + B * case["D"] * 4, "flops": 2 * n}
    d, Hq, Hk, W, S = case["d"], case["Hq"], case["Hk"], case["window"], case["sinks"]
    if case["form"] == "decode":
        slots = min(N + 1, S + W)
        return {"bytes": 2 * B * Hk * slots * d * e + 2 * B * (Hq + 2 * Hk) * d * e, "flops": 4 * B * Hq * slots * d}
    rows, keys, pairs = B * Hq * N * d * e, B * Hk * N * d * e, B * Hq * _visible(N, W, S)
    if case["form"] == "forward":
        return {"bytes": 2 * rows + 2 * keys + B * Hq * N * 4, "flops": 4 * d * pairs}
    return {"bytes": 4 * rows + 4 * keys + B * Hq * N * 4, "flops": 10 * d * pairs}


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits: rotations as complex products, the recurrence token by
    token (long ones in runs), attention over the whole masked square of one head at a time."""
    if case["op"] == "window" and case["form"] != "decode" and case["N"] > 8192:
        return None
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return [_rotary_exact(s[n], s, case) for n in ("q", "k")]
    if case["op"] == "recurrence":
        return _recurrence_exact(s, case)
    if case["form"] == "decode":
        return _decode_exact(s, case)
    return _window_exact(s, case)


def _rotary_exact(x, s, case):
    o, N, rot = s["options"], case["N"], case["rot"]
    freq = []
    for i in range(rot // 2):
        base = o["base"] * (o["factor"] ** (rot / max(rot - 2, 1)) if o["scaling"] == "ntk" else 1.0)
        f = math.exp(-2.0 * i / rot * math.log(base))
        if o["scaling"] == "linear":
            f /= o["factor"]
        elif o["scaling"] == "ramp":
            turns = o["original"] * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - o["ramp"][0]) / (o["ramp"][1] - o["ramp"][0])))
            f = keep * f + (1 - keep) * f / o["factor"]
        freq.append(-f if case["backward"] else f)
    pos = s["positions"]
    pos = pos.double() if pos is not None else s["offset"] + torch.arange(N, device="cuda", dtype=torch.float64)[None]
    angle = pos[:, None, :, None] * torch.tensor(freq, device="cuda", dtype=torch.float64)
    turn = torch.polar(torch.full_like(angle, o["amplitude"]), angle)
    y = x.double()
    head = y[..., :rot]
    if o["layout"] == "half":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        out = torch.cat((z.real, z.imag), -1)
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        out = torch.view_as_real(z).reshape(head.shape)
    return torch.cat((out, y[..., rot:]), -1)


def _runs_exact(a, x, first):
    """h_t = a_t h_{t-1} + x_t from `first`, in 64 bits: all runs of 256 tokens side by side from zero,
    with the products of their gates, then the runs one after the other."""
    B, N, D = x.shape
    L = min(N, 256)
    runs = -(-N // L)
    if runs * L > N:
        a = torch.cat((a, a.new_ones(B, runs * L - N, D)), 1)
        x = torch.cat((x, x.new_zeros(B, runs * L - N, D)), 1)
    h, p = x.double().view(B, runs, L, D), a.double().view(B, runs, L, D).clone()
    for t in range(1, L):
        h[:, :, t] += p[:, :, t] * h[:, :, t - 1]
        p[:, :, t] *= p[:, :, t - 1]
    carry = torch.zeros((B, D), device="cuda", dtype=torch.float64) if first is None else first.double()
    for r in range(runs):
        h[:, r] += p[:, r] * carry[:, None]
        carry = h[:, r, -1]
    return h.view(B, runs * L, D)[:, :N]


def _recurrence_exact(s, case):
    a = s["alpha"]
    if case["form"] == "step":
        h = torch.addcmul(s["x"].double(), a.double(), s["h0"].double())
        return h, h
    if case["form"] == "forward":
        h = _runs_exact(a, s["x"].double(), s["h0"])
        return h, h[:, -1]
    g = _runs_exact(torch.cat((torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]), 1), s["dh"].double().flip(1), s["dhN"])
    g = g.flip(1)
    da = torch.empty_like(g)
    da[:, 1:] = g[:, 1:] * s["h"][:, :-1].double()
    da[:, 0] = 0.0 if s["h0"] is None else g[:, 0] * s["h0"].double()
    return g, da, None if s["h0"] is None else a[:, 0].double() * g[:, 0]


def _window_exact(s, case):
    B, Hq, Hk, N, d, W, S = (case[n] for n in ("B", "Hq", "Hk", "N", "d", "window", "sinks"))
    i = torch.arange(N, device="cuda")
    see = (i[None, :] <= i[:, None]) & ((i[:, None] - i[None, :] < W) | (i[None, :] < S))
    back = case["form"] == "backward"
    o = torch.zeros((B, Hq, N, d), device="cuda", dtype=torch.float64)
    lse = torch.full((B, Hq, N), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros((B, Hk, N, d), device="cuda", dtype=torch.float64) for _ in "kv")
    for b in range(B):
        n = N if s["lens"] is None else int(s["lens"][b])
        for h in range(Hq if n else 0):
            kv = h // (Hq // Hk)
            q, k, v = s["q"][b, h, :n].double(), s["k"][b, kv, :n].double(), s["v"][b, kv, :n].double()
            z = torch.where(see[:n, :n], q @ k.T / math.sqrt(d), -math.inf)
            if not back:
                lse[b, h, :n] = torch.logsumexp(z, -1)
                o[b, h, :n] = torch.softmax(z, -1) @ v
                continue
            p = torch.exp(z - s["lse"][b, h, :n, None].double())
            do = s["dout"][b, h, :n].double()
            dv[b, kv, :n] += p.T @ do
            p *= (do @ v.T - (do * s["o"][b, h, :n].double()).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[b, h, :n] = p @ k
            dk[b, kv, :n] += p.T @ q
    return (dq, dk, dv) if back else (o, lse)


def _decode_exact(s, case):
    B, Hq, Hk, d, W, S = (case[n] for n in ("B", "Hq", "Hk", "d", "window", "sinks"))
    pos = s["pos"].tolist()
    o = torch.empty((B, Hq, d), device="cuda", dtype=torch.float64)
    kc, vc = s["kc"].double(), s["vc"].double()
    for b in range(B):
        tokens = [t for t in range(min(S, pos[b] + 1))] + list(range(max(S, pos[b] - W + 1), pos[b] + 1))
        slots = torch.tensor([t if t < S else S + (t - S) % W for t in tokens], device="cuda")
        kc[b, :, slots[-1]], vc[b, :, slots[-1]] = s["k"][b].double(), s["v"][b].double()
        k, v = (x[b][:, slots].repeat_interleave(Hq // Hk, 0) for x in (kc, vc))
        p = torch.softmax((k @ s["q"][b].double()[:, :, None])[..., 0] / math.sqrt(d), -1)
        o[b] = (p[:, None, :] @ v)[:, 0]
    return o, kc, vc
