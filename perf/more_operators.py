"""Measured cases of the gated delta rule and of group norm with an activation.

The delta rule is the linear-attention state with a correcting write: a token's value is stored less
what the decayed state already answers for its key.  Behind it, as behind the decayed forms, stands
a group norm of each token's heads with a gate; the same norm over positions and channels, channels
last, serves convolutional layers.  Each case is one pass through one operator as a training step
or a serving loop calls it.  ``own`` false: plain forms in elementary torch operations, 32 bits.
``own`` true: the library's entry points.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a single sequence through a small layer: latency alone
        dict(name="delta_step_one", op="delta", form="step", dtype="bf16", B=1, Hk=8, H=8, N=1, dk=64, dv=64, initial=True),
        # one decode step of 128 sequences, keys shared two to one
        dict(name="delta_step", op="delta", form="step", dtype="bf16", B=128, Hk=16, H=32, N=1, dk=128, dv=128, initial=True),
        # an ordinary training batch
        dict(name="delta_fwd", op="delta", form="forward", dtype="bf16", B=4, Hk=8, H=8, N=2048, dk=64, dv=64, initial=False),
        # the prefill of one long prompt's segment, continued from the state before it, a ragged length
        dict(name="delta_long_fwd", op="delta", form="forward", dtype="bf16", B=2, Hk=16, H=32, N=16381, dk=128, dv=128,
             initial=True),
        # 32 bits, narrow keys, wide values, a ragged length
        dict(name="delta_fwd_odd_f32", op="delta", form="forward", dtype="f32", B=3, Hk=5, H=5, N=1021, dk=32, dv=64,
             initial=True),
        # gradients of a training batch, keys shared two to one
        dict(name="delta_bwd", op="delta", form="backward", dtype="bf16", B=4, Hk=8, H=16, N=4096, dk=128, dv=128,
             initial=False),
        # gradients in 32 bits, no power of two in the lengths, through the first state and the last
        dict(name="delta_bwd_odd_f32", op="delta", form="backward", dtype="f32", B=2, Hk=3, H=6, N=509, dk=64, dv=32,
             initial=True),
        # the heads of a training batch behind the delta rule: a token's heads each by their root mean square, gated
        dict(name="norm_heads_fwd", op="norm", form="forward", dtype="bf16", B=4, L=4096, G=16, D=128, per_token=True,
             heads_first=True, center=False, gate=True, act="silu"),
        # its gradients
        dict(name="norm_heads_bwd", op="norm", form="backward", dtype="bf16", B=4, L=4096, G=16, D=128, per_token=True,
             heads_first=True, center=False, gate=True, act="silu"),
        # feature maps of 64 x 64 positions, channels last
        dict(name="norm_map_fwd", op="norm", form="forward", dtype="bf16", B=16, L=4096, G=32, D=16, per_token=False,
             heads_first=False, center=True, gate=False, act="silu"),
        # gradients of feature maps of 32 x 32 positions
        dict(name="norm_map_bwd", op="norm", form="backward", dtype="bf16", B=16, L=1024, G=32, D=40, per_token=False,
             heads_first=False, center=True, gate=False, act="silu"),
        # gradients in 32 bits, no power of two anywhere
        dict(name="norm_odd_bwd_f32", op="norm", form="backward", dtype="f32", B=3, L=777, G=11, D=30, per_token=False,
             heads_first=False, center=True, gate=False, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(hi, lo))))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if rng.random() < 0.55:
        form = rng.choice(("forward", "forward", "backward", "backward", "step"))
        Hk = rng.choice((1, 2, 3, 4, 8))
        H = Hk * rng.choice((1, 1, 2, 4))
        dk, dv = rng.choice((32, 64, 128)), rng.choice((32, 64, 128))
        B = _log(rng, 1, 128 if form == "step" else 4)
        tokens = (1 << 18 if dtype == "bf16" else 1 << 16) // (B * H)  # heads times tokens
        N = 1 if form == "step" else _log(rng, 1, min(16384, tokens))
        return dict(op="delta", form=form, dtype=dtype, B=B, Hk=Hk, H=H, N=N, dk=dk, dv=dv,
                    initial=True if form == "step" else rng.random() < 0.5)
    form = rng.choice(("forward", "backward"))
    per_token = rng.random() < 0.5
    if per_token:
        D, G = rng.choice((32, 64, 128, _log(rng, 8, 512))), _log(rng, 1, 32)
    else:
        D, G = rng.choice((8, 10, 16, 20, 30, 40, 64)), rng.choice((1, 4, 8, 32))
    B = _log(rng, 1, 16)
    return dict(op="norm", form=form, dtype=dtype, B=B, L=_log(rng, 1, min(16384, (1 << 25) // (B * G * D))), G=G, D=D,
                per_token=per_token, heads_first=per_token and rng.random() < 0.5, center=rng.random() < 0.6,
                gate=rng.random() < 0.5, act=rng.choice(("silu", "silu", "none")))


# ---------------------------------------------------------------------------------- the inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


def prepare(case, seed):
    dev, t = "cuda", _TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    B = case["B"]
    if case["op"] == "norm":
        L, G, D = case["L"], case["G"], case["D"]
        C = G * D
        s = dict(case=case, w=1.0 + 0.2 * normal(C), b=0.1 * normal(C) if case["center"] else None, gate=None)
        x = 1.5 * normal(B, L, G, D) + 0.3 * normal(B, 1, G, 1) + 0.2
        s["x"] = (x.transpose(1, 2) if case["heads_first"] else x.reshape(B, L, C)).contiguous().to(t)
        if case["gate"]:
            s["gate"] = normal(B, L, C).to(t)
        if case["form"] == "backward":  # the statistics that the forward pass left
            s["dy"] = normal(B, L, C).to(t)
            s["mean"], s["rstd"] = (y.contiguous() for y in _statistics(_by_group(s["x"].float(), case), case))
        return s
    Hk, H, N, dk, dv = (case[i] for i in ("Hk", "H", "N", "dk", "dv"))
    one = case["form"] == "step"

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(t)

    tokens = (B, H) if one else (B, H, N)
    s = dict(case=case, scale=dk ** -0.5, q=unit(*((B, Hk, dk) if one else (B, Hk, N, dk))),
             k=unit(*((B, Hk, dk) if one else (B, Hk, N, dk))), v=normal(*tokens, dv).to(t),
             beta=torch.sigmoid(normal(*tokens)))
    # a head's own rate times the token's step: gates from almost open to nearly closed
    rate = torch.exp(torch.rand((1, H) if one else (1, H, 1), device=dev, generator=gen) * math.log(16.0))
    s["g"] = -rate * torch.nn.functional.softplus(normal(*tokens) - 3.0)
    if not one:  # a document boundary now and then starts a new state
        s["g"].masked_fill_(torch.rand((B, 1, N), device=dev, generator=gen) < 0.0005, -math.inf)
    s["S0"] = 0.3 * normal(B, H, dk, dv) if case["initial"] else None
    if case["form"] == "backward":
        s["do"] = normal(*tokens, dv).to(t)
        s["dSN"] = 0.3 * normal(B, H, dk, dv) if case["initial"] else None
    return s


# ---------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "norm":
        return _norm_forward(s, case) if case["form"] == "forward" else _norm_backward(s, case)
    return {"step": _delta_step, "forward": _delta_forward, "backward": _delta_backward}[case["form"]](s)


def _run_own(s, case):
    import causal_kernelized_attention_gb300 as la
    if case["op"] == "norm":
        options = dict(w=s["w"], b=s["b"], gate=s["gate"], act=case["act"], eps=_EPS, per_token=case["per_token"],
                       heads_first=case["heads_first"], center=case["center"])
        if case["form"] == "forward":
            y, mean, rstd = la.la_group_norm_forward(s["x"], case["G"], **options)
            return dict(y=y, mean=mean if case["center"] else None, rstd=rstd)
        dx, dgate, dw, db = la.la_group_norm_backward(s["x"], case["G"], s["mean"], s["rstd"], s["dy"], **options)
        return dict(dx=dx, dgate=dgate, dw=dw, db=db)
    if case["form"] == "step":
        o = la.la_delta_step(s["S0"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"])
        return dict(o=o, S=s["S0"])
    if case["form"] == "forward":
        o, SN = la.la_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s["S0"], scale=s["scale"])
        return dict(o=o, SN=SN)
    got = la.la_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], S0=s["S0"], dSN=s["dSN"],
                               scale=s["scale"])
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got))


# ---------------------------------------------------------------------------------- plain: the delta rule
_C = 64  # tokens a chunk


def _shared(x, H):
    """Rows of the key heads, in 32 bits, for each of the H heads that read them."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _summed(x, Hk):
    """Gradients of the key heads: the sum over the heads that share them."""
    return x.reshape(x.shape[0], Hk, -1, *x.shape[2:]).sum(2)


def _delta_step(s):
    S, q, k = s["S0"], _shared(s["q"], s["v"].shape[1]), _shared(s["k"], s["v"].shape[1])
    S.mul_(s["g"].exp()[..., None, None])
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(2))
    S.add_(k[..., None] * u[:, :, None])
    return dict(o=((q[..., None] * S).sum(2) * s["scale"]).to(s["v"].dtype), S=S)


def _chunks(x):
    """[B, H, N, ...] as [B, H, chunks, _C, ...], zeros behind the last token."""
    n = -(-x.shape[2] // _C)
    y = x.new_zeros(x.shape[0], x.shape[1], n * _C, *x.shape[3:])
    y[:, :, :x.shape[2]] = x
    return y.reshape(x.shape[0], x.shape[1], n, _C, *x.shape[3:])


def _local(s):
    """What a chunk needs apart from the states: its rows, its decays, and (I + N diag(beta))^-1 with
    N_ij = exp(G_i - G_j) k_i . k_j below the diagonal (a product of powers, as N diag(beta) is nilpotent)."""
    H = s["v"].shape[1]
    q, k, v, beta = (_chunks(x) for x in (_shared(s["q"], H), _shared(s["k"], H), s["v"].float(), s["beta"]))
    G = _chunks(s["g"].clamp(min=-200.0).double()).cumsum(-1)  # sums in 64 bits: differences of large ones follow
    D = (G[..., :, None] - G[..., None, :]).float().exp().tril()
    N = (D * (k @ k.transpose(-1, -2))).tril(-1)
    A = N * beta[..., None, :]
    eye = torch.eye(_C, device=q.device)
    T, P, n = eye - A, A @ A, 2
    while n < _C:
        T, P, n = T + T @ P, P @ P, 2 * n
    first, last = G.float().exp(), (G[..., -1:] - G).float().exp()
    return q, k, v, beta, D, N, T, first, last, G[..., -1].float().exp()


def _states(k, v, beta, T, first, last, whole, S):
    """The state before each chunk, the errors E that the chunk writes (times beta), and the last state."""
    before, errors = [], []
    for c in range(k.shape[2]):
        before.append(S)
        E = T[:, :, c] @ (v[:, :, c] - first[:, :, c, :, None] * (k[:, :, c] @ S))
        S = whole[:, :, c, None, None] * S + k[:, :, c].transpose(-1, -2) @ ((last * beta)[:, :, c, :, None] * E)
        errors.append(E)
    return torch.stack(before, 2), torch.stack(errors, 2), S


def _initial(s, name):
    B, H, dv = s["v"].shape[0], s["v"].shape[1], s["v"].shape[-1]
    return s["v"].new_zeros((B, H, s["k"].shape[-1], dv), dtype=torch.float32) if s[name] is None else s[name]


def _rows(x, N):
    return x.flatten(2, 3)[:, :, :N]


def _delta_forward(s):
    q, k, v, beta, D, _, T, first, last, whole = _local(s)
    before, E, S = _states(k, v, beta, T, first, last, whole, _initial(s, "S0"))
    o = first[..., None] * (q @ before) + (D * (q @ k.transpose(-1, -2))) @ (beta[..., None] * E)
    return dict(o=(_rows(o, s["v"].shape[2]) * s["scale"]).to(s["v"].dtype), SN=S)


def _delta_backward(s):
    t, Hk, n = s["v"].dtype, s["k"].shape[1], s["v"].shape[2]
    q, k, v, beta, D, N, T, first, last, whole = _local(s)
    before, E, _ = _states(k, v, beta, T, first, last, whole, _initial(s, "S0"))
    do, dS = _chunks(s["do"].float()) * s["scale"], _initial(s, "dSN")
    QK = D * (q @ k.transpose(-1, -2))
    U = beta[..., None] * E
    # X = diag(beta) (v - first k S), U = (I + diag(beta) N)^-1 X: dX by the transposed inverse, which is
    # dU - N^T dY with dY = diag(beta) dX = (I + N diag(beta))^-T diag(beta) dU
    after, dX, dY = [], [], []
    for c in reversed(range(k.shape[2])):
        after.append(dS)
        dU = QK[:, :, c].transpose(-1, -2) @ do[:, :, c] + last[:, :, c, :, None] * (k[:, :, c] @ dS)
        y = T[:, :, c].transpose(-1, -2) @ (beta[:, :, c, :, None] * dU)
        dX.append(dU - N[:, :, c].transpose(-1, -2) @ y)
        dY.append(y)
        f = first[:, :, c, :, None]
        dS = whole[:, :, c, None, None] * dS + q[:, :, c].transpose(-1, -2) @ (f * do[:, :, c]) - k[:, :, c].transpose(-1, -2) @ (f * y)
    after, dX, dY = (torch.stack(x[::-1], 2) for x in (after, dX, dY))
    dP = (do @ U.transpose(-1, -2)).tril()
    dN = -(dY @ U.transpose(-1, -2)).tril(-1)
    rq = first[..., None] * (do @ before.transpose(-1, -2))
    rk = -first[..., None] * (dY @ before.transpose(-1, -2))
    wk = last[..., None] * (U @ after.transpose(-1, -2))
    M = D * dN
    dq = rq + (D * dP) @ k
    dk = rk + wk + (D * dP).transpose(-1, -2) @ q + M @ k + M.transpose(-1, -2) @ k
    # g_t stands in every decay that crosses from before t to t or later
    R = (QK * dP).tril(-1) + N * dN
    pairs = torch.nn.functional.pad(R.cumsum(-1), (1, 0))[..., :_C].tril().sum(-2)  # column t: sum over i >= t > j
    reads = ((q * rq).sum(-1) + (k * rk).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    writes = torch.nn.functional.pad((k * wk).sum(-1).cumsum(-1), (1, 0))[..., :_C]
    dg = pairs + reads + writes + (whole * (before * after).sum((-1, -2)))[..., None]
    return dict(dq=_summed(_rows(dq, n), Hk).to(t), dk=_summed(_rows(dk, n), Hk).to(t), dv=_rows(dY, n).to(t),
                dg=_rows(dg, n).contiguous(), dbeta=_rows((dX * E).sum(-1), n).contiguous(),
                dS0=None if s["S0"] is None else dS)


# ---------------------------------------------------------------------------------- plain: group norm
def _by_group(x, case):
    """[B, L, G, D] of either layout."""
    return x.transpose(1, 2) if case["heads_first"] else x.reshape(case["B"], case["L"], case["G"], case["D"])


def _statistics(x, case):
    """mean and 1 / sqrt(var + eps) of x [B, L, G, D]: [B, G], or [B, L, G] for each token alone."""
    over = (3,) if case["per_token"] else (1, 3)
    m = x.mean(over, keepdim=True) if case["center"] else torch.zeros_like(x.mean(over, keepdim=True))
    r = ((x - m).square().mean(over, keepdim=True) + _EPS).rsqrt()
    keep = (0, 1, 2) if case["per_token"] else (0, 2)
    return tuple(y.reshape([x.shape[i] for i in keep]) for y in (m, r))


def _spread(y, case):
    return y[..., None] if case["per_token"] else y[:, None, :, None]


def _act(z, case):
    return z * torch.sigmoid(z) if case["act"] == "silu" else z


def _act_slope(z, case):
    if case["act"] != "silu":
        return torch.ones_like(z)
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _norm_forward(s, case):
    x = _by_group(s["x"].float(), case)
    m, r = _statistics(x, case)
    z = ((x - _spread(m, case)) * _spread(r, case)).flatten(2) * s["w"]
    z = z if s["b"] is None else z + s["b"]
    y = _act(z, case) if s["gate"] is None else z * _act(s["gate"].float(), case)
    return dict(y=y.to(s["x"].dtype), mean=m if case["center"] else None, rstd=r)


def _norm_backward(s, case):
    t, m, r = s["x"].dtype, _spread(s["mean"], case), _spread(s["rstd"], case)
    h = (_by_group(s["x"].float(), case) - m) * r
    flat, dy = h.flatten(2), s["dy"].float()
    z = flat * s["w"] if s["b"] is None else flat * s["w"] + s["b"]
    if s["gate"] is None:
        dz, dgate = dy * _act_slope(z, case), None
    else:
        gate = s["gate"].float()
        dz, dgate = dy * _act(gate, case), (dy * z * _act_slope(gate, case)).to(t)
    dh = (dz * s["w"]).reshape(h.shape)
    over = (3,) if case["per_token"] else (1, 3)
    dx = dh - h * (dh * h).mean(over, keepdim=True)
    if case["center"]:
        dx = dx - dh.mean(over, keepdim=True)
    dx = (dx * r).to(t)
    dx = dx.transpose(1, 2).contiguous() if case["heads_first"] else dx.flatten(2)
    return dict(dx=dx, dgate=dgate, dw=(dz * flat).sum((0, 1)), db=None if s["b"] is None else dz.sum((0, 1)))


# ---------------------------------------------------------------------------------- the work of a pass
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["B"] * case["L"] * case["G"] * case["D"]
        if case["form"] == "forward":
            return dict(bytes=n * e * (3 if case["gate"] else 2), flops=10 * n)
        return dict(bytes=n * e * (5 if case["gate"] else 3), flops=20 * n)
    B, Hk, H, N, dk, dv = (case[i] for i in ("B", "Hk", "H", "N", "dk", "dv"))
    state = B * H * dk * dv * 4
    keys, values, gates = B * Hk * N * dk * e, B * H * N * dv * e, B * H * N * 4
    if case["form"] == "step":
        return dict(bytes=2 * state + 2 * keys + 2 * values + 2 * gates, flops=6 * B * H * dk * dv)
    if case["form"] == "forward":
        return dict(bytes=2 * keys + 2 * values + 2 * gates + (2 if case["initial"] else 1) * state,
                    flops=6 * B * H * N * dk * dv)
    return dict(bytes=4 * keys + 3 * values + 4 * gates + (3 if case["initial"] else 0) * state,
                flops=16 * B * H * N * dk * dv)


# ---------------------------------------------------------------------------------- 64 bits, by definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s, case)
    B, H, N, dk, dv = (case[i] for i in ("B", "H", "N", "dk", "dv"))
    if N * (1 if case["form"] == "forward" else 3) > 70000:
        return None
    wide = {i: None if x is None else x.double() for i, x in s.items() if i not in ("case", "scale")}
    for i in ("q", "k"):  # head h reads key head h // (H / Hk)
        wide[i] = torch.stack([wide[i][:, h // (H // case["Hk"])] for h in range(H)], 1)
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64, device="cuda") if wide["S0"] is None else wide["S0"].clone()
    alpha = wide["g"].exp()

    def token(t):
        pick = (slice(None), slice(None)) if case["form"] == "step" else (slice(None), slice(None), t)
        return [x[pick] for x in (wide["q"], wide["k"], wide["v"], wide["beta"], alpha)]

    def write(S, t):
        _, k, v, b, a = token(t)
        S = a[..., None, None] * S
        error = v - torch.einsum("bhk,bhkv->bhv", k, S)
        return S + torch.einsum("bhk,bhv->bhkv", k, b[..., None] * error), error

    if case["form"] != "backward":
        o = []
        for t in range(N):
            S, _ = write(S, t)
            o.append(torch.einsum("bhk,bhkv->bhv", token(t)[0], S) * s["scale"])
        return dict(o=o[0], S=S) if case["form"] == "step" else dict(o=torch.stack(o, 2), SN=S)
    marks, run_of = [], 64  # the state before every 64th token; the run between is made again on the way back
    for t in range(N):
        if t % run_of == 0:
            marks.append(S)
        S, _ = write(S, t)
    R = torch.zeros_like(S) if wide["dSN"] is None else wide["dSN"].clone()
    grads = [[] for _ in range(5)]
    for start in reversed(range(0, N, run_of)):
        run, S = [], marks.pop()
        for t in range(start, min(N, start + run_of)):
            after, error = write(S, t)
            run.append((t, S, after, error))
            S = after
        for t, S, after, error in reversed(run):
            q, k, _, b, a = token(t)
            do = wide["do"][:, :, t] * s["scale"]
            R = R + torch.einsum("bhk,bhv->bhkv", q, do)
            dq = torch.einsum("bhkv,bhv->bhk", after, do)
            dw = torch.einsum("bhk,bhkv->bhv", k, R)  # of the written value b * error
            decayed = a[..., None, None] * S
            derr = b[..., None] * dw
            dk = torch.einsum("bhkv,bhv->bhk", R, b[..., None] * error) - torch.einsum("bhkv,bhv->bhk", decayed, derr)
            Q = R - torch.einsum("bhk,bhv->bhkv", k, derr)
            for where, x in zip(grads, (dq, dk, derr, (Q * decayed).sum((-1, -2)), (dw * error).sum(-1))):
                where.append(x)
            R = a[..., None, None] * Q
    dq, dk, dv, dg, db = (torch.stack(x[::-1], 2) for x in grads)
    n = H // case["Hk"]
    dq, dk = (torch.stack([x[:, h:h + n].sum(1) for h in range(0, H, n)], 1) for x in (dq, dk))
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, dS0=None if wide["S0"] is None else R)


def _norm_exact(s, case):
    B, L, G, D = (case[i] for i in ("B", "L", "G", "D"))
    x = s["x"].double()
    x = x.permute(0, 2, 1, 3) if case["heads_first"] else x.view(B, L, G, D)
    over = (3,) if case["per_token"] else (1, 3)
    count = D if case["per_token"] else L * D
    w = s["w"].double().view(G, D)
    b = 0.0 if s["b"] is None else s["b"].double().view(G, D)
    gate = None if s["gate"] is None else s["gate"].double().view(B, L, G, D)

    def act(u):
        return u / (1 + torch.exp(-u)) if case["act"] == "silu" else u

    def slope(u):
        if case["act"] != "silu":
            return torch.ones_like(u)
        e = torch.exp(-u)
        return 1 / (1 + e) + u * e / (1 + e) ** 2

    if case["form"] == "forward":
        m = x.sum(over, keepdim=True) / count * (1.0 if case["center"] else 0.0)
        r = 1 / torch.sqrt(((x - m) ** 2).sum(over, keepdim=True) / count + _EPS)
        z = (x - m) * r * w + b
        y = act(z) if gate is None else z * act(gate)
        flat = (lambda u: u.reshape(B, L, G)) if case["per_token"] else (lambda u: u.reshape(B, G))
        return dict(y=y.reshape(B, L, G * D), mean=flat(m) if case["center"] else None, rstd=flat(r))
    shape = (B, L, G, 1) if case["per_token"] else (B, 1, G, 1)
    m, r = (s[i].double().view(shape) for i in ("mean", "rstd"))
    h = (x - m) * r
    z, dy = h * w + b, s["dy"].double().view(B, L, G, D)
    dz = dy * slope(z) if gate is None else dy * act(gate)
    dgate = None if gate is None else (dy * z * slope(gate)).reshape(B, L, G * D)
    dh = dz * w
    dx = dh - h * ((dh * h).sum(over, keepdim=True) / count)
    if case["center"]:
        dx = dx - dh.sum(over, keepdim=True) / count
    dx = dx * r
    return dict(dx=dx.permute(0, 2, 1, 3).contiguous() if case["heads_first"] else dx.reshape(B, L, G * D), dgate=dgate,
                dw=(dz * h).sum((0, 1)).reshape(-1), db=None if s["b"] is None else dz.sum((0, 1)).reshape(-1))
