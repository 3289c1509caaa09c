"""The gated delta rule's and group norm's entry points refuse bad arguments before touching the GPU (CPU only:
every call here fails validation or is an empty problem, so no pointer is followed), and the float64 forms that the GPU
tests compare with agree with differences."""
import ctypes

import pytest

import causal_kernelized_attention_gb300 as la
from causal_kernelized_attention_gb300 import build as la_build
from causal_kernelized_attention_gb300._binding import GroupNormSpec

torch = pytest.importorskip("torch")

from delta_ref import delta, delta_inputs, norm_backward, norm_forward  # noqa: E402

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
F32, BF16 = 0, 1
NAN, INF = float("nan"), float("inf")


def at(i):
    """Made-up addresses 16 MB apart, never followed."""
    return 0x10000000 + i * 0x1000000


@pytest.fixture(scope="module")
def lib():
    la_build.build()
    return la.load_library()


def forward(lib, **kw):
    f = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), S0=at(5), o=at(6), SN=at(7), B=1, Hk=2, H=4, N=100, dk=64, dv=64,
             scale=0.125, dtype=BF16)
    f.update(kw)
    return lib.la_delta_forward(*f.values(), None)


def backward(lib, **kw):
    f = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), S0=at(5), dout=at(6), dSN=at(7), dq=at(8), dk=at(9), dv=at(10),
             dg=at(11), dbeta=at(12), dS0=at(13), B=1, Hk=2, H=4, N=100, d_k=64, d_v=64, scale=0.125, dtype=BF16)
    f.update(kw)
    return lib.la_delta_backward(*f.values(), None)


def step(lib, **kw):
    f = dict(S=at(0), q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), o=at(6), B=2, Hk=2, H=4, dk=64, dv=64, scale=1.0, dtype=BF16)
    f.update(kw)
    return lib.la_delta_step(*f.values(), None)


def test_delta_forward(lib):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(o=None), dict(B=-1), dict(N=-1),
                dict(H=-4), dict(Hk=3), dict(Hk=0), dict(dtype=2), dict(scale=NAN), dict(scale=INF), dict(o=at(2)), dict(SN=at(5)),
                dict(o=at(0) + 64), dict(SN=at(6) + 16), dict(SN=at(3))):
        assert forward(lib, **bad) == INVALID, bad
    for bad in (dict(q=at(0) + 8), dict(o=at(6) + 2), dict(S0=at(5) + 4), dict(g=at(3) + 2), dict(beta=at(4) + 1)):
        assert forward(lib, **bad) == MISALIGNED, bad
    for bad in (dict(dk=48), dict(dv=256), dict(dk=16), dict(N=(1 << 30) + 1), dict(B=1 << 20, H=1 << 10, Hk=1 << 10)):
        assert forward(lib, **bad) == UNSUPPORTED, bad
    for empty in (dict(B=0), dict(H=0, Hk=0), dict(dk=0), dict(dv=0), dict(N=0, SN=None)):
        assert forward(lib, q=None, k=None, v=None, g=None, beta=None, o=None, **empty) == OK, empty


def test_delta_backward(lib):
    for name in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta"):
        assert backward(lib, **{name: None}) == INVALID, name
    for bad in (dict(dq=at(0)), dict(dk=at(8)), dict(dv=at(6)), dict(dg=at(3)), dict(dbeta=at(11) + 4), dict(dS0=at(7)), dict(dS0=at(5)),
                dict(scale=NAN), dict(Hk=3), dict(dtype=7), dict(N=-5)):
        assert backward(lib, **bad) == INVALID, bad
    for bad in (dict(dq=at(8) + 8), dict(dS0=at(13) + 4), dict(dg=at(11) + 2), dict(dSN=at(7) + 8)):
        assert backward(lib, **bad) == MISALIGNED, bad
    for bad in (dict(d_k=33), dict(d_v=512)):
        assert backward(lib, **bad) == UNSUPPORTED, bad
    none = {n: None for n in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta")}
    for empty in (dict(B=0), dict(d_k=0), dict(d_v=0), dict(N=0, dS0=None)):
        assert backward(lib, **none, **empty) == OK, empty


def test_delta_step(lib):
    for name in ("S", "q", "k", "v", "g", "beta", "o"):
        assert step(lib, **{name: None}) == INVALID, name
    for bad in (dict(o=at(3)), dict(o=at(0) + 32), dict(S=at(1)), dict(Hk=3), dict(dtype=-1), dict(scale=INF)):
        assert step(lib, **bad) == INVALID, bad
    assert step(lib, S=at(0) + 4) == MISALIGNED and step(lib, beta=at(5) + 2) == MISALIGNED
    assert step(lib, dk=96) == UNSUPPORTED
    assert step(lib, B=0) == OK and step(lib, dv=0) == OK


def spec(**kw):
    f = dict(groups=4, per_token=0, heads_first=0, center=1, act=1, eps=1e-5)
    f.update(kw)
    return GroupNormSpec(*f.values())


def norm(lib, s=None, **kw):
    f = dict(x=at(0), gate=at(1), w=at(2), b=at(3), y=at(4), mean=at(5), rstd=at(6))
    z = dict(B=2, L=10, C=64, dtype=BF16)
    f.update({k: v for k, v in kw.items() if k in f})
    z.update({k: v for k, v in kw.items() if k in z})
    return lib.la_group_norm_forward(*f.values(), ctypes.byref(spec() if s is None else s), *z.values(), None)


def norm_back(lib, s=None, **kw):
    f = dict(x=at(0), gate=at(1), w=at(2), b=at(3), mean=at(4), rstd=at(5), dy=at(6), dx=at(7), dgate=at(8), dw=at(9), db=at(10))
    z = dict(B=2, L=10, C=64, dtype=BF16)
    f.update({k: v for k, v in kw.items() if k in f})
    z.update({k: v for k, v in kw.items() if k in z})
    return lib.la_group_norm_backward(*f.values(), ctypes.byref(spec() if s is None else s), *z.values(), None)


def test_group_norm(lib):
    for call in (norm, norm_back):
        for bad in (dict(groups=0), dict(groups=5), dict(per_token=2), dict(heads_first=1), dict(center=-1), dict(act=2), dict(eps=-1.0),
                    dict(eps=NAN), dict(eps=INF)):
            assert call(lib, spec(**bad)) == INVALID, (call, bad)
        for bad in (dict(x=None), dict(B=-1), dict(L=-1), dict(C=-64), dict(dtype=3)):
            assert call(lib, **bad) == INVALID, (call, bad)
        assert call(lib, x=at(0) + 8) == MISALIGNED and call(lib, w=at(2) + 2) == MISALIGNED
        assert call(lib, spec(groups=1, per_token=1, heads_first=1), C=1024) == UNSUPPORTED
        assert call(lib, L=(1 << 30) + 1) == UNSUPPORTED
    for bad in (dict(y=None), dict(y=at(0)), dict(y=at(1) + 16), dict(mean=at(6)), dict(rstd=at(2))):
        assert norm(lib, **bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dx=None), dict(rstd=None), dict(mean=None), dict(dgate=None), dict(dx=at(6)), dict(dgate=at(7)),
                dict(dw=at(10)), dict(db=at(5))):
        assert norm_back(lib, **bad) == INVALID, bad
    assert lib.la_group_norm_forward(at(0), None, None, None, at(4), None, None, None, 1, 1, 4, F32, None) == INVALID
    for empty in (dict(B=0), dict(L=0), dict(C=0)):
        assert norm(lib, x=None, y=None, **empty) == OK, empty
        assert norm_back(lib, x=None, dy=None, dx=None, dgate=None, dw=None, db=None, **empty) == OK, empty


def test_python_checks_shapes_and_types():
    f32, bf = torch.float32, torch.bfloat16
    q, v, g = torch.zeros(1, 2, 8, 64, dtype=bf), torch.zeros(1, 4, 8, 32, dtype=bf), torch.zeros(1, 4, 8)
    for bad in (dict(k=q[:, :1]), dict(v=v[:, :, :4]), dict(g=g[:, :2]), dict(beta=g.double()), dict(S0=torch.zeros(1, 4, 64, 64)),
                dict(q=q[0])):
        a = dict(q=q, k=q, v=v, g=g, beta=g, S0=None)
        a.update(bad)
        with pytest.raises(ValueError):
            la.la_delta_forward(**a)
    with pytest.raises(ValueError):  # on the CPU
        la.la_delta_forward(q, q, v, g, g)
    x = torch.zeros(2, 5, 12, dtype=f32)
    for bad in (dict(groups=0), dict(act="relu"), dict(w=torch.zeros(3)), dict(gate=x[:, :2]), dict(heads_first=True)):
        with pytest.raises(ValueError):
            la.la_group_norm_forward(x, **{"groups": 3, **bad})
    with pytest.raises(ValueError):
        la.la_group_norm_backward(x, 3, None, torch.zeros(2, 3), x)
    with pytest.raises(TypeError):
        la.la_group_norm_forward(x, 2.5)


def test_reference_gradients_agree_with_differences():
    s = delta_inputs(1, 1, 1, 2, 9, 4, 3, torch.float64, True, (4,))
    s = {n: None if x is None else x.double() for n, x in s.items()}
    r = delta(s, 0.5)

    def loss(changed):
        o = delta(changed, 0.5, backward=False)
        return float((o["o"] * s["dout"]).sum() + (o["SN"] * s["dSN"]).sum())

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("S0", "dS0"), ("g", "dg")):
        for i in range(0, s[name].numel(), 5):
            if name == "g" and i % 9 == 4:
                continue  # the reset: -inf has no neighbours
            x = [s[name].clone() for _ in range(2)]
            x[0].view(-1)[i] += 1e-6
            x[1].view(-1)[i] -= 1e-6
            d = (loss({**s, name: x[0]}) - loss({**s, name: x[1]})) / 2e-6
            assert abs(d - float(r[grad].reshape(-1)[i])) < 1e-7 * (1 + abs(d)), (name, i)


@pytest.mark.parametrize("per_token,heads_first,center,gated", [(True, True, False, True), (True, False, True, False), (False, False, True, True)])
def test_norm_reference_gradients_agree_with_autograd(per_token, heads_first, center, gated):
    gen = torch.Generator().manual_seed(3)
    B, L, G, D = 2, 3, 2, 4
    x = torch.randn((B, G, L, D) if heads_first else (B, L, G * D), generator=gen, dtype=torch.float64).requires_grad_()
    w, b = (torch.randn(G * D, generator=gen, dtype=torch.float64).requires_grad_() for _ in range(2))
    gate = torch.randn((B, L, G * D), generator=gen, dtype=torch.float64).requires_grad_() if gated else None
    dy = torch.randn((B, L, G * D), generator=gen, dtype=torch.float64)
    (y, _), (mean, _), (rstd, _) = norm_forward(x, G, w, b, gate, "silu", 1e-5, per_token, heads_first, center)
    y.backward(dy)
    dx, dgate, dw, db = norm_backward(x.detach(), G, mean.detach(), rstd.detach(), dy, w.detach(), b.detach(),
                                      None if gate is None else gate.detach(), "silu", per_token, heads_first, center)
    for got, want in ((dx, x.grad), (dw, w.grad), (db, b.grad)) + (((dgate, gate.grad),) if gated else ()):
        assert torch.allclose(got[0], want, rtol=1e-9, atol=1e-9)
