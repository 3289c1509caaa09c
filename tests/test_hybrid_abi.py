"""The hybrid-layer entry points refuse bad arguments before touching the GPU (CPU only: every call
here fails validation or is an empty problem, so no pointer is followed)."""
import ctypes

import pytest

import causal_kernelized_attention_gb300 as la
from causal_kernelized_attention_gb300 import build as la_build
from causal_kernelized_attention_gb300._binding import RotarySpec

torch = pytest.importorskip("torch")

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


def spec(**kw):
    f = dict(rot=64, layout=0, scaling=0, original=0, base=10000.0, factor=1.0, ramp_lo=1.0, ramp_hi=32.0, amplitude=1.0)
    f.update(kw)
    return RotarySpec(**f)


def rotary(lib, name="la_rotary_forward", s=None, **kw):
    f = dict(q=at(0), k=at(1), oq=at(2), ok=at(3), pos=None, offset=0, B=1, Hq=2, Hk=2, N=8, d=64, dtype=BF16)
    f.update(kw)
    s = spec() if s is None else s
    return getattr(lib, name)(f["q"], f["k"], f["oq"], f["ok"], f["pos"], f["offset"], ctypes.byref(s), f["B"], f["Hq"],
                              f["Hk"], f["N"], f["d"], f["dtype"], None)


@pytest.mark.parametrize("name", ["la_rotary_forward", "la_rotary_backward"])
def test_rotary(lib, name):
    r = lambda s=None, **kw: rotary(lib, name, s, **kw)  # noqa: E731
    for bad in (dict(rot=3), dict(rot=66), dict(rot=-2), dict(layout=2), dict(scaling=4), dict(scaling=-1), dict(base=0.0),
                dict(base=NAN), dict(amplitude=INF), dict(scaling=1, factor=0.0), dict(scaling=2, factor=NAN),
                dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, original=4096, ramp_lo=32.0)):
        assert r(spec(**bad)) == INVALID, bad
    assert getattr(lib, name)(at(0), at(1), at(2), at(3), None, 0, None, 1, 2, 2, 8, 64, BF16, None) == INVALID
    for bad in (dict(q=None), dict(ok=None), dict(B=-1), dict(N=-1), dict(dtype=2), dict(oq=at(0) + 16), dict(ok=at(0)),
                dict(oq=at(2), ok=at(2)), dict(oq=at(1)), dict(pos=at(2) + 4)):
        assert r(**bad) == INVALID, bad
    assert r(q=at(0) + 8) == MISALIGNED and r(pos=at(4) + 2) == MISALIGNED
    assert r(spec(rot=12), d=12) == UNSUPPORTED and r(d=264) == UNSUPPORTED
    for empty in (dict(B=0), dict(N=0), dict(Hq=0, Hk=0)):
        assert r(q=None, k=None, oq=None, ok=None, **empty) == OK
    assert r(spec(rot=0), d=0) == OK


def test_recurrence(lib):
    def fwd(x=at(0), a=at(1), h0=None, h=at(2), hN=at(3), B=2, N=8, D=64, dtype=BF16):
        return lib.la_recurrence_forward(x, a, h0, h, hN, B, N, D, dtype, None)

    for bad in (dict(x=None), dict(a=None), dict(h=None), dict(B=-1), dict(D=-1), dict(N=-1), dict(dtype=9), dict(h=at(0)),
                dict(h=at(1) + 1024), dict(hN=at(2)), dict(h0=at(3))):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(x=at(0) + 4), dict(a=at(1) + 4), dict(h=at(2) + 8), dict(hN=at(3) + 4), dict(h0=at(4) + 4)):
        assert fwd(**bad) == MISALIGNED, bad
    assert fwd(x=None, a=None, h=None, hN=None, B=0) == OK and fwd(x=None, a=None, h=None, hN=None, N=0) == OK

    def bwd(a=at(0), h=at(1), dh=at(2), h0=None, dhN=None, dx=at(3), da=at(4), dh0=None, B=2, N=8, D=64, dtype=F32):
        return lib.la_recurrence_backward(a, h, dh, h0, dhN, dx, da, dh0, B, N, D, dtype, None)

    for bad in (dict(a=None), dict(h=None), dict(dh=None), dict(dx=None), dict(da=None), dict(dx=at(2)), dict(da=at(0)),
                dict(dx=at(4)), dict(dh0=at(5), dhN=at(5)), dict(dtype=-1), dict(N=-3)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(dh=at(2) + 8) == MISALIGNED and bwd(dh0=at(5) + 8) == MISALIGNED
    assert bwd(a=None, h=None, dh=None, dx=None, da=None, N=0) == OK

    def step(s=at(0), x=at(1), a=at(2), h=at(3), B=2, D=64, dtype=BF16):
        return lib.la_recurrence_step(s, x, a, h, B, D, dtype, None)

    for bad in (dict(s=None), dict(x=None), dict(a=None), dict(h=None), dict(h=at(0)), dict(s=at(2)), dict(h=at(1)), dict(D=-1)):
        assert step(**bad) == INVALID, bad
    assert step(s=at(0) + 4) == MISALIGNED
    assert step(s=None, x=None, a=None, h=None, D=0) == OK


SIZES = dict(B=1, Hq=4, Hk=2, Nq=8, Nk=8, d=64, window=4, sinks=1, scale=0.125, dtype=BF16)


def sized(f):
    return (f["B"], f["Hq"], f["Hk"], f["Nq"], f["Nk"], f["d"], f["window"], f["sinks"], ctypes.c_float(f["scale"]), f["dtype"],
            None)


BAD_SIZES = (dict(B=-1), dict(Hq=-4), dict(Hq=3), dict(Hk=0), dict(Nq=9), dict(Nq=-1), dict(window=0), dict(window=-5),
             dict(sinks=-1), dict(scale=0.0), dict(scale=1e-38), dict(scale=1e35), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(dtype=5))


def test_window_forward(lib):
    def fwd(q=at(0), k=at(1), v=at(2), o=at(3), lse=at(4), lens=None, **kw):
        return lib.la_window_forward(q, k, v, o, lse, lens, *sized({**SIZES, **kw}))

    for bad in BAD_SIZES + (dict(q=None), dict(lse=None), dict(o=at(0)), dict(o=at(4)), dict(lse=at(1)), dict(lens=at(3))):
        assert fwd(**bad) == INVALID, bad
    for d in (16, 48, 256):
        assert fwd(d=d) == UNSUPPORTED
    assert fwd(v=at(2) + 8) == MISALIGNED and fwd(lens=at(5) + 1) == MISALIGNED and fwd(lse=at(4) + 4) == MISALIGNED
    none = dict(q=None, k=None, v=None, o=None, lse=None)
    for empty in (dict(B=0), dict(Nq=0), dict(d=0), dict(Hq=0, Hk=0), dict(Hq=0)):
        assert fwd(**none, **empty) == OK


def test_window_backward(lib):
    def bwd(q=at(0), k=at(1), v=at(2), o=at(3), lse=at(4), go=at(5), dq=at(6), dk=at(7), dv=at(8), lens=None, **kw):
        return lib.la_window_backward(q, k, v, o, lse, go, dq, dk, dv, lens, *sized({**SIZES, **kw}))

    for bad in BAD_SIZES + (dict(go=None), dict(dq=None), dict(dk=None), dict(dv=at(7)), dict(dq=at(0)), dict(dk=at(4))):
        if bad != dict(Hk=0):
            assert bwd(**bad) == INVALID, bad
    assert bwd(Hk=0) == INVALID and bwd(d=40) == UNSUPPORTED and bwd(lse=at(4) + 4) == MISALIGNED
    assert bwd(B=0, dk=None, dv=None) == OK and bwd(Nq=0, Nk=0, dk=None, dv=None) == OK


def test_window_cache_and_decode(lib):
    def fill(k=at(0), v=at(1), kc=at(2), vc=at(3), lens=None, B=1, Hk=2, N=8, d=64, window=4, sinks=1, dtype=BF16):
        return lib.la_window_cache(k, v, kc, vc, lens, B, Hk, N, d, window, sinks, dtype, None)

    for bad in (dict(k=None), dict(vc=None), dict(kc=at(3)), dict(vc=at(1)), dict(window=0), dict(sinks=-1), dict(N=-1), dict(dtype=3)):
        assert fill(**bad) == INVALID, bad
    assert fill(d=24) == UNSUPPORTED and fill(window=2 ** 31 - 1, sinks=1) == UNSUPPORTED
    assert fill(kc=at(2) + 8) == MISALIGNED and fill(k=None, v=None, N=0) == OK

    def step(kc=at(0), vc=at(1), q=at(2), k=at(3), v=at(4), o=at(5), pos=at(6), **kw):
        f = {**SIZES, **kw}
        return lib.la_window_decode_step(kc, vc, q, k, v, o, pos, f["B"], f["Hq"], f["Hk"], f["d"], f["window"], f["sinks"],
                                         ctypes.c_float(f["scale"]), f["dtype"], None)

    for bad in (dict(kc=None), dict(pos=None), dict(o=at(2)), dict(kc=at(1)), dict(vc=at(3)), dict(Hq=3), dict(window=0),
                dict(scale=-1.0), dict(dtype=2), dict(pos=at(5))):
        assert step(**bad) == INVALID, bad
    assert step(d=80) == UNSUPPORTED and step(pos=at(6) + 2) == MISALIGNED and step(window=2 ** 31 - 1) == UNSUPPORTED
    assert step(kc=None, vc=None, B=0) == OK


def test_python_refusals():
    """Shapes, types and devices, before the library is called."""
    x = torch.zeros((1, 2, 4, 64))
    with pytest.raises(ValueError):
        la.la_rotary_forward(x)  # not on a GPU
    with pytest.raises(ValueError):
        la.la_rotary_forward(torch.zeros((2, 64)))
    with pytest.raises(ValueError):
        la.la_recurrence_forward(torch.zeros((4, 64)), torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        la.la_window_forward(x, x, x, 4)
    with pytest.raises(ValueError):
        la.la_window_forward(x, torch.zeros((1, 2, 4, 32)), x, 4)
    with pytest.raises(ValueError):
        la.la_window_cache(x, x, 0)
    with pytest.raises(ValueError):
        la.la_window_decode_step(x, x, x, x, x, x, 4)


@pytest.mark.parametrize("name", ["la_rotary_forward", "la_rotary_backward"])
def test_rotary_frequencies_that_overflow(lib, name):
    """A base or factor next to 0 leaves pairs without a finite frequency."""
    for bad in (dict(scaling=1, factor=1e-310), dict(scaling=2, factor=1e-300, rot=4, base=1e-20), dict(base=1e-320, scaling=1, factor=1e-10),
                dict(scaling=3, factor=1e-310, original=4096)):
        assert rotary(lib, name, spec(**bad)) == INVALID, bad


def test_whole_numbers_are_not_bent():
    """A window of 4.7 is no window of 4, an offset past 64 bits none modulo them."""
    x, y = torch.zeros((1, 2, 4, 64)), torch.zeros((1, 2, 64))
    lse, pos = torch.zeros((1, 2, 4)), torch.zeros(1, dtype=torch.int32)
    for kw in (dict(window=4.7), dict(window=4, sinks=1.5), dict(window="4"), dict(window=float("nan")), dict(window=None)):
        for call in (lambda: la.la_window_forward(x, x, x, **kw), lambda: la.la_window_backward(x, x, x, x, lse, x, **kw),
                     lambda: la.la_window_cache(x, x, **kw), lambda: la.la_window_decode_step(x, x, y, y, y, pos, **kw)):
            with pytest.raises(TypeError, match="whole number"):
                call()
    for kw in (dict(rot=32.5), dict(offset=float("inf")), dict(offset=0.5), dict(scaling="ramp", original=4096.5)):
        for call in (la.la_rotary_forward, la.la_rotary_backward):
            with pytest.raises(TypeError, match="whole number"):
                call(x, **kw)
    for kw, bits in ((dict(offset=2 ** 63), 64), (dict(offset=-2 ** 63 - 1), 64), (dict(rot=2 ** 31), 32)):
        with pytest.raises(ValueError, match="%d bits" % bits):
            la.la_rotary_forward(x, **kw)
    with pytest.raises(ValueError, match="CUDA device"):  # numbers of other kinds that are whole
        la.la_window_forward(x, x, x, torch.tensor(4), sinks=2.0)


def test_sizes_that_pass_32_bits():
    """Every size that the library takes as 32 bits, none modulo them; empty tensors too."""
    big = 2 ** 32 + 5
    wide = lambda *shape: torch.zeros(1).expand(shape)  # noqa: E731
    x, one = wide(1, 1, 8, 64), wide(1, 1, 64)
    pos = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: la.la_window_forward(wide(1, 1, big, 64), x, x, 4), lambda: la.la_window_forward(wide(1, big, 8, 64), x, x, 4),
                 lambda: la.la_window_forward(x, wide(1, 1, big, 64), wide(1, 1, big, 64), 4),
                 lambda: la.la_window_backward(wide(1, 1, big, 64), x, x, x, x, x, 4),
                 lambda: la.la_window_cache(wide(big, 0, 8, 64), wide(big, 0, 8, 64), 4),
                 lambda: la.la_window_decode_step(x, x, wide(1, big, 64), one, one, pos, 4),
                 lambda: la.la_window_decode_step(x, x, one, wide(1, big, 64), one, pos, 4),
                 lambda: la.la_rotary_forward(wide(1, big, 64)), lambda: la.la_rotary_forward(wide(big, 0, 8, 64), wide(big, 1, 8, 64)),
                 lambda: la.la_rotary_forward(x, wide(1, big, 8, 64)),
                 lambda: la.la_recurrence_forward(wide(big, 0, 8), wide(big, 0, 8)), lambda: la.la_recurrence_step(one[0], wide(1, big), one[0])):
        with pytest.raises(ValueError, match="fit 32 bits"):
            call()
