"""Refusals of the operators beside the delta rules, before anything reaches a
GPU: the C ABI's error codes and the binding's checks (no GPU needed)."""
import ctypes

import pytest

import delta_rule_linear_kron_b200 as kd
from delta_rule_linear_kron_b200 import build as kbuild

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(256)   # aligned, non-null, never dereferenced: every call here is refused
ODD = ctypes.c_void_p(260)
INV, UNS, WS = kd.KD_ERR_INVALID_ARG, kd.KD_ERR_UNSUPPORTED, kd.KD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kd.lib()


def _with(defaults, over):
    a = dict(defaults)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


ROT = dict(q=P, k=P, freqs=P, pos=None, qo=P, ko=P, B=1, T=4, H=2, Hk=1, d=64, rot=64, inter=0, inv=0, scale=1.0,
           dtype=1, stream=None)


@pytest.mark.parametrize("over,code,word", [
    (dict(q=None), INV, b"q must not"), (dict(freqs=None), INV, b"freqs"), (dict(qo=None), INV, b"q_out"),
    (dict(k=None), INV, b"Hk"), (dict(Hk=0), INV, b"Hk"), (dict(B=0), INV, b"B, T, H"), (dict(T=-3), INV, b"B, T, H"),
    (dict(d=48), UNS, b"32, 64 or 128"), (dict(rot=63), INV, b"rot"), (dict(rot=66), INV, b"rot"),
    (dict(rot=0), INV, b"rot"), (dict(inter=2), INV, b"interleaved"), (dict(scale=float("nan")), INV, b"scale"),
    (dict(dtype=2), UNS, b"dtype"), (dict(q=ODD), INV, b"aligned"), (dict(pos=ODD), INV, b"aligned"),
    (dict(B=65536, T=65536), INV, b"too large"), (dict(qo=ctypes.c_void_p(512)), INV, b"overlaps"),
])
def test_rotary_refusals(L, over, code, word):
    assert L.kron_delta_rotary(*_with(ROT, over)) == code
    assert word in L.kron_delta_last_error()


FWD = dict(q=P, k=P, v=P, out=P, lse=P, B=1, T=100, H=4, Hk=2, d=64, window=8, sinks=2, scale=0.1, dtype=1, ws=None,
           ws_bytes=0, save=0, stream=None)
SHAPES = [(dict(B=0), INV, b"B, T, H"), (dict(H=3), INV, b"multiple"), (dict(Hk=0), INV, b"B, T, H"),
          (dict(d=96), UNS, b"32, 64 or 128"), (dict(window=0), INV, b"window"), (dict(sinks=-1), INV, b"sinks"),
          (dict(sinks=129), UNS, b"sinks"), (dict(window=2 ** 31 - 100), INV, b"window"), (dict(dtype=5), UNS, b"dtype"),
          (dict(scale=0.0), INV, b"scale"), (dict(scale=float("inf")), INV, b"scale"), (dict(k=None), INV, b"k must"),
          (dict(v=ctypes.c_void_p(8)), INV, b"aligned"), (dict(B=70000), INV, b"65535")]


@pytest.mark.parametrize("over,code,word", SHAPES + [
    (dict(T=0), INV, b"B, T, H"), (dict(T=2 ** 30 + 1), INV, b"2^30"), (dict(lse=None), INV, b"lse"),
    (dict(save=2), INV, b"save"), (dict(save=1), WS, b"workspace"),
    (dict(save=1, ws=ctypes.c_void_p(16), ws_bytes=1 << 30), WS, b"256-byte"),
])
def test_swa_fwd_refusals(L, over, code, word):
    assert L.kron_delta_swa_fwd(*_with(FWD, over)) == code
    assert word in L.kron_delta_last_error()


BWD = dict(q=P, k=P, v=P, out=P, lse=P, dO=P, dq=P, dk=P, dv=P, B=1, T=100, H=4, Hk=2, d=64, window=8, sinks=2,
           scale=0.1, dtype=1, fws=P, fws_bytes=1 << 40, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code,word", SHAPES + [
    (dict(dO=None), INV, b"dO"), (dict(dv=None), INV, b"dv"), (dict(fws=None), WS, b"forward"),
    (dict(fws_bytes=1 * 100 * 4 * 64 * 2 - 1), WS, b"forward"), (dict(ws_bytes=256), WS, b"backward"),
    (dict(ws=None), WS, b"backward"),
])
def test_swa_bwd_refusals(L, over, code, word):
    assert L.kron_delta_swa_bwd(*_with(BWD, over)) == code
    assert word in L.kron_delta_last_error()


DEC = dict(q=P, k=P, v=P, kc=P, vc=P, pos=P, out=P, B=1, H=4, Hk=2, d=64, window=8, sinks=2, scale=0.1, dtype=1,
           ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("over,code,word", SHAPES + [
    (dict(kc=None), INV, b"k_cache"), (dict(pos=None), INV, b"pos"), (dict(pos=ODD), INV, b"aligned"),
    (dict(window=20000), WS, b"decode workspace"),
])
def test_swa_decode_refusals(L, over, code, word):
    assert L.kron_delta_swa_decode(*_with(DEC, over)) == code
    assert word in L.kron_delta_last_error()


FILL = dict(k=P, v=P, lens=P, kc=P, vc=P, B=1, T=100, Hk=2, d=64, window=8, sinks=2, dtype=1, stream=None)


@pytest.mark.parametrize("over,code,word", [
    (dict(T=0), INV, b"B, T, H"), (dict(lens=None), INV, b"lens"), (dict(vc=ODD), INV, b"aligned"),
    (dict(d=16), UNS, b"32, 64 or 128"), (dict(sinks=200), UNS, b"sinks"),
    (dict(window=2 ** 31 - 200, B=60000, Hk=8, d=128), INV, b"too large"),
])
def test_swa_fill_refusals(L, over, code, word):
    assert L.kron_delta_swa_fill(*_with(FILL, over)) == code
    assert word in L.kron_delta_last_error()


GF = dict(x=P, i=P, f=P, a=P, h0=None, out=P, hT=None, B=1, T=10, D=16, dtype=1, ws=None, ws_bytes=0, save=0,
          stream=None)
GSHAPES = [(dict(B=0), INV, b"B, T, D"), (dict(D=12), UNS, b"multiple of 8"), (dict(dtype=9), UNS, b"dtype"),
           (dict(x=None), INV, b"x must"), (dict(a=ODD), INV, b"aligned"), (dict(B=65536), INV, b"65535")]


@pytest.mark.parametrize("over,code,word", GSHAPES + [
    (dict(T=0), INV, b"B, T, D"), (dict(out=None), INV, b"out"), (dict(save=1), WS, b"workspace"),
    (dict(save=-1), INV, b"save"),
])
def test_glr_fwd_refusals(L, over, code, word):
    assert L.kron_delta_glr_fwd(*_with(GF, over)) == code
    assert word in L.kron_delta_last_error()


GB = dict(x=P, i=P, f=P, a=P, dh=P, dhT=None, dx=P, di=P, df=P, da=P, dh0=None, B=1, T=10, D=16, dtype=1, fws=P,
          fws_bytes=1 << 40, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code,word", GSHAPES + [
    (dict(dh=None), INV, b"dh"), (dict(da=None), INV, b"da_log"), (dict(fws_bytes=63), WS, b"forward"),
    (dict(ws_bytes=63), WS, b"backward"),
])
def test_glr_bwd_refusals(L, over, code, word):
    assert L.kron_delta_glr_bwd(*_with(GB, over)) == code
    assert word in L.kron_delta_last_error()


@pytest.mark.parametrize("over,code,word", GSHAPES + [(dict(h=None), INV, b"h must")])
def test_glr_decode_refusals(L, over, code, word):
    d = dict(x=P, i=P, f=P, a=P, h=P, out=P, B=1, D=16, dtype=1, stream=None)
    assert L.kron_delta_glr_decode(*_with(d, over)) == code
    assert word in L.kron_delta_last_error()


def test_workspace_sizes(L):
    assert kd.swa_workspace_size(kd.KD_SWA_WS_SAVE, 2, 100, 4, 2, 64, 8, 2, 1) == 2 * 100 * 4 * 64 * 2
    assert kd.swa_workspace_size(kd.KD_SWA_WS_SAVE, 2, 100, 4, 2, 64, 8, 2, 0) == 0  # none needed, no error
    # lse and delta per head, tokens rounded up to 128; first tokens add their parts
    base = kd.swa_workspace_size(kd.KD_SWA_WS_BWD, 2, 100, 4, 2, 64, 8, 0, 1)
    assert base == 2 * (2 * 4 * 128 * 4)
    assert kd.swa_workspace_size(kd.KD_SWA_WS_BWD, 2, 100, 4, 2, 64, 8, 2, 1) > base
    assert kd.swa_workspace_size(kd.KD_SWA_WS_BWD, 2, 100, 4, 2, 64, 100, 2, 1) == base  # the window is the sequence
    assert kd.swa_workspace_size(kd.KD_SWA_WS_DECODE, 512, 1, 16, 4, 128, 64, 0, 1) == 0
    assert kd.swa_workspace_size(kd.KD_SWA_WS_DECODE, 1, 1, 16, 4, 128, 4096, 4, 1) == 0  # a cluster joins the parts
    assert kd.swa_workspace_size(kd.KD_SWA_WS_DECODE, 1, 1, 16, 4, 128, 20000, 4, 1) > 0
    assert kd.glr_workspace_size(kd.KD_GLR_WS_SAVE, 3, 65, 16, 1) == 3 * 2 * 16 * 4
    for bad in (lambda: kd.swa_workspace_size(7, 1, 1, 1, 1, 32, 1, 0, 1),
                lambda: kd.swa_workspace_size(kd.KD_SWA_WS_SAVE, 1, 0, 1, 1, 32, 1, 0, 0),
                lambda: kd.glr_workspace_size(5, 1, 1, 8, 1), lambda: kd.glr_workspace_size(0, 1, 1, 9, 1)):
        with pytest.raises(kd.KronDeltaError):
            bad()


def test_binding_refuses_host_tensors_and_wrong_ranks():
    x = torch.zeros(1, 4, 2, 32)
    with pytest.raises(kd.KronDeltaError, match="CUDA tensor"):
        kd.swa_fwd(x, x, x, 4)
    with pytest.raises(kd.KronDeltaError, match="4 dimensions"):
        kd.swa_fwd(x[0], x, x, 4)
    with pytest.raises(kd.KronDeltaError, match="CUDA tensor"):
        kd.rotary_fwd(x, None, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(kd.KronDeltaError, match="3 dimensions"):
        kd.glr_fwd(x, x, x, x)


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.5),
                                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, factor=0.5),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0),
                                dict(rotary_dim=2, scaling="ntk", factor=2.0)])
def test_rotary_freqs_refusals(kw):
    with pytest.raises(kd.KronDeltaError):
        kd.rotary_freqs(**kw, device="cpu")


def test_rotary_freqs_values():
    w, s = kd.rotary_freqs(8, 10000.0, device="cpu")
    assert w.dtype == torch.float64 and s == 1.0
    assert torch.allclose(w, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    lin, _ = kd.rotary_freqs(8, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, w / 4)
    ntk, _ = kd.rotary_freqs(8, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and torch.allclose(ntk[-1], w[-1] / 4)
    # over 1000 positions the pairs turn 159, 16, 1.6 and 0.16 times
    yarn, s = kd.rotary_freqs(8, scaling="yarn", factor=4.0, trained_len=1000, low=1.0, high=32.0, device="cpu")
    assert yarn[0] == w[0] and torch.allclose(yarn[3], w[3] / 4) and w[1] / 4 < yarn[1] < w[1]
    assert abs(s - 1.1386294361119891) < 1e-12


@pytest.mark.parametrize("fn,defaults,outs,ins", [
    ("rotary", ROT, ["qo", "ko"], ["q", "k"]), ("swa_fwd", FWD, ["out", "lse"], ["q", "k", "v"]),
    ("swa_bwd", BWD, ["dq", "dk", "dv", "ws"], ["q", "k", "v", "out", "lse", "dO", "fws"]),
    ("swa_decode", DEC, ["out", "kc", "vc"], ["q", "k", "v", "pos"]), ("swa_fill", FILL, ["kc", "vc"], ["k", "v", "lens"]),
    ("glr_fwd", GF, ["out", "hT"], ["x", "i", "f", "a", "h0"]),
    ("glr_bwd", GB, ["dx", "di", "df", "da", "dh0", "ws"], ["x", "i", "f", "a", "dh", "dhT", "fws"]),
    ("glr_decode", dict(x=P, i=P, f=P, a=P, h=P, out=P, B=1, D=16, dtype=1, stream=None), ["h", "out"], ["x", "i", "f", "a"]),
])
def test_outputs_that_overlap_are_refused(L, fn, defaults, outs, ins):
    a = dict(defaults)
    for n, name in enumerate(outs + ins):
        a[name] = ctypes.c_void_p((n + 1) << 24)
    a["B"] = 4
    call = getattr(L, "kron_delta_" + fn)
    for o in outs:
        for other in outs + ins:
            if other == o or (fn == "rotary" and (o, other) in (("qo", "q"), ("ko", "k"))):
                continue
            for shift in (0, 16):  # the other's last bytes too: every tensor here holds more than 16
                b = dict(a)
                b[o] = ctypes.c_void_p(a[other].value + shift) if (o, shift) != ("ws", 16) else a[other]
                assert call(*b.values()) == INV, (o, other)
                assert b"overlaps" in L.kron_delta_last_error()
