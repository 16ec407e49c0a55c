"""Arguments of the operators beside the delta rules that are refused before
anything reaches a GPU, or that must be understood (no GPU needed)."""
import ctypes

import pytest

import delta_rule_linear_kron_b200 as kd
from delta_rule_linear_kron_b200 import build as kbuild

torch = pytest.importorskip("torch")


def at(n):
    return ctypes.c_void_p(n)   # aligned, never dereferenced: every call here is refused


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kd.lib()


@pytest.mark.parametrize("with_k", [True, False])
@pytest.mark.parametrize("out", ["qo", "ko"])
@pytest.mark.parametrize("other", ["freqs", "pos"])
def test_rotary_outputs_over_frequencies_or_positions_are_refused(L, out, other, with_k):
    """Also where only the last bytes of either meet the first of the other."""
    if out == "ko" and not with_k:
        return
    a = dict(q=at(1 << 24), k=at(2 << 24), freqs=at(3 << 24), pos=at(4 << 24), qo=at(5 << 24), ko=at(6 << 24), B=2, T=5, H=2,
             Hk=1, d=64, rot=64, inter=0, inv=0, scale=1.0, dtype=1, stream=None)
    if not with_k:
        a.update(k=None, ko=None, Hk=0)
    size = {"freqs": 32 * 8, "pos": 2 * 5 * 8, "qo": 2 * 5 * 2 * 64 * 2, "ko": 2 * 5 * 64 * 2}
    base = a[other].value
    for shift in (0, size[other] - 16, 16 - size[out]):
        b = dict(a)
        b[out] = at(base + shift)
        assert L.kron_delta_rotary(*b.values()) == kd.KD_ERR_INVALID_ARG
        assert b"overlaps " + other.encode() in L.kron_delta_last_error()


class StreamOfCuda:
    device = torch.device("cuda", 0)


def test_a_stream_is_held_against_the_first_tensor_wherever_it_stands():
    """Arguments by name come in any order, numbers before tensors."""
    x = torch.zeros(1, 4, 2, 32)
    for call in (lambda **k: kd.swa_fwd(window=3, q=x, k=x, v=x, **k), lambda **k: kd.swa_fwd(x, x, x, 3, **k),
                 lambda **k: kd.rotary_fwd(interleaved=True, k=None, q=x, freqs=x, **k),
                 lambda **k: kd.glr_fwd(save=True, h0=None, x=x, i_pre=x, f_pre=x, a_log=x, **k)):
        with pytest.raises(kd.KronDeltaError, match="stream belongs to cuda:0 but the call's tensors are on cpu"):
            call(stream=StreamOfCuda())


def test_a_window_beyond_32_bits_is_all_of_the_sequence():
    """Not its lowest 32 bits; what a call has to refuse stays refused."""
    def size(kind, window, sinks=2):
        return kd.swa_workspace_size(kind, 2, 100, 4, 2, 64, window, sinks, kd.KD_BF16)
    for kind in (kd.KD_SWA_WS_SAVE, kd.KD_SWA_WS_BWD):
        for window in (2 ** 31 - 128, 2 ** 31, 2 ** 32 + 8, 2 ** 63 - 1):
            assert size(kind, window) == size(kind, 100)
    assert size(kd.KD_SWA_WS_BWD, 8) > size(kd.KD_SWA_WS_BWD, 100)  # a narrow window's first tokens have parts
    for window, sinks in ((-2 ** 32 + 8, 2), (0, 2), (8, 2 ** 32 + 2), (8, -2 ** 32 + 2), (8, 2 ** 31)):
        for kind in (kd.KD_SWA_WS_SAVE, kd.KD_SWA_WS_BWD, kd.KD_SWA_WS_DECODE):
            with pytest.raises(kd.KronDeltaError, match="must be"):
                size(kind, window, sinks)
    with pytest.raises(kd.KronDeltaError, match="window < 2"):  # a cache of so many slots
        size(kd.KD_SWA_WS_DECODE, 2 ** 32 + 8)
