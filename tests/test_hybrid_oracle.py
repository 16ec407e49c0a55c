"""Pins of the fp64 oracles of rotary positions, sliding-window attention and
the gated linear recurrence: closed forms and central differences."""
import numpy as np
import pytest

from oracle import hybrid as O

RNG = np.random.default_rng


def test_rotary_closed_forms():
    x = RNG(0).standard_normal((1, 3, 2, 8))
    f, pos = np.array([np.pi / 2, 0.25]), np.array([[0, 1, -2]])
    y = O.rotary(x, f, pos)
    assert np.allclose(y[0, 0], x[0, 0]) and np.allclose(y[..., 4:], x[..., 4:])
    # a quarter turn: (x1, x2) -> (-x2, x1), pairs (0, 2)
    assert np.allclose(y[0, 1, :, 0], -x[0, 1, :, 2]) and np.allclose(y[0, 1, :, 2], x[0, 1, :, 0])
    z = O.rotary(x, f, pos, interleaved=True)
    assert np.allclose(z[0, 1, :, 0], -x[0, 1, :, 1]) and np.allclose(z[0, 1, :, 1], x[0, 1, :, 0])
    # back and forth, and scores that depend on the distance alone
    assert np.allclose(O.rotary(y, f, pos, inverse=True), x)
    a, b = RNG(1).standard_normal((2, 1, 1, 1, 4))
    s = [np.sum(O.rotary(a, f, [[p]]) * O.rotary(b, f, [[p + 5]])) for p in (0, 7, 1000)]
    assert np.allclose(s, s[0])


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (50, 0), (2, 9)])
def test_swa_matches_rows_one_by_one(window, sinks):
    r = RNG(3)
    q, k, v = r.standard_normal((1, 9, 4, 3)), r.standard_normal((1, 9, 2, 3)), r.standard_normal((1, 9, 2, 3))
    got = O.swa(q, k, v, window, sinks, 0.7)
    for t in range(9):
        seen = [j for j in range(t + 1) if t - j < window or j < sinks]
        for h in range(4):
            x = np.array([0.7 * q[0, t, h] @ k[0, j, h // 2] for j in seen])
            w = np.exp(x) / np.exp(x).sum()
            assert np.allclose(got["out"][0, t, h], w @ v[0, seen, h // 2])
            assert np.isclose(got["lse"][0, t, h], np.log(np.exp(x).sum()))


def _differences(fn, args, names, grads, rel=1e-6):
    r = RNG(11)
    for n in names:
        d = r.standard_normal(args[n].shape)
        step = 1e-6
        up, down = (fn({**args, n: args[n] + s * step * d}) for s in (1, -1))
        assert np.isclose((up - down) / (2 * step), np.sum(grads[n] * d), rtol=rel, atol=1e-8), n


def test_swa_gradients_by_differences():
    r = RNG(4)
    a = {n: r.standard_normal((2, 7, h, 4)) for n, h in (("q", 4), ("k", 2), ("v", 2))}
    dO = r.standard_normal((2, 7, 4, 4))
    g = O.swa(**a, window=3, sinks=1, scale=0.5, dO=dO)
    _differences(lambda x: np.sum(O.swa(**x, window=3, sinks=1, scale=0.5)["out"] * dO), a, "qkv",
                 {"q": g["dq"], "k": g["dk"], "v": g["dv"]})


def test_ring_slots_hold_exactly_what_a_query_sees():
    for window, sinks in ((1, 0), (4, 0), (4, 3), (3, 5)):
        cache = {}
        for p in range(20):
            cache[O.ring_slot(p, window, sinks)] = p
            seen = {j for j in range(p + 1) if p - j < window or j < sinks}
            assert set(cache.values()) == seen
            assert set(cache) == set(range(min(p + 1, window + sinks)))


def test_glr_closed_forms():
    x, one = np.ones((1, 50, 1)), np.ones((1, 50, 1))
    # constant gates: h_t = b (1 - f^t) / (1 - f)
    f = O.sigmoid(2.0) ** np.exp(0.3)
    b = np.sqrt(1 - f * f) * O.sigmoid(-0.5)
    got = O.glr(x, -0.5 * one, 2.0 * one, np.array([0.3]))["out"][0, :, 0]
    assert np.allclose(got, b * (1 - f ** np.arange(1, 51)) / (1 - f))
    # f = 0 starts again; f = 1 keeps the state and writes nothing
    z = 2.0 * one
    z[0, 20] = -np.inf
    y = O.glr(x, -0.5 * one, z, np.array([0.3]))["out"][0, :, 0]
    assert np.isclose(y[20], O.sigmoid(-0.5)) and np.allclose(y[:20], got[:20])
    z[0, 20] = 800.0
    y = O.glr(x, -0.5 * one, z, np.array([0.3]))["out"][0, :, 0]
    assert y[20] == y[19]


def test_glr_gradients_by_differences():
    r = RNG(5)
    a = dict(x=r.standard_normal((2, 6, 3)), i_pre=r.standard_normal((2, 6, 3)),
             f_pre=r.standard_normal((2, 6, 3)) + 1, a_log=r.uniform(-1, 1, 3), h0=r.standard_normal((2, 3)))
    dh, dhT = r.standard_normal((2, 6, 3)), r.standard_normal((2, 3))
    g = O.glr(**a, dh=dh, dhT=dhT)

    def loss(v):
        y = O.glr(**v)
        return np.sum(y["out"] * dh) + np.sum(y["hT"] * dhT)
    _differences(loss, a, a, {"x": g["dx"], "i_pre": g["di_pre"], "f_pre": g["df_pre"], "a_log": g["da_log"],
                              "h0": g["dh0"]})
