"""Edges of rotary positions, sliding-window attention and the gated linear
recurrence on the GPU: what is not a number, what overflows, tensors at the
least alignment that is allowed."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import delta_rule_linear_kron_b200 as kd  # noqa: E402
from oracle import hybrid as O  # noqa: E402
from tests.test_gpu_hybrid import check_glr, draw, glr_inputs, host, run_glr  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    kd.lib()


# ---- what is not a number ---------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "i_pre", "f_pre", "a_log", "h0", "dh", "dhT"])
def test_glr_nan_reaches_what_depends_on_it(name, dtype):
    """One NaN: the results are NaN where the formulas' are, and everything
    else is bitwise what it is without it."""
    t, r = glr_inputs(2, 700, 72, dtype, 11)
    clean = run_glr(t)
    at = {1: (37,), 2: (1, 37), 3: (1, 333, 37)}[t[name].dim()]
    t[name][at] = r[name][at] = float("nan")
    got, ref = run_glr(t), O.glr(**r)
    for n, x in got.items():
        bad = np.isnan(ref[n])
        assert bad.any() == (n in NAN_IN[name]), n
        assert np.array_equal(np.isnan(host(x)), bad), n
        ok = torch.from_numpy(~bad).cuda()
        assert torch.equal(x[ok], clean[n][ok]), n


# what one NaN in an input reaches
NAN_IN = {"x": {"out", "hT", "di_pre", "df_pre", "da_log"},
          "i_pre": {"out", "hT", "dx", "di_pre", "df_pre", "da_log"},
          "f_pre": {"out", "hT", "dx", "di_pre", "df_pre", "da_log", "dh0"},
          "a_log": {"out", "hT", "dx", "di_pre", "df_pre", "da_log", "dh0"},
          "h0": {"out", "hT", "df_pre", "da_log"},
          "dh": {"dx", "di_pre", "df_pre", "da_log", "dh0"}, "dhT": {"dx", "di_pre", "df_pre", "da_log", "dh0"}}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "i_pre", "f_pre", "a_log", "h"])
def test_glr_decode_nan_reaches_what_depends_on_it(name, dtype):
    t, _ = glr_inputs(3, 1, 40, dtype, 12)
    a = {n: t[n][:, 0].contiguous() for n in ("x", "i_pre", "f_pre")}
    a.update(a_log=t["a_log"], h=t["h0"])
    clean = {n: x.clone() for n, x in a.items()}
    want = kd.glr_decode(**clean)
    at = (slice(None), 7) if name == "a_log" else (1, 7)
    a[name][at[-1:] if name == "a_log" else at] = float("nan")
    got = kd.glr_decode(**a)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[at] = True
    for x, y in ((got, want), (a["h"], clean["h"])):
        assert torch.equal(torch.isnan(x), bad) and torch.equal(x[~bad], y[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [40, 3000, 9000, 40000])
def test_swa_decode_nan_reaches_what_depends_on_it(window, dtype):
    """In one CTA, in a cluster's parts and in parts through the workspace: a
    NaN in a query makes its head NaN, one in a key its group's heads, one in a
    value its channel of them; an idle sequence's out is zero."""
    H, Hk, d, sinks = 4, 2, 64, 3
    rng = np.random.default_rng(window)
    B = 6
    q, k, v = (draw(rng, (B, h, d), dtype)[0] for h in (H, Hk, Hk))
    kc, vc = (draw(rng, (B, window + sinks, Hk, d), dtype)[0] for _ in range(2))
    pos = torch.tensor([-1, 5, window + sinks + 7, window + sinks, window // 2, 0], device="cuda")
    want = kd.swa_decode(q, k, v, kc.clone(), vc.clone(), pos, window, sinks)
    nan = float("nan")
    q[:3, 1, 9] = nan          # idle, its start, wrapped
    k[3, 1, 0] = nan           # the new key
    kc[4, 2, 0, 5] = nan       # a first token's
    v[5, 0, 11] = nan          # the only value
    vc[2, 4, 1, 3] = nan
    got = kd.swa_decode(q, k, v, kc, vc, pos, window, sinks)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1:3, 1] = True
    bad[3, 2:] = True
    bad[4, :2] = True
    bad[5, :2, 11] = True
    bad[2, 2:, 3] = True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])
    assert not got[0].any()


# ---- what overflows -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [300, 3000, 9000])
def test_swa_decode_scores_of_minus_infinity_weigh_nothing(window, dtype):
    """Keys whose scores are -infinity (by an infinite channel, or by overflow)
    drop out, also where they are all that a warp or a part has seen so far."""
    H, Hk, d, sinks, B = 4, 2, 64, 2, 2
    rng = np.random.default_rng(window)
    n = window + sinks
    (q, qh), (k, kh), (v, vh) = (draw(rng, (B, h, d), dtype) for h in (H, Hk, Hk))
    q[..., 0] = qh[..., 0] = 2.0
    (kc, kch), (vc, vch) = (draw(rng, (B, n, Hk, d), dtype) for _ in range(2))
    low = torch.finfo(kc.dtype).min
    gone = np.zeros((B, n), dtype=bool)
    gone[0, :n - 5] = True                      # all but the last slots
    gone[1] = rng.random(n) < 0.7
    pos = torch.tensor([n - 1, n + 3], device="cuda")
    slots = [O.ring_slot(int(p), window, sinks) for p in pos]
    for b, s in enumerate(slots):
        gone[b, s] = False
        kch[b, s], vch[b, s] = kh[b], vh[b]
    at = torch.from_numpy(gone).cuda()
    kc[..., 0][at] = -float("inf")
    kc[0, : n // 2, :, 0] = low                 # times 2: beyond fp32
    got = host(kd.swa_decode(q, k, v, kc, vc, pos, window, sinks))
    for b in range(B):
        for h in range(H):
            kk, vv = kch[b, ~gone[b], h // 2], vch[b, ~gone[b], h // 2]
            x = kk @ qh[b, h] / np.sqrt(d)
            w = np.exp(x - x.max())
            w /= w.sum()
            # scores d + 8 roundings of sum |q||k|, twice; sums of n terms; the output's rounding
            e = 2 * (d + 8) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qh[b, h])).max() / np.sqrt(d) + (2 * n + 32) * 2.0 ** -24
            ref, u = w @ vv, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            assert (np.abs(got[b, h] - ref) <= e * (w @ np.abs(vv)) + u * np.abs(ref) + 1e-30).all(), (b, h)


def test_swa_decode_last_position_of_64_bits():
    """The largest position sees a full cache and stores its token."""
    window, sinks, p = 20, 3, 2 ** 63 - 1
    q, k, v = torch.randn(1, 2, 32, device="cuda"), torch.randn(1, 1, 32, device="cuda"), torch.randn(1, 1, 32, device="cuda")
    kc, vc = (torch.randn(1, window + sinks, 1, 32, device="cuda") for _ in range(2))
    near = sinks + (p - sinks) % window + window * 1000  # a position of the same slot
    a, b = [kc.clone(), vc.clone()], [kc.clone(), vc.clone()]
    got = kd.swa_decode(q, k, v, *a, torch.tensor([p], device="cuda"), window, sinks)
    want = kd.swa_decode(q, k, v, *b, torch.tensor([near], device="cuda"), window, sinks)
    assert want.any() and torch.equal(got, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [70, 128, 1000])
def test_glr_exponents_beyond_fp32(T, dtype):
    """e^{a_log} beyond fp32: each gate forgets all, and a sequence that ends
    inside a chunk of tokens keeps its last state and passes dhT on."""
    t, r = glr_inputs(2, T, 72, dtype, T)
    for c, a in ((3, 88.0), (4, 89.0), (40, 120.0), (71, 300.0)):
        t["a_log"][c] = r["a_log"][c] = a
    check_glr(t, r, dtype)
    f = kd.glr_fwd(t["x"], t["i_pre"], t["f_pre"], t["a_log"], t["h0"])[1]
    t["a_log"][71] = float("inf")
    assert torch.equal(kd.glr_fwd(t["x"], t["i_pre"], t["f_pre"], t["a_log"], t["h0"])[1], f)


# ---- the least alignment ------------------------------------------------------------


class Placed:
    """Tensors 16 bytes behind a 256-byte boundary, the memory around them marked."""

    def __init__(self):
        self.bufs = []

    def __call__(self, t):
        n = t.numel() * t.element_size()
        buf = torch.full((256 + n + 256,), 0x5a, dtype=torch.uint8, device="cuda")
        at = -buf.data_ptr() % 256 + 16
        x = buf[at:at + n].view(t.dtype).view(t.shape)
        x.copy_(t)
        assert x.data_ptr() % 256 == 16
        self.bufs.append((buf, at, n))
        return x

    def untouched(self):
        return all((b[:a] == 0x5a).all() and (b[a + n:] == 0x5a).all() for b, a, n in self.bufs)


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("dtype,d", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 128)])
@pytest.mark.parametrize("window", [40, 300])
def test_swa_tensors_at_16_bytes(dtype, d, window):
    """Every tensor of the attention at the least alignment that the C entry
    points take, first tokens with far queries among them."""
    B, T, H, Hk, sinks = 2, 700, 4, 2, 70
    rng = np.random.default_rng(d + window)
    q, k, v, g = (draw(rng, (B, T, h, d), dtype)[0] for h in (H, Hk, Hk, H))
    out, lse, ws = kd.swa_fwd(q, k, v, window, sinks, save=True)
    ref = dict(out=out, lse=lse, **kd.swa_bwd(q, k, v, out, lse, g, window, sinks, fwd_workspace=ws))
    place, L, s = Placed(), kd.lib(), torch.cuda.current_stream().cuda_stream
    q, k, v, g = (place(x) for x in (q, k, v, g))
    got = {n: place(torch.zeros_like(x)) for n, x in ref.items()}
    dt, nb = (kd.KD_BF16 if dtype == "bf16" else kd.KD_F32), 0 if ws is None else ws.numel()
    shape = (B, T, H, Hk, d, window, sinks, d ** -0.5, dt)
    assert L.kron_delta_swa_fwd(ptr(q), ptr(k), ptr(v), ptr(got["out"]), ptr(got["lse"]), *shape, ptr(ws), nb, 1, s) == kd.KD_OK
    n = kd.swa_workspace_size(kd.KD_SWA_WS_BWD, B, T, H, Hk, d, window, sinks, dt)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert L.kron_delta_swa_bwd(*(ptr(x) for x in (q, k, v, got["out"], got["lse"], g, got["dq"], got["dk"], got["dv"])),
                                *shape, ptr(ws), nb, ptr(scratch), n, s) == kd.KD_OK
    torch.cuda.synchronize()
    for n, x in ref.items():
        assert torch.equal(got[n], x), n
    assert place.untouched()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_tensors_at_16_bytes(dtype):
    """The same of rotary, the one-token step and the fill of its cache, and the
    recurrence."""
    rng = np.random.default_rng(1)
    place = Placed()
    q, k = (draw(rng, (2, 30, h, 64), dtype)[0] for h in (3, 1))
    f, _ = kd.rotary_freqs(48)
    for inter in (False, True):
        want = kd.rotary_fwd(q, k, f, interleaved=inter)
        a, b = place(q), place(k)
        got = kd.rotary_fwd(a, b, place(f), interleaved=inter, out=(a, b))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    for window in (40, 9000):
        kc, vc = (draw(rng, (2, window + 2, 1, 64), dtype)[0] for _ in range(2))
        lens, pos = torch.tensor([30, 11], device="cuda"), torch.tensor([window + 30, 11], device="cuda")
        ca, cb = place(kc), place(vc)
        v = draw(rng, (2, 30, 1, 64), dtype)[0]
        kd.swa_fill(k, v, lens, kc, vc, window, 2)
        kd.swa_fill(place(k), place(v), place(lens), ca, cb, window, 2)
        one = [x[:, 7].contiguous() for x in (q, k, v)]
        want = kd.swa_decode(*one, kc, vc, pos, window, 2)
        got = kd.swa_decode(*(place(x) for x in one), ca, cb, place(pos), window, 2, out=place(torch.zeros_like(want)))
        assert torch.equal(got, want) and torch.equal(ca, kc) and torch.equal(cb, vc)
    t, _ = glr_inputs(2, 150, 72, dtype, 5)
    want, p = run_glr(t), {n: place(x) for n, x in t.items()}
    B, T, D, dt = 2, 150, 72, kd.KD_BF16 if dtype == "bf16" else kd.KD_F32
    L, s = kd.lib(), torch.cuda.current_stream().cuda_stream
    got = {n: place(torch.zeros_like(x)) for n, x in want.items()}
    sizes = [kd.glr_workspace_size(kind, B, T, D, dt) for kind in (kd.KD_GLR_WS_SAVE, kd.KD_GLR_WS_BWD)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    ins = [ptr(p[n]) for n in ("x", "i_pre", "f_pre", "a_log")]
    assert L.kron_delta_glr_fwd(*ins, ptr(p["h0"]), ptr(got["out"]), ptr(got["hT"]), B, T, D, dt, ptr(ws[0]), sizes[0], 1,
                                s) == kd.KD_OK
    assert L.kron_delta_glr_bwd(*ins, *(ptr(p[n]) for n in ("dh", "dhT")),
                                *(ptr(got[n]) for n in ("dx", "di_pre", "df_pre", "da_log", "dh0")), B, T, D, dt, ptr(ws[0]),
                                sizes[0], ptr(ws[1]), sizes[1], s) == kd.KD_OK
    one = [place(t[n][:, 3].contiguous()) for n in ("x", "i_pre", "f_pre")]
    h, h2 = place(t["h0"]), t["h0"].clone()
    assert torch.equal(kd.glr_decode(*one, p["a_log"], h, out=place(torch.zeros_like(one[0]))),
                       kd.glr_decode(*(x.clone() for x in one), t["a_log"], h2)) and torch.equal(h, h2)
    torch.cuda.synchronize()
    for n, x in want.items():
        assert torch.equal(got[n], x), n
    assert place.untouched()


# ---- how calls are made ---------------------------------------------------------------


def test_arguments_by_name_in_any_order_on_a_stream():
    q, k = torch.randn(1, 40, 2, 32, device="cuda"), torch.randn(1, 40, 1, 32, device="cuda")
    f, _ = kd.rotary_freqs(32)
    want = kd.swa_fwd(q, k, k, 9, 1)[0], kd.rotary_fwd(q, None, f)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kd.swa_fwd(sinks=1, window=9, v=k, k=k, q=q, stream=s)[0], kd.rotary_fwd(k=None, freqs=f, q=q, stream=s)[0]
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_swa_windows_beyond_32_bits():
    """Plain causal attention, forward and backward, with first tokens as without."""
    q, k, g = (torch.randn(1, 300, h, 32, device="cuda") for h in (2, 1, 2))
    want = kd.swa_fwd(q, k, k, 300, save=True)
    grads = kd.swa_bwd(q, k, k, *want[:2], g, 300, fwd_workspace=want[2])
    for window in (2 ** 31, 2 ** 32 + 3, 2 ** 63 - 1):
        got = kd.swa_fwd(q, k, k, window, 1, save=True)
        r = kd.swa_bwd(q, k, k, *got[:2], g, window, 1, fwd_workspace=got[2])
        assert torch.equal(got[0], want[0]) and all(torch.equal(r[n], x) for n, x in grads.items())
