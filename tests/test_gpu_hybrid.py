"""GPU parity of rotary positions, sliding-window attention and the gated
linear recurrence against their fp64 oracles, element by element.

Tolerances follow from the arithmetic.  A rounding to bf16 is off by at most
2^-8 of the value, one to fp32 by 2^-24 (eps / 2).
  rotary  two products and a sum of fp32 table values that are within 2^-22 of
          the sine and cosine (sincospi's 2 ulp and the fraction's rounding):
          4 * 2^-22 of |x1| + |x2|, and the output's rounding.
  swa     oracle.hybrid.swa_bounds, where p and dS are rounded to bf16 before
          their products on the tensor-core path (bf16).
  glr     h is a sum of terms prod f * m i x.  e^{-|z|} carries the rounding of
          its argument (|z| 2^-24, twice with the hardware exponential's own),
          so l = log f is within (6 + 2 |z|) 2^-24 of itself, and f = e^l is
          off by |l| times that, plus 2^-24 for its own rounding.  Over a term's
          steps the l add up: a sum beyond 16 makes the term negligible (e^-16),
          but for its first step, which may have any l (a gate that forgets
          almost all at once, whose small f is all there is).  So a term is off
          by 2^-24 (16 + 2 steps) + (6 + 2 max |z|) 2^-24 (16 + max |l|) of
          itself, steps <= min(T, 16 / min |l|); |l| > 200 gives 0 on both sides.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import delta_rule_linear_kron_b200 as kd  # noqa: E402
from oracle import hybrid as O  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    kd.lib()


def draw(rng, shape, dtype, scale=1.0, mean=0.0):
    """A device tensor of `dtype` and its exact values in fp64."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale + mean).to("cuda", TYPES[dtype])
    return t, host(t)


def host(t):
    return t.detach().double().cpu().numpy()


def within(x, ref, bound, name):
    x = host(x)
    assert np.isfinite(x).all(), name
    bad = np.abs(x - ref) > bound
    at = np.argwhere(bad)[0] if bad.any() else None
    assert not bad.any(), f"{name}: {int(bad.sum())} of {x.size} off, first at {at}: {x[tuple(at)]} {ref[tuple(at)]}"


# ---- rotary positions ---------------------------------------------------------


def check_rotary(B, T, H, Hk, d, rot, dtype, interleaved, start=0, scale=1.0, in_place=False, seed=0):
    rng = np.random.default_rng(seed)
    q, qh = draw(rng, (B, T, H, d), dtype)
    k, kh = draw(rng, (B, T, Hk, d), dtype) if Hk else (None, None)
    freqs = torch.from_numpy(10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)).cuda()
    pos = torch.from_numpy(start + rng.integers(-5, 5, (B, 1)) + np.arange(T)).cuda()
    for fn, inverse in ((kd.rotary_fwd, False), (kd.rotary_bwd, True)):
        a, b = q.clone(), None if k is None else k.clone()
        y = fn(a, b, freqs, pos, interleaved=interleaved, scale=scale, out=(a, b) if in_place else None)
        torch.cuda.synchronize()
        for got, x, name in ((y[0], qh, "q"), (y[1], kh, "k")):
            if x is None:
                assert got is None
                continue
            ref = O.rotary(x, host(freqs), pos.cpu().numpy(), interleaved, scale, inverse)
            size = O.rotary(np.abs(x), 0 * host(freqs), pos.cpu().numpy())  # |x1|, |x2| of a pair
            both = np.array(size)
            half = rot // 2
            i, j = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
            both[..., i] = both[..., j] = size[..., i] + size[..., j]
            bound = 4 * 2.0 ** -22 * scale * both + ROUND[dtype] * np.abs(ref)
            bound[..., rot:] = 0.0  # copied
            within(got, ref, bound, name)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(32, 32), (64, 16), (64, 48), (128, 128), (128, 2), (128, 126), (32, 10)])
def test_rotary_shapes(d, rot, dtype, interleaved):
    check_rotary(2, 37, 5, 3, d, rot, dtype, interleaved, seed=d + rot)


@pytest.mark.parametrize("B,T,H,Hk", [(1, 1, 1, 1), (256, 1, 4, 1), (1, 4097, 2, 1), (3, 33, 7, 0)])
def test_rotary_sizes_and_far_positions(B, T, H, Hk):
    check_rotary(B, T, H, Hk, 64, 64, "f32", False, start=2 ** 33 if T == 1 else 10 ** 6, scale=1.3, seed=T)


def test_rotary_in_place():
    check_rotary(2, 50, 4, 2, 128, 64, "bf16", True, in_place=True)
    check_rotary(2, 50, 4, 2, 128, 64, "bf16", False, in_place=True)


def test_rotary_default_positions_and_one_token_form():
    q = torch.randn(2, 9, 3, 64, device="cuda")
    k = torch.randn(2, 9, 1, 64, device="cuda")
    f, _ = kd.rotary_freqs(64)
    pos = torch.arange(9, device="cuda").expand(2, 9).contiguous()
    a, b = kd.rotary_fwd(q, k, f), kd.rotary_fwd(q, k, f, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = kd.rotary_fwd(q[:, 4].contiguous(), k[:, 4].contiguous(), f, pos[:, 4].contiguous())
    assert torch.equal(one[0], a[0][:, 4]) and torch.equal(one[1], a[1][:, 4])


def test_rotary_autograd_of_queries_alone():
    q = torch.randn(1, 9, 2, 32, device="cuda", requires_grad=True)
    freqs, _ = kd.rotary_freqs(32)
    y, none = kd.RotaryFunction.apply(q, None, freqs)
    g = torch.randn_like(y)
    assert none is None
    assert torch.equal(torch.autograd.grad(y, q, g)[0], kd.rotary_bwd(g, None, freqs)[0])


def test_rotary_autograd():
    q, k = (torch.randn(1, 6, 2, 32, device="cuda", requires_grad=True) for _ in range(2))
    f, s = kd.rotary_freqs(16, scaling="yarn", factor=4.0, trained_len=64)
    y = kd.RotaryFunction.apply(q, k, f, None, True, s)
    w = torch.randn_like(y[0])
    (y[0] * w).sum().backward()
    g = kd.rotary_bwd(w, torch.zeros_like(k), f, interleaved=True, scale=s)
    assert torch.equal(q.grad, g[0]) and not k.grad.any()


# ---- sliding-window attention ---------------------------------------------------


def on_tensor_cores(dtype, d):
    return dtype == "bf16"


def check_swa(B, T, H, Hk, d, window, sinks, dtype, seed=0, size=1.0, scale=None):
    rng = np.random.default_rng(seed)
    (q, qh), (k, kh), (v, vh), (g, gh) = (draw(rng, (B, T, h, d), dtype, size if i < 2 else 1.0)
                                          for i, h in enumerate((H, Hk, Hk, H)))
    out, lse, ws = kd.swa_fwd(q, k, v, window, sinks, scale=scale, save=True)
    r = kd.swa_bwd(q, k, v, out, lse, g, window, sinks, scale=scale, fwd_workspace=ws)
    torch.cuda.synchronize()
    kd.device_status()
    s = scale or d ** -0.5
    ref = O.swa(qh, kh, vh, window, sinks, s, gh)
    bound = O.swa_bounds(qh, kh, vh, window, sinks, s, ref, 2.0 ** -8 if on_tensor_cores(dtype, d) else 0.0,
                         ROUND[dtype], gh)
    for name, x in dict(out=out, lse=lse, **r).items():
        within(x, ref[name], bound[name], name)
    return out, lse, r


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128), ("f32", 64), ("f32", 32)])
@pytest.mark.parametrize("T", [1, 2, 63, 65, 128, 129, 257])
def test_swa_lengths(dtype, d, T):
    check_swa(1, T, 2, 1, d, 50, 2, dtype, seed=T + d)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 128), (2, 3), (64, 0), (127, 1), (128, 4), (129, 65),
                                          (200, 128), (299, 5), (300, 0), (2 ** 31 - 129, 128)])
def test_swa_windows_and_first_tokens(dtype, d, window, sinks):
    check_swa(1, 300, 2, 2, d, window, sinks, dtype, seed=window % 1000 + sinks)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("B,H,Hk", [(2, 3, 3), (2, 6, 2), (1, 8, 1), (3, 5, 1)])
def test_swa_grouped_heads(dtype, d, B, H, Hk):
    check_swa(B, 190, H, Hk, d, 70, 3, dtype, seed=H)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 32)])
def test_swa_sharp_scores(dtype, d):
    """Large scores: probabilities near one-hot, running maxima that move a lot."""
    check_swa(1, 200, 2, 1, d, 90, 2, dtype, seed=1, size=4.0)


@pytest.mark.parametrize("B,T,H,Hk,window,sinks", [(2, 300, 4, 2, 299, 128), (1, 700, 3, 3, 500, 5), (2, 190, 8, 1, 70, 3),
                                                   (1, 2300, 2, 1, 30, 5), (1, 2300, 2, 2, 400, 70)])
def test_swa_heads_of_32(B, T, H, Hk, window, sinks):
    """Half a tile's channels lie outside the tensors: nothing of them is read
    or written (the neighbours in memory are other heads, checked too)."""
    check_swa(B, T, H, Hk, 32, window, sinks, "bf16", seed=T + H)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 32)])
def test_swa_far_queries_of_first_tokens(dtype, d):
    """Longer than one item of far queries (2048): parts are joined."""
    check_swa(1, 2300, 2, 1, d, 30, 5, dtype, seed=9)


def test_swa_one_key_rows_have_exact_gradients():
    """The first query (and every query of a window of one) has one key: out is
    its value and no gradient reaches q and k."""
    rng = np.random.default_rng(2)
    for dtype, d in (("bf16", 128), ("f32", 64)):
        q, k, v, g = (draw(rng, (1, 70, 2, d), dtype)[0] for _ in range(4))
        out, lse, ws = kd.swa_fwd(q, k, v, 1, save=True)
        r = kd.swa_bwd(q, k, v, out, lse, g, 1, fwd_workspace=ws)
        assert torch.equal(out, v) and not r["dq"].any() and not r["dk"].any()
        r = kd.swa_bwd(q, k, v, *kd.swa_fwd(q, k, v, 9, save=True)[:2], g, 9,
                       fwd_workspace=kd.swa_fwd(q, k, v, 9, save=True)[2])
        assert not r["dq"][:, 0].any()


def test_swa_is_reproducible_and_runs_on_another_stream():
    rng = np.random.default_rng(3)
    q, k, v, g = (draw(rng, (2, 400, h, 128), "bf16")[0] for h in (4, 2, 2, 4))

    def both(stream=None):
        out, lse, ws = kd.swa_fwd(q, k, v, 100, 4, save=True, stream=stream)
        r = kd.swa_bwd(q, k, v, out, lse, g, 100, 4, fwd_workspace=ws, stream=stream)
        return [out, lse, r["dq"], r["dk"], r["dv"]]
    a = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = both()
    c = both(s)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_swa_autograd_with_broadcast_key_heads():
    """Gradients of key heads that query heads share: as with repeated heads."""
    T, d = 90, 64
    q = torch.randn(1, T, 4, d, device="cuda", requires_grad=True)
    k, v = (torch.randn(1, T, 2, d, device="cuda", requires_grad=True) for _ in range(2))
    w = torch.randn(1, T, 4, d, device="cuda")
    g = torch.autograd.grad((kd.SwaFunction.apply(q, k, v, 20, 2, None) * w).sum(), (q, k, v))
    kk, vv = k.repeat_interleave(2, 2), v.repeat_interleave(2, 2)
    h = torch.autograd.grad((kd.SwaFunction.apply(q, kk, vv, 20, 2, None) * w).sum(), (q, k, v))
    # the same terms in another order: T * 2 sums of fp32 values
    for x, y in zip(g, h):
        assert torch.allclose(x, y, rtol=0, atol=float(y.abs().max()) * 2 * T * 2 ** -24 * 4)
    with pytest.raises(kd.KronDeltaError):
        kd.SwaFunction.apply(q, k[:, :, :1].expand(1, T, 2, d), v, 20, 2, None)  # not contiguous: refused


# ---- the one-token step and its cache -------------------------------------------


def filled_cache(k, v, lens, window, sinks, fill=float("nan")):
    B, _, Hk, d = k.shape
    kc = torch.full((B, window + sinks, Hk, d), fill, dtype=k.dtype, device="cuda")
    vc = torch.full_like(kc, fill)
    kd.swa_fill(k, v, torch.tensor(lens, device="cuda"), kc, vc, window, sinks)
    return kc, vc


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (16, 0), (30, 7)])
def test_swa_fill_takes_the_newest_token_of_each_slot(window, sinks, dtype):
    rng = np.random.default_rng(window)
    T, lens = 40, [0, 1, 3, 17, 39, 40, 55, -2]
    (k, kh), (v, vh) = (draw(rng, (len(lens), T, 2, 32), dtype) for _ in range(2))
    kc, vc = filled_cache(k, v, lens, window, sinks, fill=7.0)
    ref_k, ref_v = np.full(kc.shape, 7.0), np.full(kc.shape, 7.0)
    for b, n in enumerate(lens):
        for p in range(min(max(n, 0), T)):
            ref_k[b, O.ring_slot(p, window, sinks)], ref_v[b, O.ring_slot(p, window, sinks)] = kh[b, p], vh[b, p]
    # tokens that are neither first nor in the last window are overwritten in the loop above
    assert np.array_equal(host(kc), ref_k) and np.array_equal(host(vc), ref_v)


def check_decode(H, Hk, d, window, sinks, dtype, positions, seed=0):
    """Against the oracle's last row over each sequence's own tokens; slots
    not yet in use hold NaN."""
    rng = np.random.default_rng(seed)
    B, T = len(positions), max(max(positions), 0) + 1
    (q, qh), (k, kh), (v, vh) = (draw(rng, (B, T, h, d), dtype) for h in (H, Hk, Hk))
    kc, vc = filled_cache(k, v, [max(p, 0) for p in positions], window, sinks)
    old = kc.clone(), vc.clone()
    at = torch.tensor([max(p, 0) for p in positions], device="cuda")
    rows = torch.arange(B, device="cuda")
    out = kd.swa_decode(q[rows, at], k[rows, at], v[rows, at], kc, vc, torch.tensor(positions, device="cuda"), window,
                        sinks)
    torch.cuda.synchronize()
    u = ROUND[dtype]
    for b, p in enumerate(positions):
        if p < 0:
            assert not out[b].any()
            assert all(torch.equal(x[b].view(torch.uint8), y[b].view(torch.uint8)) for x, y in zip((kc, vc), old))
            continue
        slot = O.ring_slot(p, window, sinks)
        assert torch.equal(kc[b, slot], k[b, p]) and torch.equal(vc[b, slot], v[b, p])
        seen = [j for j in range(p + 1) if p - j < window or j < sinks]
        n = len(seen)
        for h in range(H):
            kk, vv, qq = kh[b, seen, h // (H // Hk)], vh[b, seen, h // (H // Hk)], qh[b, p, h]
            x = kk @ qq / np.sqrt(d)
            w = np.exp(x - x.max())
            w /= w.sum()
            # scores d + 8 roundings of sum |q||k|, twice; sums of n terms; the output's rounding
            e = 2 * (d + 8) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qq)).max() / np.sqrt(d) + (2 * n + 32) * 2.0 ** -24
            within(out[b, h], w @ vv, e * (w @ np.abs(vv)) + u * np.abs(w @ vv) + 1e-30, f"b {b} h {h}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (3, 1), (5, 1), (16, 2), (20, 1)])
def test_swa_decode_heads(dtype, d, H, Hk):
    check_decode(H, Hk, d, 40, 3, dtype, [0, 1, 2, 3, 41, 42, 43, 44, 100, -1], seed=H + d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 128), (7, 0), (500, 4), (1000, 1), (3000, 2), (9000, 3)])
def test_swa_decode_windows(window, sinks, dtype):
    """One CTA, a cluster's parts, and (9000) parts through the workspace."""
    check_decode(4, 1, 64, window, sinks, dtype, [0, window - 1, window, window + sinks, 2 * window + sinks + 3, -7], seed=window)


def test_swa_decode_far_position():
    """A position beyond 32 bits lands in its slot."""
    window, sinks, p = 11, 3, 2 ** 40 + 5
    k, v = torch.randn(2, 1, 2, 32, device="cuda"), torch.randn(2, 1, 2, 32, device="cuda")
    q = torch.randn(1, 4, 32, device="cuda")
    kc, vc = torch.randn(1, 14, 2, 32, device="cuda"), torch.randn(1, 14, 2, 32, device="cuda")
    ref_k, ref_v = kc.clone(), vc.clone()
    slot = sinks + (p - sinks) % window
    ref_k[0, slot], ref_v[0, slot] = k[0, 0], v[0, 0]
    out = kd.swa_decode(q, k[0], v[0], kc, vc, torch.tensor([p], device="cuda"), window, sinks)
    assert torch.equal(kc, ref_k) and torch.equal(vc, ref_v)
    x = torch.einsum("hd,shd->hs", q[0].double(), ref_k[0].double().repeat_interleave(2, 1)) / 32 ** 0.5
    ref = torch.einsum("hs,shd->hd", torch.softmax(x, -1), ref_v[0].double().repeat_interleave(2, 1))
    assert torch.allclose(out[0].double(), ref, rtol=1e-5, atol=1e-5)


def test_swa_decode_captured_graphs_with_their_own_workspaces():
    """Two captured steps, replayed in turn and on two streams, each with its
    own workspace, equal the eager steps."""
    args = []
    for seed in (0, 1):
        torch.manual_seed(seed)
        B, H, Hk, d, window, sinks = 2, 4, 2, 128, 9000, 4
        a = dict(q=torch.randn(B, H, d, device="cuda").bfloat16(), k=torch.randn(B, Hk, d, device="cuda").bfloat16(),
                 v=torch.randn(B, Hk, d, device="cuda").bfloat16(),
                 k_cache=torch.randn(B, window + sinks, Hk, d, device="cuda").bfloat16(),
                 v_cache=torch.randn(B, window + sinks, Hk, d, device="cuda").bfloat16(),
                 pos=torch.tensor([12000, 350], device="cuda"), window=window, sinks=sinks)
        n = kd.swa_workspace_size(kd.KD_SWA_WS_DECODE, B, 1, H, Hk, d, window, sinks, kd.KD_BF16)
        assert n > 0  # a split cache
        a["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        a["out"] = torch.empty_like(a["q"])
        args.append(a)
    ref = [kd.swa_decode(**a).clone() for a in args]
    torch.cuda.synchronize()
    graphs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kd.swa_decode(**a)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for a in args:
        a["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, r in zip(args, ref):
        assert torch.equal(a["out"], r)


# ---- gated linear recurrence ------------------------------------------------------


def glr_inputs(B, T, D, dtype, seed, h0=True, mean=3.0):
    rng = np.random.default_rng(seed)
    t, r = {}, {}
    for n in ("x", "i_pre", "f_pre", "dh"):
        t[n], r[n] = draw(rng, (B, T, D), dtype, mean=mean if n == "f_pre" else 0.0)
    t["a_log"], r["a_log"] = draw(rng, (D,), "f32", scale=0.5)
    for n in ("h0", "dhT"):
        t[n], r[n] = draw(rng, (B, D), "f32") if h0 else (None, None)
    return t, r


def run_glr(t):
    a = (t["x"], t["i_pre"], t["f_pre"], t["a_log"], t["h0"])
    out, hT, ws = kd.glr_fwd(*a, save=True)
    g = kd.glr_bwd(*a, t["dh"], t["dhT"], fwd_workspace=ws)
    torch.cuda.synchronize()
    return dict(out=out, hT=hT, **g)


def check_glr(t, r, dtype):
    got, ref = run_glr(t), O.glr(**r)
    T = r["x"].shape[1]
    l, f, m, i = O.glr_gates(r["f_pre"], r["i_pre"], r["a_log"])
    steps = np.minimum(T, 16 / np.maximum(-l.max((0, 1)), 1e-9))           # [D]
    z, lmax = np.abs(np.clip(r["f_pre"], -100, 100)).max(), np.minimum(-l, 200).max()
    e = 2.0 ** -24 * (16 + 2 * steps + (6 + 2 * z) * (16 + lmax))
    absr = dict(r, x=np.abs(r["x"]), dh=np.abs(r["dh"]), h0=None if r["h0"] is None else np.abs(r["h0"]),
                dhT=None if r["dhT"] is None else np.abs(r["dhT"]))
    mag = O.glr(**absr)                                                     # the sums of magnitudes
    u = ROUND[dtype]
    within(got["out"], ref["out"], e * mag["out"] + u * np.abs(ref["out"]) + 1e-30, "out")
    within(got["hT"], ref["hT"], e * mag["hT"] + 1e-30, "hT")
    within(got["dh0"], ref["dh0"], e * mag["dh0"] + 1e-30, "dh0")
    # each gradient is g (and h_{t-1}) times gate factors within 16 * 2^-24
    for n, factor in (("dx", m * i), ("di_pre", m * np.abs(r["x"]) * i * O.sigmoid(-r["i_pre"]))):
        within(got[n], ref[n], 2 * e * mag["g"] * factor + u * np.abs(ref[n]) + 1e-30, n)
    before = np.concatenate([np.zeros_like(mag["out"][:, :1]) if r["h0"] is None else absr["h0"][:, None],
                             mag["out"][:, :-1]], 1)
    dm = np.divide(f * f, m, out=np.zeros_like(m), where=m > 0)
    terms = mag["g"] * (before * f + i * absr["x"] * dm)
    a = np.exp(r["a_log"]) * O.sigmoid(-r["f_pre"])
    within(got["df_pre"], ref["df_pre"], 4 * e * terms * a + u * np.abs(ref["df_pre"]) + 1e-30, "df_pre")
    n = r["x"].shape[0] * T
    within(got["da_log"], ref["da_log"], (4 * e + n * 2.0 ** -24) * (terms * np.abs(np.maximum(l, -1e30))).sum((0, 1))
           + 1e-30, "da_log")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 63, 64, 65, 513, 1000])
def test_glr_lengths(dtype, T):
    check_glr(*glr_inputs(2, T, 72, dtype, T, h0=T % 2 == 0), dtype)


@pytest.mark.parametrize("B,D", [(1, 8), (3, 64), (1, 136), (5, 1000)])
def test_glr_sizes(B, D):
    check_glr(*glr_inputs(B, 150, D, "bf16", D), "bf16")


@pytest.mark.parametrize("mean", [-8.0, 0.0, 7.0])
def test_glr_gate_ranges(mean):
    """Gates that forget at once, and gates that keep for thousands of steps."""
    check_glr(*glr_inputs(1, 700, 64, "f32", 3, mean=mean), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_glr_extreme_gates(dtype):
    """f_pre at -inf and at the type's lowest value starts a new sequence, at
    the largest it keeps the state; saturated input gates."""
    t, r = glr_inputs(1, 200, 64, dtype, 4)
    low, high = torch.finfo(TYPES[dtype]).min, torch.finfo(TYPES[dtype]).max
    for at, v in ((0, -np.inf), (10, low), (64, -np.inf), (65, low), (127, 300.0), (130, high), (199, high)):
        t["f_pre"][:, at] = v
        r["f_pre"][:, at] = float(t["f_pre"][0, at, 0])
    t["i_pre"][:, 20], r["i_pre"][:, 20] = -np.inf, -np.inf
    t["i_pre"][:, 21], r["i_pre"][:, 21] = high, high
    with np.errstate(over="ignore", invalid="ignore"):
        check_glr(t, r, dtype)
    # packed sequences: a reset makes what follows independent of what came before
    a = (t["i_pre"], t["f_pre"], t["a_log"])
    one = kd.glr_fwd(t["x"], *a, t["h0"])[0]
    x = t["x"].clone()
    x[:, :10] = 5.0
    assert torch.equal(kd.glr_fwd(x, *a, None)[0][:, 10:], one[:, 10:])


def test_glr_steps_equal_the_sequence():
    t, _ = glr_inputs(3, 40, 64, "f32", 6)
    out, hT, _ = kd.glr_fwd(t["x"], t["i_pre"], t["f_pre"], t["a_log"], t["h0"])
    h = t["h0"].clone()
    for n in range(40):
        o = kd.glr_decode(*(t[k][:, n].contiguous() for k in ("x", "i_pre", "f_pre")), t["a_log"], h)
        # the same fp32 steps, combined in another order: 40 roundings of the magnitudes
        assert torch.allclose(o, out[:, n], rtol=0, atol=80 * 2 ** -24 * 8)
    assert torch.allclose(h, hT, rtol=0, atol=80 * 2 ** -24 * 8)


def test_glr_autograd_and_reproducible():
    t, _ = glr_inputs(2, 300, 136, "bf16", 8)
    a = [t[n].clone().requires_grad_() for n in ("x", "i_pre", "f_pre", "a_log", "h0")]
    out, hT = kd.GlrFunction.apply(*a)
    torch.autograd.backward([out, hT], [t["dh"], t["dhT"]])
    one, two = run_glr(t), run_glr(t)
    for n in one:
        assert torch.equal(one[n], two[n])
    for x, n in zip(a, ("dx", "di_pre", "df_pre", "da_log", "dh0")):
        assert torch.equal(x.grad, one[n])


# ---- a layer's run of them ----------------------------------------------------------


def test_prefill_then_steps_equal_the_whole_sequence():
    """Rotary, window attention and the recurrence over a prompt, then token by
    token over the caches: the same rows as over the whole sequence."""
    torch.manual_seed(0)
    B, T, P, H, Hk, d, window, sinks = 2, 150, 100, 4, 2, 64, 40, 3
    q, k, v = (torch.randn(B, T, h, d, device="cuda") for h in (H, Hk, Hk))
    zi, zf = (torch.randn(B, T, H * d, device="cuda") + m for m in (0, 3))
    a_log = torch.rand(H * d, device="cuda")
    freqs, s = kd.rotary_freqs(d, scaling="yarn", factor=4.0, trained_len=64)

    def mix(q, k, v, pos):
        return (*kd.rotary_fwd(q, k, freqs, pos, scale=s), v)
    pos = torch.arange(T, device="cuda").expand(B, T).contiguous()
    qr, kr, _ = mix(q, k, v, pos)
    whole = kd.swa_fwd(qr, kr, v, window, sinks)[0]
    y = kd.glr_fwd(whole.view(B, T, H * d), zi, zf, a_log)[0]
    kc, vc = (torch.full((B, window + sinks, Hk, d), float("nan"), device="cuda") for _ in range(2))
    kd.swa_fill(kr[:, :P].contiguous(), v[:, :P].contiguous(), torch.tensor([P, P], device="cuda"), kc, vc, window, sinks)
    h = kd.glr_fwd(whole[:, :P].reshape(B, P, H * d).contiguous(), zi[:, :P].contiguous(), zf[:, :P].contiguous(), a_log)[1]
    for n in range(P, T):
        qn, kn, vn = mix(*(x[:, n].contiguous() for x in (q, k, v)), pos[:, n].contiguous())
        o = kd.swa_decode(qn, kn, vn, kc, vc, pos[:, n].contiguous(), window, sinks)
        # both are within the fp32 bounds of the exact row: (d + 8) roundings of the scores' magnitudes
        e = 4 * (d + 8) * 2 ** -24 * float((q[:, n].abs().amax() * k.abs().amax()) * d ** 0.5) * s * s * 2
        assert torch.allclose(o, whole[:, n], rtol=0, atol=e * float(v.abs().max()))
        o = kd.glr_decode(whole[:, n].reshape(B, H * d).contiguous(), zi[:, n].contiguous(), zf[:, n].contiguous(), a_log, h)
        assert torch.allclose(o, y[:, n], rtol=0, atol=200 * 2 ** -24 * float(y.abs().max()) * 4)


def test_training_step_through_the_layer_by_differences():
    """Gradients of rotary -> attention -> recurrence against central
    differences of the loss, summed in 64 bits: the differences' own error is
    the loss's fp32 error over the step."""
    torch.manual_seed(1)
    B, T, H, Hk, d = 1, 70, 2, 1, 32
    q, k, v = (torch.randn(B, T, h, d, device="cuda", requires_grad=True) for h in (H, Hk, Hk))
    zi, zf = (torch.randn(B, T, H * d, device="cuda", requires_grad=True) for _ in range(2))
    a_log = torch.zeros(H * d, device="cuda", requires_grad=True)
    freqs, _ = kd.rotary_freqs(d)
    w = torch.randn(B, T, H * d, device="cuda")

    def loss():
        a, b = kd.RotaryFunction.apply(q, k, freqs)
        o = kd.SwaFunction.apply(a, b, v, 20, 2)
        y, _ = kd.GlrFunction.apply(o.view(B, T, H * d), zi, zf, a_log)
        return y, (y.double() * w.double()).sum()
    y, l = loss()
    grads = torch.autograd.grad(l, (q, k, v, zi, zf, a_log))
    size = float((y.detach().double().abs() * w.double().abs()).sum())
    for x, g in zip((q, k, v, zi, zf, a_log), grads):
        assert torch.isfinite(g).all()
        u = torch.randn_like(x)
        step = 1e-2 / float(u.norm())
        with torch.no_grad():
            x.add_(step * u)
            up = loss()[1]
            x.sub_(2 * step * u)
            down = loss()[1]
            x.add_(step * u)
        want, got = float((up - down) / (2 * step)), float((g.double() * u.double()).sum())
        # fp32 noise of the two losses over the step; the third-order term of a 1e-2 step is below 1e-3
        assert abs(want - got) <= 1e-3 * float((g.double() ** 2).sum() ** 0.5 * u.norm()) + 64 * 2 ** -24 * size / step


def test_a_thread_without_a_context_can_call():
    """The first CUDA work of a fresh thread is one of these calls."""
    import threading
    t, _ = glr_inputs(1, 70, 64, "bf16", 1)
    a = (t["x"], t["i_pre"], t["f_pre"], t["a_log"], t["h0"])
    q = torch.randn(1, 70, 2, 64, device="cuda").bfloat16()
    want = kd.glr_fwd(*a)[0], kd.swa_fwd(q, q, q, 9)[0]
    torch.cuda.synchronize()
    outs = torch.empty_like(a[0]), torch.empty_like(q)
    lib, stream, p = kd.lib(), torch.cuda.current_stream().cuda_stream, lambda x: x.data_ptr()  # noqa: E731
    lse = torch.empty(1, 70, 2, device="cuda")
    rc = []

    def work():
        rc.append(lib.kron_delta_glr_fwd(*(p(x) for x in a), p(outs[0]), None, 1, 70, 64, 1, None, 0, 0, stream))

    def more():
        rc.append(lib.kron_delta_swa_fwd(p(q), p(q), p(q), p(outs[1]), p(lse), 1, 70, 2, 2, 64, 9, 0, 0.125, 1, None, 0,
                                         0, stream))
    for f in (work, more):
        th = threading.Thread(target=f)
        th.start()
        th.join()
    torch.cuda.synchronize()
    assert rc == [kd.KD_OK, kd.KD_OK]
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_captured_training_step_replays_on_new_inputs(dtype):
    """Forward and backward of all three in one graph, by their functions and
    by autograd: replayed after the inputs changed, it gives the eager results."""
    B, T, H, Hk, d, window, sinks = 2, 300, 4, 2, 64, 30, 3
    rng = np.random.default_rng(5)
    shapes = [(B, T, H, d), (B, T, Hk, d), (B, T, Hk, d), (B, T, H * d), (B, T, H * d), (B, T, H * d)]
    new = [draw(rng, s, dtype)[0] for s in shapes]
    x = [n.clone() for n in new]
    a_log = torch.rand(H * d, device="cuda")
    freqs, _ = kd.rotary_freqs(d)

    def calls():
        q, k, v, zi, zf, g = x
        qr, kr = kd.rotary_fwd(q, k, freqs)
        o, lse, ws = kd.swa_fwd(qr, kr, v, window, sinks, save=True)
        y, _, gw = kd.glr_fwd(o.view(B, T, H * d), zi, zf, a_log, save=True)
        r = kd.glr_bwd(o.view(B, T, H * d), zi, zf, a_log, None, g, fwd_workspace=gw)
        s = kd.swa_bwd(qr, kr, v, o, lse, r["dx"].view(B, T, H, d), window, sinks, fwd_workspace=ws)
        return [y, r["di_pre"], r["df_pre"], r["da_log"], s["dv"], *kd.rotary_bwd(s["dq"], s["dk"], freqs)]

    def graded():
        leaves = [t.detach().requires_grad_() for t in x[:5]] + [a_log.detach().requires_grad_()]
        q, k, v, zi, zf, a = leaves
        qr, kr = kd.RotaryFunction.apply(q, k, freqs)
        y, _ = kd.GlrFunction.apply(kd.SwaFunction.apply(qr, kr, v, window, sinks).view(B, T, H * d), zi, zf, a)
        dq, dk, dv, di, df, da = torch.autograd.grad(y, leaves, x[5])
        return [y.detach(), di, df, da, dv, dq, dk]
    for fn in (calls, graded):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fn()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fn()
        for _ in range(2):
            for a, n in zip(x, new):
                a.copy_(n.roll(1, 1))
            new = [n.roll(1, 1) for n in new]
            want = fn()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        assert kd.device_status() is None
