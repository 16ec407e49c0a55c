"""Sliding-window attention and the gated linear recurrence at the shapes of
real layers, against their fp64 oracles: loops long enough that every ring,
barrier phase and carry comes round again.

Tolerances: those of test_gpu_hybrid, with the attention's at
tests.test_hybrid_bounds.tight_bounds (which says why, and shows that the
kernels' extra parts cannot be lost within them)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import delta_rule_linear_kron_b200 as kd  # noqa: E402
from oracle import hybrid as O  # noqa: E402
from tests.test_gpu_hybrid import ROUND, check_glr, draw, glr_inputs, within  # noqa: E402
from tests.test_hybrid_bounds import tight_bounds  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    kd.lib()


# ---- the recurrence: more steps than a step's buffers ------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", [
    (1, 2600, 72),     # clusters of 8: 41 chunks in 6 steps, the last with one chunk
    (2, 2100, 264),    # clusters of 8: 33 chunks in 5 steps
    (3, 1100, 1000),   # clusters of 4 (48 channel blocks): 18 chunks in 5 steps
    (5, 600, 1000),    # clusters of 2 (80): 10 chunks in 5 steps
    (10, 330, 1000),   # no clusters (160): 6 chunks, the last with 10 tokens
    (2, 500, 4800),    # no clusters (150): 8 chunks
])
def test_glr_long_sequences(B, T, D, dtype):
    check_glr(*glr_inputs(B, T, D, dtype, T, h0=T % 200 != 0), dtype)


# ---- the attention: layers' shapes -----------------------------------------------------


def check_swa(B, T, H, Hk, d, window, sinks, dtype, seed=0):
    rng = np.random.default_rng(seed)
    (q, qh), (k, kh), (v, vh), (g, gh) = (draw(rng, (B, T, h, d), dtype) for h in (H, Hk, Hk, H))
    out, lse, ws = kd.swa_fwd(q, k, v, window, sinks, save=True)
    r = kd.swa_bwd(q, k, v, out, lse, g, window, sinks, fwd_workspace=ws)
    torch.cuda.synchronize()
    kd.device_status()
    a = (qh, kh, vh, window, sinks, d ** -0.5)
    ref = O.swa(*a, gh)
    if dtype == "bf16":
        bound = tight_bounds(*a, ref, fine=min(window + sinks, T) <= 256, u_out=ROUND[dtype], dO=gh)
    else:
        bound = O.swa_bounds(*a, ref, 0.0, ROUND[dtype], gh)
    for name, x in dict(out=out, lse=lse, **r).items():
        within(x, ref[name], bound[name], name)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (50, 2), (127, 1), (128, 4), (128, 128), (255, 1), (300, 0)])
def test_swa_rows_of_few_keys_keep_both_parts(window, sinks, d):
    """Rows of at most 256 keys (and the first that have more)."""
    check_swa(1, 300, 2, 1, d, window, sinks, "bf16", seed=window + sinks)


@pytest.mark.parametrize("T", [1, 2, 65, 128, 129, 256, 257])
def test_swa_short_sequences_keep_both_parts(T):
    check_swa(1, T, 2, 1, 128, 2 ** 30, 0, "bf16", seed=T)


WRAPS = (1, 1500, 4, 2, 600, 4)    # ring of tiles wraps, grouped heads, far queries of first tokens
PIECES = (1, 2300, 2, 1, 400, 70)  # two far pieces
FEW = (1, 2300, 2, 1, 30, 5)       # the same with rows of few keys
MEET = (2, 1100, 3, 3, 1023, 128)  # band and far queries meet in the last tile
CAUSAL = (1, 1400, 5, 1, 1400, 0)


@pytest.mark.parametrize("d,dtype,B,T,H,Hk,window,sinks", [(128, "bf16", *c) for c in (WRAPS, PIECES, FEW, MEET, CAUSAL)] +
                         [(64, "bf16", *c) for c in (WRAPS, MEET)] + [(128, "f32", *c) for c in (WRAPS, MEET)])
def test_swa_layers(B, T, H, Hk, window, sinks, d, dtype):
    check_swa(B, T, H, Hk, d, window, sinks, dtype, seed=T + window)


# ---- the one-token step: rings that come round, every width -----------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,H,Hk,window,sinks", [
    (150, 2, 2, 600, 4),    # one CTA to a cache: up to 10 tiles of each warp
    (40, 10, 2, 900, 3),    # three parts
    (2, 4, 1, 3000, 2),     # a cluster of 8, or parts through the workspace
    (1, 16, 4, 9000, 0),    # the workspace
    (2, 20, 1, 40000, 1),   # more heads than a product's rows
])
def test_swa_decode_long_caches(B, H, Hk, window, sinks, d, dtype):
    """Against softmax in 64 bits over the slots in use; the others hold NaN."""
    rng = np.random.default_rng(B + window)
    n = window + sinks
    (q, _), (k, _), (v, _) = (draw(rng, (B, h, d), dtype) for h in (H, Hk, Hk))
    kc, vc = (torch.randn(B, n, Hk, d, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).to(q.dtype)
              for s in (1, 2))
    pos = torch.from_numpy(rng.integers(0, 2 * n, B)).cuda()
    pos[0] = n - 1
    pos[B // 2] = n + 17
    used = (pos + 1).clamp(max=n)
    unused = torch.arange(n, device="cuda")[None] >= used[:, None]
    slot = torch.where(pos < sinks, pos, sinks + (pos - sinks) % window)
    unused[torch.arange(B), slot] = True  # the new token's slot is written, not read
    kc[unused] = vc[unused] = float("nan")
    got = kd.swa_decode(q, k, v, kc, vc, pos, window, sinks).double()
    rows = torch.arange(B, device="cuda")
    assert torch.equal(kc[rows, slot], k) and torch.equal(vc[rows, slot], v)
    G, scale = H // Hk, d ** -0.5
    for b in range(B):
        kk, vv = (c[b, :used[b]].double().permute(1, 0, 2) for c in (kc, vc))       # [Hk, slots, d]
        qq = q[b].double().view(Hk, G, d)
        p = torch.softmax(qq @ kk.transpose(1, 2) * scale, -1)
        ref, mag = p @ vv, p @ vv.abs()
        # as test_gpu_hybrid.check_decode: d + 8 roundings of the scores' magnitudes, twice; sums of the slots in use;
        # weights in two bf16 parts; a product that tensor cores cut off counts two roundings
        worst = (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale
        e = 2 * (2 * (d + 8) * 2.0 ** -24 * worst + (2 * float(used[b]) + 32) * 2.0 ** -24)
        if dtype == "bf16":
            e = e + 2.0 ** -16
        assert bool(((got[b].view(Hk, G, d) - ref).abs() <= e * mag + ROUND[dtype] * ref.abs() + 1e-30).all()), b


# ---- offsets that pass 32 bits ------------------------------------------------------------


@pytest.fixture
def memory():
    yield
    torch.cuda.empty_cache()


FAR = 2 ** 20  # 2^20 tokens of 16 heads of 128: 2^31 elements


def randn(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(*shape, device="cuda", dtype=dtype, generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("dtype,Hk", [("bf16", 16), ("f32", 2)])
def test_swa_offsets_beyond_32_bits(memory, dtype, Hk):
    """The rows behind 2^31 elements are bitwise those of a sequence that starts
    256 tokens before them (a window of 64, the same tiles)."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, g = (randn(1, FAR + 300, h, 128, dtype=t, seed=i) for i, h in enumerate((16, Hk, Hk, 16)))

    def both(q, k, v, g):
        out, lse, ws = kd.swa_fwd(q, k, v, 64, save=True)
        return dict(out=out, lse=lse, **kd.swa_bwd(q, k, v, out, lse, g, 64, fwd_workspace=ws))
    want = both(*(x[:, FAR - 256:].contiguous() for x in (q, k, v, g)))
    got = both(q, k, v, g)
    for n, x in want.items():
        assert torch.isfinite(x[:, 256:]).all() and torch.equal(got[n][:, FAR:], x[:, 256:]), n
    kd.device_status()


def test_rotary_and_glr_offsets_beyond_32_bits(memory):
    q = randn(1, FAR + 300, 16, 128)
    f, _ = kd.rotary_freqs(128)
    pos = torch.arange(FAR, FAR + 300, device="cuda")[None]
    got = kd.rotary_fwd(q, None, f, out=(q, None))[0][:, FAR:].clone()
    q = randn(1, FAR + 300, 16, 128)[:, FAR:].contiguous()
    assert torch.equal(got, kd.rotary_fwd(q, None, f, pos)[0])
    del q
    x, i, z = (randn(1, FAR + 300, 2048, seed=s) for s in (1, 2, 3))
    z[:, FAR - 512] = -float("inf")  # a new sequence, at the start of a step of its cluster
    a, g = torch.zeros(2048, device="cuda"), randn(1, FAR + 300, 2048, seed=4)

    def both(x, i, z, g):
        out, hT, ws = kd.glr_fwd(x, i, z, a, save=True)
        r = kd.glr_bwd(x, i, z, a, None, g, fwd_workspace=ws)
        return dict(out=out, hT=hT[:, None].expand(1, 812, 2048), dx=r["dx"], di_pre=r["di_pre"], df_pre=r["df_pre"])
    want = both(*(y[:, FAR - 512:].contiguous() for y in (x, i, z, g)))
    got = both(x, i, z, g)
    for n, y in want.items():
        assert torch.isfinite(y).all() and torch.equal(got[n][:, -300:], y[:, -300:]), n
    kd.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swa_decode_offsets_beyond_32_bits(memory, dtype):
    """Caches on both sides of 2^31 elements: their fill, and full ones whose
    first and last slots alone have weight."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Hk, d, window = 3, 8, 128, 2 ** 20 + 7  # 2^30 elements and some to a sequence
    kc, vc = (torch.zeros(B, window, Hk, d, dtype=t, device="cuda") for _ in range(2))
    k, v = randn(B, 40, Hk, d, dtype=t, seed=1), randn(B, 40, Hk, d, dtype=t, seed=2)
    q1, k1, v1 = (randn(B, Hk, d, dtype=t, seed=s) for s in (3, 4, 5))
    small = [torch.zeros(B, 64, Hk, d, dtype=t, device="cuda") for _ in range(2)]
    lens = torch.full((B,), 40, device="cuda")
    kd.swa_fill(k, v, lens, kc, vc, window)
    kd.swa_fill(k, v, lens, *small, 64)
    assert torch.equal(kc[:, :64], small[0]) and torch.equal(vc[:, :64], small[1]) and not kc[:, 64:].any()
    # full caches: 40 keys at the front, 41 at the end, the last one the new token; all the others weigh nothing
    kc[:, 40:, :, 0] = -float("inf")
    kc[:, -41:-1], vc[:, -41:-1] = k, v
    q1[..., 0] = 1.0
    pos = torch.full((B,), window - 1, device="cuda")
    got = kd.swa_decode(q1, k1, v1, kc, vc, pos, window).double()
    assert torch.equal(kc[:, -1], k1) and torch.equal(vc[:, -1], v1)
    kk, vv = (torch.cat((x, x, y[:, None]), 1).double().transpose(1, 2) for x, y in ((k, k1), (v, v1)))  # [B, Hk, 81, d]
    p = torch.softmax((kk @ q1.double()[..., None])[..., 0] * d ** -0.5, -1)
    ref, mag = (p[..., None, :] @ vv)[..., 0, :], (p[..., None, :] @ vv.abs())[..., 0, :]
    # scores of d + 8 roundings of their magnitudes, twice; 81 keys; weights in two bf16 parts; all but those taken twice
    worst = (kk.abs() @ q1.double().abs()[..., None])[..., 0].amax(-1)[..., None] * d ** -0.5
    e = 2 * (2 * (d + 8) * 2.0 ** -24 * worst + (2 * 81 + 32) * 2.0 ** -24) + 2.0 ** -16
    assert bool(((got - ref).abs() <= e * mag + ROUND[dtype] * ref.abs()).all())
