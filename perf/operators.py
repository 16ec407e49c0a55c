"""What is measured of the hybrid-stack operators, and their plain forms.

Three token mixers' operators that stand beside the Kronecker delta rule in a hybrid stack:

rotary   rotary positions of q and k (half or interleaved pairs, part of the head, scaled frequencies, far positions),
         and the backward rotation.
swa      causal attention over a sliding window with a few first tokens that stay visible: query t sees key j when
         j <= t and (t - j < window or j < sinks).  Grouped heads; forward, training step, the one-token step over a
         ring cache of sinks + window slots, and the fill of that cache after a prefill.
glr      the element-wise gated linear recurrence h_t = f_t h_{t-1} + sqrt(1 - f_t^2) sigmoid(i_pre_t) x_t with
         f_t = sigmoid(f_pre_t)^exp(a_log): forward, training step, one-token step.

`run` computes them in elementary torch operations in 32 bits (angles in 64), or through the package where `own` is
set.  `exact` computes them in 64 bits, apart from the plain forms.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kd():
    import delta_rule_linear_kron_b200 as kd
    return kd


# ---- cases -----------------------------------------------------------------------------------------------------------

def _rotary(name, **kw):
    c = dict(op="rotary", dir="fwd", B=1, T=1, H=16, Hk=4, d=128, rot=128, interleaved=False, dtype="bf16",
             base=10000.0, scaling="none", factor=1.0, start=0, far=0)
    c.update(kw)
    return _named(name, c)


def _swa(name, **kw):
    c = dict(op="swa", dir="fwd", B=1, T=1, H=16, Hk=4, d=128, window=2048, sinks=4, dtype="bf16")
    c.update(kw)
    return _named(name, c)


def _glr(name, **kw):
    c = dict(op="glr", dir="fwd", B=1, T=1, D=2048, h0=True, dtype="bf16")
    c.update(kw)
    return _named(name, c)


def _named(name, c):
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the queries and keys of one long prompt, frequencies stretched for a context eight times the trained one
        _rotary("rotary-prefill-16k", T=16384, scaling="yarn", factor=8.0),
        # one token of each of 256 requests, at far positions; a quarter of the head turns, in interleaved pairs
        _rotary("rotary-step-256", B=256, T=1, rot=32, interleaved=True, far=1 << 20),
        # gradients of a training batch kept in 32 bits, ragged length
        _rotary("rotary-back-f32", dir="bwd", B=3, T=2047, H=8, Hk=8, d=64, rot=64, dtype="f32", start=5),
        # the prefill of a long prompt in the layer of a hybrid stack whose window is 2048
        _swa("swa-prefill-16k", T=16384),
        # the same layer's training step at the benchmark's length
        _swa("swa-train-16k", dir="train", T=16384, Hk=16),
        # a ragged training batch of short documents, narrow window, one first token kept
        _swa("swa-train-ragged", dir="train", B=3, T=1357, H=8, Hk=2, d=64, window=200, sinks=1),
        # the tiny 32-bit setting that the repository's parity runs use
        _swa("swa-train-f32-tiny", dir="train", T=256, H=2, Hk=2, d=32, window=64, sinks=3, dtype="f32"),
        # serving: one token of each of 256 requests, caches partly and wholly filled
        _swa("swa-step-256", dir="decode", B=256, T=6000),
        # serving: a single request, where the call's own latency counts
        _swa("swa-step-1", dir="decode", T=6000),
        # the recurrence's training step at the benchmark's length and width (16 heads of 128)
        _glr("glr-train-16k", dir="train", T=16384),
        # a ragged prefill in 32 bits, without a first state
        _glr("glr-prefill-f32", B=3, T=999, D=264, h0=False, dtype="f32"),
        # serving: one token of each of 256 requests
        _glr("glr-step-256", dir="decode", B=256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 4, 5, 8])
    op = rng.choice(["rotary", "swa", "swa", "glr"])
    if op == "rotary":
        direction = rng.choice(["fwd", "bwd"])
        B = _log(rng, 1, 256)
        T = _log(rng, 1, max(1, 16384 * 20 * 128 // (B * (H + Hk) * d)))
        T = min(T, 16384)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return _rotary("", dir=direction, B=B, T=T, H=H, Hk=Hk, d=d, rot=rng.choice([d // 4, d // 2, 3 * d // 4, d]),
                       interleaved=rng.random() < 0.5, dtype=dtype, base=rng.choice([10000.0, 500000.0]),
                       scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                       start=rng.choice([0, 0, 17, 100003]), far=rng.choice([0, 0, 1 << 20]))
    if op == "swa":
        direction = rng.choice(["fwd", "train", "decode", "fill"])
        window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 3, 4, 16, 63, 128])
        if direction in ("fwd", "train"):
            # 32-bit values and heads of 32 channels do not reach the tensor cores: an eighth of the work for them
            most = 16 * 16384 * 2048 // (1 if dtype == "bf16" and d >= 64 else 8)
            B = _log(rng, 1, 4)
            T = _log(rng, 1, 16384)
            while B * H * T * min(T, window + sinks + 256) > most:
                T = T * 3 // 4
        else:
            B = _log(rng, 1, 256)
            T = _log(rng, 1, 9000)
            while B * Hk * d * (window + sinks + (T if direction == "fill" else 0)) > 256 * 4 * 128 * 2052:
                window, T, B = max(1, window // 2), max(1, T * 3 // 4), max(1, B * 3 // 4)
        return _swa("", dir=direction, B=B, T=T, H=H, Hk=Hk, d=d, window=window, sinks=sinks, dtype=dtype)
    direction = rng.choice(["fwd", "train", "decode"])
    D = 8 * _log(rng, 1, 512)
    if direction == "decode":
        return _glr("", dir=direction, B=_log(rng, 1, 256), D=D, dtype=dtype)
    B = _log(rng, 1, 16)
    T = min(16384, _log(rng, 1, max(1, 16384 * 2048 // (B * D))))
    return _glr("", dir=direction, B=B, T=T, D=D, h0=rng.random() < 0.5, dtype=dtype)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    if case["op"] == "rotary":
        n = B * T * (case["H"] + case["Hk"])
        return {"bytes": 2 * es * n * case["d"] + 8 * B * T, "flops": 3 * n * case["rot"]}
    if case["op"] == "swa":
        H, Hk, d, W, S = case["H"], case["Hk"], case["d"], case["window"], case["sinks"]
        if case["dir"] == "fill":
            n = sum(min(p + 1, W + S) for p in _positions(case))
            return {"bytes": 4 * es * n * Hk * d, "flops": 0}
        if case["dir"] == "decode":
            n = sum(min(p + 1, W + S) for p in _positions(case) if p >= 0)
            return {"bytes": 2 * es * n * Hk * d + 2 * es * B * (H + 2 * Hk) * d, "flops": 4 * n * H * d}
        pairs = sum(min(t + 1, W + min(S, max(0, t + 1 - W))) for t in range(T)) * B * H
        q, k = B * T * H * d * es, B * T * Hk * d * es
        if case["dir"] == "fwd":
            return {"bytes": 2 * q + 2 * k + 4 * B * T * H, "flops": 4 * pairs * d}
        return {"bytes": 4 * q + 4 * k, "flops": 14 * pairs * d}
    n = B * T * case["D"]
    if case["dir"] == "decode":
        return {"bytes": (4 * es + 8) * B * case["D"], "flops": 30 * B * case["D"]}
    if case["dir"] == "fwd":
        return {"bytes": 4 * es * n, "flops": 30 * n}
    return {"bytes": 8 * es * n, "flops": 75 * n}


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _positions(case):
    """The position of each request's new token: most caches wrapped, some filling, the first one at its start."""
    B, T = case["B"], case["T"]
    return [T - 1] if B == 1 else [(T - 1) * i // (B - 1) for i in range(B)]


def _freqs(case):
    """Angular frequencies of the pairs, in 64 bits, and the factor on the rotated values."""
    rot, base, kind, factor = case["rot"], case["base"], case["scaling"], case["factor"]
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if kind == "ntk":
        base = base * factor ** (rot / max(rot - 2, 1))
    w = base ** (-2.0 * j / rot)
    if kind == "linear":
        return w / factor, 1.0
    if kind == "yarn":
        turns = 4096.0 * w / (2 * math.pi)  # turns of a pair over the trained length
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return w * keep + w / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return w, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    B, T = case["B"], case["T"]

    def normal(*shape, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "rotary":
        s["q"], s["k"] = normal(B, T, case["H"], case["d"]), normal(B, T, case["Hk"], case["d"])
        s["freqs"], s["scale"] = _freqs(case)
        first = torch.full((B, 1), case["start"], dtype=torch.int64, device="cuda")
        if case["far"]:
            first += torch.randint(0, case["far"], (B, 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(T, device="cuda")).contiguous()
    elif case["op"] == "swa":
        H, Hk, d, R = case["H"], case["Hk"], case["d"], case["window"] + case["sinks"]
        if case["dir"] in ("fwd", "train"):
            s["q"], s["k"], s["v"] = normal(B, T, H, d), normal(B, T, Hk, d), normal(B, T, Hk, d)
            if case["dir"] == "train":
                s["dO"] = normal(B, T, H, d)
        elif case["dir"] == "decode":
            s["q"], s["k"], s["v"] = normal(B, H, d), normal(B, Hk, d), normal(B, Hk, d)
            s["k_cache"], s["v_cache"] = normal(B, R, Hk, d), normal(B, R, Hk, d)
            s["pos"] = torch.tensor(_positions(case), dtype=torch.int64, device="cuda")
        else:
            s["k"], s["v"] = normal(B, T, Hk, d), normal(B, T, Hk, d)
            s["k_cache"], s["v_cache"] = normal(B, R, Hk, d), normal(B, R, Hk, d)
            s["lens"] = torch.tensor([p + 1 for p in _positions(case)], dtype=torch.int64, device="cuda")
    else:
        D = case["D"]
        shape = (B, D) if case["dir"] == "decode" else (B, T, D)
        s["x"], s["i_pre"], s["f_pre"] = normal(*shape), normal(*shape), normal(*shape, mean=3.0)
        s["a_log"] = torch.rand(D, generator=g, device="cuda") * 2 - 1
        if case["dir"] == "decode":
            s["h"] = normal(B, D, dtype=torch.float32)
        else:
            s["h0"] = normal(B, D, dtype=torch.float32) if case["h0"] else None
            if case["dir"] == "train":
                s["dh"], s["dhT"] = normal(*shape), normal(B, D, dtype=torch.float32)
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)(c["op"], c["dir"], c, s)


def _run_own(op, direction, c, s):
    kd = _kd()
    if op == "rotary":
        f = kd.rotary_fwd if direction == "fwd" else kd.rotary_bwd
        q, k = f(s["q"], s["k"], s["freqs"], s["pos"], interleaved=c["interleaved"], scale=s["scale"])
        return {"q": q, "k": k}
    if op == "swa":
        W, S = c["window"], c["sinks"]
        if direction == "decode":
            out = kd.swa_decode(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pos"], W, S)
            return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if direction == "fill":
            kd.swa_fill(s["k"], s["v"], s["lens"], s["k_cache"], s["v_cache"], W, S)
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if direction == "fwd":
            out, lse, _ = kd.swa_fwd(s["q"], s["k"], s["v"], W, S)
            return {"out": out, "lse": lse}
        out, lse, ws = kd.swa_fwd(s["q"], s["k"], s["v"], W, S, save=True)
        g = kd.swa_bwd(s["q"], s["k"], s["v"], out, lse, s["dO"], W, S, fwd_workspace=ws)
        return {"out": out, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if direction == "decode":
        return {"out": kd.glr_decode(s["x"], s["i_pre"], s["f_pre"], s["a_log"], s["h"]), "h": s["h"]}
    a = (s["x"], s["i_pre"], s["f_pre"], s["a_log"], s["h0"])
    if direction == "fwd":
        out, hT, _ = kd.glr_fwd(*a)
        return {"out": out, "hT": hT}
    out, hT, ws = kd.glr_fwd(*a, save=True)
    g = kd.glr_bwd(*a, s["dh"], s["dhT"], fwd_workspace=ws, want_dh0=c["h0"])
    r = {"out": out, "hT": hT, "dx": g["dx"], "di_pre": g["di_pre"], "df_pre": g["df_pre"], "da_log": g["da_log"]}
    if c["h0"]:
        r["dh0"] = g["dh0"]
    return r


def _run_plain(op, direction, c, s):
    if op == "rotary":
        back = direction == "bwd"
        return {n: _plain_rotary(s[n], s["freqs"], s["pos"], s["scale"], c["interleaved"], back) for n in ("q", "k")}
    if op == "swa":
        if direction == "decode":
            return _plain_step(c, s)
        if direction == "fill":
            return _plain_fill(c, s)
        return _plain_swa(c, s, direction == "train")
    if direction == "decode":
        f, m, i = _plain_gates(s["f_pre"], s["i_pre"], s["a_log"])[:3]
        s["h"].copy_(f * s["h"] + m * i * s["x"].float())
        return {"out": s["h"].to(s["x"].dtype), "h": s["h"]}
    return _plain_glr(s, direction == "train")


def _plain_rotary(x, freqs, pos, scale, interleaved, back):
    rot = 2 * freqs.numel()
    angle = pos.double()[:, :, None, None] * freqs
    if back:
        angle = -angle
    cos, sin = torch.cos(angle).float() * scale, torch.sin(angle).float() * scale
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _visible(t, j, W, S):
    return (j[None, :] <= t[:, None]) & ((t[:, None] - j[None, :] < W) | (j[None, :] < S))


def _plain_swa(c, s, train):
    """Blocks of queries against the keys that any of them sees."""
    W, S, dt = c["window"], c["sinks"], s["q"].dtype
    B, T, H, d = s["q"].shape
    Hk = s["k"].shape[2]
    G, scale = H // Hk, 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, T, Hk, G, d).permute(0, 2, 3, 1, 4)   # B, Hk, G, T, d
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))
    out, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
    if train:
        dO = s["dO"].float().view(B, T, Hk, G, d).permute(0, 2, 3, 1, 4)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    block = max(64, min(1024, (1 << 27) // (B * H * min(T, W + S + 1024))))
    for t0 in range(0, T, block):
        t1 = min(T, t0 + block)
        lo = max(0, t0 - W + 1)
        j = torch.arange(lo, t1, device="cuda")
        if min(S, lo):
            j = torch.cat((torch.arange(min(S, lo), device="cuda"), j))
        t = torch.arange(t0, t1, device="cuda")
        kj, vj, qt = k[..., j, :], v[..., j, :], q[..., t0:t1, :]
        x = torch.matmul(qt, kj.transpose(-1, -2)) * scale
        x = x.masked_fill(~_visible(t, j, W, S), float("-inf"))
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        p = p / total
        lse[..., t0:t1] = (top + torch.log(total))[..., 0]
        out[..., t0:t1, :] = torch.matmul(p, vj)
        if train:
            g = dO[..., t0:t1, :]
            dp = torch.matmul(g, vj.transpose(-1, -2))
            dx = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
            dq[..., t0:t1, :] = torch.matmul(dx, kj)
            dk.index_add_(3, j, torch.matmul(dx.transpose(-1, -2), qt).sum(2, keepdim=True))
            dv.index_add_(3, j, torch.matmul(p.transpose(-1, -2), g).sum(2, keepdim=True))

    def back(y):
        return y.permute(0, 3, 1, 2, 4).reshape(B, T, -1, d).to(dt)
    if not train:
        return {"out": back(out), "lse": lse.permute(0, 3, 1, 2).reshape(B, T, H).contiguous()}
    return {"out": back(out), "dq": back(dq), "dk": back(dk), "dv": back(dv)}


def _slot(p, W, S):
    return torch.where(p < S, p, S + (p - S) % W)


def _plain_step(c, s):
    W, S = c["window"], c["sinks"]
    q, kc, vc, pos = s["q"], s["k_cache"], s["v_cache"], s["pos"]
    B, H, d = q.shape
    R, Hk = kc.shape[1], kc.shape[2]
    rows, slot = torch.arange(B, device="cuda"), _slot(pos, W, S)
    kc[rows, slot], vc[rows, slot] = s["k"], s["v"]
    x = torch.matmul(q.float().view(B, Hk, H // Hk, d), kc.float().permute(0, 2, 3, 1)) / math.sqrt(d)
    gone = torch.arange(R, device="cuda")[None, :] > pos[:, None]
    x = x.masked_fill(gone[:, None, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    out = torch.matmul(p / p.sum(-1, keepdim=True), vc.float().permute(0, 2, 1, 3))
    return {"out": out.reshape(B, H, d).to(q.dtype), "k_cache": kc, "v_cache": vc}


def _plain_fill(c, s):
    W, S, T = c["window"], c["sinks"], c["T"]
    r = torch.arange(W + S, device="cuda")[None, :]
    n = s["lens"][:, None]
    p = torch.where(r < S, r, n - 1 - (n - 1 - r) % W)  # the newest position below n that the slot holds
    there = (p >= r) & (p < n)
    p = p.clamp(0, T - 1)[..., None, None]
    for cache, new in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        rows = torch.take_along_dim(new, p, 1)
        cache.copy_(torch.where(there[..., None, None], rows, cache))
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_gates(f_pre, i_pre, a_log):
    z, a = f_pre.float(), torch.exp(a_log)
    soft = torch.clamp(-z, min=0) + torch.log1p(torch.exp(-z.abs()))  # -log sigmoid
    logf = -a * soft
    f, m = torch.exp(logf), torch.sqrt(-torch.expm1(2 * logf))
    return f, m, 1 / (1 + torch.exp(-i_pre.float())), logf, a


def _scan(f, b):
    """y_t = f_t y_{t-1} + b_t along dim 1, by doubling."""
    T, step = f.shape[1], 1
    f, b = f.clone(), b.clone()
    while step < T:
        b = torch.cat((b[:, :step], b[:, step:] + f[:, step:] * b[:, :-step]), 1)
        f = torch.cat((f[:, :step], f[:, step:] * f[:, :-step]), 1)
        step *= 2
    return b


def _plain_glr(s, train):
    dt, x = s["x"].dtype, s["x"].float()
    f, m, i, logf, a = _plain_gates(s["f_pre"], s["i_pre"], s["a_log"])
    first = torch.zeros_like(x[:, 0]) if s["h0"] is None else s["h0"]
    b = m * i * x
    b[:, 0] += f[:, 0] * first
    h = _scan(f, b)
    r = {"out": h.to(dt), "hT": h[:, -1].clone()}
    if not train:
        return r
    dh = s["dh"].float()
    dh[:, -1] += s["dhT"]
    after = torch.cat((f[:, 1:], torch.zeros_like(f[:, :1])), 1)  # g_t = dh_t + f_{t+1} g_{t+1}
    g = _scan(after.flip(1), dh.flip(1)).flip(1)
    before = torch.cat((first[:, None], h[:, :-1]), 1)
    dm = torch.where(m > 0, f * f / m, torch.zeros_like(m))
    dlog = g * (before * f - i * x * dm)
    r["dx"] = (g * m * i).to(dt)
    r["di_pre"] = (g * m * x * i / (1 + torch.exp(s["i_pre"].float()))).to(dt)
    r["df_pre"] = (dlog * a / (1 + torch.exp(s["f_pre"].float()))).to(dt)
    r["da_log"] = (dlog * logf).double().sum((0, 1)).float()
    if s["h0"] is not None:
        r["dh0"] = f[:, 0] * g[:, 0]
    return r


# ---- in 64 bits, from the definitions --------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "swa": _exact_swa, "glr": _exact_glr}[case["op"]](case, s)


def _exact_rotary(c, s):
    sign = -1.0 if c["dir"] == "bwd" else 1.0
    turn = torch.polar(torch.full_like(s["pos"], s["scale"], dtype=torch.float64)[..., None].expand(-1, -1, c["rot"] // 2)
                       .contiguous(), sign * s["pos"].double()[..., None] * s["freqs"])[:, :, None]
    r = {}
    for n in ("q", "k"):
        y = s[n].double()
        head = y[..., :c["rot"]]
        pairs = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., :c["rot"]] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        r[n] = y
    return r


def _exact_swa(c, s):
    W, S, B, T, H, Hk = (c[n] for n in ("window", "sinks", "B", "T", "H", "Hk"))
    G, root = H // Hk, math.sqrt(c["d"])
    if c["dir"] == "fill":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, n in enumerate(s["lens"].tolist()):
            # only the newest position of each slot is written
            old = list(range(min(S, n))) + list(range(max(S, n - W), n))
            p = torch.tensor(old, dtype=torch.int64, device="cuda")
            to = torch.tensor([i if i < S else S + (i - S) % W for i in old], dtype=torch.int64, device="cuda")
            kc[b, to], vc[b, to] = s["k"][b, p].double(), s["v"][b, p].double()
        return {"k_cache": kc, "v_cache": vc}
    if c["dir"] == "decode":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, p in enumerate(s["pos"].tolist()):
            at = p if p < S else S + (p - S) % W
            kc[b, at], vc[b, at] = s["k"][b].double(), s["v"][b].double()
            n = min(p + 1, W + S)
            for h in range(H):
                w = torch.softmax(kc[b, :n, h // G] @ s["q"][b, h].double() / root, 0)
                out[b, h] = w @ vc[b, :n, h // G]
        return {"out": out, "k_cache": kc, "v_cache": vc}
    train = c["dir"] == "train"
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    key = torch.arange(T, device="cuda")
    for b in range(B):
        for h in range(H):
            kh, vh = k[b, :, h // G], v[b, :, h // G]
            for t0 in range(0, T, 2048):
                t1 = min(T, t0 + 2048)
                seen = ((key[:t1] > t0 - W) | (key[:t1] < S)).nonzero()[:, 0]
                qt, kt, vt = q[b, t0:t1, h], kh[seen], vh[seen]
                if train:
                    qt, kt, vt = (y.clone().requires_grad_() for y in (qt, kt, vt))
                t = key[t0:t1, None]
                hide = (seen > t) | ((seen <= t - W) & (seen >= S))
                with torch.set_grad_enabled(train):
                    z = torch.where(hide, -math.inf, qt @ kt.T / root)
                    o = torch.softmax(z, -1) @ vt
                out[b, t0:t1, h] = o.detach()
                lse[b, t0:t1, h] = torch.logsumexp(z.detach(), -1)
                if train:
                    gq, gk, gv = torch.autograd.grad(o, (qt, kt, vt), s["dO"][b, t0:t1, h].double())
                    dq[b, t0:t1, h] = gq
                    dk[b, :, h // G].index_add_(0, seen, gk)
                    dv[b, :, h // G].index_add_(0, seen, gv)
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _exact_glr(c, s):
    x, zi, zf, al = (s[n].double() for n in ("x", "i_pre", "f_pre", "a_log"))
    a, i = al.exp(), torch.sigmoid(zi)
    logf = a * torch.nn.functional.logsigmoid(zf)
    f, m = logf.exp(), (-torch.special.expm1(2 * logf)).sqrt()
    if c["dir"] == "decode":
        h = f * s["h"].double() + m * i * x
        return {"out": h, "h": h.clone()}
    T = x.shape[1]
    h = torch.zeros_like(x[:, 0]) if s["h0"] is None else s["h0"].double()
    h0, out = h, torch.empty_like(x)
    for t in range(T):
        h = f[:, t] * h + m[:, t] * i[:, t] * x[:, t]
        out[:, t] = h
    r = {"out": out, "hT": h}
    if c["dir"] == "fwd":
        return r
    g, gs = s["dhT"].double(), torch.empty_like(x)
    for t in reversed(range(T)):
        g = g + s["dh"][:, t].double()
        gs[:, t] = g
        g = g * f[:, t]
    before = torch.cat((h0[:, None], out[:, :-1]), 1)
    dlog = gs * (before * f - i * x * f * f / m)
    r.update(dx=gs * m * i, di_pre=gs * m * x * i * (1 - i), df_pre=dlog * a * torch.sigmoid(-zf),
             da_log=(dlog * logf).sum((0, 1)))
    if s["h0"] is not None:
        r["dh0"] = g
    return r
