"""fp64 numpy oracles of the operators beside the delta rules: rotary
positions, attention over a sliding window with first tokens kept, and the
element-wise gated linear recurrence.  Written from the definitions, without
the package; the *_bounds functions turn a kernel's roundings into bounds on
its outputs' errors, term by term."""
import numpy as np


def sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


# ---- rotary positions ---------------------------------------------------------


def rotary(x, freqs, pos, interleaved=False, scale=1.0, inverse=False):
    """x [B,T,H,d], freqs [r/2], pos [B,T] -> rotated x."""
    half = len(freqs)
    y = np.array(x, dtype=np.float64)
    theta = np.asarray(pos, np.float64)[:, :, None, None] * np.asarray(freqs, np.float64)
    if inverse:
        theta = -theta
    c, s = scale * np.cos(theta), scale * np.sin(theta)
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    return y


# ---- attention over a sliding window with first tokens kept -----------------


def swa_mask(T, window, sinks):
    t, j = np.arange(T)[:, None], np.arange(T)[None, :]
    return (j <= t) & ((t - j < window) | (j < sinks))


def _heads(k, H):
    return np.repeat(np.asarray(k, np.float64), H // k.shape[2], axis=2)


def swa(q, k, v, window, sinks, scale, dO=None):
    """q [B,T,H,d], k, v [B,T,Hk,d].  Returns dict out, lse, p (and dq, dk, dv
    with dO), with p [B,H,T,T]."""
    q = np.asarray(q, np.float64)
    B, T, H, d = q.shape
    Hk = k.shape[2]
    kk, vv = _heads(k, H), _heads(v, H)
    x = scale * np.einsum("bthd,bjhd->bhtj", q, kk)
    x = np.where(swa_mask(T, window, sinks), x, -np.inf)
    top = x.max(-1, keepdims=True)
    e = np.exp(x - top)
    total = e.sum(-1, keepdims=True)
    p = e / total
    r = dict(p=p, out=np.einsum("bhtj,bjhd->bthd", p, vv),
             lse=(top + np.log(total))[..., 0].transpose(0, 2, 1))
    if dO is not None:
        dO = np.asarray(dO, np.float64)
        dp = np.einsum("bthd,bjhd->bhtj", dO, vv)
        ds = p * (dp - (p * dp).sum(-1, keepdims=True))
        r["ds"] = ds
        r["dq"] = scale * np.einsum("bhtj,bjhd->bthd", ds, kk)
        dk = scale * np.einsum("bhtj,bthd->bjhd", ds, q)
        dv = np.einsum("bhtj,bthd->bjhd", p, dO)
        r["dk"], r["dv"] = (y.reshape(B, T, Hk, H // Hk, d).sum(3) for y in (dk, dv))
    return r


def swa_bounds(q, k, v, window, sinks, scale, r, u_w, u_out, dO=None):
    """Bounds on |kernel - oracle| per element, from the arithmetic.  u: fp32
    rounding 2^-24; u_w: rounding of p and dS before their products (2^-8 for
    bf16 operands, 0 for fp32); u_out: rounding of the outputs.
      scores: (d + 8) u sum |q||k| scale, and e^x moves p by twice that (its own
      and the sum's); a sum of n terms adds n u of their magnitudes; delta =
      dO.out takes out's error (its fp32 value, before the last rounding, which
      the saved remainder restores to 2^-16 of it)."""
    u = 2.0 ** -24
    q, kk, vv = np.abs(np.asarray(q, np.float64)), np.abs(_heads(k, q.shape[2])), np.abs(_heads(v, q.shape[2]))
    B, T, H, d = q.shape
    Hk = k.shape[2]
    p = r["p"]
    seen = p > 0
    dx = np.where(seen, (d + 8) * u * scale * np.einsum("bthd,bjhd->bhtj", q, kk), 0.0)
    worst = dx.max(-1, keepdims=True) + (T + 16) * u
    ep = p * (dx + worst + 8 * u)                      # error of p in fp32
    wp = ep + u_w * p                                  # and of its rounded copy
    out32 = np.einsum("bhtj,bjhd->bthd", wp + (T + 8) * u * p, vv)
    o = {"out": out32 + u_out * np.abs(r["out"]) + 1e-30,
         "lse": np.broadcast_to(worst[..., 0].transpose(0, 2, 1), r["lse"].shape) + 4 * u * np.abs(r["lse"]) + 2 * u}
    if dO is not None:
        g = np.abs(np.asarray(dO, np.float64))
        dpa = np.einsum("bthd,bjhd->bhtj", g, vv)
        edelta = np.einsum("bthd,bthd->bht", g, out32 + (2.0 ** -16 + (d + 8) * u) * np.abs(r["out"]))[..., None]
        # p (dp - delta): each factor's error, and the difference's own rounding
        diff = np.abs(np.where(seen, r["ds"] / np.where(seen, p, 1), 0.0))
        eds = ep * diff + p * ((d + 8) * u * dpa + edelta + 2 * u * diff) + 2 * u * np.abs(r["ds"])
        eds[:, :, 0, :] = 0.0                           # the first query has one key: exactly 0
        wds = eds + u_w * np.abs(r["ds"])
        n = (T * (H // Hk) + 16) * u
        o["dq"] = scale * np.einsum("bhtj,bjhd->bthd", wds + (T + 16) * u * np.abs(r["ds"]), kk) \
            + u_out * np.abs(r["dq"]) + 1e-30
        dk = scale * np.einsum("bhtj,bthd->bjhd", wds + n * np.abs(r["ds"]), q)
        dv = np.einsum("bhtj,bthd->bjhd", wp + n * p, g)
        for name, y in (("dk", dk), ("dv", dv)):
            o[name] = y.reshape(B, T, Hk, H // Hk, d).sum(3) + u_out * np.abs(r[name]) + 1e-30
    return o


def ring_slot(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


# ---- gated linear recurrence --------------------------------------------------


def glr_gates(f_pre, i_pre, a_log):
    """log f, f, sqrt(1 - f^2), sigmoid(i_pre)."""
    z = np.asarray(f_pre, np.float64)
    a = np.exp(np.asarray(a_log, np.float64))
    l = -a * (np.maximum(-z, 0) + np.log1p(np.exp(-np.abs(z))))
    return l, np.exp(l), np.sqrt(-np.expm1(2 * l)), sigmoid(i_pre)


def glr(x, i_pre, f_pre, a_log, h0=None, dh=None, dhT=None):
    """x, i_pre, f_pre [B,T,D].  Returns dict out (h_t), hT, and with dh the
    gradients dx, di_pre, df_pre, da_log, dh0 and mag_da (the sum of da_log's
    terms' magnitudes)."""
    x = np.asarray(x, np.float64)
    B, T, D = x.shape
    l, f, m, i = glr_gates(f_pre, i_pre, a_log)
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64)
    before, out = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        before[:, t] = h
        h = f[:, t] * h + m[:, t] * i[:, t] * x[:, t]
        out[:, t] = h
    r = dict(out=out, hT=h)
    if dh is not None:
        u = np.zeros((B, D)) if dhT is None else np.asarray(dhT, np.float64)
        g = np.empty_like(x)
        for t in reversed(range(T)):
            g[:, t] = np.asarray(dh[:, t], np.float64) + u
            u = f[:, t] * g[:, t]
        # d m / d l = -f^2 / m, and 0 where f is exactly 1 (its limit times sigma(-f_pre))
        dm = np.divide(f * f, m, out=np.zeros_like(m), where=m > 0)
        dl = g * (before * f - i * x * dm)
        lf = np.maximum(l, -1e30)  # f = 0: dl is 0 and so is its product with l
        a = np.exp(np.asarray(a_log, np.float64))
        r.update(dx=g * m * i, di_pre=g * m * x * i * sigmoid(-np.asarray(i_pre, np.float64)),
                 df_pre=dl * a * sigmoid(-np.asarray(f_pre, np.float64)), da_log=(dl * lf).sum((0, 1)),
                 mag_da=(np.abs(g) * (np.abs(before) * f + i * np.abs(x) * dm) * np.abs(lf)).sum((0, 1)), dh0=u,
                 g=g)
    return r
