"""The bounds that the GPU tests hold the bf16 attention to can tell its
roundings apart: a model of the kernels' arithmetic passes with the weights in
two bf16 parts and the output's remainder, and fails with either left out (on
the CPU, the mistake planted in the model)."""
import numpy as np
import pytest

from oracle import hybrid as O


def bf16(x):
    """x rounded to bf16, to nearest and even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def two_parts(x):
    hi = bf16(x)
    return hi + bf16(x - hi)


def tight_bounds(*a, fine, u_out, dO):
    """oracle.hybrid.swa_bounds for the tensor-core kernels: p and dS are in two
    bf16 parts (2^-16 of themselves) for rows of at most 256 keys, else in one
    (2^-8).  A product that the tensor cores cut off where fp32 would round
    counts two roundings, so the fp32 terms are taken twice (all terms, the
    given ones halved)."""
    u_w = 2.0 ** -16 if fine else 2.0 ** -8
    return {n: 2 * x for n, x in O.swa_bounds(*a, u_w / 2, u_out / 2, dO).items()}


def model(q, k, v, window, sinks, scale, dO, weights, remainder):
    """What the kernels compute, in 64 bits but for the roundings to bf16: the
    weights' before their products, the output's, and the gradients'."""
    r = O.swa(q, k, v, window, sinks, scale, dO)
    H = q.shape[2]
    kk, vv = np.repeat(k, H // k.shape[2], 2), np.repeat(v, H // k.shape[2], 2)
    out32 = np.einsum("bhtj,bjhd->bthd", weights(r["p"]), vv)
    out = bf16(out32)
    seen = out + bf16(out32 - out) if remainder else out
    dp = np.einsum("bthd,bjhd->bhtj", dO, vv)
    ds = weights(r["p"] * (dp - np.einsum("bthd,bthd->bht", dO, seen)[..., None]))
    B, T, Hk, d = k.shape
    dk = scale * np.einsum("bhtj,bthd->bjhd", ds, q).reshape(B, T, Hk, H // Hk, d).sum(3)
    dv = np.einsum("bhtj,bthd->bjhd", weights(r["p"]), dO).reshape(B, T, Hk, H // Hk, d).sum(3)
    return r, dict(out=out, dq=bf16(scale * np.einsum("bhtj,bjhd->bthd", ds, kk)), dk=bf16(dk), dv=bf16(dv))


def off(window, sinks, weights, remainder, fine, T=200):
    rng = np.random.default_rng(window)
    q, k, v, dO = (bf16(rng.standard_normal((1, T, h, 64))) for h in (4, 2, 2, 4))
    r, got = model(q, k, v, window, sinks, 0.125, dO, weights, remainder)
    bound = tight_bounds(q, k, v, window, sinks, 0.125, r, fine=fine, u_out=2.0 ** -8, dO=dO)
    return {n for n, x in got.items() if (np.abs(x - r[n]) > bound[n]).any()}


@pytest.mark.parametrize("window,sinks", [(1, 1), (9, 2), (70, 3), (200, 0)])
def test_two_parts_and_the_remainder_are_within(window, sinks):
    assert not off(window, sinks, two_parts, True, True)


@pytest.mark.parametrize("window,sinks", [(9, 2), (70, 3), (200, 0)])
def test_one_part_in_their_place_is_seen(window, sinks):
    assert off(window, sinks, bf16, True, True) == {"out", "dq", "dk", "dv"}


@pytest.mark.parametrize("window,sinks", [(1, 1), (9, 2), (70, 3), (200, 0)])
def test_a_lost_remainder_is_seen(window, sinks):
    """By dq, whose rows each meet one delta; dk's bound adds up over the queries."""
    assert "dq" in off(window, sinks, two_parts, False, True)


def test_one_part_is_within_where_one_is_meant():
    assert not off(300, 4, bf16, True, False, T=400)
