"""Layer norm, 8-bit activation checkpoints and the gated product in 64 bits, from their definitions.

Everything here runs on the CPU in float64 (NumPy) and shares no code with the
library.  The error bounds count roundings: U is half a step of fp32 relative
to the value, `half_step` that of an output type.
"""
from __future__ import annotations

import math

import numpy as np
import torch
from scipy.special import erfc

U = 2.0 ** -24
BLOCK = 32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def act8(x: np.ndarray):
    """(codes int8, exponents uint8, values) of float64 entries that are exact in fp32."""
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.int8)
    scale = np.zeros((rows, -(-cols // BLOCK)), np.uint8)
    values = np.zeros((rows, cols))
    for b in range(scale.shape[1]):
        blk = x[:, BLOCK * b:BLOCK * (b + 1)]
        a = np.abs(blk).max(axis=1)
        bad = ~np.isfinite(blk).all(axis=1)
        _, e = np.frexp(np.where(bad, 1.0, a))
        e = np.where(a == 0, 0, np.maximum(e + 126, 0))
        e = np.where(bad, 255, e)
        q = np.clip(np.rint(np.ldexp(np.where(bad[:, None], 0.0, blk), (133 - e)[:, None])), -127, 127)
        codes[:, BLOCK * b:BLOCK * (b + 1)] = q
        scale[:, b] = e
        values[:, BLOCK * b:BLOCK * (b + 1)] = np.where(bad[:, None], np.nan, np.ldexp(q, (e - 133)[:, None]))
    return codes, scale, values


def act8_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    e = np.repeat(scale.astype(np.int64), BLOCK, axis=1)[:, :codes.shape[1]]
    return np.where(e == 255, np.nan, np.ldexp(codes.astype(np.float64), e - 133))


def check_act8_of(codes: np.ndarray, scale: np.ndarray, exact: np.ndarray, err: np.ndarray) -> None:
    """The checkpoint of an fp32 tensor that lies within `err` of `exact`: each block's exponent is that of a
    maximum within the error, each value within half a step (one where the clamp takes 128 steps to 127)."""
    rows, cols = exact.shape
    for b in range(scale.shape[1]):
        sl = slice(BLOCK * b, min(BLOCK * (b + 1), cols))
        hi = (np.abs(exact[:, sl]) + err[:, sl]).max(axis=1)
        lo = np.maximum(np.abs(exact[:, sl]) - err[:, sl], 0).max(axis=1)
        e = scale[:, b].astype(np.int64)
        assert (np.ldexp(1.0, e - 127) <= hi)[e > 0].all() and (lo < np.ldexp(1.0, e - 126)).all(), f"exponents of block {b}"
        step = np.ldexp(1.0, e - 133)[:, None]
        off = np.abs(np.ldexp(codes[:, sl].astype(np.float64), (e - 133)[:, None]) - exact[:, sl]) - err[:, sl]
        clamped = np.abs(exact[:, sl]) + err[:, sl] >= 127.5 * step
        assert (off <= np.where(clamped, 1.0, 0.5) * step).all(), f"values of block {b}"


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

# Additions a term passes through in a row's fp32 sum: at most 32 entries a
# thread, 6 steps across the lanes, 16 waves, with room for the products' own
# roundings.
CHAIN = 32 + 6 + 16 + 8


def norm_fwd(x, w, b, eps):
    mean = x.mean(axis=1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    xhat = c * rstd[:, None]
    y = xhat * (1.0 if w is None else w) + (0.0 if b is None else b)
    return y, mean, rstd, xhat


def norm_fwd_bounds(x, w, b, eps):
    """fp32 error bounds of (y, mean, rstd, xhat), before any rounding to an output type."""
    y, mean, rstd, xhat = norm_fwd(x, w, b, eps)
    wa = np.abs(np.ones(x.shape[1]) if w is None else w)
    d_mean = (CHAIN + 2) * U * np.abs(x).mean(axis=1)
    # x - mean: the mean's error and one rounding; squares and their sum CHAIN + 3 roundings; the mean's
    # error enters the variance twice (2 c d + d^2), sqrt and the reciprocal half of that and 4 roundings
    c = np.abs(xhat) / rstd[:, None]
    var = (c * c).mean(axis=1)
    d_var = 2 * c.mean(axis=1) * (d_mean + U * c.max(axis=1)) + d_mean ** 2 + (CHAIN + 3) * U * var
    d_rstd = rstd * (0.5 * d_var * rstd ** 2 + 4 * U)
    # relative bounds above hold while d_var is small against var + eps
    d_xhat = rstd[:, None] * (d_mean[:, None] + U * c) + c * d_rstd[:, None] + U * np.abs(xhat)
    d_y = wa * d_xhat + 2 * U * (np.abs(xhat) * wa + np.abs(y))
    return d_y, d_mean, d_rstd, d_xhat


def norm_bwd(dy, xhat, rstd, w):
    a = dy * (1.0 if w is None else w)
    m1, m2 = a.mean(axis=1), (a * xhat).mean(axis=1)
    dx = rstd[:, None] * (a - m1[:, None] - xhat * m2[:, None])
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)


def norm_bwd_bounds(dy, xhat, rstd, w):
    """fp32 error bounds of (dx, dw, db): xhat = (x - mean) rstd carries 2 roundings."""
    rows = dy.shape[0]
    a = np.abs(dy * (1.0 if w is None else w))
    xa = np.abs(xhat)
    d1 = (CHAIN + 2) * U * a.mean(axis=1)[:, None]
    d2 = (CHAIN + 5) * U * (a * xa).mean(axis=1)[:, None]
    m1, m2 = a.mean(axis=1)[:, None], (a * xa).mean(axis=1)[:, None]
    dx = rstd[:, None] * (d1 + xa * d2 + 4 * U * (a + m1) + 7 * U * xa * m2)
    # a column's terms: the rows of one of at most 512 workgroups (of up to 4 waves), then 512 / 4 sums and 8 more
    chain = min(rows, -(-rows // 512) + 512 // 4 + 12)
    return dx, (chain + 4) * U * np.abs(dy * xhat).sum(axis=0), (chain + 2) * U * np.abs(dy).sum(axis=0)


def check(name: str, got: torch.Tensor, want: np.ndarray, err: np.ndarray) -> float:
    """|got - want| within err and half a step of got's type (of the type's smallest normal step below that)."""
    g = f64(got)
    assert g.shape == want.shape, f"{name}: shape {g.shape}, expected {want.shape}"
    info = torch.finfo(got.dtype)
    tol = err + half_step(got.dtype) * (np.abs(want) + err) + info.tiny * info.eps
    off = np.abs(g - want)
    ratio = float((off / tol).max()) if off.size else 0.0
    at = np.unravel_index(np.argmax(off / tol), off.shape) if off.size else ()
    assert ratio <= 1.0, f"{name}: error {off[at]:.3g} at {at}, tolerance {tol[at]:.3g} (value {want[at]:.6g})"
    return ratio


# ---------------------------------------------------------------------------
# The gated product
# ---------------------------------------------------------------------------

def act(g, name):
    """act(g), act'(g) and bounds of their fp32 errors for an exact g (about 2 ulp per function call, the
    exponent's and erfc's arguments rounded: relative 2 |g| U and 2 g^2 U)."""
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        c = 1.0 / (1.0 + np.exp(g))
        rel = (2 * np.abs(g) + 10) * U
        return g * s, s + g * s * c, np.abs(g) * s * rel, (s + np.abs(g) * s * (c + 2 * U / np.maximum(rel, U))) * rel
    phi = 0.5 * erfc(-g / math.sqrt(2.0))
    dens = np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    rel = (2 * g * g + 20) * U
    return g * phi, phi + g * dens, np.abs(g) * phi * rel, (phi + np.abs(g) * dens) * rel


class Levels:
    """A quantised tensor: odd whole numbers `units` (2 u - L + 1) times a row's `factor` s / (L - 1)."""

    def __init__(self, codes: np.ndarray, scale: np.ndarray, bits: int):
        top = 2 ** bits - 1
        self.units = 2.0 * codes - top
        self.factor = scale.astype(np.float64) / top

    def times(self, other: "Levels") -> np.ndarray:
        """self other^T; the sum of whole numbers is exact in float64."""
        return (self.units @ other.units.T) * (self.factor[:, None] * other.factor)


def gated_fwd(qx, qg, qu, name):
    """(h, g, u, fp32 error bounds of h, g and u)."""
    g, u = qx.times(qg), qx.times(qu)
    dg, du = 4 * U * np.abs(g), 4 * U * np.abs(u)  # the sum is exact; Delta's two factors, their product, the scaling
    v, slope, dv, _ = act(g, name)
    d_act = dv + np.abs(slope) * dg + dg * dg
    return v * u, g, u, np.abs(u) * d_act + (np.abs(v) + d_act) * du + 2 * U * np.abs(v * u), dg, du


def gated_bwd(dh, g, u, name):
    v, slope, dv, ds = act(g, name)
    out = np.concatenate([dh * u * slope, dh * v], axis=1)
    err = np.concatenate([np.abs(dh * u) * (ds + 4 * U * np.abs(slope)), np.abs(dh) * (dv + 3 * U * np.abs(v))], axis=1)
    return out, err


def unpacked(codes: torch.Tensor, rows: int, cols: int, bits: int) -> np.ndarray:
    """One integer a code of the LSB-first packed stream."""
    b = np.unpackbits(codes.cpu().numpy().reshape(rows, cols * bits // 8), axis=1, bitorder="little")
    return (b.reshape(rows, cols, bits) * (1 << np.arange(bits))).sum(axis=2)
