"""The mixture-of-experts layer in 64 bits, from its definition, with the roundings of an fp32 evaluation counted.

Runs on the CPU in float64 and shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc

from oracle import quest_oracle as qo

U = 2.0 ** -24  # half a step of fp32, relative


def values(c: np.ndarray, scale: np.ndarray, bits: int) -> np.ndarray:
    return (2.0 * c + 1.0) * (scale.astype(np.float64) / (2 ** bits - 1))[..., None]


def chosen(logits: np.ndarray, top: int) -> list[list[int]]:
    """The experts of each token in the order of their rank."""
    out = []
    for row in logits:
        order = sorted((e for e in range(len(row)) if row[e] > -math.inf), key=lambda e: (-row[e], e))  # (NaN: not >)
        out.append(order[:top])
    return out


def act(g: np.ndarray, name: str):
    """(value, slope, what an fp32 evaluation of the value may be off by)."""
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        # the exponential (2 U), the sum and the quotient
        return g * s, s * (1.0 + g * (1.0 - s)), 6 * U * np.abs(g * s)
    phi = 0.5 * erfc(-g / math.sqrt(2.0))
    slope = phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    # the argument's roundings (of 1 / sqrt(2) and the product) move the tail by g^2 of them; the function a few steps
    return g * phi, slope, (2 * g * g + 16) * U * np.abs(g * phi)


def moe(x, logits, gate, up, down, top, block, h_bits, name, over_all):
    """(y, bound) for values x (n, k), gate and up (e, m, k), down (e, k, m); logits (n, e) in float64.

    The bound counts, in fp32: a product's roundings (7: the steps' factors and products, the sum, the result), the
    activation's, and for h's quantisation every entry that they may move across a level's edge, by a whole step.
    """
    n, k = x.shape
    y, bound = np.zeros((n, k)), np.zeros((n, k))
    alpha = qo.fit_alpha(h_bits)
    half = 2 ** (h_bits - 1)
    for t, experts in enumerate(chosen(logits, top)):
        if np.isnan(logits[t]).any() or np.isposinf(logits[t]).any():
            y[t] = bound[t] = np.nan
            continue
        if not experts:
            continue
        row = logits[t]
        w = np.exp(row - row[experts[0]])
        w = w / (w.sum() if over_all else w[experts].sum())
        for e in experts:
            g, u = gate[e] @ x[t], up[e] @ x[t]
            a, slope, a_err = act(g, name)
            h = a * u
            h_err = np.abs(u) * (np.abs(slope * g) * 7.1 * U + a_err) + np.abs(h) * 8.1 * U
            yt = qo.blockwise_hadamard(h[None], block)[0]
            s = alpha * math.sqrt(np.mean(h * h))
            step = 2 * s / (2 ** h_bits - 1)
            if s == 0:
                continue
            q = np.clip(np.floor(yt / step), -half, half - 1)
            # a transformed entry: its block's errors, log2(block) additions of up to the block's sum; the row's mean
            # square (m additions in chains of at most 8 m / 512 + 8) and the code's factor, as parts of the entry
            m = h.size
            mix = (h_err + np.abs(h) * math.log2(block) * U).reshape(-1, block).sum(1) / math.sqrt(block)
            rms_err = h_err.max() / max(np.abs(h).max(), 1e-300) + (m / 64 + 16) * U
            y_err = np.repeat(mix, block) + np.abs(yt) * (rms_err + 6 * U)
            edge = np.abs(yt / step - np.rint(yt / step)) * step
            near = (edge <= y_err) & (np.abs(np.rint(yt / step)) < half + 0.5)
            value = (2 * q + 1) * step / 2
            d = down[e]
            prod = d @ value
            # (the step's own error, then a whole step for each entry near an edge)
            err = np.abs(prod) * (7.1 * U + rms_err + 3 * U) + np.abs(d[:, near]).sum(1) * step
            y[t] += w[e] * prod
            # the weight: both exponentials and the quotient, their sum; adding the products up
            bound[t] += w[e] * err + w[e] * np.abs(prod) * (len(row) + 10 + top) * U
    return y, bound


def check(got: np.ndarray, eps: float, want: np.ndarray, bound: np.ndarray) -> float:
    """Every entry within the bound and the output type's half step eps; returns the largest share used."""
    assert (np.isnan(got) == np.isnan(want)).all()
    fine = ~np.isnan(want)
    err = np.abs(got - want)[fine]
    most = (bound + (np.abs(want) + bound) * eps)[fine] + 1e-300
    assert (err <= most).all(), f"{(err / most).max():.3g} of the bound"
    return float((err / most).max()) if err.size else 0.0
