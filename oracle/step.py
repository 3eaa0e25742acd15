"""Plain oracle of a step's operators (include/stage_step.h): numpy in 64 bits, test infrastructure only.

It shares no code with the CUDA path: e4m3 goes by the table of its 256 values, positions by extended precision, sums by
exactly rounded or float64 arithmetic.
"""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------------------------------- e4m3

def e4m3_values() -> np.ndarray:
    """The 256 codes' values."""
    c = np.arange(256)
    s, e, m = np.where(c & 128, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = s * np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[[0x7F, 0xFF]] = np.nan
    return v


def e4m3_codes(x) -> np.ndarray:
    """The nearest code (ties to the even one) of each number; beyond 448: 448; NaN: NaN."""
    x = np.asarray(x, np.float64)
    table = e4m3_values()[:127]                       # 0 .. 448, rising
    a = np.abs(x)
    hi = np.clip(np.searchsorted(table, np.where(np.isnan(a), 0, a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    c = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    c = np.where(a >= 448, 126, c)
    return np.where(np.isnan(x), 0x7F, c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


# ------------------------------------------------------------------------------------------- norm

def norm_f8(x, resid=None, gamma=None, eps: float = 1e-5, store=lambda h: h):
    """x, resid: float arrays [n_tok, n] of the numbers given; store: rounds the sum to the residual's type.  Returns (h, y float32, codes,
    scales [blocks, n_tok])."""
    f32 = np.float32
    with np.errstate(all="ignore"):
        h = np.asarray(x, f32) if resid is None else store(np.asarray(x, f32) + np.asarray(resid, f32)).astype(f32)
        y = h
        n_tok, n = h.shape
        if gamma is not None:
            m = np.array([math.fsum(v) if np.isfinite(v).all() else np.nan for v in h.astype(np.float64) ** 2]) / n
            r = (1.0 / np.sqrt(m + np.float64(f32(eps)))).astype(f32)
            r = np.where((m * n >= 2.0 ** 128) | (m + np.float64(f32(eps)) < 2.0 ** -256), f32(np.nan), r)   # beyond float32's range
            y = (h * r[:, None]) * np.asarray(gamma, f32)
        nb = -(-n // 128)
        codes, scales = np.zeros((n_tok, n), np.uint8), np.zeros((nb, n_tok), f32)
        for b in range(nb):
            part = y[:, 128 * b: 128 * b + 128]
            top = np.maximum(np.abs(part).max(1), f32(2.0 ** -100))   # numpy's max keeps NaN
            scales[b] = top / f32(448)
            codes[:, 128 * b: 128 * b + 128] = e4m3_codes(part * (f32(448) / top)[:, None])
    return h, y, codes, scales


# ------------------------------------------------------------------------------------------- product

def f8_gemm(a_codes, a_scale, w_codes, w_scale):
    """(y, the sum of the terms' magnitudes) in float64."""
    t = e4m3_values()
    K, N = a_codes.shape[1], w_codes.shape[0]
    a = t[a_codes] * np.repeat(np.asarray(a_scale, np.float64), 128, 0)[:K].T
    w = t[w_codes] * np.repeat(np.repeat(np.asarray(w_scale, np.float64), 128, 0)[:N], 128, 1)[:, :K]
    return a @ w.T, np.abs(a) @ np.abs(w).T


# ------------------------------------------------------------------------------------------- rope

def rope_freqs(rot, theta, kind="plain", factor=1.0, first=1.0, low=1.0, high=32.0):
    """Frequencies and scale by the definitions, pair by pair."""
    if kind == "base":
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        waves = first * f / (2 * math.pi)
        if kind == "linear":
            f = f / factor
        elif kind == "bands":
            if waves < low:
                f = f / factor
            elif waves <= high:
                s = (waves - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif kind == "parts":
            def place(w):
                return rot * math.log(first / (w * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(place(high)), 0), min(math.ceil(place(low)), rot - 1)
            ramp = min(1.0, max(0.0, (i - a) / (b - a if b > a else 1e-3)))
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if kind == "parts" else 1.0)


def rope(x, pos, freqs, interleaved=False, scale=1.0):
    """x [n_tok, heads, d] -> float64; every token is turned, whatever its position."""
    x = np.asarray(x, np.float64)
    r = 2 * len(freqs)
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    angle = np.asarray(pos).astype(np.longdouble)[:, None] * np.asarray(freqs).astype(np.longdouble)
    angle = angle - two_pi * np.floor(angle / two_pi)
    c, s = (f(angle.astype(np.float64))[:, None] * scale for f in (np.cos, np.sin))
    out = x.copy()
    at = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, v = x[..., at[0]], x[..., at[1]]
    out[..., at[0]] = u * c - v * s
    out[..., at[1]] = v * c + u * s
    return out


# ------------------------------------------------------------------------------------------- log probabilities

def logprobs(z, tokens=None, top=0):
    """dict of logprob, entropy, rank, ids, best, and (for tolerances) away = sum p |z - max|, drop = max - z[token]."""
    z = np.asarray(z, np.float64)
    n, vocab = z.shape
    out = {"logprob": np.full(n, np.nan), "entropy": np.full(n, np.nan), "rank": np.full(n, -1), "ids": np.full((n, top), -1), "best": np.full((n, top), np.nan),
           "away": np.zeros(n), "drop": np.zeros(n), "fall": np.zeros((n, top))}
    for i, row in enumerate(z):
        if np.isnan(row).any() or (row == np.inf).any() or not np.isfinite(row).any():
            continue
        d = row - row.max()
        e = np.exp(d)
        log = math.log(math.fsum(e))
        p = e / e.sum()
        some = p > 0
        out["away"][i] = (p[some] * -d[some]).sum()
        out["entropy"][i] = log + out["away"][i]
        order = np.lexsort((np.arange(vocab), -row))
        out["ids"][i], out["best"][i], out["fall"][i] = order[:top], (d - log)[order[:top]], -d[order[:top]]
        if tokens is not None and 0 <= tokens[i] < vocab:
            t = tokens[i]
            out["logprob"][i], out["drop"][i] = d[t] - log, -d[t]
            out["rank"][i] = (row > row[t]).sum() + (row[:t] == row[t]).sum()
    return out
