"""Oracle of the operators around the linear layer in a training step: 8-bit
activation checkpoints and the losses on logits, as their definitions in
numpy fp64.  Test infrastructure; shares no code with the library.
"""
from __future__ import annotations

import numpy as np

ACT8_BLOCK = 32
INT8, E4M3 = 0, 1


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 E4M3 codes (0x7f and 0xff: NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(e == 15) & (m == 7)] = np.nan
    return np.where(c >= 128, -v, v)


def _nearest_e4m3(v: np.ndarray) -> np.ndarray:
    """Code of the E4M3 value nearest to v >= 0, v <= 448 (halfway: the even code)."""
    grid = e4m3_values()[:127]
    i = np.clip(np.searchsorted(grid, v), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def act8_quantize(x: np.ndarray, fmt: int):
    """fp64 x [M, K] of bf16 values -> (codes uint8 [M, K], scale bytes uint8 [M, K / 32])."""
    M, K = x.shape
    b = x.reshape(M, K // ACT8_BLOCK, ACT8_BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -127, np.int64)
    pos = amax > 0
    top = 127.5 if fmt == INT8 else 448.0
    # the smallest exponent, from -127 on, at which the block's largest magnitude fits the codes
    for cand in range(-126, 128):
        e[pos & (amax > top * 2.0 ** (cand - 1.0))] = cand
    q = b / 2.0 ** e[..., None].astype(np.float64)
    if fmt == INT8:
        codes = np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    else:
        codes = (_nearest_e4m3(np.abs(q)) + np.where(np.signbit(q), 128, 0)).astype(np.uint8)
        codes[bad] = 0
    return codes.reshape(M, K), np.where(bad, 255, e + 127).astype(np.uint8)


def act8_values(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    """fp64 values that codes and scale bytes stand for."""
    M, K = codes.shape
    v = codes.view(np.int8).astype(np.float64) if fmt == INT8 else e4m3_values()[codes]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(M, K // ACT8_BLOCK, ACT8_BLOCK) * s[..., None]).reshape(M, K)


# ------------------------------------------------------------------ losses
def log_softmax(l: np.ndarray, tau: float) -> np.ndarray:
    """Rows of log probabilities; a row with NaN, +inf or nothing above -inf is NaN."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        x = l.astype(np.float64)
        top = x.max(-1, keepdims=True)
        x = tau * (x - np.where(np.isneginf(top), 0.0, top))
        out = x - np.log(np.exp(x).sum(-1, keepdims=True))
        out[~np.isfinite(top[:, 0])] = np.nan
    return out


def token_logprob(l, y, tau=1.0):
    """(logp [M], log probabilities [M, V], rows with a target)."""
    V = l.shape[1]
    live = (y >= 0) & (y < V)
    ls = log_softmax(np.where(live[:, None], l, 0.0), tau)
    lp = np.where(live, ls[np.arange(len(y)), np.where(live, y, 0)], 0.0)
    return lp, ls, live


def dlogits(ls, y, live, d, tau):
    """Gradient of sum_m d_m logp_m."""
    use = live & (d != 0)
    g = np.where(use[:, None], -np.exp(ls), 0.0)
    g[np.arange(len(y))[use], y[use]] += 1
    return g * np.where(use, d, 0.0)[:, None] * tau


def preference_loss(l, y, cu, ref, beta, kind, eps=0.0, margin=0.0, average=False, tau=1.0, grad_scale=1.0):
    """kind 0 sigmoid, 1 hinge, 2 ipo.  Returns (loss, rewards, logp, dlogits, d loss / d logp)."""
    lp, ls, live = token_logprob(l, y, tau)
    P, M = len(cu) // 2, len(y)
    d, rewards, losses = np.zeros(M), [], []
    for p in range(P):
        rows = [np.arange(cu[2 * p + k], cu[2 * p + k + 1]) for k in (0, 1)]
        rows = [r[live[r]] for r in rows]
        div = [max(len(r), 1) if average else 1 for r in rows]
        S = [(lp[r] - (ref[r] if ref is not None else 0.0)).sum() / n for r, n in zip(rows, div)]
        delta = S[0] - S[1]
        z = beta * delta - margin
        if kind == 0:
            losses.append((1 - eps) * np.logaddexp(0, -z) + (eps * np.logaddexp(0, z) if eps else 0.0))
            g = beta * (eps / (1 + np.exp(-z)) - (1 - eps) / (1 + np.exp(z)))
        elif kind == 1:
            losses.append(max(0.0, 1 - z))
            g = -beta if z < 1 else 0.0
        else:
            losses.append((delta - 0.5 / beta) ** 2)
            g = 2 * (delta - 0.5 / beta)
        d[rows[0]] += g / P / div[0] * grad_scale
        d[rows[1]] -= g / P / div[1] * grad_scale
        rewards += [beta * s for s in S]
    return np.mean(losses), np.array(rewards), lp, dlogits(ls, y, live, d, tau), d


def policy_loss(l, y, adv, w, old, ref, lo=0.2, hi=0.2, kl_coef=0.0, tau=1.0, grad_scale=1.0):
    """Returns (stats [4], logp, dlogits, d loss / d logp)."""
    y = np.where(w != 0, y, -1)
    lp, ls, live = token_logprob(l, y, tau)
    d, stats = np.zeros(len(y)), np.zeros(4)
    for m in np.flatnonzero(live):
        rho = np.exp(lp[m] - old[m]) if old is not None else 1.0
        free, held = rho * adv[m], np.clip(rho, 1 - lo, 1 + hi) * adv[m]
        clipped = held < free
        dist = ref[m] - lp[m] if ref is not None else 0.0
        kl = np.expm1(dist) - dist
        pol = -min(free, held)
        stats += w[m] * np.array([pol + kl_coef * kl, pol, kl, clipped])
        d[m] = w[m] * ((0.0 if clipped else -free) - kl_coef * np.expm1(dist)) * grad_scale
    return stats, lp, dlogits(ls, y, live, d, tau), d
