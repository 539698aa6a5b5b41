"""The scores of logits from their definitions, in binary64 with numpy, and how far a result of the
library may be off (``tol_*``), from the arithmetic it documents.

u = 2^-24 is half a step of fp32.  A lane forms an exponent y = x k - R with one rounding, u |y|;
k is the nearest float to log2(e) / T, whose rest is put right on average, so that a share keeps an
error of u |y - mean(y)|; R is its maximum's exponent, rounded, which every element shares.  2^y is
good to one step (2 u).  A share's relative error is then below E_j = 4 u (|z_j - max| + 2), z = x / T.
A lane adds at most `chain` shares, one at a time, and scales its sums when the maximum grows (an
exponential and a product, for which 2 chain stands); shares of lanes are joined in binary64 with one
exponential each.  The sum is off by ds = sum_j q_j E_j + (3 chain + 16) u, its logarithm by ds + 2 u.

R is up to 8 below the maximum's exponent: |y| is at most |z_j - max| log2(e) + 8 there, which adds
8 ln 2 u = 5.6 u to E_j's exponent part (4 u (.. + 2) has 8 u).

The entropy is ln S - sum_j q_j (z_j - max): the second term is off by E_j, ds and the roundings of
its own chain of additions, (chain + 4) u, of sum_j q_j (|z_j - max| + 5.6), and k's rest tilts the
shares: u times the variance of z in all.
"""
import numpy as np

from loss_reference import FLUSH, U, round_tol, rows_of


def score(x, targets, T=1.0, top=0):
    m, ln_s, lse, q, E, _ = rows_of(x, T)
    rows, V = x.shape
    chain = 4 + V // 64
    with np.errstate(all="ignore"):
        t = (x - m[:, None]) / T
        a = np.where(q > 0, np.abs(t), 0.0)
        ds = (q * E).sum(1) + (3 * chain + 16) * U
        mean = (q * a).sum(1)
        entropy = ln_s + mean
        var = (q * (a - mean[:, None]) ** 2).sum(1)
        dh = ds + 2 * U + (q * (a + 5.6) * E).sum(1) + (mean + 5.6) * (ds + (chain + 4) * U) + 2 * U * var
    live = np.ones(rows, bool) if targets is None else targets >= 0
    none = ~np.isfinite(ln_s)           # no distribution
    out = dict(lse=np.where(live, lse, 0.0), entropy=np.where(live, entropy, 0.0))
    for name in ("lse", "entropy"):
        out[name][live & none] = np.nan
    out["tol_lse"] = np.where(live, ds + 2 * U, 0.0) + round_tol(out["lse"])
    out["tol_entropy"] = np.where(live, dh, 0.0) + round_tol(out["entropy"])
    at = np.arange(rows)
    if targets is not None:
        bad = targets >= V
        xt = x[at, np.where(live & ~bad, targets, 0)]
        with np.errstate(all="ignore"):
            lp = np.where(live, np.where(bad, np.nan, (xt - m) / T - ln_s), 0.0)
        lp[live & none] = np.nan
        out["logp"] = lp
        out["tol_logp"] = np.where(live, ds + 2 * U, 0.0) + round_tol(lp)
    if top:
        k = min(top, V)
        with np.errstate(all="ignore"):
            ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
            v = np.take_along_axis(x, ids, 1)
            logp = (v - m[:, None]) / T - ln_s[:, None]
        gone = ~(live & ~none)[:, None] | ~(v > -np.inf)
        pad = ((0, 0), (0, top - k))
        out["ids"] = np.pad(np.where(gone, -1, ids), pad, constant_values=-1)
        out["values"] = np.pad(np.where(gone, -np.inf, v), pad, constant_values=-np.inf)
        out["top_logp"] = np.pad(np.where(gone, -np.inf, logp), pad, constant_values=-np.inf)
        out["tol_top_logp"] = (ds + 2 * U)[:, None] + round_tol(out["top_logp"])
    return out


def score_grad(x, targets, lse, entropy, dlogp, dentropy, T=1.0, factor=1.0, kind="fp32"):
    """The gradient from the stored lse and entropy, which count as exact here.

    log2 q = x k - lse log2(e) is one fma (fp32 adds the rests): an error of u (|log2 q|), and for
    16-bit results of u |lse| log2(e) and 2 u |x k| for the rests left out; 2^y is good to 2 u, the
    bracket h ln q + (g + h H) to 4 u of its parts.  The target's element takes expm1 and exp of
    lp, good to 2^-21."""
    rows, V = x.shape
    live = np.ones(rows, bool) if targets is None else targets >= 0
    g = np.zeros(rows) if dlogp is None else dlogp * factor / T
    h = np.zeros(rows) if dentropy is None else dentropy * factor / T
    H = np.zeros(rows) if dentropy is None else entropy
    live = live & ~((g == 0) & (h == 0))
    with np.errstate(all="ignore"):
        y = x / T - lse[:, None]
        q = np.exp(y)
        yc = np.where(q > 0, y, 0.0)
        dy = 2 * U * np.abs(yc) + 2 * U
        if kind != "fp32":
            dy = dy + 2 * U * np.abs(lse)[:, None] + 2 * U * np.where(q > 0, np.abs(x / T), 0.0)
        else:
            dy = dy + 4 * U * U * (np.abs(lse)[:, None] + np.abs(x / T))
        bracket = h[:, None] * yc + (g + h * H)[:, None]
        size = np.abs(h[:, None] * yc) + np.abs(g + h * H)[:, None] + (np.abs(g) + np.abs(h * H))[:, None]
        dx = -q * bracket
        off = q * (np.abs(bracket) * (dy + 4 * U) + np.abs(h)[:, None] * dy + 4 * U * size) + FLUSH * size
        if targets is not None and dlogp is not None:
            at = np.arange(rows)
            t = np.where(live & (targets < V), targets, 0)
            lp = y[at, t]
            part = np.where(np.exp(lp) > 0, h * np.exp(lp) * (lp + H), 0.0)
            dx[at, t] = -g * np.expm1(lp) - part
            off[at, t] += (np.abs(g * np.expm1(lp))
                           + np.abs(h) * np.exp(lp) * (np.abs(lp) + np.abs(H))) * 2.0 ** -21
            dx = np.where((targets >= V)[:, None], np.nan, dx)
        elif targets is not None:
            dx = np.where((targets >= V)[:, None], np.nan, dx)
    dx = np.where(live[:, None], dx, 0.0)
    return dx, np.where(live[:, None], off, 0.0) * 1.01 + round_tol(dx, kind)
