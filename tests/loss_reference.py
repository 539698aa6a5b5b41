"""The losses over vocabulary logits from their definitions, in binary64 with numpy.

Each function takes float64 arrays (the logits widened, already exact) and returns a dict with
the outputs, the gradient ``dx`` (times ``factor``), and ``tol_*``: how far a result of the
library may be off, from the arithmetic it documents -- statistics in fp32 joined in binary64,
results rounded once.  u = 2^-24 is half a step of fp32.

* An exponent (x - m) k is formed with three roundings and exp2 is good to one step, so a share
  q_j has a relative error of at most E_j = 4 u (|x_j - m| / T + 2) (the fp32-only correction of k
  left out for 16-bit results: k_hi is off by at most 2 u).
* A row's sum is formed by lanes that each add at most `chain` partial sums of up to 8 terms,
  rescaling as the maximum grows (exp2 and a product each time): its relative error is at most
  sum_j q_j E_j + (3 chain + 16) u =: ds.  lse and lp are then off by ds (absolutely) + 3 u (the
  logarithm), and rounded once.
* An element of the gradient is coef * q_j: relative error E_j + ds + 4 u, plus what an error of
  lp does to coef, plus the rounding to the result's type (eps / 2, or half the smallest
  subnormal).  exp2 results below 2^-126 may come out as 0.
"""
import numpy as np

U = 2.0 ** -24
FLUSH = 2.0 ** -126
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def rows_of(x, T):
    """m, ln s, lse, q, E and ds of every row."""
    with np.errstate(all="ignore"):
        m = np.max(x, axis=1, keepdims=True)
        t = (x - m) / T
        e = np.exp(t)
        s = e.sum(1, keepdims=True)
        ln_s = np.log(s)[:, 0]           # kept apart from m / T, which may be any size
        lse = m[:, 0] / T + ln_s
        q = e / s
        E = 4 * U * (np.where(np.isfinite(t), np.abs(t), 0.0) + 2.0)
        chain = 4 + x.shape[1] // 256
        ds = (q * E).sum(1) + (3 * chain + 16) * U
    return m[:, 0], ln_s, lse, q, E, ds


def round_tol(v, kind="fp32"):
    return np.abs(v) * HALF_STEP[kind] + TINY[kind]


def _target(x, targets, T):
    """lp and the shared pieces; rows without a target have lp 0."""
    m, ln_s, lse, q, E, ds = rows_of(x, T)
    live = targets >= 0
    t = np.where(live, targets, 0)
    bad = t >= x.shape[1]
    tc = np.where(bad, 0, t)
    xt = x[np.arange(len(t)), tc]
    with np.errstate(all="ignore"):
        lp = np.where(live, np.where(bad, np.nan, (xt - m) / T - ln_s), 0.0)
    return lp, lse, q, E, ds, live, tc


def target_grad(x, targets, T, coef, dcoef, factor, kind, parts):
    """factor / T * coef * (1[j = t] - q): coef = dL/dlp, dcoef its error."""
    lp, lse, q, E, ds, live, tc = parts
    onehot = np.zeros_like(x)
    onehot[np.arange(len(tc)), tc] = 1.0
    c = np.where(live, coef * factor / T, 0.0)[:, None]
    with np.errstate(all="ignore"):
        rest = onehot - q
        rest[np.arange(len(tc)), tc] = -np.expm1(lp)
        dx = np.where(live[:, None], c * rest, 0.0)
        off = np.abs(c) * q * (E + ds[:, None] + 8 * U) + np.abs(c) * onehot * 4 * U
        off += np.abs(c) * FLUSH
        off += np.abs(factor / T) * np.where(live, dcoef, 0.0)[:, None] * np.abs(rest)
        tol = np.where(live[:, None], off, 0.0) * 1.01 + round_tol(dx, kind)
    return dx, tol


def logprob(x, targets, T=1.0, dlogp=None, factor=1.0, kind="fp32"):
    parts = _target(x, targets, T)
    lp, lse, q, E, ds, live, tc = parts
    out = dict(logp=lp, lse=np.where(live, lse, 0.0))
    out["tol_logp"] = np.where(live, ds + 3 * U, 0.0) + round_tol(lp)
    out["tol_lse"] = np.where(live, ds + 3 * U, 0.0) + round_tol(out["lse"])
    if dlogp is not None:
        # from the stored lse: its rounding is an error of every exponent, and the exponent is
        # x k - lse k with one rounding of the larger part's size for 16-bit results
        extra = ds + 3 * U + np.abs(lse) * U * (4 if kind != "fp32" else 2)
        z = np.abs(x) / T
        E2 = E + (4 * U * np.where(np.isfinite(z), z, 0.0) if kind != "fp32" else 0.0)
        parts2 = (lp, lse, q, E2, extra, live, tc)
        out["dx"], out["tol_dx"] = target_grad(x, targets, T, dlogp, 0.0 * dlogp, factor, kind,
                                               parts2)
        # the target's element is -expm1(lp) with lp from the stored lse
        off = np.abs(dlogp * factor / T) * np.exp(np.minimum(lp, 0)) * extra * 2
        out["tol_dx"][np.arange(len(tc)), tc] += np.where(live, off, 0.0)
    return out


def cross_entropy(x, targets, T=1.0, w=None, factor=1.0, kind="fp32"):
    parts = _target(x, targets, T)
    lp, lse, q, E, ds, live, tc = parts
    w = np.ones_like(lp) if w is None else w
    live = live & (w != 0)
    parts = (lp, lse, q, E, ds, live, tc)
    loss = np.where(live, -w * lp, 0.0)
    out = dict(loss=loss, tol_loss=np.where(live, np.abs(w) * (ds + 3 * U), 0.0) + round_tol(loss))
    out["dx"], out["tol_dx"] = target_grad(x, targets, T, -w, 0.0 * w, factor, kind, parts)
    return out


def policy(x, targets, old, ref, adv, T=1.0, w=None, clip=(0.2, 0.2), kl_coef=0.0, factor=1.0,
           kind="fp32"):
    parts = _target(x, targets, T)
    lp, lse, q, E, ds, live, tc = parts
    w = np.ones_like(lp) if w is None else w
    live = live & (w != 0)
    parts = (lp, lse, q, E, ds, live, tc)
    with np.errstate(all="ignore"):
        rho = np.exp(lp - old)
        free = np.where(adv == 0, 0.0, rho * adv)
        cut = np.where(adv == 0, 0.0, np.clip(rho, 1 - clip[0], 1 + clip[1]) * adv)
        slope = np.where(free <= cut, -free, 0.0)
        loss = -np.minimum(free, cut)
        dl = ds + 3 * U
        err = np.abs(free) * (dl + 4 * U)
        out = {}
        dslope, dloss = err, np.where(free <= cut, err, 0.0) + np.abs(loss) * U
        if ref is not None:
            d = ref - lp
            kl = np.where(np.abs(d) < 1e-3, d * d / 2 * (1 + d / 3 * (1 + d / 4)), np.expm1(d) - d)
            out["kl"] = np.where(live, kl, 0.0)
            out["tol_kl"] = np.where(live, np.abs(np.expm1(d)) * dl + kl * 4 * U + dl * dl, 0.0) + \
                round_tol(kl)
            loss = loss + kl_coef * kl
            slope = slope - kl_coef * np.expm1(d)
            dslope = dslope + kl_coef * (np.exp(d) * dl + (np.abs(np.expm1(d)) + kl) * 4 * U)
            dloss = dloss + kl_coef * out["tol_kl"]
        out["loss"] = np.where(live, w * loss, 0.0)
        out["tol_loss"] = np.where(live, np.abs(w) * dloss, 0.0) + round_tol(out["loss"])
        out["logp"] = np.where(live, lp, 0.0)
        out["tol_logp"] = np.where(live, dl, 0.0) + round_tol(out["logp"])
        out["dx"], out["tol_dx"] = target_grad(x, targets, T, w * slope, np.abs(w) * dslope, factor,
                                               kind, parts)
        # distance of rho from the borders: within it, the branch may differ
        out["near_border"] = live & (np.minimum(abs(rho - 1 + clip[0]), abs(rho - 1 - clip[1]))
                                     <= rho * (dl + 4 * U))
    return out


def log_sigmoid(h):
    return np.minimum(h, 0.0) - np.log1p(np.exp(-np.abs(h)))


def preference(x, targets, start, ref, T=1.0, kind_of="sigmoid", beta=0.1, eps=0.0, margin=0.0,
               mean=False, factor=1.0, kind="fp32"):
    n = (len(start) - 1) // 2
    parts = _target(x, targets, T)
    lp, lse, q, E, ds, live, tc = parts
    rows = len(lp)
    base = logprob(x, targets, T)
    start = np.clip(start, 0, rows)
    pi, dpi, per = np.zeros(2 * n), np.zeros(2 * n), np.ones(2 * n)
    for i in range(2 * n):
        r = slice(start[i], max(start[i], start[i + 1]))
        if mean:
            per[i] = 1.0 / max(1, int(live[r].sum()))
        pi[i] = lp[r].sum() * per[i]
        dpi[i] = base["tol_logp"][r].sum() * per[i]
    r = np.zeros(2 * n) if ref is None else ref
    D = (pi - r)[:n] - (pi - r)[n:]
    dD = (dpi[:n] + dpi[n:]) * 1.01 + (np.abs(D) + np.abs(r[:n]) + np.abs(r[n:])) * 2.0 ** -50
    if kind_of == "sigmoid":
        h = beta * D - margin
        loss = -(1 - eps) * log_sigmoid(h) - eps * log_sigmoid(-h)
        sig = 1 / (1 + np.exp(-h))
        slope = beta * (eps * sig - (1 - eps) * (1 - sig))
        curve = beta * beta * sig * (1 - sig)
    else:
        off = D - 1 / (2 * beta)
        loss, slope, curve = off * off, 2 * off, 2.0 + 0 * D
    out = dict(loss=loss, seq_logp=pi, logp=lp, lse=base["lse"])
    out["tol_loss"] = np.abs(slope) * dD + curve * dD * dD + round_tol(loss)
    out["tol_seq_logp"] = dpi + round_tol(pi)
    out["tol_logp"], out["tol_lse"] = base["tol_logp"], base["tol_lse"]
    dlogp, ddlogp = np.zeros(rows), np.zeros(rows)
    for i in range(2 * n):
        s = slice(start[i], max(start[i], start[i + 1]))
        dlogp[s] = np.where(live[s], (1 if i < n else -1) * slope[i % n] * per[i], 0.0)
        ddlogp[s] = np.where(live[s], (curve * dD * 1.01)[i % n] * per[i], 0.0)
    out["dlogp"], out["tol_dlogp"] = dlogp, ddlogp + round_tol(dlogp)
    g = logprob(x, targets, T, dlogp, factor, kind)
    out["dx"] = g["dx"]
    with np.errstate(all="ignore"):
        slack = np.where(dlogp != 0, out["tol_dlogp"] / np.where(dlogp != 0, np.abs(dlogp), 1.0), 0.0)
    out["tol_dx"] = g["tol_dx"] + np.abs(g["dx"]) * slack[:, None] * 1.01
    return out


def distill(x, values, ids, t_lse=None, T=1.0, w=None, factor=1.0, kind="fp32"):
    m, ln_s, lse, q, E, ds = rows_of(x, T)
    rows, V = x.shape
    w = np.ones(rows) if w is None else w
    loss, dx = np.zeros(rows), np.zeros_like(x)
    tol_loss, tol_dx = np.zeros(rows), np.zeros_like(x)
    for r in range(rows):
        there = ids[r] >= 0
        if w[r] == 0 or not there.any():
            continue
        id, v = ids[r][there], values[r][there] / T
        if t_lse is None:
            top = v.max()
            norm = top + np.log(np.exp(v - top).sum())
        else:
            norm = t_lse[r]
        lp = v - norm
        with np.errstate(all="ignore"):
            p = np.exp(lp)
            lq = (x[r, id] - m[r]) / T - ln_s[r]
            term = np.where(p > 0, p * (np.where(p > 0, lp, 0.0) - lq), 0.0)
            loss[r] = w[r] * term.sum()
            # the shares: an exponent rounded to fp32, exp good to 2 steps; the teacher's own sum
            # as the student's
            ep = 4 * U * (np.where(np.isfinite(lp), np.abs(lp), 0.0) + 4)
            dn = (p * 4 * U * (np.abs(v - v.max()) + 4)).sum() if t_lse is None else 0.0
            dp = p * (ep + dn)
            tol_loss[r] = abs(w[r]) * (np.where(p > 0, dp * np.abs(lp - lq), 0.0).sum()
                                       + p.sum() * (dn + ds[r] + 4 * U))
            mass = p.sum()
            share = np.zeros(V)
            dshare = np.zeros(V)
            np.add.at(share, id, p)
            np.add.at(dshare, id, dp + p * 2 * U * len(id))
            c = w[r] * factor / T
            dx[r] = c * (q[r] * mass - share)
            tol_dx[r] = abs(c) * (q[r] * mass * (E[r] + ds[r] + ep.max() + dn + 8 * U) + dshare
                                  + (q[r] * mass + share) * 2 * U + mass * FLUSH)
    tol_loss += round_tol(loss)
    return dict(loss=loss, dx=dx, tol_loss=tol_loss, tol_dx=tol_dx * 1.01 + round_tol(dx, kind))
