"""Routing to experts from its definitions, in binary64 with numpy, and how far a result of the
library may be off (``tol_*``), from the arithmetic it documents.

Choices are by binary64 numbers rounded to 42 bits: what is equal but for the order of a sum is equal.
Without a bias and without sums of two scores the order is the logits', also where scores round alike.
A chosen expert's own exponential is binary64's.  What is summed over the experts (a softmax's sum,
the shares) may be fp32 with a relative error of E = 4 u (|z| + 2), z the logit (softmax: its difference
to the largest), u = 2^-24: an exponent of two roundings of its size, an exponential good to one step; so
is the gradient, formed in fp32.  A sum over a token's experts is then off by the mean of E over the
shares, a share by that, its own E and four roundings, and the sum over the tokens by a rounding for
each 4096 tokens (a lane's own additions, the lanes' are joined in binary64); a weight that is not divided by the chosen
ones' sum by the softmax's sum.
"""
import numpy as np

from loss_reference import U, round_tol

TINY = 1e-20


def rounded(c):
    m, e = np.frexp(c)
    with np.errstate(all="ignore"):
        return np.where(np.isfinite(c), np.ldexp(np.rint(m * 2.0 ** 43), e - 43), c)


def scores(x, sigmoid):
    with np.errstate(all="ignore"):
        if sigmoid:
            s = np.where(x < -1000 * np.log(2.0), 0.0, 1.0 / (1.0 + np.exp(-x)))
            return s, None, 4 * U * (np.where(np.isfinite(x), np.abs(x), 0.0) + 2)
        m = x.max(1, keepdims=True)
        t = x - m
        e = np.exp(t)
        total = e.sum(1, keepdims=True)
        lse = (m + np.log(total))[:, 0]
        return e / total, lse, 4 * U * (np.where(np.isfinite(t), np.abs(t), 0.0) + 2)


def route(x, bias, mask, sigmoid, top, groups=1, top_groups=1, best=1, renormalise=True, scale=1.0):
    rows, n = x.shape
    s, lse, E = scores(x, sigmoid)
    bad = np.isnan(x).any(1)
    if not sigmoid:
        bad |= np.isposinf(x).any(1) | np.isneginf(x).all(1)
    live = np.ones(rows, bool) if mask is None else mask.astype(bool)
    with np.errstate(all="ignore"):
        c = s + (0.0 if bias is None else bias)
    open_ = (x > -np.inf) & (c > -np.inf)
    by_logit = bias is None and (groups == 1 or best == 1)
    cr = x if by_logit else rounded(c)
    ids = np.full((rows, top), -1)
    w = np.zeros((rows, top))
    for r in range(rows):
        if not live[r]:
            continue
        if bad[r]:
            w[r] = np.nan
            continue
        may = open_[r].copy()
        if groups > 1:
            width = n // groups
            val = []
            for g in range(groups):
                cs = sorted(cr[r, g * width:(g + 1) * width][may[g * width:(g + 1) * width]], reverse=True)
                val.append(float(rounded(sum(cs[:best]))) if cs else -np.inf)
            order = sorted(range(groups), key=lambda g: (-val[g], g))[top_groups:]
            for g in order:
                may[g * width:(g + 1) * width] = False
        # the open ones alone: a sort with NaN among its keys has no order
        pick = sorted((e for e in range(n) if may[e]), key=lambda e: (-cr[r, e], e))[:top]
        ids[r, :len(pick)] = pick
        w[r, :len(pick)] = s[r, pick]
        if renormalise:
            w[r] /= w[r].sum() + TINY
        w[r] *= scale
    ok = live & ~bad & (ids[:, 0] >= 0)
    load = np.array([int((ids[ok] == e).sum()) for e in range(n)] + [int(ok.sum())])
    tokens = max(1, load[-1])
    total = np.where(s.sum(1) > 0, s.sum(1), 1.0)[ok][:, None]
    p = s[ok] if not sigmoid else s[ok] / total
    share = p.sum(0) / tokens if len(p) else np.zeros(n)
    aux = np.array([n * (load[:n] * share).sum() / (top * tokens),
                    (lse[ok] ** 2).sum() / tokens if not sigmoid else 0.0])
    with np.errstate(all="ignore"):
        sum_off = np.nan_to_num((s * E).sum(1) / s.sum(1)) + 2 * U
    off_w = np.abs(w) * (1e-13 if sigmoid or renormalise else sum_off[:, None])
    off_p = (p * (E[ok] + sum_off[ok][:, None] + (4 + rows // 4096) * U)).sum(0) / tokens if len(p) else 0.0 * share
    off_lse = (2 * np.abs(lse[ok]) * (sum_off[ok] + 2 * U)).sum() / tokens if not sigmoid else 0.0
    return dict(ids=ids, weights=w, load=load, share=share, aux=aux,
                tol_weights=round_tol(w) + off_w, tol_share=round_tol(share) + off_p,
                tol_aux=round_tol(aux) + np.array([
                    n * (load[:n] * (off_p + share * U)).sum() / (top * tokens) + aux[0] * 2 * U, off_lse]))


def loss(x, ids, mask, dweights, load, sigmoid, top, renormalise, scale, balance, large, factor):
    """What the gradient is of, with ids held and load as counted."""
    n = x.shape[1]
    s, lse, _ = scores(x, sigmoid)
    ok = (np.ones(len(x), bool) if mask is None else mask.astype(bool)) & (ids >= 0).any(1)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renormalise:
        w = w / (w.sum(1, keepdims=True) + TINY)
    total = (np.where(ok[:, None], w, 0.0) * scale * dweights).sum()
    tokens = max(1, int(load[n]))
    p = s if not sigmoid else s / s.sum(1, keepdims=True)
    share = p[ok].sum(0) / tokens
    total += factor * balance * n * (load[:n] * share).sum() / (top * tokens)
    if large:
        total += factor * large * (lse[ok] ** 2).sum() / tokens
    return total


def route_grad(x, ids, mask, dweights, load, sigmoid, top, renormalise, scale, balance, large, factor,
               kind="fp32"):
    rows, n = x.shape
    s, lse, E = scores(x, sigmoid)
    live = np.ones(rows, bool) if mask is None else mask.astype(bool)
    bad = np.isnan(x).any(1) | (ids >= n).any(1)
    if not sigmoid:
        bad |= np.isposinf(x).any(1) | np.isneginf(x).all(1)
    some = (ids >= 0).any(1)
    at = np.clip(ids, 0, n - 1)
    there = (ids >= 0) & (ids < n)
    dw = np.where(there, (np.zeros(ids.shape) if dweights is None else dweights) * scale, 0.0)
    tokens = 1 if load is None else max(1, int(load[n]))
    f = factor / tokens
    pull = np.zeros(n) if load is None else f * balance * n / (top * tokens) * load[:n]
    with np.errstate(all="ignore"):
        ws = np.where(there, np.take_along_axis(s, at, 1), 0.0)
        e_top = np.where(there, np.take_along_axis(E, at, 1), 0.0).max(1, keepdims=True)
        if renormalise:
            d = ws.sum(1, keepdims=True) + TINY
            mean = (dw * ws).sum(1, keepdims=True) / d
            ds = np.where(there, (dw - mean) / d, 0.0)
            dds = (np.abs(dw) + (np.abs(dw) * ws).sum(1, keepdims=True) / d) / d * (3 * e_top + 8 * U)
        else:
            ds, dds = dw, np.abs(dw) * 2 * U
        add, dadd = np.zeros_like(s), np.zeros_like(s)
        for i in range(ids.shape[1]):
            np.add.at(add, (np.arange(rows), at[:, i]), np.where(there[:, i], ds[:, i], 0.0))
            np.add.at(dadd, (np.arange(rows), at[:, i]), np.where(there[:, i], dds[:, i], 0.0))
        dadd += np.abs(add) * 2 * U
        if sigmoid:
            total = s.sum(1, keepdims=True)
            total = np.where(total > 0, total, 1.0)
            p = s / total
            base = (p * pull).sum(1, keepdims=True)
            slope = s * (1.0 - s)
            dx = slope * ((pull - base) / total + add)
            eb = (p * np.abs(pull) * (E + (p * E).sum(1, keepdims=True) + 4 * U)).sum(1, keepdims=True)
            size = (np.abs(pull) + np.abs(base)) / total
            off = slope * ((E + 8 * U) * 2 * (size + np.abs(add)) + eb / total + dadd
                           + size * (p * E).sum(1, keepdims=True))
        else:
            to = pull + add
            es = (s * E).sum(1, keepdims=True)          # the sum's own
            base = 2.0 * f * large * lse[:, None] - (s * to).sum(1, keepdims=True)
            eb = (s * np.abs(to) * (E + es + 4 * U) + s * dadd).sum(1, keepdims=True)
            eb = eb + np.abs(2.0 * f * large) * (4 * U + 4 * U * np.abs(lse[:, None])) + np.abs(base) * U
            dx = s * (to + base)
            size = np.abs(pull) + np.abs(add) + np.abs(base)
            off = s * ((E + es + 8 * U) * size + eb + dadd)
    on = live & some & ~bad
    dx = np.where(on[:, None], dx, 0.0)
    dx[live & bad] = np.nan
    return dx, np.where(on[:, None], off, 0.0) * 1.01 + round_tol(dx, kind) + 2.0 ** -126 * 10
