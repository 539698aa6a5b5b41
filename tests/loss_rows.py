"""Rows of logits in binary64 with torch, on the tensors' own device: cross-entropy, and how far a
result of the library may be off by the additions that a lane makes.

u = 2^-24 is half a step of fp32.  A row is shared by at least 64 lanes, from 512 vectors on by 256;
a lane adds its vectors in pairs -- the 2 E elements of a pair one after another, then to its running
sum, which is rescaled (exp2: 2 u, a product: u, the sum: u) -- and up to four single ones (a head or
tail element, the vectors that are left over).  That bounds a row's sum by

    chain = (2 E + 4 (ceil(vectors / (2 lanes)) + 5) + 8) u

relative, the 8 for the joins.  An exponent has three roundings, exp2 one step: E_j = 4 u (|z_j| + 2) of
a share, z = (x - m) / T, so a sum is off by at most ds = sum_j q_j E_j + chain, and so is lp, besides
3 u of the logarithm.  At 128256 16-bit logits chain is 1.0e-5, where eight average logits are 6e-5.
"""
import math

import torch

from loss_reference import FLUSH, HALF_STEP, TINY, U

E = {"bf16": 8, "fp16": 8, "fp32": 4}


def chain_of(V, kind):
    nvec = V // E[kind]
    lanes = 64 if nvec <= 512 else 256
    return (2 * E[kind] + 4 * (-(-nvec // (2 * lanes)) + 5) + 8) * U


def reference(x, t, kind, factor, T=1.0, from_lse=False):
    """Cross-entropy of the rows of a tensor in binary64: loss, lse, dx and how far each may be off.
    from_lse: dx formed of an lse that was rounded to fp32, as mp_token_logprob_grad's is."""
    x = x.double()
    rows, V = x.shape
    at = torch.arange(rows, device=x.device)
    m = x.amax(1, keepdim=True)
    z = (x - m) / T
    e = torch.exp(z)
    s = e.sum(1, keepdim=True)
    q = e / s
    ln_s = torch.log(s)[:, 0]
    lse = m[:, 0] / T + ln_s
    live = t >= 0
    tt = t.clamp(min=0)
    chain = chain_of(V, kind)
    Ej = 4 * U * (z.abs() + 2.0)
    ds = (q * Ej).sum(1) + chain
    lp = z[at, tt] - ln_s
    r = dict(loss=torch.where(live, -lp, 0.0), lse=torch.where(live, lse, 0.0))
    r["tol_loss"] = torch.where(live, ds + 3 * U + lp.abs() * U, 0.0)
    r["tol_lse"] = torch.where(live, ds + 3 * U + lse.abs() * U, 0.0)
    if from_lse:
        # lse's rounding is an error of every exponent; for 16-bit results the exponent has one more
        # rounding of the size of x / T, and k's own correction is left out (2 u)
        ds = ds + 3 * U + lse.abs() * U * (4 if kind != "fp32" else 2)
        if kind != "fp32":
            Ej = Ej + 4 * U * x.abs() / T
    c = factor / T
    dx = c * q
    tol = abs(c) * q * (Ej + ds[:, None] + 8 * U) + abs(c) * FLUSH
    dx[at, tt] = c * torch.expm1(lp)
    tol[at, tt] += abs(c) * (4 * U + (2 * torch.exp(lp) * ds if from_lse else 0.0))
    r["dx"] = torch.where(live[:, None], dx, 0.0)
    r["tol_dx"] = torch.where(live[:, None], tol * 1.01, 0.0) + r["dx"].abs() * HALF_STEP[kind] + TINY[kind]
    return r


def near(name, got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                 float((off / tol.clamp(min=1e-300)).max()))
    assert bool(torch.isfinite(want).all())


def borders(V, kind):
    """Where a row is cut: its ends, and the borders of every lane count's vectors."""
    per = E[kind]
    at = set(range(min(V, per + 2))) | set(range(max(0, V - 2 * per - 2), V))
    for lanes in (64, 256, 512, 1024):
        step = lanes * per
        n = V // step
        for j in {1, 2, n // 2, n - 1, n}:
            at |= {j * step - 1, j * step, j * step + per - 1}
    return sorted(p for p in at if 0 <= p < V)


def planted(x, kind):
    """Into rows of normally distributed logits, one for each border, a logit there that holds about
    half of the row's mass.  Left out of the statistics it moves the loss by ln 2."""
    at = borders(x.shape[1], kind)
    high = round(math.log(1.65 * x.shape[1]) * 4) / 4
    x[torch.arange(len(at), device=x.device), torch.tensor(at, device=x.device)] = high
    return at
