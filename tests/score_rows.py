"""Scores of logits in binary64 with torch, on the tensors' own device, and how far a result of the
library may be off by the additions that a lane makes in the form that a call takes.

u = 2^-24 is half a step of fp32, z = (x - max) / T.  A row's vectors are dealt to 64, 128 or 256 lanes, or
to parts of 256 lanes each; a lane adds its elements one at a time (`chain` counts them, pairs of vectors whole, and
8 for single ones and what is added when the reference is raised).  A share's exponent is off by u (|z| + 5.6) for its
rounding (the reference may lie 8 below it, 8 ln 2 = 5.6) and u |z| for the rest of log2(e) / T, 2^y by 2 u; each of up
to three joins scales by a power of two of a rounded difference, u (|z| + 5.6) + 2 u.  In all below

    E_j = 5 u (|z_j| + 6.3),

a sum is off by ds = sum_j q_j E_j + chain u, its logarithm by 2 u more.  The entropy ln S - sum_j q_j z_j has the
second sum's own roundings besides: E_j, ds and chain + 8 of them, of |z_j| + 5.6.
"""
import torch

from loss_reference import U

E = {"bf16": 8, "fp16": 8, "fp32": 4}
WORKSPACE = 1 << 20


def parts_of(V, kind, rows, top):
    """Parts of a row and vectors of a part where few long rows are split, or None."""
    nvec = V // E[kind]
    if rows > 128 or nvec < 10000:
        return None
    most = min(64, 2048 // top) if top else 64
    most = min(most, WORKSPACE // ((32 + 8 * top) * rows))
    parts = min(512 // rows, -(-nvec // 512))
    parts = min(max(parts, -(-nvec // 1024)), most)
    if parts < 2:
        return None
    vecs = -(-nvec // parts)
    return -(-nvec // vecs), vecs


def lanes_of(V, kind, rows, top):
    nvec, many = V // E[kind], rows >= 2048
    if nvec <= (1024 if many else 512) and top <= 64:
        return 64
    return 128 if nvec <= (4096 if many else 512) else 256


def chain_of(V, kind, rows, top, with_ws):
    cut = parts_of(V, kind, rows, top) if with_ws else None
    vecs, lanes = (cut[1], 256) if cut else (V // E[kind], lanes_of(V, kind, rows, top))
    return (2 * E[kind] * -(-vecs // (2 * lanes)) + 8) * U


def reference(x, T, chain):
    """lse and entropy of the rows of a tensor, the log-probability of every logit, and how far
    each may be off."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    z = (x - m) / T
    e = torch.exp(z)
    s = e.sum(1, keepdim=True)
    q = e / s
    ln_s = torch.log(s)
    a = torch.where(q > 0, z.abs(), 0.0)
    Ej = 5 * U * (a + 6.3)
    ds = (q * Ej).sum(1) + chain
    mean = (q * a).sum(1)
    var = (q * (a - mean[:, None]) ** 2).sum(1)
    r = dict(lse=(m / T + ln_s)[:, 0], entropy=ln_s[:, 0] + mean, logp=z - ln_s)
    r["tol_lse"] = ds + 2 * U + r["lse"].abs() * U
    r["tol_logp"] = (ds + 2 * U)[:, None] + r["logp"].abs() * U
    r["tol_entropy"] = (ds + 2 * U + (q * (a + 5.6) * Ej).sum(1) + (mean + 5.6) * (ds + chain + 8 * U) + 2 * U * var
                        + r["entropy"] * U)
    return r


def entries(x, top):
    """The ids of the largest logits in order, the lower id first of equal ones."""
    return torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top]


def borders(V, kind, rows, top, with_ws):
    """Where a call cuts its rows: elements at the ends, and, counted from the first whole vector, the first and
    last of what a lane, the unrolled part, its remainder and the parts of a split row go over."""
    per, nvec = E[kind], V // E[kind]
    cut = parts_of(V, kind, rows, top) if with_ws else None
    ends = sorted({p for p in list(range(per + 2)) + list(range(V - 2 * per - 2, V)) if 0 <= p < V})
    at = set()
    lanes = 256 if cut else lanes_of(V, kind, rows, top)
    pieces, vecs = cut if cut else (1, nvec)
    for p in {0, 1, pieces // 2, pieces - 1}:
        lo, hi = p * vecs, min((p + 1) * vecs, nvec)
        unrolled = (hi - lo) // (4 * lanes) * 4 * lanes
        for v in {lo, lo + lanes, lo + 2 * lanes, lo + 3 * lanes, lo + unrolled, lo + unrolled + lanes,
                  lo + unrolled + 2 * lanes, hi}:
            at |= {v * per - 1, v * per}
    return ends, sorted(g for g in at if 0 <= g < nvec * per)


def planted(x, places):
    """Into rows of normally distributed logits, one for each place, a logit there that holds about half
    of the row's mass."""
    high = round(float(torch.log(torch.tensor(1.65 * x.shape[1]))) * 4) / 4
    x[torch.arange(len(places), device=x.device), torch.tensor(places, device=x.device)] = high
