"""Distillation where logits are masks or far from 0: only differences of logits count, on either
side, so a common offset (the type's lowest value for all is one) changes nothing."""
import numpy as np
import pytest

from loss_reference import FLUSH, U, round_tol
from loss_rows import chain_of
from test_gpu_losses import KINDS, check, dev, empty, f32, gen, mp, state_for, ttype, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def definition(x, v, ids, t_lse, T, w, factor, kind):
    """loss and dx of every row in binary64 from differences of logits, and how far each may be off:
    a share p_e has the error of its exponent (4 u (|log p_e| + 4), its own normaliser's dn besides),
    log q that of the row's sum (ds) -- see loss_rows.py -- and sums of shares are formed in binary64.
    A share of 0 adds 0, whatever stands beside it."""
    rows, V = x.shape
    loss, dx, tol_loss, tol_dx = np.zeros(rows), np.zeros((rows, V)), np.zeros(rows), np.zeros((rows, V))
    for r in range(rows):
        there = ids[r] >= 0
        if w[r] == 0 or not there.any():
            continue
        with np.errstate(all="ignore"):
            m = x[r].max()
            z = (x[r] - m) / T
            ln_s = np.log(np.exp(z).sum())
            q = np.exp(z - ln_s)
            Ej = 4 * U * (np.where(np.isfinite(z), np.abs(z), 0.0) + 2.0)
            ds = (q * Ej).sum() + chain_of(V, kind)
            id, top = ids[r][there], v[r][there].max()
            d = (v[r][there] - top) / T
            norm = np.log(np.exp(d).sum()) if t_lse is None else t_lse[r] - top / T
            lp = d - norm
            p = np.exp(lp)
            some = p > 0
            size = np.where(some, np.abs(lp), 0.0)
            dn = (p * 4 * U * (size + 4)).sum() if t_lse is None else 0.0
            dp = p * (4 * U * (size + 4) + dn)
            lq = z[id] - ln_s
            gap = np.where(some, np.where(some, lp, 0.0) - lq, 0.0)
            loss[r] = w[r] * np.where(some, p * gap, 0.0).sum()
            tol_loss[r] = abs(w[r]) * (np.where(some, dp * np.abs(gap), 0.0).sum()
                                       + p.sum() * (dn + ds + 4 * U))
            # the largest share's logit against the largest of the list, in binary64
            tol_loss[r] += abs(w[r]) * np.where(some, p * np.abs(gap), 0.0).sum() * 2.0 ** -50
            mass, c = p.sum(), w[r] * factor / T
            share, dshare = np.zeros(V), np.zeros(V)
            np.add.at(share, id, p)
            np.add.at(dshare, id, dp + p * 2 * U * len(id))
            dx[r] = c * (q * mass - share)
            tol_dx[r] = abs(c) * (q * mass * (Ej + ds + dn + 4 * U * (size.max() + 4) + 8 * U) + dshare
                                  + (q * mass + share) * 2 * U + mass * FLUSH)
    assert not np.isnan(tol_loss[np.isfinite(loss)]).any() and not np.isnan(tol_dx).any()
    # a loss is an fp32 number: w p 3.4e38 with w p past 1 is past its largest, and rounds to inf
    past = np.abs(loss) > np.finfo(np.float32).max
    loss[past] = np.sign(loss[past]) * np.inf
    return dict(loss=loss, dx=dx, tol_loss=tol_loss + round_tol(loss),
                tol_dx=tol_dx * 1.01 + round_tol(dx, kind))


def run(mp, x, v, ids, t_lse, T, w, kind, ws):  # noqa: F811
    import torch
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws)
    tv, ti = dev(v, ttype(kind)), dev(ids)
    loss, alone = empty(len(x)), empty(len(x))
    teacher = mp.teacher(tv, ti, None if t_lse is None else dev(t_lse, torch.float32))
    mp.mp_distill_loss(lx, teacher, dev(w, torch.float32), loss, lg)
    mp.mp_distill_loss(lx, teacher, dev(w, torch.float32), alone)
    r = definition(x, v, ids, t_lse, T, w, factor, kind)
    check("loss", loss, r["loss"], r["tol_loss"])
    check("loss alone", alone, r["loss"], r["tol_loss"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    assert bx.untouched() and bd.untouched()
    del keep
    return loss


ROWS = 9


def rows_of(kind, V, k, key):
    import torch
    rng = gen(70, key, V, k)
    low = float(torch.finfo(ttype(kind)).min)

    def held(a):
        return torch.as_tensor(a).to(ttype(kind)).double().numpy()
    x, v = held(rng.normal(0, 2, (ROWS, V))), held(rng.normal(1, 2, (ROWS, k)))
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(ROWS)])
    x[1] = low                              # the student knows nothing: uniform
    v[2] = low                              # the teacher's list is uniform
    x[3], v[3] = low, low
    x[4], v[4] = held(x[4] + 4000.0), held(v[4] - 3000.0)
    v[5, ::2] = -np.inf                     # entries that the teacher masks ...
    x[5, ids[5, ::2]] = -np.inf             # ... where the student may mask them, too
    x[6, ids[6]] = -np.inf                  # the student masks the whole list: an infinite loss
    x[7, ids[7, 0]] = low                   # one entry of the list next to nothing
    v[8, 1:] = low                          # all of the share on one entry
    return x, v, ids, rng


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,k,with_ws", [(40, 3, False), (700, 3, False), (700, 65, False), (9001, 7, False),
                                         (9001, 300, False), (60001, 5, False), (60001, 5, True),
                                         (60001, 300, True), (300007, 3, False)])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_only_differences_of_logits_count(mp, kind, V, k, with_ws, T):  # noqa: F811
    x, v, ids, rng = rows_of(kind, V, k, 0)
    w = f32(rng.uniform(0.5, 2, ROWS))
    loss = run(mp, x, v, ids, None, T, w, kind, workspace(mp) if with_ws else None)
    assert loss[6] == np.inf


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,k,with_ws", [(700, 5, False), (9001, 300, False), (60001, 5, True)])
def test_with_the_teachers_normaliser(mp, kind, V, k, with_ws):  # noqa: F811
    """The same with a given lse (rounded to fp32: at the lowest value it holds no log k)."""
    x, v, ids, rng = rows_of(kind, V, k, 1)
    top = v.max(1)
    lse = f32(top + np.log(np.exp(v - top[:, None]).sum(1)) + 0.1)
    run(mp, x, v, ids, lse, 1.0, f32(rng.uniform(0.5, 2, ROWS)), kind, workspace(mp) if with_ws else None)


@pytest.mark.parametrize("kind", KINDS)
def test_an_offset_changes_nothing(mp, kind):  # noqa: F811
    """Logits on a grid of 1/4 within +-16, which hold after adding 0, 32 or -32 in every type: the
    losses agree with each other to their rounding, not to that of the offset."""
    rng = gen(71)
    x = np.round(rng.normal(0, 1, (5, 3000)) * 4) / 4
    v = np.round(rng.normal(0, 1, (5, 20)) * 4) / 4
    ids = np.stack([rng.choice(3000, 20, replace=False) for _ in range(5)])
    w = np.ones(5)
    base = run(mp, x, v, ids, None, 1.0, w, kind, None)
    for a, b in ((32.0, -32.0), (-32.0, 32.0), (32.0, 32.0)):
        if kind == "bf16":
            a, b = a / 16, b / 16
        got = run(mp, x + a, v + b, ids, None, 1.0, w, kind, None)
        assert bool(((got - base).abs() <= 4 * U * base.abs()).all()), (a, b, got - base)
