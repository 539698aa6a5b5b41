"""Every logit of a row counts, in every shape of the row kernels, and the variants that read large
logits past the caches: against binary64, with tolerances from the additions that a lane makes.

u = 2^-24 is half a step of fp32.  A row is shared by at least 64 lanes, from 512 vectors on by 256;
a lane adds its vectors in pairs -- the 2 E elements of a pair one after another, then to its running
sum, which is rescaled (exp2: 2 u, a product: u, the sum: u) -- and up to four single ones (a head or
tail element, the vectors that are left over).  That bounds a row's sum by

    chain = (2 E + 4 (ceil(vectors / (2 lanes)) + 5) + 8) u

relative, the 8 for the joins.  An exponent has three roundings, exp2 one step: E_j = 4 u (|z_j| + 2) of
a share, z = (x - m) / T, so a sum is off by at most ds = sum_j q_j E_j + chain, and so is lp, besides
3 u of the logarithm.  At 128256 16-bit logits chain is 1.0e-5, where eight average logits are 6e-5.
"""
import numpy as np
import pytest

from loss_reference import FLUSH, HALF_STEP, TINY, U
from test_gpu_losses import KINDS, LAYOUTS, Buf, empty, gen, mp, ttype, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

E = {"bf16": 8, "fp16": 8, "fp32": 4}


def reference(x, t, kind, factor, T=1.0, from_lse=False):
    """Cross-entropy of the rows of a device tensor in binary64: loss, lse, dx and how far each may
    be off.  from_lse: dx formed of an lse that was rounded to fp32, as mp_token_logprob_grad's is."""
    import torch
    x = x.double()
    rows, V = x.shape
    at = torch.arange(rows, device="cuda")
    m = x.amax(1, keepdim=True)
    z = (x - m) / T
    e = torch.exp(z)
    s = e.sum(1, keepdim=True)
    q = e / s
    ln_s = torch.log(s)[:, 0]
    lse = m[:, 0] / T + ln_s
    live = t >= 0
    tt = t.clamp(min=0)
    nvec = V // E[kind]
    lanes = 64 if nvec <= 512 else 256
    chain = (2 * E[kind] + 4 * (-(-nvec // (2 * lanes)) + 5) + 8) * U
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
    import torch
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


def planted(V, kind, layout, key):
    """A row for each border, with a logit there that holds about half of the row's mass; the target
    is elsewhere.  Left out of the statistics it would move the loss by ln 2."""
    import torch
    at = borders(V, kind)
    rows = len(at)
    g = torch.Generator(device="cuda").manual_seed(key)
    lay = {k: v for k, v in layout.items() if k in ("pad", "shift")}
    bx = Buf(rows, V, kind, **lay)
    bx.t.copy_(torch.randn(rows, V, generator=g, device="cuda"))
    p = torch.tensor(at, device="cuda")
    bx.t[torch.arange(rows, device="cuda"), p] = float(np.round(np.log(1.65 * V) * 4) / 4)
    t = (p + 1 + torch.randint(V - 1, (rows,), generator=g, device="cuda")) % V
    return bx, t


# one V for every lane count and number of vectors a lane, odd ends on most, and rows longer than what
# is held
SHAPES = {"bf16": [40, 1003, 1900, 3999, 8190, 12003, 16385, 20011, 31001, 40003, 49155, 57001, 65541,
                   81001, 98003, 114000, 131001, 163001, 170003, 524291],
          "fp32": [20, 500, 1003, 2001, 4003, 6001, 8190, 16001, 24001, 32001, 40003, 48005, 57000,
                   65531, 81001, 90003, 262147]}
CASES = [(k, V) for k, vs in SHAPES.items() for V in vs] + [("fp16", V) for V in (1003, 50305, 128256)]


@pytest.mark.parametrize("kind,V", CASES)
def test_no_logit_is_left_out(mp, kind, V):  # noqa: F811
    i = CASES.index((kind, V))
    layout = LAYOUTS[i % 4]
    bx, t = planted(V, kind, layout, 50 + i)
    x = bx.t.clone()
    rows = x.shape[0]
    r = reference(x, t, kind, 2.0)
    out = lambda: Buf(rows, V, kind, layout.get("dpad", 0), layout.get("dshift", 0))  # noqa: E731
    lx = mp.logits(bx.t)
    # with a gradient (each row by one workgroup), and the losses alone
    bd, loss = out(), empty(rows)
    mp.mp_cross_entropy(lx, t, None, loss, mp.logits_grad(bd.t, 2.0))
    near("loss", loss, r["loss"], r["tol_loss"])
    near("dx", bd.t, r["dx"], r["tol_dx"])
    assert bd.untouched()
    loss = empty(rows)
    mp.mp_cross_entropy(lx, t, None, loss)
    near("loss alone", loss, r["loss"], r["tol_loss"])
    # a teacher of one entry, the target at the student's own logit: the same loss and gradient
    vals = x.gather(1, t[:, None]).float()
    bd, loss = out(), empty(rows)
    mp.mp_distill_loss(lx, mp.teacher(vals, t[:, None].contiguous()), None, loss,
                       mp.logits_grad(bd.t, 2.0))
    near("distill loss", loss, r["loss"], r["tol_loss"])
    near("distill dx", bd.t, r["dx"], r["tol_dx"])
    # the log-probability and its gradient
    lp, lse, bd = empty(rows), empty(rows), out()
    mp.mp_token_logprob(lx, t, lp, lse)
    near("logp", -lp, r["loss"], r["tol_loss"])
    near("lse", lse, r["lse"], r["tol_lse"])
    mp.mp_token_logprob_grad(lx, t, lse, empty(rows, -1.0), mp.logits_grad(bd.t, 2.0))
    rg = reference(x, t, kind, 2.0, from_lse=True)
    near("logprob dx", bd.t, rg["dx"], rg["tol_dx"])
    assert bd.untouched() and bx.untouched()
    # few rows at a time, split over workgroups where they are long, in place
    ws = workspace(mp)
    for a in range(0, rows, 30):
        b = min(a + 30, rows)
        loss = empty(b - a)
        mp.mp_cross_entropy(mp.logits(bx.t[a:b], 1.0, ws), t[a:b], None, loss,
                            mp.logits_grad(bx.t[a:b], 2.0))
        near("split loss", loss, r["loss"][a:b], r["tol_loss"][a:b])
    near("split dx", bx.t, r["dx"], r["tol_dx"])
    assert bx.untouched()


# logits of just over 256 MiB, in a row shape of one wave, of several, and past what is held
STREAMED = [("fp16", 140001, 1003), ("bf16", 2700, 50305), ("fp32", 1400, 50305), ("fp32", 700, 98311)]


@pytest.mark.parametrize("kind,rows,V", STREAMED)
def test_logits_larger_than_the_cache(mp, kind, rows, V):  # noqa: F811
    """Past 256 MiB (the gradient of log-probabilities: 128) the logits are read another way: every
    call, at odd row starts, out of place and in place, a sample of rows against binary64."""
    import torch
    assert rows * V * torch.finfo(ttype(kind)).bits // 8 > 256 << 20
    g = torch.Generator(device="cuda").manual_seed(rows)
    bx = Buf(rows, V, kind, pad=1, shift=1)
    bx.t.copy_(torch.randn(rows, V, generator=g, device="cuda", dtype=ttype(kind)) * 2)
    t = torch.randint(V, (rows,), generator=g, device="cuda")
    bx.t[torch.arange(rows, device="cuda"), t] += 4.0
    t[torch.rand(rows, generator=g, device="cuda") < 0.2] = -100
    some = torch.unique(torch.cat([torch.tensor([0, 1, rows - 2, rows - 1], device="cuda"),
                                   torch.randint(rows, (40,), generator=g, device="cuda")]))
    assert bool((t[some] < 0).any()) and bool((t[some] >= 0).any())
    x, ts = bx.t[some].clone(), t[some]
    T = float(np.float32(0.7))
    r, rg = reference(x, ts, kind, 2.0, T), reference(x, ts, kind, 2.0, T, from_lse=True)
    lx = mp.logits(bx.t, T)
    loss, lp, lse = empty(rows), empty(rows), empty(rows)
    bd = Buf(rows, V, kind, pad=3, shift=3)
    lg = mp.logits_grad(bd.t, 2.0)
    mp.mp_cross_entropy(lx, t, None, loss, lg)
    near("loss", loss[some], r["loss"], r["tol_loss"])
    near("dx", bd.t[some], r["dx"], r["tol_dx"])
    mp.mp_cross_entropy(lx, t, None, loss)
    near("loss alone", loss[some], r["loss"], r["tol_loss"])
    mp.mp_token_logprob(lx, t, lp, lse)
    near("logp", -lp[some], r["loss"], r["tol_loss"])
    near("lse", lse[some], r["lse"], r["tol_lse"])
    bd.t.fill_(1.0)
    mp.mp_token_logprob_grad(lx, t, lse, empty(rows, -1.0), lg)
    near("logprob dx", bd.t[some], rg["dx"], rg["tol_dx"])
    vals = bx.t.gather(1, t.clamp(min=0)[:, None]).float()
    ids = t[:, None].contiguous()
    bd.t.fill_(1.0)
    mp.mp_distill_loss(lx, mp.teacher(vals, ids), None, loss, lg)
    near("distill loss", loss[some], r["loss"], r["tol_loss"])
    near("distill dx", bd.t[some], r["dx"], r["tol_dx"])
    mp.mp_distill_loss(lx, mp.teacher(vals, ids), None, loss)
    near("distill loss alone", loss[some], r["loss"], r["tol_loss"])
    assert bx.untouched() and bd.untouched()
    keep = bx.flat.clone()
    mp.mp_cross_entropy(lx, t, None, loss, mp.logits_grad(bx.t, 2.0))
    near("loss in place", loss[some], r["loss"], r["tol_loss"])
    near("dx in place", bx.t[some], r["dx"], r["tol_dx"])
    bx.flat.copy_(keep)
    mp.mp_token_logprob_grad(lx, t, lse, empty(rows, -1.0), mp.logits_grad(bx.t, 2.0))
    near("logprob dx in place", bx.t[some], rg["dx"], rg["tol_dx"])
    assert bx.untouched()
    del bx, bd, keep, vals
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("V,with_ws", [(1000, False), (60001, False), (60001, True)])
@pytest.mark.parametrize("with_grad", [False, True])
def test_digits_of_a_probability_near_one(mp, kind, V, with_ws, with_grad):  # noqa: F811
    """The target g above a single runner-up, everything else masked: the loss is log(1 + e^-g).
    Where the two lie in different lanes it keeps its relative precision (sums are joined in
    binary64: down to 2^-52); in one lane's vector an fp32 sum holds both, and the loss and the
    target's gradient are right to chain, absolutely."""
    gaps = np.array([8.0, 12.0, 20.0, 28.0])
    per = E[kind]
    chain = (2 * per + 4 * (-(-(V // per) // 512) + 5) + 8) * U if V > 1000 else (2 * per + 4 * 9 + 8) * U
    import torch
    for far in (True, False):
        x = torch.full((4, V), float("-inf"), dtype=ttype(kind), device="cuda")
        t = torch.tensor([0, 8, 504, 504], device="cuda")       # first of a vector each
        other = t + (3 * per if far else 1)
        x[torch.arange(4), t] = torch.tensor(gaps, dtype=ttype(kind), device="cuda")
        x[torch.arange(4), other] = 0.0
        loss, dx = empty(4), torch.empty_like(x)
        lx = mp.logits(x, 1.0, workspace(mp) if with_ws else None)
        mp.mp_cross_entropy(lx, t, None, loss, mp.logits_grad(dx) if with_grad else None)
        want = np.log1p(np.exp(-gaps))
        rel = 4 * U * (gaps + 2) + 8 * U
        tol = want * rel + 2.0 ** -52 if far else np.full(4, chain)
        got = loss.double().cpu().numpy()
        assert (np.abs(got - want) <= tol).all(), (far, got, want, tol)
        if not with_grad:
            continue
        q = np.exp(-gaps) / (1 + np.exp(-gaps))
        dt = dx[torch.arange(4), t].double().cpu().numpy()
        do = dx[torch.arange(4), other].double().cpu().numpy()
        step = HALF_STEP[kind]
        assert (np.abs(dt + q) <= (q * rel + 2.0 ** -52 if far else chain) + q * step).all(), (far, dt, -q)
        assert (np.abs(do - q) <= q * (rel + chain + step)).all(), (far, do, q)
