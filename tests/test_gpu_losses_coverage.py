"""Every logit of a row counts, in every shape of the row kernels, and the variants that read large
logits past the caches: against binary64, with tolerances from the additions that a lane makes
(loss_rows.py)."""
import numpy as np
import pytest

from loss_rows import HALF_STEP, U, E, borders, chain_of, near, planted, reference
from test_gpu_losses import KINDS, LAYOUTS, Buf, empty, mp, ttype, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def planted_rows(V, kind, layout, key):
    """planted() in a guarded tensor; the targets are elsewhere."""
    import torch
    rows = len(borders(V, kind))
    g = torch.Generator(device="cuda").manual_seed(key)
    bx = Buf(rows, V, kind, layout.get("pad", 0), layout.get("shift", 0))
    bx.t.copy_(torch.randn(rows, V, generator=g, device="cuda"))
    p = torch.tensor(planted(bx.t, kind), device="cuda")
    t = (p + 1 + torch.randint(V - 1, (rows,), generator=g, device="cuda")) % V
    return bx, t


# one V for every lane count and number of vectors a lane, odd ends on most, and rows longer than what
# is held
SHAPES = {"bf16": [40, 1003, 1900, 3999, 8190, 12003, 16385, 20011, 31001, 40003, 49155, 57001, 65541,
                   81001, 98003, 114000, 131001, 163001, 170003, 524291],
          "fp32": [20, 500, 1003, 2001, 4003, 6001, 8190, 16001, 24001, 32001, 40003, 48005, 57000,
                   65531, 81001, 90003, 262147]}
CASES = [(k, V) for k, vs in SHAPES.items() for V in vs] + [("fp16", V) for V in (1003, 50305, 128256)]
assert {k for k, _ in CASES} == set(KINDS)


@pytest.mark.parametrize("kind,V", CASES)
def test_no_logit_is_left_out(mp, kind, V):  # noqa: F811
    i = CASES.index((kind, V))
    layout = LAYOUTS[i % 4]
    bx, t = planted_rows(V, kind, layout, 50 + i)
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
    per, chain = E[kind], chain_of(V, kind)
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
