"""Losses of a probability of zero: a target, or a reference's token, whose logit or log-probability
is -inf or the type's lowest value.  What is infinite by its formula is infinite, what is finite is
finite, and the gradient is the formula's."""
import numpy as np
import pytest

import loss_reference as ref
from test_gpu_losses import KINDS, check, dev, empty, f32, gen, make_x, mp, state_for, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("eps", [0.0, 0.05])
@pytest.mark.parametrize("V,with_ws", [(700, False), (60001, True)])
def test_preference_with_a_masked_target(mp, kind, eps, V, with_ws):  # noqa: F811
    """Pair 0 is ordinary; pair 1's chosen and pair 2's rejected sequence hold a target of
    probability 0, so that h is -inf and +inf: losses of +inf, and of 0 (smoothed: +inf); slopes
    -beta (1 - eps) and beta eps.  Both are exact but for dlogp's rounding to fp32."""
    x, t = make_x(gen(41, V), 12, V, kind)
    start = np.arange(0, 13, 2)
    rf = f32(gen(42).normal(-10, 3, 6))
    beta, margin, eps = 0.25, 0.5, float(np.float32(eps))
    factor = 3.0 * 2.0 / 7
    plain = ref.preference(x, t, start, rf, 1.0, "sigmoid", beta, 0.05, margin, False, factor, kind)
    if eps == 0.0:                  # the reference's smoothing term, left out: its factor is 0
        h = beta * ((plain["seq_logp"] - rf)[:3] - (plain["seq_logp"] - rf)[3:]) - margin
        loss0, slope0 = -ref.log_sigmoid(h[0]), -beta / (1 + np.exp(h[0]))
    else:
        plain = ref.preference(x, t, start, rf, 1.0, "sigmoid", beta, eps, margin, False, factor, kind)
        loss0, slope0 = plain["loss"][0], plain["dlogp"][0]
    x[2, t[2]] = -np.inf            # sequence 1: pair 1's chosen
    x[11, t[11]] = -np.inf          # sequence 5: pair 2's rejected
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=workspace(mp) if with_ws else None)
    o = dict(loss=empty(3), seq_logp=empty(6), logp=empty(12), lse=empty(12), dlogp=empty(12))
    mp.mp_preference_loss(lx, dev(t), 3, dev(start), dev(rf),
                          mp.preference_cfg(0, beta, eps, margin), *o.values(), lg)
    # pair 0's tolerance does not depend on the smoothing to first order: |slope| <= beta
    dD = plain["tol_seq_logp"][0] + plain["tol_seq_logp"][3]
    check("loss", o["loss"], np.array([loss0, np.inf, 0.0 if eps == 0.0 else np.inf]),
          np.array([2 * beta * dD + ref.round_tol(loss0), 0.0, 0.0]))
    want = plain["seq_logp"].copy()
    want[[1, 5]] = -np.inf
    check("seq_logp", o["seq_logp"], want, plain["tol_seq_logp"])
    slope = np.array([slope0, -beta * (1 - eps), beta * eps])
    dlogp = np.repeat(np.concatenate([slope, -slope]), 2)
    off = np.repeat(np.tile([beta * beta * dD * 1.01, 0.0, 0.0], 2), 2)
    check("dlogp", o["dlogp"], dlogp, off + ref.round_tol(dlogp))
    d = o["dlogp"].double().cpu().numpy()
    r = ref.logprob(x, t, 1.0, d, factor, kind)
    check("logp", o["logp"], r["logp"], r["tol_logp"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    assert bx.untouched() and bd.untouched()
    del keep


@pytest.mark.parametrize("kind", KINDS)
def test_squared_preference_with_a_masked_target(mp, kind):  # noqa: F811
    """(D - 1/(2 beta))^2 of an infinite D is +inf on either side."""
    x, t = make_x(gen(43), 8, 700, kind)
    x[0, t[0]] = x[7, t[7]] = -np.inf
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind)
    o = [empty(2), empty(4), empty(8), empty(8), empty(8)]
    mp.mp_preference_loss(lx, dev(t), 2, dev(np.arange(0, 9, 2)), None, mp.preference_cfg(1), *o, lg)
    assert o[0].tolist() == [np.inf, np.inf]
    assert o[1][0] == -np.inf and o[1][3] == -np.inf
    del keep, bx, bd, factor


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,with_ws", [(700, False), (60001, True)])
@pytest.mark.parametrize("low", [-np.inf, -3.4028234663852886e38, -1e18, -1e4])
def test_policy_whose_reference_gives_the_token_nothing(mp, kind, V, with_ws, low):  # noqa: F811
    """d = ref_logp - lp far below 0: exp(d) = 0, so kl = -d - 1 (infinite or finite as ref_logp is)
    and its slope is kl_coef exactly; A = 0 leaves that alone, other rows add the policy's own."""
    rows, kl_coef = 6, 0.25
    x, t = make_x(gen(44, V), rows, V, kind)
    parts = ref._target(x, t, 1.0)
    lp, ds = parts[0], parts[4]
    old, adv = f32(lp + 0.05), f32([0.0, 1.0, -1.0, 0.0, 0.5, -0.5])
    w = f32([1.0, 1.0, 2.0, -1.0, 0.5, 1.0])
    rf = np.full(rows, f32(low))
    with np.errstate(all="ignore"):
        kl = -(rf - lp) - 1.0
    rho = np.exp(lp - old)          # e^-0.05: inside 0.8 .. 1.25, the ratio is not clipped
    free, dl = rho * adv, ds + 3 * U
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=workspace(mp) if with_ws else None)
    loss, lp_out, kl_out = empty(rows), empty(rows), empty(rows)
    mp.mp_policy_loss(lx, dev(t), dev(old), dev(rf), dev(adv), dev(w),
                      mp.policy_cfg(0.2, 0.25, kl_coef), loss, lp_out, kl_out, lg)
    err = np.abs(free) * (dl + 4 * U)
    with np.errstate(all="ignore"):
        check("kl", kl_out, kl, dl + ref.round_tol(kl))
        want = w * (kl_coef * kl - free)
        check("loss", loss, want, np.abs(w) * (err + kl_coef * dl) + ref.round_tol(want))
    check("logp", lp_out, lp, dl + ref.round_tol(lp))
    # the slope: kl_coef without an error of its own (1 - exp(d) is 1 to 2^-53)
    dx, tol = ref.target_grad(x, t, 1.0, w * (kl_coef - free), np.abs(w) * err, factor, kind, parts)
    check("dx", bd.t, dx, tol)
    assert bx.untouched() and bd.untouched()
    del keep


def test_policy_kl_slope_over_its_range(mp):  # noqa: F811
    """kl and its slope on both sides of |d| = 1/2 and far out, where A = 0: the target's element of
    the gradient is kl_coef (1 - exp(d)) (1 - q_t), read back relative to its own size.  lp's error
    dl (an exponential's (|t| + 2) 4u a term, the sum's and the logarithm's) enters d as it is; exp's
    own is 2^-23 of exp(d), the series' below 2^-22 of its sum."""
    V = 300
    ds = np.concatenate([[0.5, -0.5], np.linspace(-0.75, 0.75, 31), [-2.0, 2.0, -9.0, 9.0, -40.0, 40.0]])
    rows = len(ds)
    x, t = make_x(gen(45), rows, V, "fp32", 1.0)
    parts = ref._target(x, t, 1.0)
    lp, dl = parts[0], parts[4] + 3 * U
    rf = f32(lp + ds)
    d = rf - lp
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "fp32")
    loss, kl = empty(rows), empty(rows)
    zero = dev(np.zeros(rows))
    mp.mp_policy_loss(lx, dev(t), zero, dev(rf), zero, None, mp.policy_cfg(0.2, 0.2, 0.5), loss, None,
                      kl, lg)
    want = np.where(np.abs(d) < 1e-3, d * d / 2 * (1 + d / 3 * (1 + d / 4)), np.expm1(d) - d)
    slope_err = np.exp(d) * (dl + 2 * U) + np.where(np.abs(d) < 0.6, want * 4 * U, 0.0)
    tol = np.abs(np.expm1(d)) * dl + np.exp(np.maximum(d, 0)) * (dl * dl + 2 * U) * (np.abs(d) > 0.49)
    check("kl", kl, want, tol + want * 4 * U + dl * dl + ref.round_tol(want))
    dx, tol = ref.target_grad(x, t, 1.0, -0.5 * np.expm1(d), 0.5 * slope_err, factor, "fp32", parts)
    check("dx", bd.t, dx, tol)
    assert bx.untouched() and bd.untouched()
    del keep, loss


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,with_ws", [(9, False), (1000, False), (9001, False), (60001, True)])
def test_log_probabilities_under_a_mask(mp, kind, V, with_ws):  # noqa: F811
    """-inf and the type's lowest value at half of the ids, one id left, the target masked: the
    log-probability, and its gradient from the stored lse, in place, too."""
    import torch
    from test_gpu_losses import ttype
    rng = gen(46, V)
    x, t = make_x(rng, 4, V, kind)
    mask = rng.random((4, V)) < 0.5
    mask[np.arange(4), t] = False
    x[0][mask[0]] = -np.inf
    x[1][mask[1]] = float(torch.finfo(ttype(kind)).min)
    x[2], x[2, t[2]] = -np.inf, 3.0
    x[3, t[3]] = -np.inf
    d = f32(rng.normal(0, 1, 4))
    for inplace in (False, True):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, 0.5, inplace=inplace, pad=1, dpad=1,
                                                 ws=workspace(mp) if with_ws else None)
        lp, lse = empty(4), empty(4)
        mp.mp_token_logprob(lx, dev(t), lp, lse)
        mp.mp_token_logprob_grad(lx, dev(t), lse, dev(d), lg)
        r = ref.logprob(x, t, 0.5, d, factor, kind)
        for k, v in (("logp", lp), ("lse", lse), ("dx", bd.t)):
            assert not np.isnan(r["tol_" + k]).any()
            check(k, v, r[k], r["tol_" + k])
        assert lp[3] == -np.inf and bx.untouched() and bd.untouched()
        del keep
