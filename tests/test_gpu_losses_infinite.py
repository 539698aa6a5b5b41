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
