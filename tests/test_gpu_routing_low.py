"""Tokens that a sigmoid router likes no expert of: all their logits far below 0, where the scores leave fp32's range
but their shares p = s / sum s do not -- the shares' means, the balance loss and its gradient against binary64."""
import numpy as np
import pytest

import route_reference as ref
from test_gpu_losses import KINDS, Buf, check, dev, f32, gen, ttype
from test_gpu_routing import check_route, mp  # noqa: F401

pytestmark = pytest.mark.gpu

# below fp32's normal numbers from -87 on, below its smallest from -104, below 2^-1000 (where s counts as 0) from -693
LEVELS = [-20.0, -31.0, -33.0, -60.0, -80.0, -90.0, -95.0, -100.0, -110.0, -400.0, -600.0, -690.0, -693.0, -720.0]


def low(rng, level, rows, n, kind):
    """Router logits around a level that the type holds exactly."""
    import torch
    x = level + rng.normal(0, 2.0, (rows, n))
    return torch.as_tensor(x).to(ttype(kind)).double().numpy()


def check_shares(mp, kind, n, bias, **groups):  # noqa: F811
    """Calls of low tokens alone, and of some among ordinary ones."""
    rng = gen(60, n)
    for level in LEVELS:
        _, _, want = check_route(mp, low(rng, level, 21, n, kind), kind, min(n, 4), True, bias, **groups)
        assert want["load"][n] == 21
        if level > -690:
            assert abs(want["share"].sum() - 1.0) < 1e-12
    x = low(rng, 0.0, 40, n, kind)
    x[7:7 + len(LEVELS)] = np.concatenate([low(rng, v, 1, n, kind) for v in LEVELS])
    check_route(mp, x, kind, min(n, 4), True, bias, **groups)
    check_route(mp, x, kind, min(n, 12), True, bias, rng.random(40) < 0.8, **groups)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 60, 100, 256, 400, 1000])
def test_shares_of_low_tokens_by_a_bias(mp, kind, n):  # noqa: F811
    check_shares(mp, kind, n, f32(0.05 * gen(59, n).normal(0, 1, n)))
    if n % 4 == 0:                      # sums of two scores are binary64 too
        check_shares(mp, kind, n, None, groups=4, top_groups=2, best=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 60, 100, 256, 400, 1000])
def test_shares_of_low_tokens_by_logits(mp, kind, n):  # noqa: F811
    check_shares(mp, kind, n, None)
    if n % 4 == 0:
        check_shares(mp, kind, n, None, groups=4, top_groups=2, best=1)


@pytest.mark.parametrize("biased", [True, False])
def test_a_low_token_does_not_change_others(mp, biased):  # noqa: F811
    """The choice and the weights of the tokens that share a wave with low ones."""
    rng = gen(62)
    x = low(rng, 0.0, 64, 60, "bf16")
    bias = f32(0.05 * rng.normal(0, 1, 60)) if biased else None
    a, _, _ = check_route(mp, x, "bf16", 6, True, bias)
    y = x.copy()
    y[::3] = low(rng, -100.0, 22, 60, "bf16")
    b, _, _ = check_route(mp, y, "bf16", 6, True, bias)
    keep = np.arange(64) % 3 != 0
    assert np.array_equal(a.ids.cpu().numpy()[keep], b.ids.cpu().numpy()[keep])


# --- the gradient ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [3, 60, 100, 256, 400, 1000])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_of_low_tokens(mp, kind, n, renormalise):  # noqa: F811
    """With factors up to an ordinary loss scale: a product of 1 / sum s and the pull of a balance loss would leave
    fp32's range where the gradient is an ordinary number."""
    rng = gen(61, n)
    top, balance = min(n, 4), float(np.float32(0.01))
    for level in LEVELS[:-2]:
        for scale, with_dw in ((65536.0, False), (65536.0, True), (2.0 ** -10, False), (1.0, True)):
            x = low(rng, level, 9, n, kind)
            r = ref.route(x, None, None, True, top, renormalise=renormalise)
            dw = f32(rng.normal(0, 1, (9, top)) * scale) if with_dw else None
            b, bd = Buf(9, n, kind, 0, 0, x), Buf(9, n, kind, 3, 1)
            g = mp.logits_grad(bd.t, 1.0, dev_scale=dev(np.float32([scale])))
            mp.mp_route_grad(mp.logits(b.t), None, mp.route_cfg(top, 1, renormalise=renormalise), dev(r["ids"]),
                             None if dw is None else dev(dw), dev(r["load"]), balance, 0.0, g)
            # what has a sigmoid below 2^-126 adds nothing to the chosen weights' part
            want, tol = ref.route_grad(x, r["ids"], None, dw, r["load"], True, top, renormalise, 1.0, balance,
                                       0.0, scale, kind)
            check(("dx", level, scale, with_dw), bd.t, want, tol)
            if not with_dw and n > 8 and scale > 1:
                assert np.abs(want).max() > 100 * tol.max()
            assert b.untouched() and bd.untouched()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("level", [0.0, -20.0, -29.0, -50.0])
def test_gradient_of_large_factors(mp, kind, level):  # noqa: F811
    """A pull near 2^102, which 1 / sum s would take past fp32's range."""
    rng = gen(63)
    x = low(rng, level, 9, 60, kind)
    r = ref.route(x, None, None, True, 4)
    b, bd, scale = Buf(9, 60, kind, init=x), Buf(9, 60, kind), 2.0 ** 112
    g = mp.logits_grad(bd.t, 1.0, dev_scale=dev(np.float32([scale])))
    balance = float(np.float32(0.01))
    mp.mp_route_grad(mp.logits(b.t), None, mp.route_cfg(4, 1), dev(r["ids"]), None,
                     dev(r["load"]), balance, 0.0, g)
    want, tol = ref.route_grad(x, r["ids"], None, None, r["load"], True, 4, True, 1.0, balance, 0.0, scale, kind)
    assert 2.0 ** 90 < np.abs(want).max() < 2.0 ** 110
    check("dx", bd.t, want, tol)
    assert bd.untouched()
