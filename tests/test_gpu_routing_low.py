"""Tokens that a sigmoid router likes no expert of: all their logits far below 0, where the scores leave fp32's range
but their shares p = s / sum s do not -- the shares' means, the balance loss and its gradient against binary64."""
import numpy as np
import pytest

from test_gpu_losses import KINDS, f32, gen, ttype
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
