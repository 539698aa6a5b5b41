"""The tolerances of loss_rows.py would see logits left out of a row's statistics: here the mistake is
planted in the reference, on the CPU."""
import numpy as np
import pytest
import torch

from loss_rows import E, borders, chain_of, planted, reference


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [40, 1003, 8190, 50305, 131072])
def test_a_left_out_border_shows(kind, V):
    at = borders(V, kind)
    per = E[kind]
    assert {0, 1, V - 2, V - 1} <= set(at)
    for lanes in (64, 256, 512, 1024):
        step = lanes * per
        assert V <= step or {step - 1, step, (V - 1) // step * step} <= set(at)
    x = torch.randn(len(at), V, generator=torch.Generator().manual_seed(V))
    t = torch.tensor([(p + V // 2) % V for p in planted(x, kind)])
    whole = reference(x, t, kind, 2.0)
    less = x.clone()
    less[torch.arange(len(at)), torch.tensor(at)] = -np.inf
    off = (reference(less, t, kind, 2.0)["loss"] - whole["loss"]).abs()
    assert bool((off > 0.1).all()) and bool((off > 1000 * whole["tol_loss"]).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1003, 8190, 50305, 131072])
def test_left_out_average_logits_show(kind, V):
    """Any eight neighbours that hold their share of the mass: at 131072 still a few tolerances."""
    x = torch.randn(1, V, generator=torch.Generator().manual_seed(V))
    t = torch.tensor([V // 3])
    whole = reference(x, t, kind, 2.0)
    q = torch.softmax(x[0].double(), 0)
    mass = q[:V // 8 * 8].reshape(-1, 8).sum(1)
    at = 8 * int((mass - 8 / V).abs().argmin())
    assert not at <= V // 3 < at + 8
    less = x.clone()
    less[0, at:at + 8] = -np.inf
    off = (reference(less, t, kind, 2.0)["loss"] - whole["loss"]).abs()
    assert bool((off > 2 * whole["tol_loss"]).all())


def test_reference_is_cross_entropy():
    """The same numbers as torch's own in binary64, masked rows and a temperature among them."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 501, generator=g, dtype=torch.float64).float()
    t = torch.tensor([3, -100, 500, 0, 77, -1, 250])
    z = x.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(z / 0.5, t.clamp(min=-1), ignore_index=-1, reduction="none")
    loss.sum().backward()
    r = reference(x, t, "fp32", 1.0, 0.5)
    assert torch.allclose(r["loss"], loss.detach(), rtol=1e-13, atol=1e-13)
    assert torch.allclose(r["dx"], z.grad, rtol=1e-12, atol=1e-15)
    live = t >= 0
    assert torch.allclose(r["lse"][live], torch.logsumexp(x.double() / 0.5, 1)[live], rtol=1e-14)
    assert 0 < chain_of(128256, "bf16") < 1.1e-5
