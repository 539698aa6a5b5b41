"""The balancing bias of a skipped step stays to the bit."""
import pytest

from test_gpu_routing import mp  # noqa: F401

pytestmark = pytest.mark.gpu


def test_bias_of_a_skipped_step_keeps_its_bits(mp):  # noqa: F811
    import torch
    model = mp.ModelState([8], mp.MP_BF16)
    state = mp.mp_state_create(mp.scaler_cfg(init_scale=1.0))
    for x in (*model.master, *model.m, *model.v):
        x.zero_()
    g = torch.full((8,), float("inf"), dtype=torch.bfloat16, device="cuda")
    grads = model.gradset([g])
    hp = mp.adamw_hparams(lr=1e-3)
    mp.mp_update_step_group(model.plan, state, [grads], [1.0], True, 1.0, hp)
    torch.cuda.synchronize()
    assert mp.read_stats(state)["found_inf"] == 1
    bias = torch.tensor([-0.0, 0.0, 1.5, -1e-42, float("-inf"), float("inf"), float("nan"), -2.0], device="cuda")
    load = torch.arange(9, dtype=torch.int64, device="cuda")
    for speed in (0.5, 0.0):
        out = torch.full_like(bias, 7.0)
        mp.mp_route_bias_update(bias, load, speed, out, state=state)
        assert torch.equal(out.view(torch.int32), bias.view(torch.int32))
        one = bias.clone()
        mp.mp_route_bias_update(one, load, speed, state=state)
        assert torch.equal(one.view(torch.int32), bias.view(torch.int32))
    mp.mp_gradset_destroy(grads)
    mp.mp_state_destroy(state)
    model.close()
