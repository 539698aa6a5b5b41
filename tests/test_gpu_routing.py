"""Routing to experts on the GPU against its definitions in binary64 (route_reference.py, which also
derives how far each result may be off)."""
import numpy as np
import pytest

import route_reference as ref
from test_gpu_losses import KINDS, Buf, check, dev, f32, gen, host, ttype
from test_gpu_scores import held

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    import torch
    assert torch.cuda.is_available()
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


def workspace(mp):
    import torch
    return torch.full((mp.MP_ROUTE_WORKSPACE_BYTES,), 0xAB, dtype=torch.uint8, device="cuda")


def router(rng, rows, n, kind):
    """Router logits that the type holds exactly, some experts liked more than others."""
    import torch
    x = rng.normal(0, 1.2, (rows, n)) + 0.5 * rng.normal(0, 1, n)
    return torch.as_tensor(x).to(ttype(kind)).double().numpy()


class Out:
    def __init__(self, mp, rows, top, n=None, ws=None):
        import torch
        self.w = torch.full((rows * top + 4,), -55.0, device="cuda")
        self.i = torch.full((rows * top + 4,), -55, dtype=torch.int64, device="cuda")
        self.weights, self.ids = self.w[:-4].view(rows, top), self.i[:-4].view(rows, top)
        self.load = self.share = self.aux = None
        if n is not None:
            self.load = torch.full((n + 1,), -55, dtype=torch.int64, device="cuda")
            self.share, self.aux = torch.full((n,), -55.0, device="cuda"), torch.full((2,), -55.0, device="cuda")
            ws = workspace(mp) if ws is None else ws
        self.struct = mp.routed(self.weights, self.ids, self.load, self.share, self.aux,
                                ws if n is not None else None)

    def untouched(self):
        return bool((self.w[-4:] == -55).all()) and bool((self.i[-4:] == -55).all())


def check_route(mp, x, kind, top, sigmoid=False, bias=None, mask=None, groups=1, top_groups=1, best=1,
                renormalise=True, scale=1.0, pad=0, shift=0, train=True):
    import torch
    rows, n = x.shape
    scale = float(np.float32(scale))
    b, o = Buf(rows, n, kind, pad, shift, x), Out(mp, rows, top, n if train else None)
    cfg = mp.route_cfg(top, int(sigmoid), groups, top_groups, best, renormalise, scale)
    m = None if mask is None else torch.as_tensor(mask, dtype=torch.bool, device="cuda")
    mp.mp_route(mp.logits(b.t), None if bias is None else dev(bias), m, cfg, o.struct)
    want = ref.route(x, bias, mask, sigmoid, top, groups, top_groups, best, renormalise, scale)
    assert np.array_equal(o.ids.cpu().numpy(), want["ids"])
    check("weights", o.weights, want["weights"], want["tol_weights"])
    if train:
        assert np.array_equal(o.load.cpu().numpy(), want["load"])
        check("share", o.share, want["share"], want["tol_share"])
        check("aux", o.aux, held(want["aux"]), want["tol_aux"])
    assert o.untouched() and b.untouched()
    return o, cfg, want


EXPERTS = [1, 2, 3, 7, 8, 9, 16, 33, 60, 64, 65, 96, 128, 160, 255, 256, 257, 384, 512, 513, 1000, 1024]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", EXPERTS)
def test_experts(mp, kind, n, sigmoid):
    rng = gen(40, n)
    for rows, top, biased, pad, shift in ((5, 1, False, 0, 0), (67, min(n, 8), True, 3, 1),
                                          (130, min(n, 16), False, 0, 1), (33, min(n, 3), True, 8, 0)):
        x = router(rng, rows, n, kind)
        bias = f32(0.05 * rng.normal(0, 1, n)) if biased else None
        mask = rng.random(rows) < 0.8 if rows == 67 else None
        check_route(mp, x, kind, top, sigmoid, bias, mask, renormalise=rows != 33, scale=1.0 + rows,
                    pad=pad, shift=shift, train=rows != 5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n,groups", [(4, 2), (6, 3), (60, 5), (64, 8), (64, 64), (128, 16), (160, 8),
                                      (256, 8), (256, 2), (264, 11), (512, 16), (1024, 64), (1000, 4)])
def test_groups(mp, n, groups, sigmoid):
    rng = gen(41, n, groups)
    for best, keep in ((1, 1), (2, max(1, groups // 2)), (2, groups)):
        x = router(rng, 70, n, "fp32")
        x[3, :n // groups] = -np.inf                     # a closed group
        x[4, 1:] = -np.inf                               # one open expert
        bias = f32(0.1 * rng.normal(0, 1, n))
        if n > 8:
            bias[5] = -np.inf
            bias[6] = np.nan
        top = min(16, n // groups * keep)
        check_route(mp, x, "fp32", top, sigmoid, bias, None, groups, keep, best, True, 2.5)
        check_route(mp, x, "fp32", max(1, top // 2), sigmoid, None, None, groups, keep, best, False)


@pytest.mark.parametrize("rows", [1, 2, 3, 255, 256, 257, 4093, 20011])
def test_tokens(mp, rows):
    rng = gen(42, rows)
    x = router(rng, rows, 64, "bf16")
    check_route(mp, x, "bf16", 6, mask=rng.random(rows) < 0.7)
    check_route(mp, x, "bf16", 2, True, f32(rng.normal(0, 0.1, 64)), None, 8, 3, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,groups,top,tokens", [(60, 1, 4, 80), (64, 4, 9, 80), (128, 8, 8, 60), (256, 8, 8, 30),
                                                 (512, 1, 12, 20), (1000, 1, 6, 10)])
def test_more_tokens_than_are_at_work_at_once(mp, kind, n, groups, top, tokens):
    """A wave's second and later tokens, in every form: `tokens` times 1009 that are alike."""
    import torch
    x = router(gen(52, n), 1009, n, kind)
    bias = f32(0.05 * gen(53, n).normal(0, 1, n))
    rows = 1009 * tokens
    b = Buf(rows, n, kind, 8, 0, np.resize(x, (rows, n)))
    mask = np.arange(1009) % 7 != 3
    m = torch.as_tensor(np.resize(mask, rows), device="cuda")
    for given, sigmoid, keep, best in ((None, False, max(1, groups // 2), 1), (bias, True, max(1, groups // 2), 2)):
        want = ref.route(x, given, mask, sigmoid, top, groups, keep, best, True, 1.0)
        cfg = mp.route_cfg(top, int(sigmoid), groups, keep, best, True, 1.0)
        for train in (False, True):
            o = Out(mp, rows, top, n if train else None)
            mp.mp_route(mp.logits(b.t), None if given is None else dev(given), m, cfg, o.struct)
            assert np.array_equal(o.ids.cpu().numpy(), np.resize(want["ids"], (rows, top)))
            check("weights", o.weights, np.resize(want["weights"], (rows, top)),
                  np.resize(want["tol_weights"], (rows, top)))
            if train:
                assert np.array_equal(o.load.cpu().numpy(), want["load"] * tokens)
                # a lane adds up at most ten tokens, of a thousand and more at once; they count in fp32
                more = 10 * 2.0 ** -24 * want["share"]
                check("share", o.share, want["share"], want["tol_share"] + more)
            assert o.untouched() and b.untouched()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n", [8, 60, 256, 600])
def test_equal_scores_take_the_lowest_number(mp, n, sigmoid):
    rng = gen(43, n)
    x = np.round(rng.normal(0, 1, (40, n)))
    x[0] = 0.0
    x[1] = np.where(rng.random(n) < 0.5, -0.0, 0.0)
    x[2] = 5.0 - np.arange(n) % 3
    for groups, keep, best in ((1, 1, 1), (4, 2, 2), (4, 3, 1)):
        check_route(mp, x, "bf16", min(8, n // groups * keep), sigmoid, None, None, groups, keep, best)
        check_route(mp, x, "fp32", 2, sigmoid, np.zeros(n) - 3.0, None, groups, keep, best)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_closed_experts_and_bad_tokens(mp, kind, sigmoid):
    import torch
    rng = gen(44)
    n, rows = 60, 14
    x = router(rng, rows, n, kind)
    lowest = float(torch.finfo(ttype(kind)).min)
    x[0, 3:] = -np.inf               # fewer open than chosen
    x[1, :] = -np.inf                # none
    x[2, 5] = np.nan
    x[3, 59] = np.inf
    x[4, 2:] = lowest
    x[5] = lowest
    x[6, ::2] = -np.inf
    x[7] = np.nan                    # of a token that is not routed
    x[8] *= 1000.0 if kind != "fp16" else 100.0
    x = torch.as_tensor(x).to(ttype(kind)).double().numpy()      # what the type holds of the last
    mask = np.ones(rows, bool)
    mask[7] = mask[9] = False
    bias = f32(rng.normal(0, 0.1, n))
    bias[10], bias[11], bias[12] = -np.inf, np.nan, 1e30
    # x[3] of a sigmoid is a score of 1, of a softmax no distribution
    for b in (None, bias):
        for groups, keep in ((1, 1), (6, 3)):
            check_route(mp, x, kind, 8, sigmoid, b, mask, groups, keep, 2)
    check_route(mp, x, kind, 8, sigmoid, None, np.zeros(rows, bool))


def test_no_tokens_clear_the_sums(mp):
    import torch
    o = Out(mp, 1, 2, 8)
    x = mp.Logits(None, 0, 8, 8, mp.MP_FP32, 1.0, None)
    mp.mp_route(x, None, None, mp.route_cfg(2), o.struct)
    assert not o.load.any() and not o.share.any() and not o.aux.any()
    assert bool((o.ids == -55).all())


def test_near_scores_are_told_apart(mp):
    """Scores that fp32 arithmetic would find equal: sigmoids of neighbouring logits above 8."""
    n = 64
    base = np.float32(9.0)
    steps = np.arange(n, dtype=np.float64) * 2.0 ** -20       # exact in fp32 next to 9
    x = np.stack([base + steps, base + steps[::-1], np.where(np.arange(n) % 2, 9.0, 9.0 + 2.0 ** -20)])
    check_route(mp, x, "fp32", 16, True)
    check_route(mp, x, "fp32", 16, True, np.zeros(n) + 0.25)
    check_route(mp, -x, "fp32", 16, True, np.zeros(n) - 0.25)
    check_route(mp, x, "fp32", 16, False, np.zeros(n) + 0.25)


# --- the gradient ---------------------------------------------------------------------------

def check_grad(mp, x, kind, top, sigmoid=False, mask=None, renormalise=True, scale=1.0, balance=0.02,
               large=0.003, with_dw=True, ids=None, pad=0, shift=0, inplace=False, seed=0):
    import torch
    rows, n = x.shape
    rng = gen(50, n, rows, seed)
    scale, balance, large = (float(np.float32(v)) for v in (scale, balance, 0.0 if sigmoid else large))
    r = ref.route(x, None, mask, sigmoid, top, renormalise=renormalise, scale=scale)
    ids = r["ids"] if ids is None else ids
    load = r["load"] if balance or large else None
    dw = f32(rng.normal(0, 1, (rows, top))) if with_dw else None
    if dw is not None:
        dw[np.isnan(r["weights"])] = 1.0
    b = Buf(rows, n, kind, pad, shift, x)
    bd = b if inplace else Buf(rows, n, kind, pad + 3, shift + 1)
    g = mp.logits_grad(bd.t, 3.0, dev_scale=dev(np.float32([256.0])), dev_count=dev(np.int64([2])))
    cfg = mp.route_cfg(top, int(sigmoid), renormalise=renormalise, scale=scale)
    m = None if mask is None else torch.as_tensor(mask, dtype=torch.uint8, device="cuda")
    mp.mp_route_grad(mp.logits(b.t), m, cfg, dev(ids), None if dw is None else dev(dw),
                     None if load is None else dev(load), balance, large, g)
    want, tol = ref.route_grad(x, ids, mask, dw, load, sigmoid, top, renormalise, scale, balance, large,
                               384.0, kind)
    check("dx", bd.t, want, tol)
    assert b.untouched() and bd.untouched()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", EXPERTS)
def test_gradient(mp, kind, n, sigmoid):
    rng = gen(45, n)
    for i, (rows, top, kw) in enumerate((
            (67, min(n, 8), dict()), (5, 1, dict(renormalise=False, pad=3, shift=1, inplace=True)),
            (130, min(n, 16), dict(balance=0.0, large=0.0, scale=2.5)),
            (40, min(n, 4), dict(with_dw=False, pad=8)), (257, min(n, 2), dict(renormalise=False)))):
        x = router(rng, rows, n, kind)
        mask = rng.random(rows) < 0.8 if i != 1 else None
        check_grad(mp, x, kind, top, sigmoid, mask, seed=i, **kw)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_of_chosen_lists(mp, sigmoid):
    """Lists that routing would not make: absent entries between others, an expert twice, none, an
    expert that is not there, a bad token."""
    rng = gen(46)
    n, rows, top = 60, 12, 6
    x = router(rng, rows, n, "fp32")
    ids = np.stack([rng.permutation(n)[:top] for _ in range(rows)])
    ids[0, 2] = -1
    ids[1] = -1
    ids[2, 3] = n
    ids[3, 1] = ids[3, 4]
    ids[4] = 7
    ids[5, :] = [-1, -1, -1, -1, -1, 3]
    ids[6, 0] = 1 << 40
    x[7, 9] = np.nan
    x[8, ids[8, 0]] = -np.inf
    x[9] = -np.inf
    mask = np.ones(rows, bool)
    mask[10] = False
    x[10] = np.nan
    for renormalise in (False, True):
        check_grad(mp, x, "fp32", top, sigmoid, mask, renormalise, ids=ids)


# --- the bias ---------------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 7, 64, 256, 1000])
def test_bias_update(mp, n):
    import torch
    rng = gen(47, n)
    for layers, loads in ((1, 1), (3, 1), (58, 4)):
        bias = rng.normal(0, 1, (layers, n)).astype(np.float32)
        load = rng.integers(0, 40, (loads, layers, n + 1))
        load[..., 0] += 1 << 40
        load[:, 0, :n] = 5                               # balanced: nothing moves
        total = load[..., :n].sum(0)
        want = bias + np.sign(total.sum(1, keepdims=True) - total * n).astype(np.float32) * np.float32(0.001)
        b, out = dev(bias), torch.empty(layers, n, device="cuda")
        mp.mp_route_bias_update(b, dev(load), 0.001, out)
        assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(b.cpu().numpy(), bias)
        mp.mp_route_bias_update(b, dev(load), 0.001)     # in place
        assert np.array_equal(b.cpu().numpy(), want)
    one = dev(bias[0])
    mp.mp_route_bias_update(one, dev(load[:, 0]), 0.001)
    assert np.array_equal(one.cpu().numpy(), want[0])


# --- how they run -------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,n", [(3, 64), (5000, 256)])
def test_same_bits_every_time(mp, rows, n):
    import torch
    x = router(gen(48), rows, n, "bf16")
    b, outs = Buf(rows, n, "bf16", init=x), []
    for _ in range(3):
        o = Out(mp, rows, 8, n)
        mp.mp_route(mp.logits(b.t), None, None, mp.route_cfg(8), o.struct)
        outs.append(o)
    for o in outs[1:]:
        for name in ("w", "i", "load", "share", "aux"):
            assert torch.equal(getattr(o, name), getattr(outs[0], name)), name


def test_captured_and_replayed(mp):
    """Two graphs that share a workspace, replayed on new inputs with eager work between."""
    import torch
    rows, n, top, ws = 3000, 64, 6, workspace(mp)
    x = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    mask = torch.ones(rows, dtype=torch.bool, device="cuda")
    bias = torch.zeros(n, device="cuda")
    dw, dx = torch.randn(rows, top, device="cuda"), torch.empty_like(x)
    cfg = mp.route_cfg(top, mp.MP_ROUTE_SIGMOID, 8, 4, 2, True, 2.5)

    def work(o, new):
        mp.mp_route(mp.logits(x), bias, mask, cfg, o.struct)
        mp.mp_route_grad(mp.logits(x), mask, cfg, o.ids, dw, o.load, 0.01, 0.0, mp.logits_grad(dx))
        mp.mp_route_bias_update(bias, o.load, 0.001, new)

    outs = [Out(mp, rows, top, n, ws) for _ in range(2)]
    news = [torch.empty_like(bias) for _ in range(2)]
    graphs, side = [], torch.cuda.Stream()
    for o, new in zip(outs, news):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            work(o, new)
        graphs.append(g)
    for i in range(4):
        x.copy_(torch.as_tensor(router(gen(49, i), rows, n, "bf16")))
        mask.copy_(torch.as_tensor(gen(49, i).random(rows) < 0.7))
        bias.copy_(torch.as_tensor(gen(49, 9, i).normal(0, 0.1, n)))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        o, got = outs[i % 2], {}
        for name in ("w", "i", "load", "share", "aux"):
            got[name] = getattr(o, name).clone()
        got_dx, got_new = dx.clone(), news[i % 2].clone()
        e, new = Out(mp, rows, top, n, ws), torch.empty_like(bias)
        work(e, new)
        torch.cuda.synchronize()
        for name in got:
            assert torch.equal(got[name], getattr(e, name)), name
        assert torch.equal(got_dx, dx) and torch.equal(got_new, new)


def test_two_streams_at_once(mp):
    import torch
    streams, data = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        x = router(gen(51, i), 6000, 128, "fp16")
        data.append((x, Buf(6000, 128, "fp16", init=x), Out(mp, 6000, 4, 128)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (x, b, o) in zip(streams, data):
            mp.mp_route(mp.logits(b.t), None, None, mp.route_cfg(4), o.struct, stream=s)
    torch.cuda.synchronize()
    for x, b, o in data:
        want = ref.route(x, None, None, False, 4)
        assert np.array_equal(o.ids.cpu().numpy(), want["ids"])
        assert np.array_equal(o.load.cpu().numpy(), want["load"])


def test_binding_refuses_what_does_not_fit(mp):
    import torch
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        mp.mp_route(mp.logits(x), None, None, mp.route_cfg(3), Out(mp, 4, 2).struct)
    with pytest.raises(ValueError, match="rows"):
        mp.mp_route(mp.logits(x), None, None, mp.route_cfg(2), Out(mp, 3, 2).struct)
    with pytest.raises(ValueError, match="load"):
        mp.mp_route(mp.logits(x), None, None, mp.route_cfg(2), Out(mp, 4, 2, 7).struct)
    h = torch.zeros(4, 8).pin_memory()
    lx = mp.Logits(h.data_ptr(), 4, 8, 8, mp.MP_FP32, 1.0, None)
    with pytest.raises(mp.MpError, match="device memory"):
        mp.mp_route(lx, None, None, mp.route_cfg(2), Out(mp, 4, 2).struct)


def test_binding_refuses_lists_of_another_length(mp):
    import torch
    x, dx = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    ids, dw = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.zeros(4, 3, device="cuda")
    for i, d, name in ((ids, dw[:, :2].contiguous(), "ids"), (ids[:, :2].contiguous(), dw, "dweights")):
        with pytest.raises(ValueError, match=name + " must have 2 columns"):
            mp.mp_route_grad(mp.logits(x), None, mp.route_cfg(2), i, d, None, 0.0, 0.0, mp.logits_grad(dx))


# --- together, as a training program uses them ------------------------------------------------------

@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_step_of_a_small_mixture(mp, sigmoid):
    """Two micro-batches through a router and its experts, the router's gradient through autograd, the
    update step and the balancing bias with it -- and a third step that overflows, which leaves masters,
    weights and bias as they were."""
    import torch
    torch.manual_seed(5)
    dim, n, top, tokens = 32, 16, 4, 96
    router_w = (torch.randn(n, dim, device="cuda") * 0.3).to(torch.bfloat16).requires_grad_()
    experts = torch.randn(n, dim, dim, device="cuda") * 0.2
    numels = [n * dim]
    model = mp.ModelState(numels, mp.MP_BF16)
    model.master[0].copy_(router_w.detach().float().view(-1))
    model.w16[0].copy_(router_w.detach().view(-1))
    state = mp.mp_state_create(mp.scaler_cfg(init_scale=16.0))
    bias = torch.zeros(n, device="cuda")
    loads = torch.zeros(2, n + 1, dtype=torch.int64, device="cuda")
    cfg = mp.route_cfg(top, int(sigmoid), 4, 2, 2, True, 1.5)
    scale = mp.mp_state_scale_ptr(state)
    ws, hp = workspace(mp), mp.adamw_hparams(lr=1e-2)
    sets = None
    for step in range(3):
        grads, before = [], (model.master[0].clone(), bias.clone())
        for i in range(2):
            h = torch.randn(tokens, dim, device="cuda").to(torch.bfloat16)
            mask = torch.rand(tokens, device="cuda") < 0.9
            w = model.w16[0].view(n, dim).detach().requires_grad_()
            z = h @ w.t()
            o = Out(mp, tokens, top, n, ws)
            x = mp.logits(z.detach())
            o.struct.load = loads[i].data_ptr()
            mp.mp_route(x, bias, mask, cfg, o.struct)
            weights = o.weights.detach().requires_grad_()
            picked = experts[o.ids.clamp(min=0)]                         # tokens, top, dim, dim
            y = (weights[..., None] * (picked @ h.float()[:, None, :, None])[..., 0]).sum(1)
            loss = (y * y).mean() * mp.read_stats(state)["scale"]
            dw, = torch.autograd.grad(loss, weights)
            if step == 2 and i == 1:
                dw[0, 0] = float("inf")
                mask[0] = True
            dz = torch.empty_like(z)
            mp.mp_route_grad(x, mask, cfg, o.ids, dw, loads[i], 0.01, 0.0 if sigmoid else 0.001,
                             mp.logits_grad(dz, dev_scale=scale))
            # against autograd in binary64, from the same bits
            if step == 0:
                want, tol = ref.route_grad(host(z), o.ids.cpu().numpy(), mask.cpu().numpy(), host(dw),
                                           loads[i].cpu().numpy(), sigmoid, top, True, 1.5,
                                           float(np.float32(0.01)),
                                           0.0 if sigmoid else float(np.float32(0.001)), 16.0, "bf16")
                check("dz", dz, want, tol)
            g, = torch.autograd.grad(z, w, dz)
            grads.append(g.reshape(-1).contiguous())
        if step == 2:
            grads[1][3] = float("inf")
        if sets is None:
            sets = [model.gradset([g]) for g in grads]
        else:
            for s, g in zip(sets, grads):
                mp.mp_gradset_update(s, [g])
        torch.cuda.synchronize()
        mp.mp_update_step_group(model.plan, state, sets, mp.mp_token_weights([tokens, tokens]), True, 1.0, hp)
        mp.mp_route_bias_update(bias, loads, 0.05, state=state)
        st = mp.read_stats(state)
        if step < 2:
            total = loads[:, :n].sum(0)
            assert st["found_inf"] == 0 and not torch.equal(model.master[0], before[0])
            assert torch.equal(bias, before[1] + 0.05 * torch.sign(total.sum() - total * n).float())
            assert int(total.sum()) == top * int(loads[:, n].sum())
        else:
            assert st["found_inf"] == 1
            assert torch.equal(model.master[0], before[0]) and torch.equal(bias, before[1])
    for s in sets:
        mp.mp_gradset_destroy(s)
    mp.mp_state_destroy(state)
    model.close()
