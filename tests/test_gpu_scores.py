"""The scores of logits on the GPU against their definitions in binary64 (score_reference.py, which
also derives how far each result may be off)."""
import numpy as np
import pytest

import score_reference as ref
from test_gpu_losses import KINDS, Buf, check, dev, f32, gen, host, make_x, ttype

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
    return torch.zeros(mp.MP_SCORE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def held(a):
    """What fp32 holds of it: values past its range round to infinity."""
    with np.errstate(over="ignore"):
        return np.where(np.isinf(f32(a)), f32(a), a)


class Out:
    """The outputs of a score with a guard behind each."""

    def __init__(self, mp, rows, top, ws=None):
        import torch
        self.flat = {n: torch.full((rows + 8,), -55.0, device="cuda") for n in ("logp", "lse", "entropy")}
        for n in ("top_logp", "top_values"):
            self.flat[n] = torch.full((rows * top + 8,), -55.0, device="cuda")
        self.flat["top_ids"] = torch.full((rows * top + 8,), -55, dtype=torch.int64, device="cuda")
        self.rows, self.top = rows, top
        for n, t in self.flat.items():
            setattr(self, n, t[:rows] if n in ("logp", "lse", "entropy") else t[:rows * top].view(rows, top))
        lists = (self.top_ids, self.top_logp, self.top_values) if top else ()
        self.struct = mp.score(self.logp, self.lse, self.entropy, *lists, workspace=ws)

    def untouched(self):
        return all(bool((t[-8:] == -55).all()) for t in self.flat.values())


def check_score(mp, x, targets, kind, T=1.0, top=0, pad=0, shift=0, ws=None, logits=None):
    """Scores x (rows x V, float64, exact in `kind`) and checks every output; returns them."""
    T = float(np.float32(T))              # what the struct holds
    rows, V = x.shape
    b = logits if logits is not None else Buf(rows, V, kind, pad, shift, x)
    o = Out(mp, rows, top, ws)
    if targets is None:
        o.struct.logp = None
    mp.mp_token_score(mp.logits(b.t, T), None if targets is None else dev(targets), o.struct)
    want = ref.score(x, targets, T, top)
    for name in ("lse", "entropy") + (("logp",) if targets is not None else ()):
        check(name, getattr(o, name), held(want[name]), want["tol_" + name])
    if top:
        assert np.array_equal(o.top_ids.cpu().numpy(), want["ids"])
        assert np.array_equal(host(o.top_values), want["values"])
        check("top_logp", o.top_logp, held(want["top_logp"]), want["tol_top_logp"])
    assert o.untouched() and b.untouched()
    return o


SIZES = [(1, 1, 1), (3, 2, 4), (5, 7, 7), (4, 8, 3), (6, 9, 20), (3, 63, 64), (9, 64, 5), (7, 65, 128),
         (5, 511, 20), (3, 513, 1), (17, 1000, 128), (6, 2048, 8), (5, 2049, 64), (4, 4097, 127),
         (33, 8192, 20), (3, 16385, 33), (5, 32001, 5), (4, 50304, 64), (3, 65537, 128),
         (3, 128256, 20), (2, 131075, 100), (2, 300007, 17)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,V,top", SIZES)
def test_sizes(mp, kind, rows, V, top):
    rng = gen(1, V, top)
    x, t = make_x(rng, rows, V, kind)
    t = np.where(rng.random(rows) < 0.2, -100, t)
    for T, pad, shift, ws in ((1.0, 0, 0, None), (0.7, 5, 3, workspace(mp)), (2.0, 8, 8, workspace(mp))):
        check_score(mp, x, t, kind, T, top, pad, shift, ws)


@pytest.mark.parametrize("kind", KINDS)
def test_without_targets_or_lists(mp, kind):
    x, t = make_x(gen(2), 7, 3000, kind)
    check_score(mp, x, None, kind, 1.3, 9)
    check_score(mp, x, None, kind, 1.0, 0)
    check_score(mp, x, t, kind, 1.0, 0, ws=workspace(mp))


def test_each_output_alone(mp):
    import torch
    x, t = make_x(gen(3), 5, 1111, "bf16")
    b = Buf(5, 1111, "bf16", init=x)
    whole = check_score(mp, x, t, "bf16", 1.0, 6)
    for name in ("logp", "lse", "entropy", "top_ids"):
        o = Out(mp, 5, 6)
        s = mp.score(**{name: getattr(o, name)})
        mp.mp_token_score(mp.logits(b.t), dev(t), s)
        for n in ("logp", "lse", "entropy", "top_ids", "top_logp", "top_values"):
            if n == name:
                assert torch.equal(getattr(o, n), getattr(whole, n))
            else:
                assert bool((o.flat[n] == -55).all()), n


@pytest.mark.parametrize("rows", [1, 2, 31, 100, 256, 257, 5000])
def test_rows(mp, rows):
    for V, top in ((50304, 20), (999, 3)):
        if rows * V > 3e7:
            continue
        x, t = make_x(gen(4, rows), rows, V, "bf16")
        a = check_score(mp, x, t, "bf16", 1.0, top)
        b = check_score(mp, x, t, "bf16", 1.0, top, ws=workspace(mp))
        assert np.array_equal(a.top_ids.cpu().numpy(), b.top_ids.cpu().numpy())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vectors,top", [(1000, 7), (1030, 65), (1700, 20), (1700, 0), (4100, 9)])
def test_many_rows(mp, kind, vectors, top):
    """Rows of which workgroups of 64, 128 and 256 lanes are taken, where there are many: 2100 that
    repeat 20."""
    V = vectors * (4 if kind == "fp32" else 8) + 3
    x, t = make_x(gen(18, V), 20, V, kind)
    t = np.where(np.arange(20) % 5 == 3, -100, t)
    T = float(np.float32(0.9))
    want = ref.score(x, t, T, top)
    b = Buf(2100, V, kind, init=np.resize(x, (2100, V)))
    o = Out(mp, 2100, top)
    mp.mp_token_score(mp.logits(b.t, T), dev(np.resize(t, 2100)), o.struct)
    for name in ("logp", "lse", "entropy"):
        check(name, getattr(o, name), np.resize(held(want[name]), 2100), np.resize(want["tol_" + name], 2100))
    if top:
        assert np.array_equal(o.top_ids.cpu().numpy(), np.resize(want["ids"], (2100, top)))
        assert np.array_equal(host(o.top_values), np.resize(want["values"], (2100, top)))
        check("top_logp", o.top_logp, np.resize(held(want["top_logp"]), (2100, top)),
              np.resize(want["tol_top_logp"], (2100, top)))
    assert o.untouched() and b.untouched()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,top", [(40, 64), (5000, 50), (70001, 128)])
def test_equal_logits_come_in_the_order_of_their_ids(mp, kind, V, top):
    import torch
    rng = gen(5, V)
    x = np.stack([np.zeros(V), np.where(rng.random(V) < 0.5, -0.0, 0.0),
                  np.round(rng.normal(0, 1, V)), np.full(V, -7.0), np.arange(V) % 5 * 1.0,
                  np.sort(rng.normal(0, 3, V)), -np.sort(rng.normal(0, 3, V)),
                  np.where(np.arange(V) == V - 1, 3.0, -2.0),
                  np.where(np.arange(V) % 2048 < 9, 5.0 + rng.normal(0, 1, V), rng.normal(0, 0.1, V)),
                  # the largest in few lanes' share of the row, many of them
                  np.where(np.arange(V) % 2048 < 2, 4.0 + rng.random(V), -rng.random(V)),
                  np.where(np.arange(V) // 8 % 256 == 7, 4.0, -1.0)])
    x = torch.as_tensor(x).to(ttype(kind)).double().numpy()
    for ws in (None, workspace(mp)):
        check_score(mp, x, None, kind, 1.0, top, ws=ws)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [300, 8192, 128256])
def test_masks(mp, kind, V):
    """-inf, the type's lowest value, and the customary large negative numbers in masked places."""
    import torch
    rng = gen(6, V)
    lowest = float(torch.finfo(ttype(kind)).min)
    rows = []
    for value in (-np.inf, lowest, -1e4, -3e4 if kind == "fp16" else -1e9):
        for keep in (1, 3, 25, V // 2):
            x = rng.normal(0, 2, V)
            gone = rng.permutation(V)[keep:]
            x[gone] = value
            rows.append(x)
    rows.append(np.where(np.arange(V) < 7, lowest, -np.inf))
    rows.append(np.full(V, lowest))
    x = torch.as_tensor(np.stack(rows)).to(ttype(kind)).double().numpy()
    t = np.argmax(x, 1)
    t[::3] = rng.integers(0, V, len(t[::3]))       # some of them masked: -inf
    for top, ws in ((20, None), (64, workspace(mp))):
        check_score(mp, x, t, kind, 1.0, top, ws=ws)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 70, 5000, 128256])
def test_rows_without_a_distribution(mp, kind, V):
    rng = gen(7, V)
    x, t = make_x(rng, 8, V, kind)
    x[1, V // 2] = np.nan
    x[2] = -np.inf
    x[3, V - 1] = np.inf
    x[4] = np.nan
    x[5, 0] = -np.nan
    t[6] = -1
    x[6] = np.nan
    t[0] = V + 5          # past the vocabulary: its log-probability alone is NaN
    for ws in (None, workspace(mp)):
        check_score(mp, x, t, kind, 1.0, 5, ws=ws)


@pytest.mark.parametrize("kind", KINDS)
def test_large_logits_and_temperatures(mp, kind):
    import torch
    rng = gen(8)
    x = rng.normal(0, 2, (8, 9000))
    top = dict(bf16=1e38, fp16=6e4, fp32=1e38)[kind]
    x[1] += 6e4 if kind == "fp16" else 1e7        # an offset that all share
    x[2] -= 6e4 if kind == "fp16" else 1e6
    x[3] *= 1e3
    x[4] = rng.uniform(-top, top, 9000)
    x[5, 77] = top
    x[6, :20] = -top
    x = torch.as_tensor(x).to(ttype(kind)).double().numpy()
    t = rng.integers(0, 9000, 8)
    for T in (1.0, 2.0 ** -20, 2.0 ** 20, 1e-3):
        check_score(mp, x, t, kind, T, 30)
        check_score(mp, x, t, kind, T, 30, ws=workspace(mp))


def test_confident_rows(mp):
    """Nearly all of the probability on one entry: the entropy keeps the digits its sum has."""
    for kind in KINDS:
        x = np.zeros((6, 1000))
        for r, big in enumerate((5, 12, 20, 30, 200, 1000)):
            x[r, 500 + r] = big
        check_score(mp, x, np.arange(500, 506), kind, 1.0, 3)


def test_offsets_beyond_32_bits(mp):
    import torch
    rows, V, stride = 4, 5003, (1 << 30) + 1027
    flat = torch.empty((rows - 1) * stride + V, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(flat, (rows, V), (stride, 1))
    x, t = make_x(gen(9), rows, V, "bf16")
    view.copy_(torch.as_tensor(x))

    class B:
        t = view

        @staticmethod
        def untouched():
            return True
    for ws in (None, workspace(mp)):
        o = check_score(mp, x, t, "bf16", 1.0, 9, ws=ws, logits=B)
    dx = torch.as_strided(torch.empty_like(flat), (rows, V), (stride, 1))
    d = torch.ones(rows, device="cuda")
    mp.mp_token_score_grad(mp.logits(view), dev(t), o.lse, o.entropy, d, d, mp.logits_grad(dx))
    want, tol = ref.score_grad(x, t, host(o.lse), host(o.entropy), np.ones(rows), np.ones(rows), kind="bf16")
    check("dx", dx, want, tol)


# --- the gradient ---------------------------------------------------------------------------

def check_grad(mp, x, t, kind, T=1.0, part="both", pad=0, shift=0, inplace=False):
    import torch
    T = float(np.float32(T))
    rows, V = x.shape
    rng = gen(20, rows, V)
    s = ref.score(x, t, T)
    lse, H = f32(s["lse"]), f32(s["entropy"])
    dl = f32(rng.normal(0, 1, rows)) if part != "entropy" else None
    dh = f32(rng.normal(0, 1, rows)) if part != "logp" else None
    for r, zero in ((0, (dl, dh)), (1, (dl,)), (2, (dh,))):
        if rows > 3:
            for d in zero:
                if d is not None:
                    d[r] = 0.0
    b = Buf(rows, V, kind, pad, shift, x)
    bd = b if inplace else Buf(rows, V, kind, pad + 3, shift + 1)
    scale, count = torch.full((1,), 2.0, device="cuda"), torch.full((1,), 7, device="cuda")
    g = mp.logits_grad(bd.t, 3.0, dev_scale=scale, dev_count=count)
    mp.mp_token_score_grad(mp.logits(b.t, T), None if t is None else dev(t), dev(lse),
                           dev(H) if dh is not None else None,
                           dev(dl) if dl is not None else None, dev(dh) if dh is not None else None, g)
    want, tol = ref.score_grad(x, t, lse, H, dl, dh, T, 6.0 / 7.0, kind)
    check("dx", bd.t, want, tol)
    assert b.untouched() and bd.untouched()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,V", [(1, 1), (5, 2), (4, 9), (6, 63), (9, 513), (5, 2049), (33, 8192),
                                    (4, 32001), (5, 128256), (2, 300007), (3000, 40)])
def test_gradient(mp, kind, rows, V):
    rng = gen(10, V)
    x, t = make_x(rng, rows, V, kind)
    t = np.where(rng.random(rows) < 0.2, -100, t)
    for T, part, pad, shift, inplace in ((1.0, "both", 0, 0, False), (0.7, "both", 5, 3, True),
                                         (2.0, "entropy", 8, 8, False), (1.0, "logp", 0, 1, False)):
        check_grad(mp, x, t, kind, T, part, pad, shift, inplace)
    check_grad(mp, x, None, kind, 1.0, "entropy")


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_of_masks_and_confident_rows(mp, kind):
    import torch
    rng = gen(11)
    V = 4000
    x, t = make_x(rng, 9, V, kind)
    lowest = float(torch.finfo(ttype(kind)).min)
    x[3, 100:] = -np.inf
    t[3] = 5
    x[4, 100:] = lowest
    t[4] = 7
    x[5, 100:] = -np.inf
    t[5] = 200                  # the target itself is masked
    x[6] = 0.0
    x[7, 9] = 40.0
    t[7] = 9
    check_grad(mp, x, t, kind)


def test_gradient_of_bad_rows_is_nan(mp):
    import torch
    V = 700
    x, t = make_x(gen(12), 6, V, "bf16")
    t[0] = V
    x[1, 3] = np.nan
    x[2] = -np.inf
    t[3] = -5
    x[3] = np.nan
    b, o = Buf(6, V, "bf16", init=x), Out(mp, 6, 0)
    mp.mp_token_score(mp.logits(b.t), dev(t), o.struct)
    dx = torch.full((6, V), -77.0, dtype=torch.bfloat16, device="cuda")
    d = torch.ones(6, device="cuda")
    mp.mp_token_score_grad(mp.logits(b.t), dev(t), o.lse, o.entropy, d, d, mp.logits_grad(dx))
    assert bool(dx[:3].isnan().all()) and bool((dx[3] == 0).all()) and bool(dx[4:].isfinite().all())


# --- how they run -------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,V", [(1, 128256), (7, 50304), (300, 5000)])
def test_same_bits_every_time(mp, rows, V):
    import torch
    x, t = make_x(gen(13), rows, V, "bf16")
    b, ws = Buf(rows, V, "bf16", init=x), workspace(mp)
    outs = []
    for _ in range(4):
        o = Out(mp, rows, 20, ws)
        ws.random_()
        mp.mp_token_score(mp.logits(b.t), dev(t), o.struct)
        outs.append(o)
    for o in outs[1:]:
        for n in o.flat:
            assert torch.equal(o.flat[n], outs[0].flat[n]), n


@pytest.mark.parametrize("rows,V", [(1, 128256), (40, 9000), (600, 700)])
def test_captured_and_replayed(mp, rows, V):
    """Two graphs that share a workspace, replayed on new inputs with eager work between."""
    import torch
    ws, top = workspace(mp), 12
    x, t = make_x(gen(14), rows, V, "bf16")
    b, tt = Buf(rows, V, "bf16", init=x), dev(t)
    dx = torch.empty_like(b.t)
    d = torch.linspace(-1, 1, rows, device="cuda")
    side = torch.cuda.Stream()

    def work(o):
        mp.mp_token_score(mp.logits(b.t), tt, o.struct)
        mp.mp_token_score_grad(mp.logits(b.t), tt, o.lse, o.entropy, d, d, mp.logits_grad(dx))

    outs, graphs = [Out(mp, rows, top, ws) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            work(o)
        graphs.append(g)
    for i in range(4):
        x, t = make_x(gen(15, i), rows, V, "bf16")
        b.t.copy_(torch.as_tensor(x))
        tt.copy_(torch.as_tensor(t))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in outs[i % 2].flat.items()}
        got_dx = dx.clone()
        o = Out(mp, rows, top, ws)
        work(o)
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], o.flat[n]), n
        assert torch.equal(got_dx, dx)


def test_on_another_stream_and_two_at_once(mp):
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = []
    for i, s in enumerate(streams):
        x, t = make_x(gen(16, i), 30, 60001, "fp16")
        data.append((x, t, Buf(30, 60001, "fp16", init=x), Out(mp, 30, 10, workspace(mp)), dev(t)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (x, t, b, o, tt) in zip(streams, data):
            mp.mp_token_score(mp.logits(b.t), tt, o.struct, stream=s)
    torch.cuda.synchronize()
    for x, t, b, o, tt in data:
        want = ref.score(x, t, 1.0, 10)
        assert np.array_equal(o.top_ids.cpu().numpy(), want["ids"])
        check("entropy", o.entropy, want["entropy"], want["tol_entropy"])


def test_places_are_checked(mp):
    import torch
    h = torch.zeros(4, 10).pin_memory()
    o = Out(mp, 4, 2)
    x = mp.Logits(h.data_ptr(), 4, 10, 10, mp.MP_FP32, 1.0, None)
    with pytest.raises(mp.MpError, match="device memory"):
        mp.mp_token_score(x, None, mp.Score(None, o.lse.data_ptr(), None, None, None, None, None, 0))
    g = torch.zeros(4, 10, device="cuda")
    with pytest.raises(ValueError, match="rows"):
        mp.mp_token_score(mp.logits(g), None, Out(mp, 3, 2).struct)


# --- together, as a training program uses them ------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_a_student_distilled_from_the_lists_of_a_score(mp, kind):
    """Teacher's logits -> lists -> distillation loss and gradient, against the definitions."""
    import torch
    import loss_reference
    rows, V, top, T = 9, 5000, 32, 2.0
    xt, _ = make_x(gen(17), rows, V, kind)
    xs, _ = make_x(gen(18), rows, V, kind)
    xt[2, 10:] = -np.inf                          # ten entries alone
    bt, bs, o = Buf(rows, V, kind, init=xt), Buf(rows, V, kind, init=xs), Out(mp, rows, top)
    mp.mp_token_score(mp.logits(bt.t, T), None, mp.score(lse=o.lse, top_ids=o.top_ids,
                                                        top_values=o.top_values))
    dx, loss = torch.empty_like(bs.t), torch.empty(rows, device="cuda")
    mp.mp_distill_loss(mp.logits(bs.t, T), mp.teacher(o.top_values, o.top_ids, o.lse), None, loss,
                       mp.logits_grad(dx))
    s = ref.score(xt, None, T, top)
    values = np.where(s["ids"] >= 0, s["values"], 0.0)
    want = loss_reference.distill(xs, values, s["ids"], f32(s["lse"]), T, None, kind=kind)
    # the teacher's lse is the library's own: off by tol_lse, and every share by that
    extra = s["tol_lse"] * 4
    check("loss", loss, want["loss"], want["tol_loss"] + extra * (np.abs(want["loss"]) + 1))
    check("dx", dx, want["dx"], want["tol_dx"] + extra[:, None] / T)


def test_an_entropy_bonus_through_autograd(mp):
    """A model's logits -> scores -> a loss of log-probabilities and entropies, its gradient by the
    library, against torch's own in binary64."""
    import torch
    torch.manual_seed(3)
    rows, dim, V = 40, 32, 1500
    h = torch.randn(rows, dim, device="cuda")
    w = (torch.randn(V, dim, device="cuda") * 0.3).requires_grad_()
    t = torch.randint(V, (rows,), device="cuda")
    t[::7] = -100
    a = torch.randn(rows, device="cuda")
    z = h @ w.t()
    o, dz = Out(mp, rows, 0), torch.empty(rows, V, device="cuda")
    x = mp.logits(z.detach())
    mp.mp_token_score(x, t, o.struct)
    mp.mp_token_score_grad(x, t, o.lse, o.entropy, -a, torch.full_like(a, -0.05), mp.logits_grad(dz))
    z.backward(dz)
    w64 = w.detach().double().requires_grad_()
    logq = torch.log_softmax(h.double() @ w64.t(), 1)
    live = t >= 0
    lp = logq.gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = (live * (-a * lp + 0.05 * (logq.exp() * logq).sum(1))).sum()
    want, = torch.autograd.grad(loss, w64)
    # fp32 products of 32 and 40 terms: a few 2^-24 of the sums of magnitudes, which are below 200
    assert float((w.grad.double() - want).abs().max()) < 200 * 40 * 2.0 ** -24
