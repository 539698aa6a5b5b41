"""The losses over vocabulary logits on the GPU against their definitions in binary64
(loss_reference.py, which also derives how far each result may be off)."""
import numpy as np
import pytest

import loss_reference as ref

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp16", "fp32"]
# one lane's head and tail alone, whole vectors, ragged ends, one wave's and one workgroup's worth
# and past them, the workloads' vocabularies, and rows longer than any on-chip share
SMALL_V = [1, 2, 7, 8, 9, 15, 63, 64, 65, 511, 513, 1000, 2049, 4097, 8192, 16385]
LARGE_V = [32001, 50304, 65537, 98311, 128256, 131075, 200003, 300007]


@pytest.fixture(scope="module")
def mp():
    import torch
    assert torch.cuda.is_available()
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


def ttype(kind):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[kind]


def gen(*key):
    return np.random.default_rng([20261206, *key])


class Buf:
    """A [rows, vocab] device tensor inside a larger one: rows `pad` elements apart and the first
    `shift` elements past a 256-byte boundary, with a pattern around that has to stay."""

    def __init__(self, rows, vocab, kind, pad=0, shift=0, init=None):
        import torch
        self.flat = torch.full((shift + rows * (vocab + pad) + 16,), -77.0, dtype=ttype(kind),
                               device="cuda")
        self.t = torch.as_strided(self.flat, (rows, vocab), (vocab + pad, 1), shift)
        if init is not None:
            self.t.copy_(torch.as_tensor(init))
        self.keep = torch.ones(self.flat.shape, dtype=torch.bool, device="cuda")
        torch.as_strided(self.keep, (rows, vocab), (vocab + pad, 1), shift).fill_(False)

    def untouched(self):
        return bool((self.flat[self.keep] == -77.0).all())


def host(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype=None):
    import torch
    a = np.asarray(a)
    if dtype is None and a.dtype == np.float64:
        a = a.astype(np.float32)
    return torch.as_tensor(a, device="cuda") if dtype is None else torch.as_tensor(
        a, dtype=dtype, device="cuda")


def check(name, got, want, tol):
    got = host(got) if not isinstance(got, np.ndarray) else got
    bad_got, bad_want = ~np.isfinite(got), ~np.isfinite(want)
    assert np.array_equal(bad_got, bad_want), (name, "non-finite where it should not be, or not")
    fine = ~bad_want
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), name
    off = np.abs(got[fine] - want[fine])
    over = off > tol[fine]
    assert not over.any(), (name, int(over.sum()), float((off / np.maximum(tol[fine], 1e-300)).max()),
                            got[fine][over][:4], want[fine][over][:4], tol[fine][over][:4])


def make_x(rng, rows, V, kind, spread=2.0):
    """Logits that the type holds exactly, and targets that stand out."""
    import torch
    x = rng.normal(0, spread, (rows, V))
    t = rng.integers(0, V, rows)
    x[np.arange(rows), t] += rng.normal(5, 2, rows)
    x = torch.as_tensor(x).to(ttype(kind)).double().numpy()
    return x, t


def f32(a):
    return np.asarray(a, np.float32).astype(np.float64)


def state_for(mp, x, kind, T=1.0, pad=0, shift=0, dpad=0, dshift=0, inplace=False, ws=None,
              scale=3.0, count=7, dev_scale=2.0):
    """Buffers, structs and the factor of a call."""
    import torch
    rows, V = x.shape
    bx = Buf(rows, V, kind, pad, shift, x)
    bd = bx if inplace else Buf(rows, V, kind, dpad, dshift)
    s = torch.full((1,), dev_scale, device="cuda")
    c = torch.full((1,), count, dtype=torch.int64, device="cuda")
    lx = mp.logits(bx.t, T, workspace=ws)
    lg = mp.logits_grad(bd.t, scale, dev_scale=s, dev_count=c)
    return bx, bd, lx, lg, scale * dev_scale / count, (s, c)


def empty(rows, fill=-55.0):
    import torch
    return torch.full((rows,), fill, device="cuda")


def workspace(mp):
    import torch
    return torch.full((mp.MP_LOSS_WORKSPACE_BYTES,), 0xA5, dtype=torch.uint8, device="cuda")


LAYOUTS = [dict(), dict(pad=3, shift=1, dpad=3, dshift=1), dict(pad=5, dpad=1, dshift=3),
           dict(inplace=True, pad=1, shift=1)]


def run_all(mp, kind, V, rows, T, layout, seed, with_ws):
    """Every fused call and the two-call form on one set of logits, against the reference."""
    import torch
    rng = gen(seed, V, rows)
    x, t = make_x(rng, rows, V, kind)
    t[rng.random(rows) < 0.25] = -100
    td = dev(t)
    ws = workspace(mp) if with_ws else None
    where = (kind, V, rows, T, layout, with_ws)

    # token log-probability, and its gradient for any dlogp
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws, **layout)
    d = f32(rng.normal(0, 1, rows))
    lp, lse = empty(rows), empty(rows)
    mp.mp_token_logprob(lx, td, lp, lse)
    mp.mp_token_logprob_grad(lx, td, lse, dev(d), lg)
    r = ref.logprob(x, t, T, d, factor, kind)
    for k, v in (("logp", lp), ("lse", lse), ("dx", bd.t)):
        check((where, "logprob", k), v, r[k], r["tol_" + k])
    assert bx.untouched() and bd.untouched(), where

    # cross-entropy, weighted
    w = f32(rng.uniform(0.5, 2, rows))
    w[rng.random(rows) < 0.2] = 0.0
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws, **layout)
    loss = empty(rows)
    mp.mp_cross_entropy(lx, td, dev(w), loss, lg)
    r = ref.cross_entropy(x, t, T, w, factor, kind)
    check((where, "xent", "loss"), loss, r["loss"], r["tol_loss"])
    check((where, "xent", "dx"), bd.t, r["dx"], r["tol_dx"])
    assert bx.untouched() and bd.untouched(), where

    # policy
    bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws, **layout)
    lpn = ref.logprob(x, t, T)["logp"]
    old, rf = f32(lpn + rng.normal(0, 0.2, rows)), f32(lpn + rng.normal(0, 0.5, rows))
    adv = f32(rng.normal(0, 1, rows))
    adv[rng.random(rows) < 0.1] = 0.0
    loss, lp, kl = empty(rows), empty(rows), empty(rows)
    r = ref.policy(x, t, old, rf, adv, T, w, (float(np.float32(0.2)), float(np.float32(0.28))),
                   float(np.float32(0.05)), factor, kind)
    assert not r["near_border"].any()
    mp.mp_policy_loss(lx, td, dev(old), dev(rf), dev(adv), dev(w), mp.policy_cfg(0.2, 0.28, 0.05),
                      loss, lp, kl, lg)
    for k, v in (("loss", loss), ("logp", lp), ("kl", kl), ("dx", bd.t)):
        check((where, "policy", k), v, r[k], r["tol_" + k])
    assert bx.untouched() and bd.untouched(), where

    # distillation: own normaliser and the teacher's, absent entries, an id twice
    for own_lse in (False, True):
        k = min(V, 5) if own_lse else min(3 * V, 37)
        ids = rng.integers(0, V, (rows, k))
        ids[rng.random((rows, k)) < 0.2] = -1
        if rows > 2:
            ids[1] = -1
        vals = torch.as_tensor(rng.normal(1, 2, (rows, k))).to(ttype(kind)).double().numpy()
        tl = f32(np.log(np.exp(vals / T).sum(1)) + 0.1) if own_lse else None
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws, **layout)
        tv, ti, tld = dev(vals, ttype(kind)), dev(ids), None if tl is None else dev(tl)
        loss = empty(rows)
        mp.mp_distill_loss(lx, mp.teacher(tv, ti, tld), dev(w), loss, lg)
        r = ref.distill(x, vals, ids, tl, T, w, factor, kind)
        check((where, "distill", k, "loss"), loss, r["loss"], r["tol_loss"])
        check((where, "distill", k, "dx"), bd.t, r["dx"], r["tol_dx"])
        assert bx.untouched() and bd.untouched(), where

    # preference over whatever sequences the rows make
    n = 1 + int(rng.integers(0, 3))
    cuts = np.sort(rng.integers(0, rows + 1, 2 * n + 1))
    pi = np.array([lpn[cuts[i]:cuts[i + 1]].sum() for i in range(2 * n)])
    rf = f32(pi + rng.normal(0, 3, 2 * n))
    for kind_of, mean in (("sigmoid", False), ("squared", True)):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, T, ws=ws, **layout)
        o = dict(loss=empty(n), seq_logp=empty(2 * n), logp=empty(rows), lse=empty(rows),
                 dlogp=empty(rows))
        cfg = mp.preference_cfg(dict(sigmoid=0, squared=1)[kind_of], 0.25, 0.125, 0.5, mean)
        mp.mp_preference_loss(lx, td, n, dev(cuts), dev(rf), cfg, o["loss"], o["seq_logp"], o["logp"],
                              o["lse"], o["dlogp"], lg)
        r = ref.preference(x, t, cuts, rf, T, kind_of, 0.25, 0.125, 0.5, mean, factor, kind)
        for k in o:
            check((where, "preference", kind_of, k), o[k], r[k], r["tol_" + k])
        check((where, "preference", kind_of, "dx"), bd.t, r["dx"], r["tol_dx"])
        assert bx.untouched() and bd.untouched(), where
    del keep


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", SMALL_V)
def test_small_vocabularies(mp, kind, V):
    for i, layout in enumerate(LAYOUTS):
        run_all(mp, kind, V, 1 + 4 * (i % 3), [1.0, 0.7, 2.0, 1.0][i], layout, i, i % 2 == 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", LARGE_V)
def test_large_vocabularies(mp, kind, V):
    i = LARGE_V.index(V) + KINDS.index(kind)
    run_all(mp, kind, V, 5, [1.0, 0.7][i % 2], LAYOUTS[i % 4], 100 + i, False)
    run_all(mp, kind, V, 2, 1.0, LAYOUTS[(i + 1) % 4], 200 + i, True)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("vecs", [128, 256, 512, 1024, 1536, 2048, 4096, 8192, 16384, 20480])
def test_rows_that_fill_their_vectors(mp, kind, vecs):
    """Exactly `vecs` 16-byte vectors, one more, and one more of which an odd start takes the first
    (so that as many as before are left): the last and the first row lengths of a shape."""
    per = 8 if kind == "bf16" else 4
    for V, shift in ((per * vecs, 0), (per * vecs, 1), (per * (vecs + 1), 0), (per * (vecs + 1), 1),
                     (per * (vecs + 1) + per - 1, per - 1)):
        rng = gen(20, V, shift)
        x, t = make_x(rng, 2, V, kind)
        t[0] = V - 1 if shift else 0
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, shift=shift, dshift=shift)
        loss = empty(2)
        mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
        r = ref.cross_entropy(x, t, 1.0, None, factor, kind)
        check((V, shift, "loss"), loss, r["loss"], r["tol_loss"])
        check((V, shift, "dx"), bd.t, r["dx"], r["tol_dx"])
        ids, vals = rng.integers(0, V, (2, 9)), f32(rng.normal(0, 1, (2, 9)))
        ids[:, 0] = V - 1
        mp.mp_distill_loss(lx, mp.teacher(dev(vals), dev(ids)), None, loss, lg)
        r = ref.distill(x, vals, ids, None, 1.0, None, factor, kind)
        check((V, shift, "distill loss"), loss, r["loss"], r["tol_loss"])
        check((V, shift, "distill dx"), bd.t, r["dx"], r["tol_dx"])
        assert bx.untouched() and bd.untouched()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [33, 257, 1031])
def test_many_rows(mp, kind, rows):
    """More rows than compute units, and row counts on both sides of any split."""
    run_all(mp, kind, 1003, rows, 1.0, LAYOUTS[rows % 4], rows, True)
    run_all(mp, kind, 4200, min(rows, 300), 0.7, LAYOUTS[0], rows, False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [49151, 49152, 50305, 66001, 131079, 1050003])
def test_few_long_rows_split_over_workgroups(mp, kind, V):
    """Rows cut into parts in the workspace: every layout; parts that end inside the row's last
    vectors; more vectors than the parts hold at once (past 2^20 logits)."""
    i = KINDS.index(kind)
    for layout in LAYOUTS if V < 1000000 else LAYOUTS[2:]:
        run_all(mp, kind, V, 1 + i, [1.0, 0.7, 2.0][i], layout, 300 + i, True)


@pytest.mark.parametrize("with_ws", [False, True])
def test_a_row_of_16_million_logits(mp, with_ws):
    rng = gen(18)
    x, t = make_x(rng, 1, (1 << 24) + 5, "bf16")
    ws = workspace(mp) if with_ws else None
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16", pad=1, shift=1, dpad=1, dshift=1, ws=ws)
    loss = empty(1)
    mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
    r = ref.cross_entropy(x, t, 1.0, None, factor, "bf16")
    check("loss", loss, r["loss"], r["tol_loss"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    assert bx.untouched() and bd.untouched()
    lp, lse = empty(1), empty(1)
    mp.mp_token_logprob(lx, dev(t), lp, lse)
    r = ref.logprob(x, t, 1.0, np.array([-0.5]), factor, "bf16")
    mp.mp_token_logprob_grad(lx, dev(t), lse, dev([-0.5]), lg)
    for k, v in (("logp", lp), ("lse", lse), ("dx", bd.t)):
        check(k, v, r[k], r["tol_" + k])


@pytest.mark.parametrize("kind", KINDS)
def test_both_sides_of_the_split(mp, kind):
    rows = 101 if kind != "fp32" else 41
    for n in (rows - 1, rows):
        x, t = make_x(gen(16, n), n, 49300, kind)
        t[::5] = -1
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=workspace(mp))
        loss = empty(n)
        mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
        r = ref.cross_entropy(x, t, 1.0, None, factor, kind)
        check((n, "loss"), loss, r["loss"], r["tol_loss"])
        check((n, "dx"), bd.t, r["dx"], r["tol_dx"])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,k", [(40, 7), (9000, 300), (60000, 70)])
def test_student_masked_where_the_teacher_is_not(mp, kind, V, k):
    """An id with a share but a student's logit of -inf: an infinite loss (whatever the order the
    entries are joined in), a finite gradient; with a share of 0 there, a finite loss."""
    import torch
    rng = gen(17, V)
    x, t = make_x(rng, 4, V, kind)
    ids = np.stack([rng.choice(V, min(k, V), replace=False) for _ in range(4)])
    vals = f32(rng.normal(0, 1, ids.shape))
    x[0, ids[0, 0]] = -np.inf
    x[1, ids[1, -1]] = -np.inf
    x[2, ids[2, 1]] = -np.inf
    vals[0, 0], vals[1, -1] = 1.0, -60.0
    vals[2, 1] = -np.inf
    for ws in (None, workspace(mp)):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        loss = empty(4)
        mp.mp_distill_loss(lx, mp.teacher(dev(vals), dev(ids)), None, loss, lg)
        r = ref.distill(x, vals, ids, None, 1.0, None, factor, kind)
        check((kind, V, "loss"), loss, r["loss"], r["tol_loss"])
        check((kind, V, "dx"), bd.t, r["dx"], r["tol_dx"])
        assert bool(torch.isinf(loss[:2]).all()) and bool(torch.isfinite(loss[2:]).all())


def test_more_rows_than_a_16_bit_grid(mp):
    """70001 rows of 24 logits; every tenth switched off."""
    import torch
    rng = gen(9)
    rows, V = 70001, 24
    x, t = make_x(rng, rows, V, "bf16")
    t[::10] = -1
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16")
    loss, n = empty(rows), torch.zeros(1, dtype=torch.int64, device="cuda")
    mp.mp_target_count(dev(t), n)
    assert int(n) == int((t >= 0).sum())
    mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
    r = ref.cross_entropy(x, t, 1.0, None, factor, "bf16")
    check("loss", loss, r["loss"], r["tol_loss"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    lp, lse = empty(rows), empty(rows)
    mp.mp_token_logprob(lx, dev(t), lp, lse)
    mp.mp_token_logprob_grad(lx, dev(t), lse, empty(rows, -1.0), lg)
    r = ref.logprob(x, t, 1.0, -np.ones(rows), factor, "bf16")
    check("dx", bd.t, r["dx"], r["tol_dx"])


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 1023, 1024, 1025, 8191, 100003])
def test_target_count(mp, n):
    import torch
    rng = gen(3, n)
    t = rng.integers(-3, 4, n)
    c = torch.full((2,), -9, dtype=torch.int64, device="cuda")
    mp.mp_target_count(dev(t) if n else torch.zeros(0, dtype=torch.int64, device="cuda"), c)
    assert c.tolist() == [int((t >= 0).sum()), -9]


def test_offsets_beyond_32_bits(mp):
    """Rows 2^31 + 8 elements apart (the third starts past 2^32 elements, 8 GiB)."""
    import torch
    V, stride = 1000, (1 << 31) + 8
    rng = gen(4)
    x, t = make_x(rng, 3, V, "bf16")
    flat = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(flat, (3, V), (stride, 1))
    view.copy_(torch.as_tensor(x))
    out = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    dx = torch.as_strided(out, (3, V), (stride, 1))
    for inplace in (False, True):
        g = view if inplace else dx
        loss = empty(3)
        mp.mp_cross_entropy(mp.logits(view), dev(t), None, loss, mp.logits_grad(g))
        r = ref.cross_entropy(x, t, kind="bf16")
        check("loss", loss, r["loss"], r["tol_loss"])
        check("dx", g, r["dx"], r["tol_dx"])
    del flat, out, view, dx, g
    torch.cuda.empty_cache()


# --- rows that are off, masks and non-finite values ----------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [5, 130, 3001, 40001])
@pytest.mark.parametrize("with_ws", [False, True])
def test_switched_off_rows_hide_what_they_hold(mp, kind, V, with_ws):
    """NaN and inf in rows without a target (weight, entry) change nothing: zeros come out."""
    import torch
    rng = gen(6, V)
    x, t = make_x(rng, 4, V, kind)
    t[0] = t[2] = -100
    x[0], x[2, ::2], x[2, 1::2] = np.nan, np.inf, -np.inf
    ws = workspace(mp) if with_ws else None
    nan = torch.full((4,), float("nan"), device="cuda")
    other = dev(np.where(t < 0, np.nan, -2.0))
    for inplace in (False, True):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, inplace=inplace, ws=ws)
        loss, lp, kl = empty(4), empty(4), empty(4)
        mp.mp_policy_loss(lx, dev(t), other, other, other, None, mp.policy_cfg(0.2, 0.2, 0.1), loss,
                          lp, kl, lg)
        for v in (loss, lp, kl):
            assert v[0] == 0 and v[2] == 0 and bool(torch.isfinite(v).all())
        assert not bd.t[0].any() and not bd.t[2].any() and bool(torch.isfinite(bd.t).all())
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, inplace=inplace, ws=ws)
        w = dev([0.0, 1.0, 0.0, 1.0], torch.float32)
        ids = dev(rng.integers(0, V, (4, 3)))
        mp.mp_distill_loss(lx, mp.teacher(dev(rng.normal(0, 1, (4, 3)), torch.float32), ids), w, loss,
                           lg)
        assert loss[0] == 0 and loss[2] == 0 and bool(torch.isfinite(loss).all())
        assert not bd.t[0].any() and not bd.t[2].any() and bool(torch.isfinite(bd.t).all())
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, inplace=inplace, ws=ws)
        ids[0] = ids[2] = -1
        mp.mp_distill_loss(lx, mp.teacher(dev(rng.normal(0, 1, (4, 3)), torch.float32), ids), None,
                           loss, lg)
        assert loss[0] == 0 and loss[2] == 0 and not bd.t[0].any() and not bd.t[2].any()
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, inplace=inplace, ws=ws)
        d = dev([np.nan, 1.0, 0.0, -1.0], torch.float32)
        lse = empty(4)
        mp.mp_token_logprob(lx, dev(t), lp, lse)
        mp.mp_token_logprob_grad(lx, dev(t), lse, d, lg)
        assert lse[0] == 0 and lp[2] == 0 and bool(torch.isfinite(bd.t).all())
        assert not bd.t[0].any() and not bd.t[2].any()
    del nan


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [9, 1000, 9001, 70001])
def test_vocabulary_masks(mp, kind, V):
    """-inf and the type's lowest value at masked ids; one id left; the target masked."""
    import torch
    rng = gen(7, V)
    x, t = make_x(rng, 6, V, kind)
    low = float(torch.finfo(ttype(kind)).min)
    mask = rng.random((6, V)) < 0.5
    mask[np.arange(6), t] = False
    x[0][mask[0]] = -np.inf
    x[1][mask[1]] = low
    x[2] = -np.inf                     # one id left
    x[2, t[2]] = 3.0
    x[3, : V // 2] = -np.inf           # the row's first half gone
    t[3] = V - 1
    x[4, t[4]] = -np.inf               # the target itself is masked: infinite loss, finite gradient
    x[5] = low                         # every logit the lowest: the uniform distribution
    for ws in (None, workspace(mp)):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        loss = empty(6)
        mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
        r = ref.cross_entropy(x, t, 1.0, None, factor, kind)
        check((kind, V, "loss"), loss, r["loss"], r["tol_loss"])
        check((kind, V, "dx"), bd.t, r["dx"], r["tol_dx"])
        k = 4
        ids = np.stack([rng.choice(np.flatnonzero(np.isfinite(x[i])), k) for i in range(6)])
        vals = f32(rng.normal(0, 1, (6, k)))
        vals[:, 1] = -np.inf           # an entry that the teacher masks
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        mp.mp_distill_loss(lx, mp.teacher(dev(vals), dev(ids)), None, loss, lg)
        r = ref.distill(x, vals, ids, None, 1.0, None, factor, kind)
        check((kind, V, "distill loss"), loss, r["loss"], r["tol_loss"])
        check((kind, V, "distill dx"), bd.t, r["dx"], r["tol_dx"])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [40, 5001, 60001])
def test_rows_without_a_distribution_and_bad_ids_give_nan(mp, kind, V):
    """All -inf, +inf, NaN, a target or a teacher's id past the vocabulary: NaN in that row, the
    other rows as ever (what the step's overflow check is there for)."""
    import torch
    rng = gen(8, V)
    x, t = make_x(rng, 6, V, kind)
    x[0], x[1, V // 2], x[2, V - 1] = -np.inf, np.inf, np.nan
    t[3] = V
    t[4] = 1 << 40
    bad = [0, 1, 2, 3, 4]
    for ws in (None, workspace(mp)):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        loss = empty(6)
        mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
        r = ref.cross_entropy(x[5:], t[5:], 1.0, None, factor, kind)
        check("loss", loss[5:], r["loss"], r["tol_loss"])
        check("dx", bd.t[5:], r["dx"], r["tol_dx"])
        assert bool(torch.isnan(loss[bad]).all()), loss
        assert bool(torch.isnan(bd.t[bad].float()).any(1).all())
        assert bool(torch.isnan(bd.t[3:5].float()).all())
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        lp, lse = empty(6), empty(6)
        mp.mp_token_logprob(lx, dev(t), lp, lse)
        assert bool(torch.isnan(lp[bad]).all()) and bool(torch.isfinite(lp[5]))
        mp.mp_token_logprob_grad(lx, dev(t), lse, empty(6, 1.0), lg)
        assert bool(torch.isnan(bd.t[bad].float()).any(1).all())
        assert bool(torch.isfinite(bd.t[5]).all())
        bx, bd, lx, lg, factor, keep = state_for(mp, x, kind, ws=ws)
        ids = rng.integers(0, V, (6, 3))
        ids[3, 1], ids[4, 2] = V, 1 << 40
        mp.mp_distill_loss(lx, mp.teacher(dev(rng.normal(0, 1, (6, 3)), torch.float32), dev(ids)),
                           None, loss, lg)
        assert bool(torch.isnan(loss[bad]).all()) and bool(torch.isfinite(loss[5]))
        assert bool(torch.isnan(bd.t[bad].float()).any(1).all())
        assert bool(torch.isfinite(bd.t[5]).all())


def test_confident_rows_keep_their_digits(mp):
    """lp near 0 (probabilities 1 - 1e-4 .. 1 - 1e-30): the loss and the target's gradient are
    small numbers with relative, not absolute, precision."""
    V = 1000
    x = np.full((6, V), -3.0)
    t = np.arange(6) * 11
    x[np.arange(6), t] = [13.0, 20.0, 30.0, 40.0, 60.0, 75.0]
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "fp32")
    loss = empty(6)
    mp.mp_cross_entropy(lx, dev(t), None, loss, lg)
    r = ref.cross_entropy(x, t, 1.0, None, factor, "fp32")
    check("loss", loss, r["loss"], r["tol_loss"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    # the sum of the others is 999 e^-t < 1: formed apart from the target's 1, it would keep its
    # digits down to 2^-24 of 1, so the first two rows' losses hold to 4 digits
    got = host(loss)
    assert abs(got[0] / r["loss"][0] - 1) < 1e-3


def test_policy_rows_at_extremes(mp):
    """A far-off old policy, A = 0 with an overflowing ratio, weights of both signs."""
    import torch
    rng = gen(12)
    x, t = make_x(rng, 6, 300, "fp32")
    lp = ref.logprob(x, t)["logp"]
    old = f32(lp + np.array([0.0, 30.0, -30.0, -900.0, 900.0, -30.0]))
    adv = f32([1.0, -1.0, 2.0, 0.0, 3.0, -1e-9])
    w = f32([1.0, -2.0, 0.5, 1.0, 1.0, 1.0])
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "fp32")
    loss, l2 = empty(6), empty(6)
    mp.mp_policy_loss(lx, dev(t), dev(old), None, dev(adv), dev(w), mp.policy_cfg(0.25, 0.5), loss, l2,
                      None, lg)
    r = ref.policy(x, t, old, None, adv, 1.0, w, (0.25, 0.5), 0.0, factor, "fp32")
    check("loss", loss, r["loss"], r["tol_loss"])
    check("dx", bd.t, r["dx"], r["tol_dx"])
    assert loss[3] == 0 and not torch.isnan(bd.t).any()


def test_policy_target_that_is_masked(mp):
    """A target's logit of -inf: lp = -inf, an infinite loss where there is a KL term (a finite one
    where there is none: rho = 0), the other rows as ever."""
    import torch
    rng = gen(19)
    x, t = make_x(rng, 4, 700, "bf16")
    lp = ref.logprob(x, t)["logp"]
    old, rf, adv = f32(lp), f32(lp + 0.1), f32([1.0, -1.0, 2.0, 1.0])
    x[0, t[0]] = x[1, t[1]] = -np.inf
    for kl_coef in (0.25, 0.0):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16")
        loss, l2, kl = empty(4), empty(4), empty(4)
        mp.mp_policy_loss(lx, dev(t), dev(old), dev(rf), dev(adv), None,
                          mp.policy_cfg(0.25, 0.5, kl_coef), loss, l2, kl, lg)
        assert bool(torch.isneginf(l2[:2]).all()) and bool(torch.isposinf(kl[:2]).all())
        r = ref.policy(x[2:], t[2:], old[2:], rf[2:], adv[2:], 1.0, None, (0.25, 0.5), kl_coef, factor,
                       "bf16")
        check("loss", loss[2:], r["loss"], r["tol_loss"])
        check("dx", bd.t[2:], r["dx"], r["tol_dx"])
        if kl_coef:
            assert bool(torch.isposinf(loss[:2]).all())
            assert not bool(torch.isfinite(bd.t[:2].float()).all(1).any())
        else:
            assert loss[0] == 0.0 and loss[1] == 0.75 and not bd.t[:2].any()


def test_preference_sequences_at_extremes(mp):
    """Empty sequences, sequences without a target, rows before, between and behind, starts out of
    range and decreasing (taken as the nearest, never followed)."""
    rng = gen(13)
    x, t = make_x(rng, 40, 500, "bf16")
    t[10:14] = -100
    rf = f32(rng.normal(0, 3, 6))
    for start in ([3, 3, 10, 14, 14, 30, 37], [0, 0, 0, 0, 0, 0, 0], [40] * 7,
                  [0, 40, 40, 40, 40, 40, 40]):
        start = np.array(start)
        for mean in (False, True):
            bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16")
            o = dict(loss=empty(3), seq_logp=empty(6), logp=empty(40), lse=empty(40), dlogp=empty(40))
            mp.mp_preference_loss(lx, dev(t), 3, dev(start), dev(rf), mp.preference_cfg(length_mean=mean),
                                  *o.values(), lg)
            r = ref.preference(x, t, start, rf, mean=mean, beta=float(np.float32(0.1)), factor=factor,
                               kind="bf16")
            for k in o:
                check((start, mean, k), o[k], r[k], r["tol_" + k])
            check((start, mean, "dx"), bd.t, r["dx"], r["tol_dx"])
    import torch
    for start in ([-5, 3, 10, 14, 20, 30, 99], [30, 20, 10, 35, 1 << 62, -(1 << 62), 4]):
        bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16")
        o = dict(loss=empty(3), seq_logp=empty(6), logp=empty(40), lse=empty(40),
                 dlogp=torch.zeros(40, device="cuda"))
        mp.mp_preference_loss(lx, dev(t), 3, dev(np.array(start)), None, mp.preference_cfg(),
                              *o.values(), lg)
        assert bool(torch.isfinite(bd.t).all()) and bd.untouched()


def test_distill_counts(mp):
    """k = 1 and k = the limit (more entries than ids, so most ids come several times)."""
    rng = gen(14)
    for V, k in ((50, mp.MP_DISTILL_MAX_K), (33000, mp.MP_DISTILL_MAX_K), (33000, 1), (700, 257)):
        x, t = make_x(rng, 3, V, "fp16")
        ids = rng.integers(-1, V, (3, k))
        ids[:, 0] = 5
        vals = f32(rng.normal(0, 1, (3, k)))
        bx, bd, lx, lg, factor, keep = state_for(mp, x, "fp16")
        loss = empty(3)
        mp.mp_distill_loss(lx, mp.teacher(dev(vals), dev(ids)), None, loss, lg)
        r = ref.distill(x, vals, ids, None, 1.0, None, factor, "fp16")
        check((V, k, "loss"), loss, r["loss"], r["tol_loss"])
        check((V, k, "dx"), bd.t, r["dx"], r["tol_dx"])


# --- forward only, streams, graphs, repeatability ------------------------------------------


@pytest.mark.parametrize("V", [100, 8192, 128256])
def test_losses_without_a_gradient_are_the_same(mp, V):
    """The same bits with and without a gradient, apart from what another order of a row's sum
    changes: within the tolerance of each."""
    rng = gen(15, V)
    x, t = make_x(rng, 4, V, "bf16")
    bx, bd, lx, lg, factor, keep = state_for(mp, x, "bf16")
    r = ref.cross_entropy(x, t, 1.0, None, factor, "bf16")
    for g in (lg, None):
        loss = empty(4)
        mp.mp_cross_entropy(lx, dev(t), None, loss, g)
        check("loss", loss, r["loss"], r["tol_loss"])
    ids, vals = rng.integers(0, V, (4, 9)), f32(rng.normal(0, 1, (4, 9)))
    r = ref.distill(x, vals, ids)
    loss = empty(4)
    mp.mp_distill_loss(lx, mp.teacher(dev(vals), dev(ids)), None, loss)
    check("distill", loss, r["loss"], r["tol_loss"])
    assert bx.untouched()


def everything(mp, st):
    """One pass of every call over preallocated buffers."""
    mp.mp_target_count(st["t"], st["count"])
    lx = mp.logits(st["x"], 1.0, workspace=st["ws"])
    lg = [mp.logits_grad(d, 1.0, dev_scale=st["scale"], dev_count=st["count"]) for d in st["dx"]]
    mp.mp_cross_entropy(lx, st["t"], None, st["loss"][0], lg[0])
    mp.mp_policy_loss(lx, st["t"], st["old"], st["ref"], st["adv"], None, mp.policy_cfg(0.2, 0.2, 0.1),
                      st["loss"][1], st["lp"], st["kl"], lg[1])
    mp.mp_distill_loss(lx, mp.teacher(st["vals"], st["ids"]), None, st["loss"][2], lg[2])
    mp.mp_preference_loss(lx, st["t"], 2, st["start"], None, mp.preference_cfg(), st["ploss"],
                          st["seq"], st["lp2"], st["lse"], st["dlogp"], lg[3])


OUTPUTS = ("count", "lp", "kl", "ploss", "seq", "lp2", "lse", "dlogp")


def fresh(mp, rows, V, kind, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(x=torch.empty(rows, V, dtype=ttype(kind), device="cuda"),
              t=torch.empty(rows, dtype=torch.int64, device="cuda"), ws=workspace(mp),
              scale=torch.empty(1, device="cuda"), vals=torch.empty(rows, 6, device="cuda"),
              ids=torch.empty(rows, 6, dtype=torch.int64, device="cuda"),
              old=empty(rows), ref=empty(rows), adv=empty(rows), lp=empty(rows), kl=empty(rows),
              lp2=empty(rows), lse=empty(rows), dlogp=empty(rows), ploss=empty(2), seq=empty(4),
              count=torch.zeros(1, dtype=torch.int64, device="cuda"),
              start=torch.tensor([0, rows // 4, rows // 2, rows // 2, rows - 1], device="cuda"),
              loss=[empty(rows) for _ in range(3)],
              dx=[torch.empty(rows, V, dtype=ttype(kind), device="cuda") for _ in range(4)])
    refill(st, g)
    return st


def refill(st, g):
    """New inputs in the same buffers (what a training loop does between replays)."""
    import torch
    rows, V = st["x"].shape
    st["x"].copy_(torch.randn(rows, V, generator=g, device="cuda") * 2)
    st["t"].copy_(torch.randint(-V // 4, V, (rows,), generator=g, device="cuda").clamp(min=-1))
    st["ids"].copy_(torch.randint(-2, V, (rows, 6), generator=g, device="cuda"))
    st["vals"].copy_(torch.randn(rows, 6, generator=g, device="cuda"))
    for k in ("old", "ref", "adv"):
        st[k].copy_(torch.randn(rows, generator=g, device="cuda") - (8 if k != "adv" else 0))
    st["scale"].copy_(torch.rand(1, generator=g, device="cuda") * 100)


def results(st):
    return [st[k].clone() for k in OUTPUTS] + [v.clone() for v in st["loss"] + st["dx"]]


def same_bits(a, b):
    import torch
    for i, (x, y) in enumerate(zip(a, b)):
        v = {2: torch.int16, 4: torch.int32, 8: torch.int64}[x.element_size()]
        assert torch.equal(x.view(v), y.view(v)), i


SHAPES = [(3, 40000), (70, 9001), (300, 1111), (600, 50304)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_same_bits_every_time(mp, rows, V, kind):
    import torch
    st = fresh(mp, rows, V, kind, 3)
    everything(mp, st)
    first = results(st)
    for _ in range(3):
        st["ws"].fill_(0x3C)
        for d in st["dx"]:
            d.fill_(1.0)
        everything(mp, st)
        torch.cuda.synchronize()
        same_bits(results(st), first)


@pytest.mark.parametrize("rows,V", SHAPES)
def test_captured_and_replayed(mp, rows, V):
    """One captured pass of every call, replayed on new inputs with eager work between: each
    replay's bits are the eager call's on the same inputs."""
    import torch
    st = fresh(mp, rows, V, "bf16", 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        everything(mp, st)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything(mp, st)
    g = torch.Generator(device="cuda").manual_seed(77)
    for _ in range(4):
        refill(st, g)
        everything(mp, st)
        want = results(st)
        torch.cuda.synchronize()
        for d in st["dx"] + st["loss"]:
            d.fill_(-3.0)
        st["count"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        same_bits(results(st), want)


def test_two_graphs_that_share_a_workspace(mp):
    """Two captured passes over different buffers and one workspace, replayed in turn on a stream."""
    import torch
    sts = [fresh(mp, 9, 60001, "bf16", 23), fresh(mp, 40, 131072, "fp16", 24)]
    sts[1]["ws"] = sts[0]["ws"]
    graphs = []
    for st in sts:
        everything(mp, st)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            everything(mp, st)
    g = torch.Generator(device="cuda").manual_seed(78)
    for _ in range(3):
        want = []
        for st in sts:
            refill(st, g)
            everything(mp, st)
            want.append(results(st))
            for d in st["dx"] + st["loss"]:
                d.fill_(-3.0)
        sts[0]["ws"].fill_(0x77)
        for i in (0, 1, 0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for st, w in zip(sts, want):
            same_bits(results(st), w)


def test_two_streams_at_once(mp):
    """Two sets of buffers, each with a workspace of its own, on two streams: the results of
    one after the other."""
    import torch
    sts = [fresh(mp, 12, 128256, "bf16", 21), fresh(mp, 45, 50304, "bf16", 22)]
    want = []
    for st in sts:
        everything(mp, st)
        want.append(results(st))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sts]
    for _ in range(5):
        for st, s in zip(sts, streams):
            with torch.cuda.stream(s):
                everything(mp, st)
        torch.cuda.synchronize()
        for st, w in zip(sts, want):
            same_bits(results(st), w)


def test_logits_that_are_not_device_memory_are_refused(mp):
    import torch
    x = torch.zeros(4, 10, dtype=torch.bfloat16)
    t, loss = dev(np.zeros(4, np.int64)), empty(4)
    for pinned in (False, True):
        y = x.pin_memory() if pinned else x
        lx = mp.Logits(y.data_ptr(), 4, 10, 10, mp.MP_BF16, 1.0, None)
        with pytest.raises(mp.MpError) as e:
            mp.mp_cross_entropy(lx, t, None, loss)
        assert e.value.status == mp.MP_ERR_INVALID
        lp = empty(4)
        with pytest.raises(mp.MpError):
            mp.mp_preference_loss(lx, t, 1, t, None, mp.preference_cfg(), loss, loss, lp, lp, lp)
        n = torch.zeros(1, dtype=torch.int64, pin_memory=pinned)
        with pytest.raises(mp.MpError):
            mp.mp_target_count(t, n.data_ptr())
        assert int(n) == 0
    torch.cuda.synchronize()
    assert bool((loss == -55.0).all())


def test_binding_refuses_what_does_not_fit(mp):
    import torch
    x = torch.zeros(4, 10, dtype=torch.bfloat16, device="cuda")
    lx = mp.logits(x)
    t, loss = dev(np.zeros(4, np.int64)), empty(4)
    with pytest.raises(ValueError, match="adjacent"):
        mp.logits(x.t())
    with pytest.raises(TypeError):
        mp.mp_cross_entropy(lx, t, None, loss, mp.logits_grad(x.float()))
    with pytest.raises(ValueError, match="shape"):
        mp.mp_cross_entropy(lx, t, None, loss, mp.logits_grad(x[:, :9]))
    with pytest.raises(TypeError):
        mp.logits(x, workspace=torch.zeros(1 << 16, device="cuda"))
    with pytest.raises(ValueError):
        mp.logits(x, workspace=torch.zeros(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mp.mp_distill_loss(lx, mp.teacher(torch.zeros(3, 2, device="cuda"),
                                          torch.zeros(3, 2, dtype=torch.int64, device="cuda")), None,
                           loss)
    with pytest.raises(mp.MpError):
        mp.logits(x, 0.0) and mp.mp_cross_entropy(mp.logits(x, 0.0), t, None, loss)


# --- together, as a training step uses them -------------------------------------------------


@pytest.mark.parametrize("fmt", ["bf16", "fp16"])
def test_a_step_from_logits_to_weights(mp, fmt):
    """Two micro-batches of a small model trained by each loss in turn: counts on the device, the
    loss scaled by the state's own S, the logits' gradient handed to autograd, token weights from
    the same counts inside the first accumulation, the update.  Every step's parameter gradients
    are those of the reference's logits gradient, and the update the oracle's on the same bits."""
    import torch
    import oracle
    import types
    from harness import compare_state
    torch.manual_seed(3)
    kind = fmt
    t16 = ttype(kind)
    V, width = 331, 64
    net = torch.nn.Sequential(torch.nn.Linear(32, width), torch.nn.Tanh(),
                              torch.nn.Linear(width, V, bias=False)).to("cuda", t16)
    params = list(net.parameters())
    master = [p.detach().float().contiguous() for p in params]
    m, v, acc = ([torch.zeros_like(x) for x in master] for _ in range(3))
    dt = mp.MP_BF16 if fmt == "bf16" else mp.MP_FP16
    plan = mp.mp_plan_create([p.numel() for p in params], dt, acc, master, m, v, params)
    scaler = (dict(init_scale=1.0, enabled=False) if fmt == "bf16" else
              dict(init_scale=2.0 ** 10, growth=2.0, backoff=0.5, interval=2, enabled=True))
    state = mp.mp_state_create(mp.scaler_cfg(**scaler))
    hpd = dict(lr=5e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    hp = mp.adamw_hparams(**hpd)
    bits = lambda p: p.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16).ravel().copy()  # noqa: E731
    odt = oracle.BF16 if fmt == "bf16" else oracle.FP16
    orc = oracle.OracleStep(odt, [x.cpu().numpy().ravel().copy() for x in master],
                            [bits(p) for p in params], scaler=oracle.make_scaler(**scaler),
                            with_acc=True)
    scale_ptr = mp.mp_state_scale_ptr(state)
    counts = torch.zeros(2, dtype=torch.int64, device="cuda")
    weights = torch.zeros(2, device="cuda")
    sets = None
    rng = gen(30)
    try:
        for step, name in enumerate(["xent", "policy", "distill", "preference", "xent"], start=1):
            S = mp.read_stats(state)["scale"]
            grads, recorded = [], []
            for i, rows in enumerate((24, 41)):
                for p in params:
                    p.grad = None
                inp = torch.as_tensor(rng.normal(0, 1, (rows, 32)), device="cuda").to(t16)
                z = net(inp)
                x = host(z)
                t = rng.integers(0, V, rows)
                t[: rows // 4] = -100
                td = dev(t)
                if name == "distill":
                    td = torch.zeros(rows, dtype=torch.int64, device="cuda")
                mp.mp_target_count(td, counts[i:i + 1])
                n = int((t >= 0).sum()) if name != "distill" else rows
                dx = torch.empty_like(z)
                lx = mp.logits(z.detach())
                g = mp.logits_grad(dx, 1.0, dev_scale=scale_ptr, dev_count=counts[i:i + 1])
                loss, factor = empty(rows), S / n
                if name == "xent":
                    mp.mp_cross_entropy(lx, td, None, loss, g)
                    r = ref.cross_entropy(x, t, 1.0, None, factor, kind)
                elif name == "policy":
                    lp, lse = empty(rows), empty(rows)
                    mp.mp_token_logprob(lx, td, lp, lse)            # the sampling policy's own
                    old = f32(host(lp) + rng.normal(0, 0.2, rows))
                    adv = f32(rng.normal(0, 1, rows))
                    mp.mp_policy_loss(lx, td, dev(old), lp, dev(adv), None, mp.policy_cfg(0.2, 0.2, 0.25),
                                      loss, None, None, g)
                    c = float(np.float32(0.2))
                    r = ref.policy(x, t, old, host(lp), adv, 1.0, None, (c, c), 0.25, factor, kind)
                    assert not r["near_border"].any()
                elif name == "distill":
                    tl = torch.as_tensor(rng.normal(0, 2, (rows, V)), device="cuda")
                    top = tl.topk(16, 1)
                    vals = top.values.float().contiguous()
                    mp.mp_distill_loss(lx, mp.teacher(vals, top.indices.contiguous()), None, loss, g)
                    r = ref.distill(x, host(vals), top.indices.cpu().numpy(), None, 1.0, None, factor,
                                    kind)
                else:
                    start = np.array([0, rows // 2, rows])
                    o = [empty(1), empty(2), empty(rows), empty(rows), empty(rows)]
                    mp.mp_preference_loss(lx, td, 1, dev(start), None, mp.preference_cfg(), *o, g)
                    r = ref.preference(x, t, start, None, beta=float(np.float32(0.1)), factor=factor,
                                       kind=kind)
                    loss = o[0]
                check((step, name, "loss"), loss, r["loss"], r["tol_loss"])
                check((step, name, "dx"), dx, r["dx"], r["tol_dx"])
                z.backward(dx)
                grads.append([p.grad for p in params])
                recorded.append([bits(p) for p in grads[-1]])
            if sets is None:
                sets = [mp.mp_gradset_create(plan, gr) for gr in grads]
            else:
                for s, gr in zip(sets, grads):
                    mp.mp_gradset_update(s, gr)
            mp.mp_accumulate_first_counts(plan, sets[:1], 2, counts, weights)
            mp.mp_update_step_group(plan, state, sets[1:], weights[1:], 0, 1.0, hp)
            torch.cuda.synchronize()
            ow = oracle.token_weights(counts.cpu().numpy())
            prev, prev_m = [a.copy() for a in orc.masters], [a.copy() for a in orc.m]
            orc.accumulate(recorded[0], ow[0], True)
            orc.unscale_check_norm(recorded[1], ow[1], False, 1.0)
            orc.adamw_step(recorded[1], ow[1], False, **hpd)
            orc.scaler_update()
            stats = mp.read_stats(state)
            assert stats["found_inf"] == int(orc.found_inf) == 0 and stats["step"] == step
            same = np.float32(stats["grad_norm"]) == np.float32(orc.norm)
            for k in range(len(params)):
                got = {"master": master[k].cpu().numpy().ravel(), "m": m[k].cpu().numpy().ravel(),
                       "v": v[k].cpu().numpy().ravel(), "w16": bits(params[k])}
                want = {"master": orc.masters[k], "m": orc.m[k], "v": orc.v[k], "w16": orc.w16[k]}
                compare_state(got, want, prev[k], prev_m[k], types.SimpleNamespace(hp=hpd), same, odt,
                              " (step %d, tensor %d)" % (step, k))
    finally:
        for s in sets or ():
            mp.mp_gradset_destroy(s)
        mp.mp_state_destroy(state)
        mp.mp_plan_destroy(plan)


def test_a_bad_target_skips_the_step(mp):
    """An id past the vocabulary makes the gradient NaN, and the update it feeds is skipped."""
    import torch
    x = torch.randn(4, 50, device="cuda", dtype=torch.bfloat16)
    t = torch.tensor([1, 50, 3, -1], device="cuda")
    dx = torch.empty_like(x)
    loss = empty(4)
    mp.mp_cross_entropy(mp.logits(x), t, None, loss, mp.logits_grad(dx))
    model = mp.ModelState([200], mp.MP_BF16)
    model.master[0].fill_(1.0)
    gs = model.gradset([dx])
    st = mp.mp_state_create(mp.scaler_cfg(init_scale=1.0, enabled=False))
    try:
        mp.mp_update_step(model.plan, st, gs, 1.0, 1, 1.0, mp.adamw_hparams())
        s = mp.read_stats(st)
        assert s["found_inf"] == 1 and s["step"] == 0 and bool((model.master[0] == 1.0).all())
    finally:
        mp.mp_gradset_destroy(gs)
        mp.mp_state_destroy(st)
        model.close()
