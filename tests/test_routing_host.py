"""Routing to experts without a GPU: refusals, the binding's checks, structs against the header, arrays
that may not overlap, the reference's gradient against differences, the kernels' resources."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import route_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 24          # addresses far enough apart; every call here returns before they are read
E, ROWS, TOP = 64, 4, 6


@pytest.fixture(scope="module")
def mp():
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


def test_structs_and_constants_match_the_header(mp, tmp_path):
    lines, want = [], []
    for c, cls in (("mp_route_cfg", mp.RouteCfg), ("mp_routed", mp.Routed)):
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        want.append(ctypes.sizeof(cls))
        for n, _ in cls._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (c, n))
            want.append(getattr(cls, n).offset)
    for c in ("MAX_EXPERTS", "MAX_GROUPS", "MAX_TOP", "WORKSPACE_BYTES", "SOFTMAX", "SIGMOID"):
        lines.append('printf("%%d\\n", MP_ROUTE_%s);' % c)
        want.append(getattr(mp, "MP_ROUTE_" + c))
    f = tmp_path / "layout.c"
    f.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"mpstep.h\"\nint main(void) {\n"
                 + "\n".join(lines) + "\nreturn 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, str(f)], check=True)
    assert [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True)
            .stdout.split()] == want


def x_of(mp, **kw):
    d = dict(data=A, rows=ROWS, vocab=E, stride=E, dtype=mp.MP_BF16, temperature=1.0, workspace=None)
    d.update(kw)
    return mp.Logits(*[d[n] for n, _ in mp.Logits._fields_])


def g_of(mp, **kw):
    d = dict(data=2 * A, stride=E, dev_scale=None, dev_count=None, scale=1.0)
    d.update(kw)
    return mp.LogitsGrad(*[d[n] for n, _ in mp.LogitsGrad._fields_])


def c_of(mp, **kw):
    d = dict(score=0, top=TOP, groups=8, top_groups=4, group_best=2, renormalise=1, scale=1.0)
    d.update(kw)
    return mp.RouteCfg(*[d[n] for n, _ in mp.RouteCfg._fields_])


def r_of(mp, **kw):
    d = dict(weights=3 * A, ids=4 * A, load=5 * A, share=6 * A, aux=7 * A, workspace=8 * A)
    d.update(kw)
    return mp.Routed(*[d[n] for n, _ in mp.Routed._fields_])


def said(mp, f, *a, status=None, **kw):
    with pytest.raises(mp.MpError) as e:
        f(*a, stream=0, **kw)
    if status is not None:
        assert e.value.status == status, str(e.value)
    return str(e.value).lower()


BAD_X = [dict(rows=-1), dict(rows=1 << 22), dict(vocab=0), dict(vocab=1025, stride=1025),
         dict(stride=63), dict(dtype=3), dict(temperature=0.7), dict(data=None)]
BAD_CFG = [dict(score=2), dict(score=-1), dict(top=0), dict(top=17), dict(top=33, groups=1, top_groups=1),
           dict(groups=0), dict(groups=7), dict(groups=65), dict(top_groups=0), dict(top_groups=9),
           dict(group_best=0), dict(group_best=3), dict(scale=float("nan")),
           dict(top=9, top_groups=1), dict(scale=float("inf"))]


def test_refusals_of_routing(mp):
    I, AL = mp.MP_ERR_INVALID, mp.MP_ERR_ALIGN

    def call(x=None, bias=9 * A, mask=10 * A, cfg=None, out=None):
        return (x or x_of(mp), bias, mask, cfg or c_of(mp), out or r_of(mp))

    for kw in BAD_X:
        said(mp, mp.mp_route, *call(x=x_of(mp, **kw)), status=I)
    for kw in BAD_CFG:
        said(mp, mp.mp_route, *call(cfg=c_of(mp, **kw)), status=I)
    for kw in (dict(weights=None), dict(ids=None), dict(load=None), dict(share=None),
               dict(workspace=None)):
        said(mp, mp.mp_route, *call(out=r_of(mp, **kw)), status=I)
    for kw in (dict(weights=3 * A + 2), dict(ids=4 * A + 4), dict(load=5 * A + 4), dict(share=6 * A + 2),
               dict(aux=7 * A + 1), dict(workspace=8 * A + 8)):
        said(mp, mp.mp_route, *call(out=r_of(mp, **kw)), status=AL)
    said(mp, mp.mp_route, *call(bias=9 * A + 2), status=AL)
    L = mp.lib()
    x, c, r = x_of(mp), c_of(mp), r_of(mp)
    assert L.mp_route(None, None, None, ctypes.byref(c), ctypes.byref(r), None) == I
    assert L.mp_route(ctypes.byref(x), None, None, None, ctypes.byref(r), None) == I
    assert L.mp_route(ctypes.byref(x), None, None, ctypes.byref(c), None, None) == I
    for a in (call(), call(bias=None, mask=None), call(mask=10 * A + 1),
              call(out=r_of(mp, aux=None)), call(out=r_of(mp, share=None, aux=None)),
              call(out=r_of(mp, load=None, share=None, aux=None, workspace=None))):
        assert "device" in said(mp, mp.mp_route, *a)


def test_refusals_of_the_gradient(mp):
    I, AL = mp.MP_ERR_INVALID, mp.MP_ERR_ALIGN

    def call(x=None, mask=10 * A, cfg=None, ids=4 * A, dw=3 * A, load=5 * A, b=0.01, z=0.001, g=0):
        return (x or x_of(mp), mask, cfg or c_of(mp), ids, dw, load, b, z, g_of(mp) if g == 0 else g)

    f, nan = mp.mp_route_grad, float("nan")
    for kw in BAD_X:
        said(mp, f, *call(x=x_of(mp, **kw)), status=I)
    for kw in BAD_CFG:
        said(mp, f, *call(cfg=c_of(mp, **kw)), status=I)
    for a in (call(ids=None), call(load=None), call(dw=None, b=0.0, z=0.0), call(b=nan), call(z=nan),
              call(b=float("inf")), call(g=None), call(cfg=c_of(mp, score=1)),
              call(g=g_of(mp, data=A + 2)), call(g=g_of(mp, stride=63))):
        said(mp, f, *a, status=I)
    for a in (call(ids=4 * A + 4), call(dw=3 * A + 2), call(load=5 * A + 4)):
        said(mp, f, *a, status=AL)
    for a in (call(), call(dw=None), call(load=None, b=0.0, z=0.0), call(cfg=c_of(mp, score=1), z=0.0),
              call(g=g_of(mp, data=A))):
        assert "device" in said(mp, f, *a)


def test_refusals_of_the_bias_update(mp):
    L, I, AL = mp.lib(), mp.MP_ERR_INVALID, mp.MP_ERR_ALIGN

    def call(layers=3, experts=E, bias=A, n=2, load=2 * A, speed=0.1, out=3 * A):
        return L.mp_route_bias_update(layers, experts, bias, n, load, speed, out, None, None)

    for kw in (dict(layers=-1), dict(layers=(1 << 20) + 1), dict(experts=0), dict(experts=1025),
               dict(n=0), dict(n=(1 << 20) + 1), dict(speed=float("nan")), dict(bias=None),
               dict(load=None), dict(out=None), dict(out=A + 16), dict(out=2 * A + 16)):
        assert call(**kw) == I, kw
    for kw in (dict(bias=A + 2), dict(load=2 * A + 4), dict(out=3 * A + 2)):
        assert call(**kw) == AL, kw
    assert call(layers=0, bias=None, load=None, out=None) == mp.MP_OK
    assert "device" in mp.mp_last_error().lower() or call() != mp.MP_OK
    assert call(out=A) != mp.MP_OK and "device" in mp.mp_last_error().lower()      # in place


ARRAYS = dict(bias=(4 * E, False), mask=(ROWS, False), weights=(4 * ROWS * TOP, True),
              ids=(8 * ROWS * TOP, True), load=(8 * (E + 1), True), share=(4 * E, True),
              aux=(8, True), workspace=(4 << 20, True))


def test_arrays_that_routing_writes_are_its_own(mp):
    base = {n: (3 + i) * A for i, n in enumerate(ARRAYS)}

    def over(a):
        r = r_of(mp, **{n: a[n] for n in a if n not in ("bias", "mask")})
        return "overlaps" in said(mp, mp.mp_route, x_of(mp), a["bias"], a["mask"], c_of(mp), r)

    assert not over(base)
    for a, (na, wa) in ARRAYS.items():
        for b, (nb, wb) in ARRAYS.items():
            if a != b:
                assert over(dict(base, **{a: base[b]})) == (wa or wb), (a, b)
                assert not over(dict(base, **{a: base[b] + -(-nb // 16) * 16})), (a, b)
        assert over(dict(base, **{a: A + 16})) == wa, a


def test_no_tokens_are_no_work(mp):
    x = x_of(mp, rows=0, data=None)
    mp.mp_route(x, None, None, c_of(mp), r_of(mp, weights=None, ids=None, load=None, share=None,
                                              aux=None), stream=0)
    mp.mp_route_grad(x, None, c_of(mp), None, 3 * A, None, 0.0, 0.0, g_of(mp, data=None), stream=0)


def test_binding_checks_its_tensors(mp):
    import torch
    f, i = torch.zeros(4, 6), torch.zeros(4, 6, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        mp.routed(f, i)
    with pytest.raises(ValueError, match="tokens"):
        mp.routed(f[:, :5], i)
    with pytest.raises(TypeError, match="bias"):
        mp.mp_route(x_of(mp), torch.zeros(E, dtype=torch.float64), None, c_of(mp), r_of(mp), stream=0)
    with pytest.raises(TypeError, match="mask"):
        mp.mp_route(x_of(mp), None, torch.zeros(4), c_of(mp), r_of(mp), stream=0)
    with pytest.raises(ValueError, match="mask"):
        mp.mp_route(x_of(mp), None, torch.zeros(3, dtype=torch.bool), c_of(mp), r_of(mp), stream=0)
    b = torch.zeros(3, E)
    for load in (torch.zeros(3, E, dtype=torch.int64), torch.zeros(2, E + 1, dtype=torch.int64),
                 torch.zeros(E + 1, dtype=torch.int64)):
        with pytest.raises(ValueError, match="load"):
            mp.mp_route_bias_update(b, load, 0.1, stream=0)


# third derivatives of these losses are below 50: h^2/6 of them 1e-9; sums below 50 are rounded to
# 7e-15, over 2e-5: 4e-10
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_reference_gradient_against_differences(sigmoid, renormalise):
    rng = np.random.default_rng(3)
    rows, n, top, h = 6, 9, 3, 1e-5
    x = rng.normal(0, 1.5, (rows, n))
    x[2, 4] = -np.inf
    mask = np.array([1, 1, 1, 0, 1, 1])
    r = ref.route(x, None, mask, sigmoid, top, renormalise=renormalise, scale=1.7)
    ids = r["ids"].copy()
    ids[4, 1] = ids[4, 0]               # the same expert twice
    ids[5, 2] = -1
    dw = rng.normal(0, 1, (rows, top))
    large = 0.0 if sigmoid else 0.3
    args = (sigmoid, top, renormalise, 1.7, 0.8, large, 2.0)
    got, _ = ref.route_grad(x, ids, mask, dw, r["load"], *args)
    for i in np.ndindex(x.shape):
        if np.isfinite(x[i]):
            y = x.copy()
            y[i] += h
            up = ref.loss(y, ids, mask, dw, r["load"], *args)
            y[i] -= 2 * h
            assert abs((up - ref.loss(y, ids, mask, dw, r["load"], *args)) / (2 * h) - got[i]) < 1e-8, i


def test_no_scratch_and_bounded_vgprs(tmp_path):
    from optimizer_step_tensor_amd import build as B
    out = str(tmp_path / "routing.s")
    src = os.path.join(ROOT, "optimizer_step_tensor_amd", "csrc", "routing.hip")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", "-o", out, src], check=True,
                   stderr=subprocess.DEVNULL)
    found = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", open(out).read(), re.S)
    assert len(found) >= 8
    for name, body in found:
        assert int(re.search(r"private_segment_fixed_size (\d+)", body).group(1)) == 0, name
        assert int(re.search(r"next_free_vgpr (\d+)", body).group(1)) <= 256, name
