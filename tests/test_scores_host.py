"""The scores of logits without a GPU: refusals, the binding's checks, the struct against the header,
arrays that may not overlap, the reference's gradient against differences, the kernels' resources."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import score_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20          # an aligned address: every call here returns before it is read


@pytest.fixture(scope="module")
def mp():
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


def test_struct_and_constants_match_the_header(mp, tmp_path):
    cls = mp.Score
    names = [n for n, _ in cls._fields_]
    lines = ['printf("%zu\\n", sizeof(mp_score));']
    lines += ['printf("%%zu\\n", offsetof(mp_score, %s));' % n for n in names]
    lines += ['printf("%%d\\n", %s);' % c for c in ("MP_SCORE_MAX_TOP", "MP_SCORE_WORKSPACE_BYTES")]
    f = tmp_path / "layout.c"
    f.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"mpstep.h\"\nint main(void) {\n"
                 + "\n".join(lines) + "\nreturn 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, str(f)], check=True)
    got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True)
           .stdout.split()]
    assert got == ([ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in names]
                   + [mp.MP_SCORE_MAX_TOP, mp.MP_SCORE_WORKSPACE_BYTES])


def x_of(mp, **kw):
    d = dict(data=A, rows=4, vocab=100, stride=128, dtype=mp.MP_BF16, temperature=1.0,
             workspace=None)
    d.update(kw)
    return mp.Logits(*[d[n] for n, _ in mp.Logits._fields_])


def g_of(mp, **kw):
    d = dict(data=2 * A, stride=128, dev_scale=None, dev_count=None, scale=1.0)
    d.update(kw)
    return mp.LogitsGrad(*[d[n] for n, _ in mp.LogitsGrad._fields_])


def s_of(mp, **kw):
    d = dict(logp=4 * A, lse=5 * A, entropy=6 * A, top_ids=7 * A, top_logp=8 * A, top_values=9 * A,
             workspace=None, top=8)
    d.update(kw)
    return mp.Score(*[d[n] for n, _ in mp.Score._fields_])


def refused(mp, status, f, *a, **kw):
    with pytest.raises(mp.MpError) as e:
        f(*a, stream=0, **kw)
    assert e.value.status == status, str(e.value)
    return str(e.value)


BAD = [dict(rows=-1), dict(rows=1 << 22), dict(vocab=0), dict(vocab=(1 << 30) + 1, stride=1 << 31),
       dict(stride=99), dict(stride=(1 << 32) + 1), dict(dtype=3), dict(temperature=0.0),
       dict(temperature=float("nan")), dict(data=None)]


def test_refusals_of_the_score(mp):
    f, x, I, AL = mp.mp_token_score, x_of(mp), mp.MP_ERR_INVALID, mp.MP_ERR_ALIGN
    for kw in BAD:
        refused(mp, I, f, x_of(mp, **kw), 3 * A, s_of(mp))
    refused(mp, AL, f, x_of(mp, data=A + 1), 3 * A, s_of(mp))
    for kw in (dict(top=-1), dict(top=mp.MP_SCORE_MAX_TOP + 1), dict(top=0), dict(top_ids=None),
               dict(top=0, logp=None, lse=None, entropy=None, top_ids=None, top_logp=None,
                    top_values=None)):
        refused(mp, I, f, x, 3 * A, s_of(mp, **kw))
    assert "targets" in refused(mp, I, f, x, None, s_of(mp))
    for kw in (dict(logp=A + 2), dict(lse=A + 2), dict(entropy=A + 1), dict(top_ids=7 * A + 4),
               dict(top_logp=8 * A + 2), dict(top_values=9 * A + 1), dict(workspace=10 * A + 8)):
        refused(mp, AL, f, x, 3 * A, s_of(mp, **kw))
    refused(mp, AL, f, x, 3 * A + 4, s_of(mp))
    assert mp.lib().mp_token_score(ctypes.byref(x), 3 * A, None, None) == I
    assert mp.lib().mp_token_score(None, 3 * A, ctypes.byref(s_of(mp)), None) == I
    # whole: it gets as far as asking for the place of the logits
    assert "device" in refused_any(mp, f, x, 3 * A, s_of(mp))
    assert "device" in refused_any(mp, f, x, None, s_of(mp, logp=None))


def refused_any(mp, f, *a):
    with pytest.raises(mp.MpError) as e:
        f(*a, stream=0)
    return str(e.value).lower()


def test_refusals_of_the_gradient(mp):
    f, x, g, I = mp.mp_token_score_grad, x_of(mp), g_of(mp), mp.MP_ERR_INVALID
    ok = dict(targets=3 * A, lse=4 * A, entropy=5 * A, dlogp=6 * A, dentropy=7 * A)

    def call(x=x, g=g, **kw):
        d = dict(ok, **kw)
        return (x, d["targets"], d["lse"], d["entropy"], d["dlogp"], d["dentropy"], g)

    for kw in BAD:
        refused(mp, I, f, *call(x=x_of(mp, **kw)))
    for kw in (dict(data=None), dict(stride=99), dict(scale=float("inf")), dict(data=A + 2),
               dict(data=A, stride=129)):
        refused(mp, I, f, *call(g=g_of(mp, **kw)))
    for kw in (dict(g=None), dict(lse=None), dict(dlogp=None, dentropy=None), dict(targets=None),
               dict(entropy=None)):
        refused(mp, I, f, *call(**kw))
    for name in ok:
        refused(mp, mp.MP_ERR_ALIGN, f, *call(**{name: ok[name] + 2}))
    for kw in (dict(), dict(dlogp=None), dict(dlogp=None, targets=None),
               dict(dentropy=None, entropy=None), dict(g=g_of(mp, data=A))):
        assert "device" in refused_any(mp, f, *call(**kw))


def test_no_rows_are_no_work(mp):
    x, g = x_of(mp, rows=0, data=None), g_of(mp, data=None)
    mp.mp_token_score(x, None, s_of(mp, logp=None), stream=0)
    mp.mp_token_score_grad(x, None, None, 5 * A, None, 7 * A, g, stream=0)


ROWS, TOP = 4, 8
SCORE = dict(targets=(8 * ROWS, False), logp=(4 * ROWS, True), lse=(4 * ROWS, True),
             entropy=(4 * ROWS, True), top_ids=(8 * ROWS * TOP, True),
             top_logp=(4 * ROWS * TOP, True), top_values=(4 * ROWS * TOP, True),
             workspace=(1 << 20, True))
GRAD = dict(targets=(8 * ROWS, False), lse=(4 * ROWS, False), entropy=(4 * ROWS, False),
            dlogp=(4 * ROWS, False), dentropy=(4 * ROWS, False), dev_scale=(4, False),
            dev_count=(8, False))


@pytest.mark.parametrize("call", ["score", "grad"])
def test_arrays_that_a_call_writes_are_its_own(mp, call):
    sizes = SCORE if call == "score" else GRAD
    base = {name: (4 + 2 * i) * A for i, name in enumerate(sizes)}

    def over(a):
        if call == "score":
            s = s_of(mp, **{n: a[n] for n in a if n != "targets"})
            return "overlaps" in refused_any(mp, mp.mp_token_score, x_of(mp), a["targets"], s)
        g = g_of(mp, dev_scale=a["dev_scale"], dev_count=a["dev_count"])
        return "overlaps" in refused_any(mp, mp.mp_token_score_grad, x_of(mp), a["targets"], a["lse"],
                                         a["entropy"], a["dlogp"], a["dentropy"], g)

    assert not over(base)
    for a, (na, wa) in sizes.items():
        for b, (nb, wb) in sizes.items():
            if a != b:
                assert over(dict(base, **{a: base[b]})) == (wa or wb), (a, b)
                assert not over(dict(base, **{a: base[b] + -(-nb // 16) * 16})), (a, b)
        # in a row of the logits (256 bytes apart, 200 used), in a gradient's
        assert over(dict(base, **{a: A + 256 + 16})) == wa, a
        if call == "grad":
            assert over(dict(base, **{a: 2 * A + 256 + 16})), a


def test_the_losses_workspace_in_the_logits_is_not_the_calls(mp):
    x = x_of(mp, workspace=4 * A)
    assert "device" in refused_any(mp, mp.mp_token_score, x, 3 * A, s_of(mp, logp=4 * A))


def test_binding_checks_its_tensors(mp):
    import torch
    with pytest.raises(ValueError, match="output"):
        mp.score()
    with pytest.raises(ValueError, match="GPU"):
        mp.score(lse=torch.zeros(4))
    with pytest.raises(ValueError, match="shape"):
        mp.score(top_ids=torch.zeros(4, 2, dtype=torch.int64), top_logp=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="shape"):
        mp.score(lse=torch.zeros(4), top_values=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="top_ids"):
        mp.score(top_ids=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="targets"):
        mp.mp_token_score(x_of(mp), torch.zeros(4), s_of(mp), stream=0)


# h = 1e-5: third derivatives below 100 leave 2e-9, the rounding of sums below 100 7e-10
@pytest.mark.parametrize("T", [1.0, 0.7])
def test_reference_gradient_against_differences(T):
    rng = np.random.default_rng(5)
    rows, V, h = 6, 11, 1e-5
    x = rng.normal(0, 2, (rows, V))
    x[3, 4] = -np.inf
    t = rng.integers(0, V, rows)
    t[2] = -100
    t[3] = 5
    dl, dh = rng.normal(0, 1, rows), rng.normal(0, 1, rows)
    s = ref.score(x, t, T)

    def f(y):
        s = ref.score(y, t, T)
        return (dl * s["logp"] + dh * s["entropy"]).sum()

    got, _ = ref.score_grad(x, t, s["lse"], s["entropy"], dl, dh, T)
    want = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        if np.isfinite(x[i]):
            y = x.copy()
            y[i] += h
            up = f(y)
            y[i] -= 2 * h
            want[i] = (up - f(y)) / (2 * h)
    assert np.abs(got - want).max() < 1e-7


def test_no_scratch_and_bounded_vgprs(tmp_path):
    from optimizer_step_tensor_amd import build as B
    out = str(tmp_path / "scores.s")
    src = os.path.join(ROOT, "optimizer_step_tensor_amd", "csrc", "scores.hip")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", "-o", out, src], check=True,
                   stderr=subprocess.DEVNULL)
    found = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", open(out).read(), re.S)
    assert len(found) >= 6
    for name, body in found:
        assert int(re.search(r"private_segment_fixed_size (\d+)", body).group(1)) == 0, name
        assert int(re.search(r"next_free_vgpr (\d+)", body).group(1)) <= 128, name
