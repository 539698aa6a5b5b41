"""The losses over vocabulary logits without a GPU: every refusal that needs no device, the
binding's checks, the structs' layouts against the header, the reference's gradients against
differences of its losses, and the kernels' resource use."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import loss_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mp():
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


# --- the structs and constants of the binding are the header's -----------------------------

STRUCTS = {"mp_logits": "Logits", "mp_logits_grad": "LogitsGrad", "mp_policy_cfg": "PolicyCfg",
           "mp_preference_cfg": "PreferenceCfg", "mp_teacher": "Teacher"}


def test_struct_layouts_match_the_header(mp, tmp_path):
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "mpstep.h"', "int main(void) {"]
    want = []
    for c, py in STRUCTS.items():
        cls = getattr(mp, py)
        src.append('printf("%%zu\\n", sizeof(%s));' % c)
        want.append(ctypes.sizeof(cls))
        for name, _ in cls._fields_:
            src.append('printf("%%zu\\n", offsetof(%s, %s));' % (c, name))
            want.append(getattr(cls, name).offset)
    src.append("return 0; }")
    f = tmp_path / "layout.c"
    f.write_text("\n".join(src))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, str(f)], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True)
           .stdout.split()]
    assert got == want


def test_constants_match_the_header(mp):
    src = open(os.path.join(ROOT, "include", "mpstep.h")).read()
    for name in ("MP_FP32", "MP_LOSS_WORKSPACE_BYTES", "MP_DISTILL_MAX_K", "MP_PREF_SIGMOID",
                 "MP_PREF_SQUARED"):
        m = re.search(r"#define\s+%s\s+(\d+)" % name, src)
        assert m and int(m.group(1)) == getattr(mp, name), name


# --- refusals (addresses that are never read: every call returns before any device work) ----

A = 1 << 20          # an aligned address


def x_of(mp, **kw):
    d = dict(data=A, rows=4, vocab=100, stride=100, dtype=mp.MP_BF16, temperature=1.0,
             workspace=None)
    d.update(kw)
    return mp.Logits(*[d[n] for n, _ in mp.Logits._fields_])


def g_of(mp, **kw):
    d = dict(data=A + (1 << 16), stride=100, dev_scale=None, dev_count=None, scale=1.0)
    d.update(kw)
    return mp.LogitsGrad(*[d[n] for n, _ in mp.LogitsGrad._fields_])


def calls(mp):
    """Each loss as f(x, g) with valid other arguments."""
    cfg, pref = mp.policy_cfg(), mp.preference_cfg()
    t = mp.Teacher(A, A, None, 8, mp.MP_FP32)
    return {
        "cross_entropy": lambda x, g: mp.mp_cross_entropy(x, A, None, A, g, stream=0),
        "logprob_grad": lambda x, g: mp.mp_token_logprob_grad(x, A, A, A, g, stream=0),
        "policy": lambda x, g: mp.mp_policy_loss(x, A, A, None, A, None, cfg, A, None, None, g,
                                                 stream=0),
        "preference": lambda x, g: mp.mp_preference_loss(x, A, 2, A, A, pref, A, A, A, A, A, g,
                                                         stream=0),
        "distill": lambda x, g: mp.mp_distill_loss(x, t, None, A, g, stream=0),
    }


NAMES = ["cross_entropy", "logprob_grad", "policy", "preference", "distill"]


def refused(mp, status, f, *a, **kw):
    with pytest.raises(mp.MpError) as e:
        f(*a, **kw)
    assert e.value.status == status, str(e.value)
    return str(e.value)


@pytest.mark.parametrize("name", NAMES)
def test_bad_logits_are_refused(mp, name):
    f = calls(mp)[name]
    inv = [dict(rows=-1), dict(rows=1 << 22), dict(vocab=0), dict(vocab=-5),
           dict(vocab=(1 << 30) + 1, stride=1 << 31), dict(stride=99), dict(stride=0),
           dict(stride=-100), dict(stride=(1 << 32) + 1), dict(dtype=3), dict(dtype=-1),
           dict(dtype=1 << 30), dict(temperature=0.0), dict(temperature=-1.0),
           dict(temperature=float("nan")), dict(temperature=float("inf")),
           dict(temperature=1e-7), dict(temperature=2e6), dict(data=None)]
    for kw in inv:
        refused(mp, mp.MP_ERR_INVALID, f, x_of(mp, **kw), g_of(mp))
    for kw in (dict(data=A + 1), dict(data=A + 2, dtype=mp.MP_FP32), dict(workspace=A + 8)):
        refused(mp, mp.MP_ERR_ALIGN, f, x_of(mp, **kw), g_of(mp))


@pytest.mark.parametrize("name", NAMES)
def test_bad_gradients_are_refused(mp, name):
    f = calls(mp)[name]
    for kw in (dict(data=None), dict(stride=99), dict(stride=0), dict(stride=(1 << 32) + 1),
               dict(scale=float("nan")), dict(scale=float("inf")),
               # overlaps without being the logits: shifted, another stride, inside, around
               dict(data=A + 2), dict(data=A, stride=101), dict(data=A + 798),
               dict(data=A - 2), dict(data=A - 798)):
        refused(mp, mp.MP_ERR_INVALID, f, x_of(mp), g_of(mp, **kw))
    for kw in (dict(data=A + (1 << 16) + 1), dict(dev_scale=A + 2), dict(dev_count=A + 4)):
        refused(mp, mp.MP_ERR_ALIGN, f, x_of(mp), g_of(mp, **kw))


def test_each_call_refuses_its_own_bad_arguments(mp):
    x, g = x_of(mp), g_of(mp)
    I, AL = mp.MP_ERR_INVALID, mp.MP_ERR_ALIGN
    refused(mp, I, mp.mp_target_count, A, A, n=-1, stream=0)
    refused(mp, I, mp.mp_target_count, None, A, n=4, stream=0)
    refused(mp, I, mp.mp_target_count, A, None, n=4, stream=0)
    refused(mp, AL, mp.mp_target_count, A + 4, A, n=4, stream=0)
    refused(mp, AL, mp.mp_target_count, A, A + 4, n=4, stream=0)
    for a in ((None, A, A), (A, None, A)):
        refused(mp, I, mp.mp_token_logprob, x, *a, stream=0)
    for a in ((A + 4, A, A), (A, A + 2, A), (A, A, A + 2)):
        refused(mp, AL, mp.mp_token_logprob, x, *a, stream=0)
    refused(mp, I, mp.mp_token_logprob_grad, x, A, A, A, None, stream=0)
    for a in ((None, A, A), (A, None, A), (A, A, None)):
        refused(mp, I, mp.mp_token_logprob_grad, x, *a, g, stream=0)
    for a in ((None, None, A), (A, None, None)):
        refused(mp, I, mp.mp_cross_entropy, x, *a, g, stream=0)
    refused(mp, AL, mp.mp_cross_entropy, x, A, A + 1, A, g, stream=0)

    def pol(cfg=mp.policy_cfg(), targets=A, old=A, r=A, adv=A, w=None, loss=A, logp=A, kl=A):
        return mp.mp_policy_loss(x, targets, old, r, adv, w, cfg, loss, logp, kl, g, stream=0)
    for kw in (dict(targets=None), dict(old=None), dict(adv=None), dict(loss=None),
               dict(r=None), dict(r=None, kl=None, cfg=mp.policy_cfg(kl_coef=0.1))):
        refused(mp, I, pol, **kw)
    nan, inf = float("nan"), float("inf")
    for c in ((-0.1, 0, 0), (1.1, 0, 0), (nan, 0, 0), (0, -1, 0), (0, inf, 0), (0, nan, 0),
              (0, 0, -1), (0, 0, nan), (0, 0, inf)):
        refused(mp, I, pol, cfg=mp.policy_cfg(*c))
    for kw in (dict(old=A + 2), dict(r=A + 1), dict(adv=A + 2), dict(w=A + 2), dict(loss=A + 2),
               dict(logp=A + 2), dict(kl=A + 2), dict(targets=A + 4)):
        refused(mp, AL, pol, **kw)

    def pref(cfg=mp.preference_cfg(), n=2, targets=A, start=A, r=A, loss=A, seq=A, logp=A, lse=A,
             dlogp=A):
        return mp.mp_preference_loss(x, targets, n, start, r, cfg, loss, seq, logp, lse, dlogp, g,
                                     stream=0)
    for kw in (dict(n=0), dict(n=-1), dict(n=1 << 22), dict(targets=None), dict(start=None),
               dict(loss=None), dict(seq=None), dict(logp=None), dict(lse=None), dict(dlogp=None),
               dict(cfg=mp.preference_cfg(2)), dict(cfg=mp.preference_cfg(-1)),
               dict(cfg=mp.preference_cfg(beta=0.0)), dict(cfg=mp.preference_cfg(beta=nan)),
               dict(cfg=mp.preference_cfg(beta=inf)),
               dict(cfg=mp.preference_cfg(label_smoothing=-0.1)),
               dict(cfg=mp.preference_cfg(label_smoothing=0.6)),
               dict(cfg=mp.preference_cfg(margin=nan))):
        refused(mp, I, pref, **kw)
    for kw in (dict(start=A + 4), dict(r=A + 2), dict(seq=A + 2), dict(dlogp=A + 1)):
        refused(mp, AL, pref, **kw)

    def dist(values=A, ids=A, lse=None, k=8, dtype=2, w=None, loss=A):
        return mp.mp_distill_loss(x, mp.Teacher(values, ids, lse, k, dtype), w, loss, g, stream=0)
    for kw in (dict(k=0), dict(k=-1), dict(k=1025), dict(dtype=3), dict(values=None),
               dict(ids=None), dict(loss=None)):
        refused(mp, I, dist, **kw)
    for kw in (dict(values=A + 2), dict(ids=A + 4), dict(lse=A + 2), dict(w=A + 2)):
        refused(mp, AL, dist, **kw)


def test_null_structs_are_refused(mp):
    L = mp.lib()
    x, g = ctypes.byref(x_of(mp)), ctypes.byref(g_of(mp))
    assert L.mp_token_logprob(None, A, A, A, None) == mp.MP_ERR_INVALID
    assert L.mp_cross_entropy(None, A, None, A, g, None) == mp.MP_ERR_INVALID
    assert L.mp_policy_loss(x, A, A, A, A, None, None, A, A, A, g, None) == mp.MP_ERR_INVALID
    assert L.mp_preference_loss(x, A, 1, A, A, None, A, A, A, A, A, g, None) == mp.MP_ERR_INVALID
    assert L.mp_distill_loss(x, None, None, A, g, None) == mp.MP_ERR_INVALID
    assert "teacher" in L.mp_last_error().decode()


def test_no_rows_are_no_work(mp):
    x, g = x_of(mp, rows=0, data=None), g_of(mp, data=None)
    for name, f in calls(mp).items():
        if name != "preference":           # its pairs are written even then
            f(x, g)


def test_binding_checks_its_tensors(mp):
    import torch
    x = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="GPU"):
        mp.logits(x)
    with pytest.raises(TypeError):
        mp.logits(torch.zeros(4, 10, dtype=torch.float64))
    with pytest.raises(TypeError):
        mp.logits(torch.zeros(10))
    with pytest.raises(ValueError, match="GPU"):
        mp.logits_grad(x)
    with pytest.raises(TypeError):
        mp.teacher(torch.zeros(4, 2, dtype=torch.float64), torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        mp.teacher(torch.zeros(4, 2), torch.zeros(4, 3, dtype=torch.int64))
    xs = x_of(mp)
    with pytest.raises(TypeError, match="targets"):
        mp.mp_cross_entropy(xs, torch.zeros(4, dtype=torch.int32), None, A, stream=0)
    with pytest.raises(ValueError, match="targets"):
        mp.mp_cross_entropy(xs, torch.zeros(3, dtype=torch.int64), None, A, stream=0)
    with pytest.raises(ValueError, match="targets"):
        mp.mp_cross_entropy(xs, torch.zeros(8, dtype=torch.int64)[::2], None, A, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        mp.mp_cross_entropy(xs, torch.zeros(4, dtype=torch.int64), None, A, stream=0)


# --- the reference's gradients against differences of its losses ---------------------------

def differences(f, x, h=1e-5):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y).sum()
        y[i] -= 2 * h
        d[i] = (up - f(y).sum()) / (2 * h)
    return d


# h = 1e-5: the third derivatives here are below 100 (h^2/6 of them: 2e-9), and the rounding of
# a sum of losses below 100 is 1.4e-14 / 2e-5 = 7e-10 per evaluation
TOL = 1e-7


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_reference_gradients_against_differences(T):
    rng = np.random.default_rng(5)
    rows, V = 6, 11
    x = rng.normal(0, 2, (rows, V))
    t = rng.integers(0, V, rows)
    t[2] = -100
    w = rng.uniform(0.5, 2, rows)
    w[4] = 0.0
    d = rng.normal(0, 1, rows)
    got = ref.logprob(x, t, T, d, 1.0)["dx"]
    assert np.abs(got - differences(lambda y: d * ref.logprob(y, t, T)["logp"], x)).max() < TOL
    got = ref.cross_entropy(x, t, T, w)["dx"]
    assert np.abs(got - differences(lambda y: ref.cross_entropy(y, t, T, w)["loss"], x)).max() < TOL
    lp = ref.logprob(x, t, T)["logp"]
    old, rf, adv = lp + rng.normal(0, 0.4, rows), lp + rng.normal(0, 0.4, rows), rng.normal(0, 1, rows)

    def pol(y):
        return ref.policy(y, t, old, rf, adv, T, w, (0.2, 0.3), 0.1)
    assert not pol(x)["near_border"].any()
    assert np.abs(pol(x)["dx"] - differences(lambda y: pol(y)["loss"], x)).max() < TOL
    for kind_of in ("sigmoid", "squared"):
        for mean in (False, True):
            def pre(y):
                return ref.preference(y, t, np.array([0, 2, 2, 3, 5]), np.array([-1.0, 2, 0.5, -3]), T,
                                      kind_of, 0.3, 0.1, 0.2, mean)
            assert np.abs(pre(x)["dx"] - differences(lambda y: pre(y)["loss"], x)).max() < TOL
    ids = rng.integers(-1, V, (rows, 5))
    ids[0, :2] = 3
    ids[1] = -1
    v = rng.normal(0, 2, (rows, 5))
    for lse in (None, rng.uniform(3, 5, rows)):
        def dis(y):
            return ref.distill(y, v, ids, lse, T, w)
        assert np.abs(dis(x)["dx"] - differences(lambda y: dis(y)["loss"], x)).max() < TOL


# --- resources ------------------------------------------------------------------------------

def test_no_scratch_and_bounded_vgprs(tmp_path):
    """No kernel spills, and every one fits the registers that its workgroup size leaves."""
    from optimizer_step_tensor_amd import build as B
    out = str(tmp_path / "losses.s")
    src = os.path.join(ROOT, "optimizer_step_tensor_amd", "csrc", "losses.hip")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", "-o", out, src], check=True,
                   stderr=subprocess.DEVNULL)
    found = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", open(out).read(), re.S)
    assert len(found) >= 8
    for name, body in found:
        assert int(re.search(r"private_segment_fixed_size (\d+)", body).group(1)) == 0, name
        assert int(re.search(r"next_free_vgpr (\d+)", body).group(1)) <= 128, name
