"""What the loss calls may be given to write: an output that shares memory with an input, another
output, the logits, the gradient or the workspace is refused, and nothing else is (no GPU needed: the
refusals come before any device work, and every address here is only compared)."""
import pytest

STEP = 1 << 20
ROWS, V, STRIDE, K, PAIRS = 4, 100, 128, 8, 2


@pytest.fixture(scope="module")
def mp():
    import optimizer_step_tensor_amd as m
    m.lib()
    return m


# every array of each call: bytes, and whether the call writes it
R4, R8 = 4 * ROWS, 8 * ROWS
SHARED = {"workspace": (65536, True), "dev_scale": (4, False), "dev_count": (8, False)}
CALLS = {
    "token_logprob": {"targets": (R8, False), "logp": (R4, True), "lse": (R4, True),
                      "workspace": (65536, True)},
    "token_logprob_grad": {"targets": (R8, False), "lse": (R4, False), "dlogp": (R4, False), **SHARED},
    "cross_entropy": {"targets": (R8, False), "weights": (R4, False), "loss": (R4, True), **SHARED},
    "policy_loss": {"targets": (R8, False), "old_logp": (R4, False), "ref_logp": (R4, False),
                    "advantage": (R4, False), "weights": (R4, False), "loss": (R4, True),
                    "logp": (R4, True), "kl": (R4, True), **SHARED},
    "preference_loss": {"targets": (R8, False), "seq_start": (8 * (2 * PAIRS + 1), False),
                        "ref_logp": (8 * PAIRS, False), "loss": (4 * PAIRS, True),
                        "seq_logp": (8 * PAIRS, True), "logp": (R4, True), "lse": (R4, True),
                        "dlogp": (R4, True), **SHARED},
    "distill_loss": {"values": (4 * ROWS * K, False), "ids": (8 * ROWS * K, False),
                     "teacher_lse": (R4, False), "weights": (R4, False), "loss": (R4, True), **SHARED},
}
X = STEP                     # the logits: 4 rows of 100 bf16, 256 bytes apart
DX = 2 * STEP


def places(call):
    return {name: (3 + i) * STEP for i, name in enumerate(CALLS[call])}


def run(mp, call, a, rows=ROWS, x=X, dx=DX, stride=STRIDE):
    lx = mp.Logits(x, rows, V, stride, mp.MP_BF16, 1.0, a["workspace"])
    g = mp.LogitsGrad(dx, stride, a.get("dev_scale"), a.get("dev_count"), 1.0)
    if call == "token_logprob":
        return mp.mp_token_logprob(lx, a["targets"], a["logp"], a["lse"], stream=0)
    if call == "token_logprob_grad":
        return mp.mp_token_logprob_grad(lx, a["targets"], a["lse"], a["dlogp"], g, stream=0)
    if call == "cross_entropy":
        return mp.mp_cross_entropy(lx, a["targets"], a["weights"], a["loss"], g, stream=0)
    if call == "policy_loss":
        return mp.mp_policy_loss(lx, a["targets"], a["old_logp"], a["ref_logp"], a["advantage"],
                                 a["weights"], mp.policy_cfg(kl_coef=0.1), a["loss"], a["logp"],
                                 a["kl"], g, stream=0)
    if call == "preference_loss":
        return mp.mp_preference_loss(lx, a["targets"], PAIRS, a["seq_start"], a["ref_logp"],
                                     mp.preference_cfg(), a["loss"], a["seq_logp"], a["logp"],
                                     a["lse"], a["dlogp"], g, stream=0)
    t = mp.Teacher(a["values"], a["ids"], a["teacher_lse"], K, mp.MP_FP32)
    return mp.mp_distill_loss(lx, t, a["weights"], a["loss"], g, stream=0)


def overlap(mp, call, a, **kw):
    """Is the call refused for an overlap?  (With addresses that are no device memory, or without a
    device, every call is refused in the end.)"""
    with pytest.raises(mp.MpError) as e:
        run(mp, call, a, **kw)
    over = "overlaps" in str(e.value)
    assert not over or e.value.status == mp.MP_ERR_INVALID
    return over


@pytest.mark.parametrize("call", CALLS)
def test_arrays_that_a_call_writes_are_its_own(mp, call):
    base, sizes = places(call), CALLS[call]
    assert not overlap(mp, call, base)
    for a in sizes:
        for b in sizes:
            if a == b:
                continue
            na, wa = sizes[a]
            nb, wb = sizes[b]
            align = 16
            # the same start; a's last bytes on b's first; a inside, where they are not alike long
            up = (na - 1) // align * align
            for shift in {0, -up}:
                got = overlap(mp, call, dict(base, **{a: base[b] + shift}))
                assert got == (wa or wb), (call, a, b, shift)
            # side by side is fine
            end = -(-nb // align) * align
            for shift in {end, -(-(-na // align) * align)}:
                assert not overlap(mp, call, dict(base, **{a: base[b] + shift})), (call, a, b, shift)


@pytest.mark.parametrize("call", CALLS)
def test_arrays_and_rows(mp, call):
    """In a row of the logits or of the gradient, and in the padding between two rows."""
    base = places(call)
    row, gap = 2 * V, 2 * (STRIDE - V)             # 200 bytes, 56 bytes
    for a, (n, written) in CALLS[call].items():
        for at in (0, 256 + 16, 3 * 256 + 192):
            assert overlap(mp, call, dict(base, **{a: X + at})) == written, (a, at)
            if call != "token_logprob":
                assert overlap(mp, call, dict(base, **{a: DX + at})), (a, at)
        before, behind = -(-(-n // 16) * 16), 3 * 256 + 208
        for at in (before, behind):
            assert not overlap(mp, call, dict(base, **{a: X + at})), (a, at)
            assert not overlap(mp, call, dict(base, **{a: DX + at})), (a, at)
        if a != "workspace":
            at = 256 + row + 8                     # 16-byte aligned, 48 bytes left
            fits = n <= gap - 8
            assert overlap(mp, call, dict(base, **{a: X + at})) == (written and not fits), a
            if call != "token_logprob":
                assert overlap(mp, call, dict(base, **{a: DX + at})) == (not fits), a


@pytest.mark.parametrize("call", CALLS)
def test_one_row_has_no_padding(mp, call):
    """With one row the stride says nothing, whatever it holds."""
    base = dict(places(call))
    for a, (n, written) in CALLS[call].items():
        if not written:
            continue
        for stride in (0, STRIDE, -5):
            assert overlap(mp, call, dict(base, **{a: X + 192}), rows=1, stride=stride), a
            assert not overlap(mp, call, dict(base, **{a: X + 208}), rows=1, stride=stride), a


def test_the_gradient_may_replace_the_logits(mp):
    for call in CALLS:
        if call != "token_logprob":
            assert not overlap(mp, call, places(call), dx=X)


def test_inputs_may_be_shared(mp):
    """One array read in two roles."""
    a = places("policy_loss")
    a["old_logp"] = a["ref_logp"]
    a["weights"] = a["advantage"]
    assert not overlap(mp, "policy_loss", a)


def test_no_rows_touch_nothing(mp):
    a = {k: 3 * STEP for k in CALLS["cross_entropy"]}
    run(mp, "cross_entropy", a, rows=0)


@pytest.mark.gpu
def test_arrays_side_by_side(mp):
    """Every per-row array a slice of one tensor, loss and logp in the padding of the logits' rows, the
    gradient in place: the results of arrays of their own, with and without a workspace."""
    import torch
    for rows, V in ((2, 60001), (2, 300)):
        g = torch.Generator(device="cuda").manual_seed(V)
        x = torch.randn(rows, V, generator=g, device="cuda")
        t = torch.randint(V, (rows,), generator=g, device="cuda")
        per_row = torch.randn(4, rows, generator=g, device="cuda")
        cfg = mp.policy_cfg(0.2, 0.2, 0.1)
        for workspace in (None, torch.zeros(mp.MP_LOSS_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")):
            want = [torch.empty(rows, device="cuda") for _ in range(3)]
            dx = torch.empty_like(x)
            mp.mp_policy_loss(mp.logits(x, 1.0, workspace), t, *per_row.clone().unbind(), cfg, *want,
                              mp.logits_grad(dx))
            wide = torch.zeros(rows, V + 8, device="cuda")
            wide[:, :V] = x
            flat = torch.cat([per_row.flatten(), torch.zeros(rows, device="cuda")])
            ins = [flat[i * rows:(i + 1) * rows] for i in range(4)]
            kl, loss, logp = flat[4 * rows:], wide[0, V:V + rows], wide[0, V + rows:V + 2 * rows]
            mp.mp_policy_loss(mp.logits(wide[:, :V], 1.0, workspace), t, *ins, cfg, loss, logp, kl,
                              mp.logits_grad(wide[:, :V]))
            for got, ref in zip((loss, logp, kl, wide[:, :V]), want + [dx]):
                assert torch.allclose(got, ref, rtol=1e-5, atol=1e-6)
            assert torch.equal(flat[:4 * rows], per_row.flatten())


def test_targets_and_their_count_live_on_one_gpu(mp):
    """The kernel runs where the count lives; targets of another GPU are refused by the binding."""
    import torch

    class OnGpu:
        dtype, is_cuda = torch.int64, True

        def __init__(self, device, n):
            self.device, self.n = torch.device("cuda", device), n

        def numel(self):
            return self.n

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 3 * STEP
    with pytest.raises(ValueError, match="one GPU"):
        mp.mp_target_count(OnGpu(1, 4), OnGpu(0, 1), stream=0)
    with pytest.raises(mp.MpError):             # as far as the library: no such memory
        mp.mp_target_count(OnGpu(0, 4), OnGpu(0, 1), stream=0)
