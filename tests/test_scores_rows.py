"""The tolerances of score_rows.py would see logits that a score leaves out or takes twice: here the mistake is
planted in the reference, on the CPU."""
import pytest
import torch

from score_rows import E, borders, chain_of, entries, lanes_of, parts_of, planted, reference

FORMS = [("bf16", 40, 7, 4, False), ("bf16", 1003, 7, 20, False), ("bf16", 20011, 9, 20, False),
         ("fp32", 32001, 3000, 5, False), ("bf16", 131075, 9, 20, False), ("bf16", 131075, 9, 20, True),
         ("fp32", 60001, 128, 128, True)]


@pytest.mark.parametrize("kind,V,rows,top,with_ws", FORMS)
def test_a_border_left_out_or_taken_twice_shows(kind, V, rows, top, with_ws):
    ends, inner = borders(V, kind, rows, top, with_ws)
    assert {0, 1, V - 2, V - 1} <= set(ends)
    places = ends + inner
    x = torch.randn(len(places), V, generator=torch.Generator().manual_seed(V))
    planted(x, places)
    chain = chain_of(V, kind, rows, top, with_ws)
    whole = reference(x, 1.0, chain)
    at = torch.arange(len(places)), torch.tensor(places)
    less = x.clone()
    less[at] = float("-inf")
    twice = torch.cat([x, x[at][:, None]], 1)
    for other in (less, twice):
        r = reference(other, 1.0, chain)
        for name in ("lse", "entropy"):
            off = (r[name] - whole[name]).abs()
            # by ln 1.5 and more; the entropy's tolerance is larger, and it moves less
            assert bool((off > (1000 if name == "lse" else 50) * whole["tol_" + name]).all()), (name, off.min())


@pytest.mark.parametrize("kind,V,rows,top,with_ws", FORMS[1:])
def test_left_out_average_logits_show(kind, V, rows, top, with_ws):
    """Any eight neighbours that hold their share of the mass, in the longest rows too."""
    x = torch.randn(1, V, generator=torch.Generator().manual_seed(V))
    chain = chain_of(V, kind, rows, top, with_ws)
    whole = reference(x, 1.0, chain)
    q = torch.softmax(x[0].double(), 0)
    mass = q[:V // 8 * 8].reshape(-1, 8).sum(1)
    at = 8 * int((mass - 8 / V).abs().argmin())
    less = x.clone()
    less[0, at:at + 8] = float("-inf")
    off = (reference(less, 1.0, chain)["lse"] - whole["lse"]).abs()
    assert bool((off > 1.4 * whole["tol_lse"]).all())


def test_forms():
    assert [lanes_of(8 * v, "bf16", r, t) for v, r, t in
            ((512, 9, 20), (513, 9, 20), (1024, 2048, 20), (1025, 2048, 20), (4097, 2048, 20), (512, 9, 65))] == \
        [64, 256, 64, 128, 256, 128]
    assert parts_of(131072, "bf16", 129, 20) is None and parts_of(79999, "bf16", 1, 20) is None
    assert parts_of(131072, "bf16", 1, 20) == (32, 512)
    assert parts_of(131072, "bf16", 128, 20) == (16, 1024)
    assert parts_of(131072, "bf16", 128, 128) == (7, 2341)          # limited by the workspace
    assert parts_of(600000, "bf16", 1, 20) == (64, 1172)            # by the joining lanes
    assert chain_of(128256, "bf16", 9, 20, False) < 3.2e-5 and chain_of(128256, "bf16", 1, 20, True) < 2e-6


def test_reference_is_the_definition():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 301, generator=g, dtype=torch.float64).float()
    x[1, ::2] = float("-inf")
    r = reference(x, 0.5, 0.0)
    p = torch.softmax(x.double() / 0.5, 1)
    assert torch.allclose(r["entropy"], torch.special.entr(p).sum(1), rtol=1e-13)
    assert torch.allclose(r["lse"], torch.logsumexp(x.double() / 0.5, 1), rtol=1e-14)
    assert entries(torch.tensor([[1.0, 3.0, -0.0, 3.0, 0.0]]), 5).tolist() == [[1, 3, 0, 2, 4]]
    assert E == {"bf16": 8, "fp16": 8, "fp32": 4}
