"""Every logit of a row counts once in every form of a score, rows split over workgroups among them: against
binary64, with tolerances from the additions that a lane makes (score_rows.py)."""
import numpy as np
import pytest

from loss_rows import near
from score_rows import U, borders, chain_of, entries, parts_of, planted, reference
from test_gpu_losses import KINDS, Buf, dev, empty, host, ttype
from test_gpu_scores import mp  # noqa: F401

pytestmark = pytest.mark.gpu


class Workspace:
    """As many bytes as a call may use, with a guard behind."""

    def __init__(self, mp):
        import torch
        self.flat = torch.full((mp.MP_SCORE_WORKSPACE_BYTES + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.t = self.flat[:-4096]

    def untouched(self):
        return bool((self.flat[-4096:] == 0xA5).all())


def run(mp, b, T, top, ws, targets, stream=None):
    import torch
    rows = b.t.shape[0]
    lp, lse, H = empty(rows), empty(rows), empty(rows)
    lists = ()
    if top:
        lists = (torch.full((rows, top), -55, dtype=torch.int64, device="cuda"), empty(rows * top).view(rows, top),
                 empty(rows * top).view(rows, top))
    s = mp.score(lp, lse, H, *lists, workspace=None if ws is None else ws.t)
    mp.mp_token_score(mp.logits(b.t, T), targets, s, stream=stream)
    return lp, lse, H, lists


def check_rows(got, x, t, T, chain, top, rows=slice(None)):
    """The outputs of some rows, whose logits are x and targets t."""
    lp, lse, H, lists = got
    r = reference(x, T, chain)
    near("lse", lse[rows], r["lse"], r["tol_lse"])
    near("entropy", H[rows], r["entropy"], r["tol_entropy"])
    near("logp", lp[rows], r["logp"].gather(1, t[:, None])[:, 0], r["tol_logp"].gather(1, t[:, None])[:, 0])
    if top:
        ids = entries(x, top)
        assert bool((lists[0][rows] == ids).all())
        assert bool((lists[2][rows] == x.gather(1, ids).float()).all())
        near("top_logp", lists[1][rows], r["logp"].gather(1, ids), r["tol_logp"].gather(1, ids))


# each number of lanes, on both sides of what it takes in one unrolled turn, with and without lists, and rows in
# parts that lanes hold and that they do not: (kind, V, rows of the call or None for as many as there are borders,
# entries, with a workspace)
FORMS = [("bf16", 40, None, 0, False), ("bf16", 1003, None, 20, False), ("fp16", 4095, None, 64, False),
         ("fp32", 2050, None, 0, False), ("bf16", 2049, None, 65, False), ("bf16", 4103, None, 20, False),
         ("bf16", 8190, None, 0, False), ("bf16", 16395, None, 33, False), ("fp32", 32003, None, 5, False),
         ("bf16", 65541, None, 0, False), ("fp16", 131077, None, 20, False),
         ("bf16", 8195, 2050, 20, False), ("bf16", 8195, 2050, 0, False), ("fp32", 16390, 2050, 0, False),
         ("bf16", 20011, 2050, 64, False), ("bf16", 33003, 2050, 0, False),
         ("bf16", 80005, 24, 20, True), ("bf16", 131075, 24, 0, True), ("fp32", 40005, 24, 20, True),
         ("fp16", 131075, 128, 128, True), ("bf16", 131075, 128, 0, True), ("fp32", 65539, 128, 128, True),
         ("bf16", 600011, 1, 20, True), ("bf16", 600011, 1, 0, True), ("fp32", 300007, 2, 128, True)]


@pytest.mark.parametrize("kind,V,rows,top,with_ws", FORMS)
def test_no_logit_is_left_out_or_taken_twice(mp, kind, V, rows, top, with_ws):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(V + top)
    T = float(np.float32(1.0))
    for pad, shift in ((0, 0), (3, 1)):
        call = rows or 64
        ends, inner = borders(V, kind, call, top, with_ws)
        # a place for each row; the first whole vector is where the row's address says
        size, turn = torch.finfo(ttype(kind)).bits // 8, rows or len(ends + inner)
        places = ends + [("from", p) for p in inner]
        while places:
            now, places = places[:turn], places[turn:]
            n = rows if rows else len(now)
            b = Buf(n, V, kind, pad, shift)
            rest = torch.randn(len(now), V, generator=g, device="cuda").to(ttype(kind)).double()
            at = []
            for r, p in enumerate(now):
                off = b.t[r].data_ptr() % 16
                head = (16 - off) % 16 // size
                at.append(p if isinstance(p, int) else min(p[1] + head, V - 1))
            planted(rest, at)
            index = torch.arange(n, device="cuda") % len(now)
            # rows that repeat have other heads: their planted logit is somewhere near a border
            b.t.copy_(rest[index])
            t = (torch.tensor(at, device="cuda")[index] + V // 2) % V
            ws = Workspace(mp) if with_ws else None
            got = run(mp, b, T, top, ws, t)
            assert (parts_of(V, kind, n, top) is not None and with_ws) == with_ws
            some = slice(0, len(now))
            check_rows(got, b.t[some], t[some], T, chain_of(V, kind, n, top, with_ws), top, some)
            if n > len(now):
                last = slice(n - min(len(now), 40), n)
                check_rows(got, b.t[last], t[last], T, chain_of(V, kind, n, top, with_ws), top, last)
            assert b.untouched() and (ws is None or ws.untouched())


@pytest.mark.parametrize("kind,V", [("bf16", 80003), ("fp16", 131075), ("fp32", 40002)])
@pytest.mark.parametrize("top", [0, 20, 128])
@pytest.mark.parametrize("rows", [1, 48, 127, 128, 129])
def test_split_rows(mp, kind, V, top, rows):  # noqa: F811
    """Up to 128 long rows are cut into parts: as without a workspace, to what the order of sums does, and some
    rows switched off."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows + top)
    T = float(np.float32(0.8))
    b = Buf(rows, V, kind, 1, 1)
    b.t.copy_(torch.randn(rows, V, generator=g, device="cuda") * 2)
    t = torch.randint(V, (rows,), generator=g, device="cuda")
    t[5::7] = -100
    ws = Workspace(mp)
    cut, whole = run(mp, b, T, top, ws, t), run(mp, b, T, top, None, t)
    live = t >= 0
    split = parts_of(V, kind, rows, top) is not None
    assert split == (rows <= 128) and bool((ws.flat[:4096] == 0xA5).all()) == (not split)
    for got, with_ws in ((cut, True), (whole, False)):
        lp, lse, H, lists = got
        for v in (lp, lse, H):
            assert not v[~live].any()
        for v, off in zip(lists, (-1, float("-inf"), float("-inf"))):
            assert bool((v[~live] == off).all())
        # in turns of 32 rows, whose binary64 forms take 32 MB each
        for a in range(0, rows, 32):
            some = torch.arange(a, min(a + 32, rows), device="cuda")
            some = some[live[some]]
            check_rows(got, b.t[some], t[some], T, chain_of(V, kind, rows, top, with_ws), top, some)
    assert ws.untouched() and b.untouched()


def test_split_rows_on_two_streams_at_once(mp):  # noqa: F811
    import torch
    rows, V, top = 30, 131075, 10
    assert parts_of(V, "fp16", rows, top)
    g = torch.Generator(device="cuda").manual_seed(3)
    data, outs = [], []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        b = Buf(rows, V, "fp16")
        b.t.copy_(torch.randn(rows, V, generator=g, device="cuda") * 2)
        data.append((s, b, torch.randint(V, (rows,), generator=g, device="cuda"), Workspace(mp)))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [run(mp, b, 1.0, top, ws, t, stream=s) for s, b, t, ws in data]
        torch.cuda.synchronize()
    for got, (s, b, t, ws) in zip(outs, data):
        check_rows(got, b.t, t, 1.0, chain_of(V, "fp16", rows, top, True), top)
        assert ws.untouched()


def test_split_rows_captured_and_replayed(mp):  # noqa: F811
    """Two graphs of split rows that share a workspace, on new inputs with eager work between."""
    import torch
    rows, V, top = 20, 90001, 12
    assert parts_of(V, "bf16", rows, top)
    g = torch.Generator(device="cuda").manual_seed(4)
    ws, b, side = Workspace(mp), Buf(rows, V, "bf16"), torch.cuda.Stream()
    t = torch.randint(V, (rows,), generator=g, device="cuda")
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(run(mp, b, 1.0, top, ws, t))
        graphs.append(graph)
    for i in range(4):
        b.t.copy_(torch.randn(rows, V, generator=g, device="cuda"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check_rows(outs[i % 2], b.t, t, 1.0, chain_of(V, "bf16", rows, top, True), top)
        eager = run(mp, b, 1.0, top, ws, t)
        torch.cuda.synchronize()
        for one, two in zip([*eager[:3], *eager[3]], [*outs[i % 2][:3], *outs[i % 2][3]]):
            assert torch.equal(one, two)
    assert ws.untouched()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1000, 9001])
def test_entropy_of_confident_rows(mp, kind, V):  # noqa: F811
    """One logit g above all others, each of which has the share q = e^-g / (1 + (V - 1) e^-g): the entropy is
    right to a small part of itself.  The lane that has the large one adds up `own` logits in fp32 next to 1:
    of each it loses at most q or u.  Its sum of y 2^y stands at the rounding of the large one's exponent
    (at most 2 u g) and at what its other logits add, and is rounded once for each of them.  All other lanes'
    logits count with an error of 5 u (g + 6.3), in both sums, and the additions; lanes are joined in binary64."""
    gaps = np.array([8.0, 12.0, 16.0, 20.0, 25.0, 30.0])
    # the large one among the first vectors of its lane, among the last, in a head and in a tail
    for place in (3, 8 * 64 - 1, V // 2, V - 9, V - 1):
        x = np.zeros((len(gaps), V))
        x[:, place] = gaps
        b = Buf(len(gaps), V, kind, 0, 1, x)
        lp, lse, H, _ = run(mp, b, 1.0, 0, None, dev(np.full(len(gaps), place)))
        chain = chain_of(V, kind, len(gaps), 0, False)
        own = round(chain / U)
        eps = (V - 1) * np.exp(-gaps)
        q = np.exp(-gaps) / (1 + eps)
        want = np.log1p(eps) + (V - 1) * q * gaps
        tol = (own * np.minimum(q, U) + own * U * (2 * U * gaps + own * q * (gaps + 5.6))
               + want * (10 * U * (gaps + 6.3) + 2 * chain + 2 * U) + 2.0 ** -50)
        off = np.abs(host(H) - want)
        assert (off <= tol).all(), (place, off / tol)
        assert (tol < want / 20).all()


@pytest.mark.parametrize("kind,V", [("bf16", 9001), ("fp32", 20001)])
@pytest.mark.parametrize("rows", [1281, 1792, 1793, 2047, 2048, 2049])
def test_rows_in_one_turn_and_in_two(mp, kind, V, rows):  # noqa: F811
    """Without lists, about the number of rows that the chip holds at once."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    b = Buf(rows, V, kind)
    b.t.copy_(torch.randn(rows, V, generator=g, device="cuda") * 2)
    t = torch.randint(V, (rows,), generator=g, device="cuda")
    t[3::5] = -100
    got = run(mp, b, 1.0, 0, None, t)
    live = t >= 0
    assert not any(v[~live].any() for v in got[:3])
    some = torch.cat([torch.arange(0, rows, 61, device="cuda"), torch.arange(rows - 9, rows, device="cuda")])
    some = some[live[some]]
    check_rows(got, b.t[some], t[some], 1.0, chain_of(V, kind, rows, 0, False), 0, some)
    assert b.untouched()
