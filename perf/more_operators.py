"""What a training step takes from rows of logits besides their loss, as cases to time and to compare.

``run`` computes a case in plain torch operations, or with ``own`` through the library's calls on
the same inputs.

Scores of a vocabulary's logits x[r, j], with z = x / T, lse = log sum_j exp(z_j), q = exp(z - lse):

* ``score``   of each row the target's log-probability lp = z_t - lse, lse, the entropy
              H = -sum_j q_j log q_j, and the k likeliest entries (ties: the lowest id first) with
              their log-probabilities and logits: what sampling reports, what an entropy bonus
              takes, and the lists that a student is distilled from
* ``bonus``   the same without entries, then the logits' gradient of sum_r (g_r lp_r + h_r H_r)
              times S / n (S the loss scale, n the number of targets, both in device memory)

Routing of tokens to experts from a router's logits x[r, e], with scores s = softmax(x) or
sigmoid(x):

* ``route``   the k experts of the largest s_e + bias_e, taken from the best groups of experts only
              (a group counts as the sum of its largest one or two), weights s_e, divided by their
              sum, times a factor; with ``train`` also how many tokens each expert got, the mean
              share of each, and the losses of the imbalance and of large logits
* ``router``  the same, the logits' gradient of all of it, and the balancing bias moved by one step

A target below 0 marks a row without scores, a token whose mask is False is not routed.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BALANCE, LARGE, SPEED = 0.01, 0.001, 0.001      # the losses' coefficients, the bias's step
TINY = 1e-20                                    # added to the sum that weights are divided by


def listed():
    return [
        # one sampled token of the 8B workload's vocabulary with its alternatives: latency alone
        dict(name="score one token", op="score", rows=1, vocab=128256, dtype="bf16",
             temperature=1.0, masked=0.0, top=20, targets=True),
        # a step of 48 sequences that are sampled together: fewer rows than compute units
        dict(name="score few long rows", op="score", rows=48, vocab=128256, dtype="bf16",
             temperature=0.8, masked=0.0, top=8, targets=True),
        # fp32 logits of an odd vocabulary, where no row but the first starts on a whole vector
        dict(name="score odd fp32", op="score", rows=1531, vocab=32001, dtype="fp32",
             temperature=0.7, masked=0.2, top=5, targets=True),
        # a teacher's lists of 64 for a micro-batch, at the distillation's temperature
        dict(name="score teacher lists", op="score", rows=4096, vocab=50304, dtype="fp16",
             temperature=2.0, masked=0.0, top=64, targets=False),
        # a scored micro-batch of the 8B workload, a prompt's positions without a target
        dict(name="score large", op="score", rows=8192, vocab=128256, dtype="bf16",
             temperature=1.0, masked=0.1, top=20, targets=True),
        # a policy's entropy bonus, small: the 10.5M-parameter workload's 512 positions
        dict(name="bonus small", op="bonus", rows=512, vocab=8192, dtype="bf16",
             temperature=1.0, masked=0.12, targets=True),
        # the same for a rollout's micro-batch of the 8B workload
        dict(name="bonus rollout", op="bonus", rows=2048, vocab=128256, dtype="bf16",
             temperature=1.0, masked=0.3, targets=True),
        # the few tokens of a decoding step: latency again
        dict(name="route few tokens", op="route", rows=7, experts=64, dtype="bf16", score="softmax",
             top=6, groups=1, top_groups=1, best=1, bias=False, renormalise=False, scale=1.0,
             masked=0.0, train=False),
        # a long prompt, the plainest router
        dict(name="route prompt", op="route", rows=131072, experts=128, dtype="bf16",
             score="softmax", top=8, groups=1, top_groups=1, best=1, bias=False, renormalise=True,
             scale=1.0, masked=0.0, train=False),
        # a training micro-batch, balanced by losses, an odd number of experts, fp32 logits
        dict(name="router by losses", op="router", rows=4093, experts=60, dtype="fp32",
             score="softmax", top=4, groups=1, top_groups=1, best=1, bias=False, renormalise=False,
             scale=1.0, masked=0.1, train=True),
        # a large one, balanced by a bias, four of eight groups of experts
        dict(name="router by bias", op="router", rows=65536, experts=256, dtype="bf16",
             score="sigmoid", top=8, groups=8, top_groups=4, best=2, bias=True, renormalise=True,
             scale=2.5, masked=0.05, train=True),
    ]


def _spread(rng, low, high):
    return int(round(low * math.exp(math.log(high / low) * rng.random())))


def draw(rng):
    op = rng.choice(["score", "score", "score", "bonus", "bonus", "route", "route", "router",
                     "router"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    masked = round(rng.choice([0.0, 0.4 * rng.random()]), 3)
    if op in ("score", "bonus"):
        vocab = rng.choice([8192, 50304, 128256, _spread(rng, 500, 140000),
                            _spread(rng, 500, 140000)])
        most = max(2, int(8192 * 128256 * 2 / BYTES[dtype] / vocab / 2))
        case = dict(op=op, rows=_spread(rng, 1, min(16384, most)), vocab=vocab, dtype=dtype,
                    temperature=rng.choice([1.0, 1.0, 0.7, 2.0]), masked=masked,
                    targets=masked > 0.0 or rng.random() < 0.7)
        if op == "score":
            case["top"] = rng.choice([0, 1, 5, 20, _spread(rng, 1, 128), _spread(rng, 1, 128)])
        return case
    score = rng.choice(["softmax", "sigmoid"])
    experts = rng.choice([8, 60, 64, 128, 256, _spread(rng, 4, 512)])
    groups = rng.choice([1, 1] + [g for g in (2, 4, 8) if experts % g == 0 and experts // g >= 4])
    keep = 1 if groups == 1 else rng.randrange(1, groups + 1)
    top = min(_spread(rng, 1, 16), experts // groups * keep)
    return dict(op=op, rows=_spread(rng, 1, 32768), experts=experts, dtype=dtype, score=score,
                top=top, groups=groups, top_groups=keep, best=rng.choice([1, 2]),
                bias=rng.random() < 0.6, renormalise=rng.random() < 0.6,
                scale=rng.choice([1.0, 2.5]), masked=masked,
                train=op == "router" or rng.random() < 0.3)


# --- inputs ----------------------------------------------------------------------------------


def prepare(case, seed):
    """Logits with the spread of trained models', and the buffers that a program keeps for results.
    Vocabularies: a target that stands out by a few units over normally distributed logits.
    Routers: some experts liked more than others, and the bias that has come to balance them."""
    width = case.get("vocab") or case["experts"]
    rows, t = case["rows"], TYPES[case["dtype"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + width * 31 + rows)
    cuda = dict(device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, **cuda)

    gone = torch.rand(rows, generator=g, **cuda) < case["masked"]
    x = torch.randn(rows, width, generator=g, dtype=t, device="cuda")
    st = dict(case=case, x=x, scale=torch.full((1,), 1024.0, **cuda))
    if case["op"] in ("score", "bonus"):
        x.mul_(2.0)
        targets = torch.randint(width, (rows,), generator=g, **cuda)
        x.scatter_add_(1, targets[:, None], (6.0 + 2.0 * normal(rows, 1)).to(t))
        st["targets"] = torch.where(gone, -100, targets) if case["targets"] else None
        st["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        for name in ("logp", "lse", "entropy"):
            st[name] = torch.empty(rows, **cuda)
        if case["op"] == "score":
            k = case["top"]
            st["top_ids"] = torch.empty(rows, k, dtype=torch.int64, device="cuda")
            st["top_logp"] = torch.empty(rows, k, **cuda)
            st["top_values"] = torch.empty(rows, k, **cuda)
        else:
            st["dlogp"] = normal(rows)
            st["dentropy"] = -0.01 * (0.5 + torch.rand(rows, generator=g, **cuda))
            st["count"] = (rows - gone.sum() * int(case["targets"])).clamp(min=1).view(1)
            st["dx"] = torch.empty_like(x)
        return st
    liked = 0.5 * normal(width)
    x.add_(liked.to(t))
    st["mask"] = ~gone if case["masked"] else None
    st["bias"] = (torch.round(-100.0 * liked + 10.0 * normal(width)) * SPEED if case["bias"]
                  else None)
    k = case["top"]
    st["weights"] = torch.empty(rows, k, **cuda)
    st["ids"] = torch.empty(rows, k, dtype=torch.int64, device="cuda")
    if case["train"]:
        st["load"] = torch.empty(width + 1, dtype=torch.int64, device="cuda")
        st["share"] = torch.empty(width, **cuda)
        st["aux"] = torch.empty(2, **cuda)
        st["workspace"] = torch.zeros(4 << 20, dtype=torch.uint8, device="cuda")
    if case["op"] == "router":
        st["dweights"] = normal(rows, k)
        st["dx"] = torch.empty_like(x)
        st["moved"] = torch.empty(width, **cuda) if case["bias"] else None
    return st


# --- the plain forms: elementary operations, 32 bits; 64 for the sums over a row and what comes of
# --- them, and for an expert's score, which lies next to others' ------------------------------


def _order(v):
    """Whole numbers that order fp32 values as they are (-0 and 0 alike)."""
    i = (v + 0.0).view(torch.int32)
    return (i ^ ((i >> 31) & 0x7FFFFFFF)).long()


def _plain_scores(st):
    case, x = st["case"], st["x"]
    z = x.float() / case["temperature"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, dtype=torch.float64)
    lse = m[:, 0].double() + torch.log(s)
    e *= z - m
    entropy = torch.log(s) - e.sum(1, dtype=torch.float64) / s
    del e
    live = torch.ones_like(lse, dtype=torch.bool) if st["targets"] is None else st["targets"] >= 0
    out = dict(lse=torch.where(live, lse, 0.0).float(),
               entropy=torch.where(live, entropy, 0.0).float())
    lp = None
    if st["targets"] is not None:
        zt = z.gather(1, st["targets"].clamp(min=0)[:, None])[:, 0].double()
        lp = torch.where(live, zt - lse, 0.0)
        out["logp"] = lp.float()
    return out, z, lse, entropy, lp, live


def _plain_score(st):
    x, k = st["x"], st["case"]["top"]
    out, z, lse, _, _, live = _plain_scores(st)
    del z
    if k:
        width = x.shape[1]
        key = _order(x.float()) << 32
        key += torch.arange(width - 1, -1, -1, device="cuda")
        best = torch.topk(key, min(k, width), dim=1, sorted=True).values
        del key
        ids = width - 1 - (best & 0xFFFFFFFF)
        if k > width:
            ids = torch.nn.functional.pad(ids, (0, k - width), value=-1)
        v = x.gather(1, ids.clamp(min=0)).float()
        ids = torch.where(live[:, None] & (ids >= 0) & (v > -math.inf), ids, -1)
        v = torch.where(ids >= 0, v, -math.inf)
        logp = (v / st["case"]["temperature"]).double() - lse[:, None]
        out.update(top_ids=ids, top_values=v, top_logp=logp.float())
    return out


def _plain_bonus(st):
    out, z, lse, entropy, lp, live = _plain_scores(st)
    c = st["scale"].double() / st["count"] / st["case"]["temperature"]
    a = torch.where(live, c * st["dlogp"], 0.0)
    b = torch.where(live, c * st["dentropy"], 0.0)
    z -= lse[:, None].float()               # log q
    if lp is None:
        a = torch.zeros_like(a)
    rest = (a + b * entropy).float()[:, None]
    d = torch.exp(z) * -(z * b.float()[:, None] + rest)
    if lp is not None:
        t = (a * -torch.expm1(lp) - b * torch.exp(lp) * (lp + entropy)).float()
        d.scatter_(1, st["targets"].clamp(min=0)[:, None], torch.where(live, t, 0.0)[:, None])
    out["dx"] = d.to(st["x"].dtype)
    return out


def _expert_scores(st):
    z = st["x"].double()
    if st["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z)), None
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    return e / total, m[:, 0] + torch.log(total[:, 0])


def _plain_route(st):
    case, x = st["case"], st["x"]
    rows, experts = x.shape
    k, live = case["top"], st["mask"]
    if live is None:
        live = torch.ones(rows, dtype=torch.bool, device="cuda")
    s, lse = _expert_scores(st)
    c = s if st["bias"] is None else s + st["bias"].double()
    if case["groups"] > 1:
        per = c.view(rows, case["groups"], -1).sort(dim=2, descending=True).values
        group = per[:, :, :case["best"]].sum(2)
        order = group.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(group, dtype=torch.bool)
        keep.scatter_(1, order[:, :case["top_groups"]], True)
        keep = keep[:, :, None].expand(-1, -1, experts // case["groups"]).reshape(rows, experts)
        c = torch.where(keep, c, -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    total = w.sum(1, keepdim=True) + TINY
    if case["renormalise"]:
        w = w / total
    out = dict(ids=torch.where(live[:, None], ids, -1),
               weights=torch.where(live[:, None], w * case["scale"], 0.0).float())
    if case["train"]:
        n = live.sum().clamp(min=1)
        load = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
        chosen = torch.zeros(rows, experts, dtype=torch.int64, device="cuda")
        chosen.scatter_(1, ids, 1)
        load[:experts] = (chosen * live[:, None]).sum(0)
        load[experts] = live.sum()
        p = s if lse is not None else s / s.sum(1, keepdim=True)
        share = torch.where(live[:, None], p, 0.0).sum(0) / n
        balance = (load[:experts] * share).sum() * experts / (k * n)
        large = torch.where(live, lse * lse, 0.0).sum() / n if lse is not None else 0.0 * balance
        out.update(load=load, share=share.float(), aux=torch.stack([balance, large]).float())
    return out, s, lse, ids, total, live


def _plain_router(st):
    case = st["case"]
    out, s, lse, ids, total, live = _plain_route(st)
    experts, n = s.shape[1], out["load"][-1].clamp(min=1)
    dw = st["dweights"].double() * case["scale"]
    if case["renormalise"]:
        mean = (dw * s.gather(1, ids)).sum(1, keepdim=True) / total
        dw = (dw - mean) / total
    factor = st["scale"].double() / n
    pull = factor * BALANCE * experts / (case["top"] * n) * out["load"][:experts].double()
    if lse is None:
        p_sum = s.sum(1, keepdim=True)
        ds = (pull - (s * pull).sum(1, keepdim=True) / p_sum) / p_sum
        ds = ds.scatter_add(1, ids, dw)
        dx = ds * s * (1.0 - s)
    else:
        ds = pull.expand_as(s).scatter_add(1, ids, dw)
        dx = s * (ds - (s * ds).sum(1, keepdim=True))
        dx += s * (2.0 * LARGE * factor * lse)[:, None]
    out["dx"] = torch.where(live[:, None], dx, 0.0).to(st["x"].dtype)
    if st["bias"] is not None:
        load = out["load"][:experts]
        out["moved"] = st["bias"] + torch.sign(load.sum() - load * experts).float() * SPEED
    return out


# --- the library's calls ------------------------------------------------------------------


def _own_scores(st):
    import optimizer_step_tensor_amd as mp
    case = st["case"]
    x = mp.logits(st["x"], case["temperature"])
    top = case.get("top", 0) > 0
    logp = st["logp"] if st["targets"] is not None else None
    score = mp.score(logp, st["lse"], st["entropy"], *(
        (st["top_ids"], st["top_logp"], st["top_values"]) if top else ()),
        workspace=st["workspace"])
    mp.mp_token_score(x, st["targets"], score)
    out = dict(lse=st["lse"], entropy=st["entropy"])
    if logp is not None:
        out["logp"] = logp
    if top:
        out.update(top_ids=st["top_ids"], top_logp=st["top_logp"], top_values=st["top_values"])
    if case["op"] == "bonus":
        g = mp.logits_grad(st["dx"], 1.0, dev_scale=st["scale"], dev_count=st["count"])
        dlogp = st["dlogp"] if logp is not None else None
        mp.mp_token_score_grad(x, st["targets"], st["lse"], st["entropy"], dlogp, st["dentropy"], g)
        out["dx"] = st["dx"]
    return out


def _own_route(st):
    import optimizer_step_tensor_amd as mp
    case = st["case"]
    kind = mp.MP_ROUTE_SOFTMAX if case["score"] == "softmax" else mp.MP_ROUTE_SIGMOID
    cfg = mp.route_cfg(case["top"], kind, case["groups"], case["top_groups"], case["best"],
                       case["renormalise"], case["scale"])
    x = mp.logits(st["x"])
    out = dict(ids=st["ids"], weights=st["weights"])
    if case["train"]:
        routed = mp.routed(st["weights"], st["ids"], st["load"], st["share"], st["aux"],
                           workspace=st["workspace"])
        out.update(load=st["load"], share=st["share"], aux=st["aux"])
    else:
        routed = mp.routed(st["weights"], st["ids"])
    mp.mp_route(x, st["bias"], st["mask"], cfg, routed)
    if case["op"] == "router":
        g = mp.logits_grad(st["dx"], 1.0, dev_scale=st["scale"])
        large = LARGE if case["score"] == "softmax" else 0.0
        mp.mp_route_grad(x, st["mask"], cfg, st["ids"], st["dweights"], st["load"], BALANCE, large,
                         g)
        out["dx"] = st["dx"]
        if st["bias"] is not None:
            mp.mp_route_bias_update(st["bias"], st["load"], SPEED, st["moved"])
            out["moved"] = st["moved"]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_scores(state) if op in ("score", "bonus") else _own_route(state)
    if op == "score":
        return _plain_score(state)
    if op == "bonus":
        return _plain_bonus(state)
    return _plain_route(state)[0] if op == "route" else _plain_router(state)


def work(case):
    """Every logit read once and, with a gradient, every gradient written once; the per-row inputs
    and outputs.  Rows that are switched off are not read, their zero gradient is written.  About
    seven operations per logit for the sums, five more per gradient; for an expert about ten."""
    rows, e = case["rows"], BYTES[case["dtype"]]
    if case["op"] in ("score", "bonus"):
        live = rows * (1.0 - (case["masked"] if case["targets"] else 0.0))
        n = live * case["vocab"]
        per_row = 8 + (8 + 4 if case["targets"] else 0) + 16 * case.get("top", 0)
        grad = case["op"] == "bonus"
        return dict(bytes=n * e + rows * per_row + (rows * (case["vocab"] * e + 8) if grad else 0),
                    flops=n * (12 if grad else 7))
    experts, k = case["experts"], case["top"]
    live = rows * (1.0 - case["masked"])
    n, per_row = live * experts, 12 * k + (1 if case["masked"] else 0)
    if case["op"] == "router":
        return dict(bytes=n * e + rows * (per_row + 4 * k + experts * e) + 20 * experts,
                    flops=20 * n)
    return dict(bytes=n * e + rows * per_row + (12 * experts if case["train"] else 0), flops=10 * n)


# --- from the definitions, in 64 bits -----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_scores(case, st) if case["op"] in ("score", "bonus") else _exact_route(case, st)


def _exact_scores(case, st):
    T, x, targets = case["temperature"], st["x"], st["targets"]
    rows, vocab = x.shape
    step = max(1, (1 << 27) // vocab)
    parts = []
    for r in range(0, rows, step):
        b = slice(r, min(r + step, rows))
        z = x[b].double() / T
        logq = z - torch.logsumexp(z, 1, keepdim=True)
        q = logq.exp()
        h = -(q * logq).sum(1)
        off = torch.zeros_like(h, dtype=torch.bool) if targets is None else targets[b] < 0
        got = dict(lse=(z - logq)[:, 0].masked_fill(off, 0.0), entropy=h.masked_fill(off, 0.0))
        if targets is not None:
            t = targets[b].clamp(min=0)[:, None]
            got["logp"] = logq.gather(1, t)[:, 0].masked_fill(off, 0.0)
        if case.get("top"):
            v, i = torch.sort(x[b].float(), dim=1, descending=True, stable=True)
            short = max(0, case["top"] - vocab)
            gone = off[:, None] | torch.zeros_like(i[:, :case["top"]], dtype=torch.bool)

            def listed_(a, fill):
                a = a[:, :case["top"]].masked_fill(gone, fill)
                return torch.nn.functional.pad(a, (0, short), value=fill)

            got.update(top_ids=listed_(i, -1), top_values=listed_(v.double(), -math.inf),
                       top_logp=listed_(logq.gather(1, i[:, :case["top"]]), -math.inf))
        if case["op"] == "bonus":
            # d lp_t / dz_j = [j = t] - q_j;  d H / dz_j = -q_j (log q_j + H)
            c = float(st["scale"][0]) / int(st["count"][0]) / T
            d = -q * (logq + h[:, None]) * st["dentropy"][b].double()[:, None]
            if targets is not None:
                a = st["dlogp"][b].double()[:, None]
                d -= a * q
                d.scatter_add_(1, t, a)
            got["dx"] = d.mul_(c).masked_fill_(off[:, None], 0.0)
        parts.append(got)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_route(case, st):
    """The gradient by automatic differentiation of the definitions."""
    x = st["x"].double().requires_grad_(case["op"] == "router")
    rows, experts = x.shape
    k, mask = case["top"], st["mask"]
    softmax = case["score"] == "softmax"
    s = torch.softmax(x, 1) if softmax else torch.sigmoid(x)
    with torch.no_grad():
        c = s.clone() if st["bias"] is None else s + st["bias"].double()
        if case["groups"] > 1:
            width = experts // case["groups"]
            top = torch.topk(c.view(rows, -1, width), min(case["best"], width), dim=2).values.sum(2)
            worst = torch.argsort(top, dim=1, descending=True, stable=True)[:, case["top_groups"]:]
            cut = torch.zeros_like(top, dtype=torch.bool).scatter_(1, worst, True)
            c[cut.repeat_interleave(width, 1)] = -math.inf
        ids = torch.argsort(c, dim=1, descending=True, stable=True)[:, :k]
    w = s.gather(1, ids)
    if case["renormalise"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    w = w * case["scale"]
    if mask is not None:
        w = w * mask[:, None]
        ids = ids.masked_fill(~mask[:, None], -1)
    out = dict(ids=ids, weights=w)
    if not case["train"]:
        return out
    live = torch.arange(rows, device="cuda") if mask is None else torch.nonzero(mask)[:, 0]
    n = max(1, len(live))
    load = torch.bincount(ids[live].reshape(-1), minlength=experts)
    p = (s if softmax else s / s.sum(1, keepdim=True))[live]
    share = p.sum(0) / n
    balance = experts * (load.double() / (k * n) * share).sum()
    large = torch.logsumexp(x, 1)[live].square().sum() / n if softmax else 0.0 * balance
    out.update(load=torch.cat([load, load.new_full((1,), n)]), share=share,
               aux=torch.stack([balance, large]))
    out["load"][-1] = len(live)
    if case["op"] == "router":
        loss = (w * st["dweights"].double()).sum()
        loss = loss + float(st["scale"][0]) * (BALANCE * balance + LARGE * large)
        out["dx"], = torch.autograd.grad(loss, x)
        if st["bias"] is not None:
            out["moved"] = st["bias"].double() + SPEED * torch.sign(load.sum() / experts - load)
    return {name: v.detach() for name, v in out.items()}
