"""Cases, plain forms and 64-bit definitions of the operators around a head that is trained, adapted and served.

* ``clip``    the norm of many gradients taken together (``max_norm`` 0: that alone), and their copies scaled to at most max_norm
* ``step``    an AdamW step by the gradients clipped so
* ``verify``  drafted tokens accepted or refused by the target's probabilities, from given random numbers
* ``adapt``   low-rank adapters of many requests added to the output of a projection that they share

Definitions:
  norm = sqrt(sum g^2), or max |g|;  factor = min(1, max_norm / (norm + 1e-6)).
  verify: p = softmax(target / T), q = softmax(draft / T) (without draft logits: 1 at the drafted token d); a request's
    drafted tokens are accepted as long as u q(d) < p(d); the first that is not gives way to one drawn from max(p - q, 0),
    and behind the last accepted one another is drawn from p: the lowest column whose running sum exceeds u times the whole.
    T = 0: accepted as long as d is the target's first largest, and that is what is drawn.
    Weights 2^((z - max z) log2(e) / T) and the differences are whole numbers of 2^-43, so that their sums have one value
    in any order, and with them every token.
  adapt: y_t + scale_a B_a (A_a x_t) with a = index[t]; -1: y_t.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
UNIT = 2.0 ** 43
LOG2E = 1.4426950408889634


# ---- cases -------------------------------------------------------------------------------------------------
def listed():
    return [
        # the norm of a model's small gradients, for a log line
        dict(name="norm-small", op="clip", tensors=64, elements=300000, dtype="fp32", norm=2.0, max_norm=0.0),
        # a model's gradients in 32 bits, many of them small
        dict(name="clip-fp32", op="clip", tensors=300, elements=131072000, dtype="fp32", norm=2.0, max_norm=1.0),
        # an lm_head's and its neighbours' in bf16
        dict(name="clip-head", op="clip", tensors=8, elements=525340672, dtype="bf16", norm=2.0, max_norm=1.0),
        # a clipped step of the same kind
        dict(name="step-clipped", op="step", tensors=24, elements=131072000, dtype="bf16", max_norm=1.0),
        # one request with four drafted tokens
        dict(name="verify-1", op="verify", requests=1, drafts=4, ragged=False, v=128256, dtype="bf16", t=1.0, q=True),
        # a batch of requests of their own temperatures, some greedy, with up to eight
        dict(name="verify-64", op="verify", requests=64, drafts=8, ragged=True, v=32000, dtype="fp32", t=-1.0, q=True),
        # tokens looked up in the prompt, which have no probabilities; odd vocabulary
        dict(name="verify-lookup", op="verify", requests=33, drafts=16, ragged=True, v=40961, dtype="bf16", t=0.7, q=False),
        # a large batch
        dict(name="verify-256", op="verify", requests=256, drafts=4, ragged=False, v=128256, dtype="bf16", t=1.0, q=True),
        # the next token of one request with an adapter on the lm_head
        dict(name="adapt-1", op="adapt", tokens=1, k=4096, n=128256, rank=16, adapters=1, runs=1, dtype="bf16"),
        # one token of each of 64 requests, each with its own
        dict(name="adapt-64", op="adapt", tokens=64, k=4096, n=128256, rank=16, adapters=64, runs=64, dtype="bf16"),
        # packed prompts of different adapters, ragged, some without
        dict(name="adapt-333", op="adapt", tokens=333, k=2048, n=40961, rank=64, adapters=5, runs=9, dtype="fp32"),
        # a batch of prompts
        dict(name="adapt-4096", op="adapt", tokens=4096, k=4096, n=128256, rank=16, adapters=8, runs=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["clip", "clip", "step", "verify", "verify", "verify", "adapt", "adapt", "adapt"])
    if op in ("clip", "step"):
        c = dict(op=op, tensors=_log(rng, 1, 500), elements=_log(rng, 20000, 100000000), dtype=rng.choice(["bf16", "fp32"]), max_norm=1.0)
        return c if op == "step" else c | dict(norm=rng.choice([2.0, 2.0, math.inf]), max_norm=rng.choice([0.0, 1.0, 1e9]))
    if op == "verify":
        dtype = rng.choice(["bf16", "fp32"])
        return dict(op=op, requests=_log(rng, 1, 128), drafts=rng.randint(1, 4), ragged=rng.random() < 0.6, v=_log(rng, 1000, 128256), dtype=dtype,
                    t=rng.choice([0.0, 0.5, 1.0, 1.0, 1.3, -1.0]), q=rng.random() < 0.7)
    tokens, adapters = _log(rng, 1, 4096), _log(rng, 1, 64)
    return dict(op=op, tokens=tokens, k=8 * _log(rng, 16, 512), n=_log(rng, 1000, 128256 if tokens < 2048 else 64000), rank=8 * rng.randint(1, 16 if adapters < 9 else 2),
                adapters=adapters, runs=rng.randint(1, tokens), dtype=rng.choice(["bf16", "fp32"]) if tokens < 1024 else "bf16")


def _sizes(case):
    """The tensors' sizes: many small ones, few that hold most of the elements, odd ones among them."""
    r = random.Random(case["tensors"] * 1000003 + case["elements"])
    w = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    top = sum(w)
    return [max(1, int(case["elements"] * x / top)) for x in w]


def _counts(case):
    """Each request's number of drafted tokens."""
    r = random.Random(case["requests"] * 7919 + case["drafts"] * 31 + case["v"])
    return [r.randint(0, case["drafts"]) if case["ragged"] else case["drafts"] for _ in range(case["requests"])]


def _runs(case):
    """(adapter, first token) of runs of neighbouring tokens; one in eight has none. Decoding requests come one by one."""
    r = random.Random(case["tokens"] * 104729 + case["adapters"] * 13 + case["runs"])
    if case["runs"] == case["tokens"] == case["adapters"]:
        return list(enumerate(range(case["tokens"])))
    at = [0] + sorted(r.sample(range(1, case["tokens"]), case["runs"] - 1))
    return [(r.randrange(case["adapters"]) if i == 0 or r.random() > 0.125 else -1, t) for i, t in enumerate(at)]


# ---- inputs ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt, s = case["op"], DT[case["dtype"]], dict(case=case)
    normal = lambda shape, std: torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)  # noqa: E731
    if op in ("clip", "step"):
        sizes = _sizes(case)
        starts = [0]  # the tensors start on 256 bytes, as an allocator's do
        for n in sizes:
            starts.append(starts[-1] + -(-n // 128) * 128)
        cut = lambda flat: [flat[i:i + n] for i, n in zip(starts, sizes)]  # noqa: E731
        live = torch.zeros(starts[-1], dtype=torch.bool, device="cuda")
        [x.fill_(True) for x in cut(live)]
        flat = {"g": normal(starts[-1], 1e-3).mul_(live).to(dt)}
        if op == "clip":
            flat["out"] = torch.zeros_like(flat["g"])
        else:
            flat["p"], flat["m"] = normal(starts[-1], 0.02).mul_(live).to(dt), normal(starts[-1], 3e-4).mul_(live)
            flat["v"] = normal(starts[-1], 3e-4).square_().add_(1e-10).mul_(live)
            s["t"] = 10  # steps taken
        s.update(flat=flat, **{x: cut(flat[x]) for x in flat})
        # the elements are so many that their norm exceeds max_norm only where it is scaled up to do so
        if case["max_norm"] == 1.0:
            flat["g"].mul_(3.0 / (1e-3 * math.sqrt(sum(sizes))))
    elif op == "verify":
        counts, v = _counts(case), case["v"]
        n, b = sum(counts), len(counts)
        ends = torch.tensor([0] + counts).cumsum(0)
        s["offsets"] = ends.cuda() if case["ragged"] else None
        z = normal((n + b, v), 3.0).to(dt)  # a deviation that trained models have
        row = torch.cat([torch.arange(int(ends[i]), int(ends[i + 1])) + i for i in range(b)]).cuda()
        s["target"], s["draft"] = z, None
        from_ = z[row].float()
        if case["q"]:  # a drafter that is near its target
            s["draft"] = (from_ + normal((n, v), 0.7)).to(dt)
            from_ = s["draft"].float()
        t = case["t"]
        if t < 0:
            s["t"] = torch.tensor([0.0, 0.7, 1.0, 1.3], device="cuda")[torch.arange(b, device="cuda") % 4]
        else:
            s["t"] = t
        each = s["t"][torch.repeat_interleave(torch.tensor(counts)).cuda()] if t < 0 else torch.full((n,), t, device="cuda")
        likely = from_.argmax(1) if n else torch.zeros(0, dtype=torch.int64, device="cuda")  # what a greedy drafter proposes
        from_ = torch.softmax(from_ / torch.where(each > 0, each, 1.0)[:, None], 1)
        s["tokens"] = torch.where(each > 0, torch.multinomial(from_, 1, generator=gen)[:, 0], likely) if n else likely
        s["u"], s["u_draw"] = torch.rand(n, device="cuda", generator=gen), torch.rand(b, device="cuda", generator=gen)
    else:
        t, k, n, r, na = (case[x] for x in ("tokens", "k", "n", "rank", "adapters"))
        s["x"] = normal((t, k), 1.0).to(torch.bfloat16)
        s["a"] = normal((na, r, k), 1 / math.sqrt(k)).to(torch.bfloat16)
        s["b"] = normal((na, n, r), 0.3 / math.sqrt(r)).to(torch.bfloat16)
        s["scales"] = torch.rand(na, device="cuda", generator=gen) + 0.5
        s["y"] = normal((t, n), 1.0).to(dt)
        runs = _runs(case)
        index = torch.empty(t, dtype=torch.int64)
        for i, (a, at) in enumerate(runs):
            index[at:] = a
        s["index"] = index.cuda()
    return s


# ---- plain forms -------------------------------------------------------------------------------------------
def _norm(flat, norm):
    return flat.abs().amax().float() if norm == math.inf else flat.double().square().sum().sqrt().float()


def _weights(z, t):
    """Weights in 32 bits relative to the row's largest, and as whole numbers (held in 64 bits, exact)."""
    c = (LOG2E / torch.where(t > 0, t, 1.0).double()).float()[:, None]
    e = torch.exp2((z - z.amax(1, keepdim=True)) * c)
    return e, torch.round(e.double() * UNIT)


def _first_largest(z):
    return torch.where(z == z.amax(1, keepdim=True), torch.arange(z.shape[1], device=z.device), z.shape[1]).amin(1)


def _verify(s):
    z, tokens, u, u_draw, dev = s["target"].float(), s["tokens"], s["u"], s["u_draw"], s["u"].device
    b, n = u_draw.shape[0], tokens.shape[0]
    kmax = s["case"]["drafts"]
    ends = s["offsets"] if s["offsets"] is not None else torch.arange(b + 1, device=dev) * kmax
    t = s["t"] if isinstance(s["t"], torch.Tensor) else torch.full((b,), s["t"], device=dev)
    of_draft = torch.searchsorted(ends, torch.arange(n, device=dev), right=True) - 1  # its request
    rows = torch.arange(n, device=dev) + of_draft
    of_row = torch.searchsorted(ends + torch.arange(b + 1, device=dev), torch.arange(n + b, device=dev), right=True) - 1
    e, w = _weights(z, t[of_row])
    total = w.to(torch.int64).sum(1).double() / UNIT
    p = e[rows].gather(1, tokens[:, None])[:, 0].double() / total[rows]
    q = torch.ones_like(p)
    if s["draft"] is not None:
        eq, wq = _weights(s["draft"].float(), t[of_draft])
        total_q = wq.to(torch.int64).sum(1).double() / UNIT
        q = eq.gather(1, tokens[:, None])[:, 0].double() / total_q
    best, greedy = _first_largest(z), t == 0
    hit = torch.where(greedy[of_draft], tokens == best[rows], u.double() * q < p)
    prob = torch.where(greedy[of_draft], hit.double(), torch.where(q > 0, p / q, (p > 0).double()).clamp(max=1.0))
    at = ends[:-1, None] + torch.arange(kmax, device=dev)
    inside = at < ends[1:, None]
    at = torch.where(inside, at, 0)
    pad = lambda x: torch.nn.functional.pad(x, (0, 1))[at]  # noqa: E731 (one more, for no drafts at all)
    accepted = (pad(hit) & inside).to(torch.int64).cumprod(1).sum(1)
    row = ends[:-1] + torch.arange(b, device=dev) + accepted
    left = accepted < ends[1:] - ends[:-1]  # one was refused
    inv = lambda d: (1.0 / d).float()[:, None]  # noqa: E731
    r = e[row] * inv(total[row])
    if n:
        refused = torch.where(left, ends[:-1] + accepted, 0)
        if s["draft"] is not None:
            other = eq[refused] * inv(total_q[refused])
        else:
            other = torch.zeros_like(r).scatter_(1, tokens[refused][:, None], 1.0)
        r2 = torch.where(left[:, None], (r - other).clamp_min(0.0), r)
        r = torch.where((r2 * UNIT).amax(1, keepdim=True) > 0.5, r2, r)
    run = torch.round(r.double() * UNIT).to(torch.int64).cumsum(1)
    want = torch.minimum((u_draw.double() * run[:, -1].double()).floor().to(torch.int64), run[:, -1] - 1)
    drawn = torch.where(greedy, best[row], (run <= want[:, None]).sum(1))
    col = torch.arange(kmax + 1, device=dev)
    known = torch.nn.functional.pad(torch.where(inside, pad(tokens), -1), (0, 1), value=-1)
    out = torch.where(col < accepted[:, None], known, torch.where(col == accepted[:, None], drawn[:, None], -1))
    return {"tokens": out, "accepted": accepted, "accept_prob": prob.float()}


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    op = c["op"]
    if op == "clip":
        flat = torch.cat([g.float() for g in s["g"]])
        norm = _norm(flat, c["norm"])
        if not c["max_norm"]:
            return {"norm": norm}
        new = flat * (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        [o.copy_(x) for o, x in zip(s["out"], new.split([g.numel() for g in s["g"]]))]
        return {"norm": norm, "out": s["flat"]["out"]}
    if op == "step":
        s["t"] += 1
        cat = lambda xs: torch.cat([x.float() for x in xs])  # noqa: E731
        g = cat(s["g"])
        norm = _norm(g, 2.0)
        g = g * (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        m, v = cat(s["m"]) * BETA1 + g * (1 - BETA1), cat(s["v"]) * BETA2 + g * (1 - BETA2) * g
        den = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** s["t"])) + EPS
        p = cat(s["p"]) * (1 - LR * DECAY) - (m / den) * (LR / (1 - BETA1 ** s["t"]))
        sizes = [x.numel() for x in s["g"]]
        [to.copy_(x) for new, olds in ((p, s["p"]), (m, s["m"]), (v, s["v"])) for x, to in zip(new.split(sizes), olds)]
        return {"norm": norm, "p": s["flat"]["p"], "m": s["flat"]["m"], "v": s["flat"]["v"]}
    if op == "verify":
        return _verify(s)
    na, r = c["adapters"], c["rank"]
    mine = torch.arange(na, device=s["x"].device) == s["index"][:, None]  # [tokens, adapters]
    low = (s["x"].float() @ s["a"].float().view(na * r, -1).T).view(-1, na, r) * s["scales"][:, None]
    low = (low * mine[:, :, None]).view(-1, na * r)
    return (s["y"].float() + low @ s["b"].float().transpose(1, 2).reshape(na * r, -1)).to(s["y"].dtype)


# ---- the framework's calls ---------------------------------------------------------------------------------
def _own(s):
    import lm_head_jsd_gb300 as fl

    c = s["case"]
    op = c["op"]
    if op == "clip":
        if not c["max_norm"]:
            return {"norm": fl.grad_norm(s["g"], norm_type=c["norm"])}
        return {"norm": fl.clip_grads(s["g"], c["max_norm"], norm_type=c["norm"], out=s["out"]), "out": s["flat"]["out"]}
    if op == "step":
        if "plan" not in s:
            s["plan"] = fl.AdamW(s["p"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, exp_avg=s["m"], exp_avg_sq=s["v"], step=s["t"])
        s["plan"].step(s["g"], max_norm=c["max_norm"])
        return {"norm": s["plan"].grad_norm, "p": s["flat"]["p"], "m": s["flat"]["m"], "v": s["flat"]["v"]}
    if op == "verify":
        r = fl.verify_drafts(s["target"], s["tokens"], s["u"], s["u_draw"], draft_logits=s["draft"], offsets=s["offsets"], max_drafts=c["drafts"],
                             temperature=s["t"])
        return {"tokens": r.tokens, "accepted": r.accepted, "accept_prob": r.accept_prob}
    return fl.low_rank_add(s["y"], s["x"], s["a"], s["b"], s["index"], s["scales"])


# ---- the work that cannot be done without ------------------------------------------------------------------
def work(case):
    op, size = case["op"], 4.0 if case["dtype"] == "fp32" else 2.0
    if op == "clip":
        n = sum(_sizes(case))
        return {"bytes": n * size * (2 if case["max_norm"] else 1), "flops": n * (3.0 if case["max_norm"] else 2.0)}
    if op == "step":
        n = sum(_sizes(case))
        return {"bytes": n * (3 * size + 16.0), "flops": 18.0 * n}
    if op == "verify":
        n, b, v = sum(_counts(case)), case["requests"], case["v"]
        rows = n + b + (n if case["q"] else 0)
        return {"bytes": rows * v * size + 16.0 * n + 8.0 * b * (case["drafts"] + 3), "flops": 4.0 * rows * v + 4.0 * b * v}
    t, k, n, r = (case[x] for x in ("tokens", "k", "n", "rank"))
    runs = _runs(case)
    ends = [at for _, at in runs[1:]] + [t]
    used, live = {a for a, _ in runs if a >= 0}, sum(e - at for (a, at), e in zip(runs, ends) if a >= 0)
    return {"bytes": 2.0 * t * n * size + 2.0 * live * k + 2.0 * len(used) * r * (k + n) + 8.0 * t, "flops": 2.0 * live * r * (k + n) + float(live) * n}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("clip", "step"):
        g = s["flat"]["g"].double()
        norm = g.abs().max() if case.get("norm", 2.0) == math.inf else torch.linalg.vector_norm(g)
        if not case["max_norm"]:
            return {"norm": norm}
        g = g * min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        if op == "clip":
            return {"norm": norm, "out": g}
        t = s["t"] + 1
        m = BETA1 * s["flat"]["m"].double() + (1 - BETA1) * g
        v = BETA2 * s["flat"]["v"].double() + (1 - BETA2) * g * g
        p = s["flat"]["p"].double()
        p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        return {"norm": norm, "p": p, "m": m, "v": v}
    if op == "verify":  # which token a number next to a border gives goes by the weights in 32 bits
        counts, prob, at = _counts(case), [], 0
        for i, n in enumerate(counts):
            t = float(s["t"][i]) if isinstance(s["t"], torch.Tensor) else s["t"]
            for j in range(n):
                z, d = s["target"][at + i].double(), int(s["tokens"][at])
                if t == 0.0:
                    prob.append(float(d == int((z == z.max()).nonzero()[0, 0])))
                else:
                    lp = float(torch.log_softmax(z / t, 0)[d])
                    lq = float(torch.log_softmax(s["draft"][at].double() / t, 0)[d]) if case["q"] else 0.0
                    prob.append(math.exp(min(0.0, lp - lq)))
                at += 1
        return {"tokens": None, "accepted": None, "accept_prob": torch.tensor(prob, dtype=torch.float64)}
    out = s["y"].double()
    for a in range(case["adapters"]):
        rows = (s["index"] == a).nonzero()[:, 0]
        if len(rows):
            out[rows] += float(s["scales"][a]) * (s["x"][rows].double() @ s["a"][a].double().T) @ s["b"][a].double().T
    return out
