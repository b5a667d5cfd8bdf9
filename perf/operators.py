"""Cases, plain forms and 64-bit definitions of the operators around an lm_head.

A model's output layer is scored, kept in 8 bits when it is frozen, trained and stepped. Five operators:

* ``head``       log probabilities of given tokens from hidden states and the lm_head weight, with the entropy
                 of each row and its most likely alternatives; nothing of size tokens x vocabulary is returned
* ``head_grad``  the same with the gradients in the hidden states and the weight
* ``logits``     the same quantities of given logits, with or without the gradient in the logits
* ``fp8``        x . W^T with W in e4m3 and one scale for each 128 x 128 block, x quantised per 1 x 128 block
* ``adamw``      one AdamW step over many tensors, with states in 32 or in 8 bits

Definitions, with z = x . W^T, s = z / T, p = softmax(s):
  lse = log sum_j e^{s_j},  logp = s_y - lse,  entropy = -sum_j p_j log p_j,
  alternatives = the k largest z_j (ties: the lowest index first) with their log probabilities,
  dz_j = (a (1[j = y] - p_j) - b p_j (log p_j + entropy)) / T for upstream gradients a (logp), b (entropy).
A row whose label is -100 has logp 0, entropy 0 and gradient 0; its alternatives are written all the same.
"""
import math
import random

import torch

own = False

IGNORE = -100
BLOCK = 128  # elements of one 8-bit block
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # blocks below it are held as zeros
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1


# ---- cases -------------------------------------------------------------------------------------------------
def listed():
    return [
        # the next token of one sequence, with the eight alternatives that a server returns beside it
        dict(name="head-1", op="head", bt=1, h=4096, v=128256, k=8, t=1.0, ignored=0.0),
        # a few packed answers, scored with the twenty alternatives that a teacher's cache keeps
        dict(name="head-333", op="head", bt=333, h=2048, v=40960, k=20, t=0.7, ignored=0.1),
        # a batch of prompts, scored
        dict(name="head-4096", op="head", bt=4096, h=4096, v=128256, k=8, t=1.0, ignored=0.05),
        # a policy-gradient step on few, ragged tokens
        dict(name="head-grad-1000", op="head_grad", bt=1000, h=4096, v=32000, t=1.0, ignored=0.1),
        # the same on a whole batch
        dict(name="head-grad-4096", op="head_grad", bt=4096, h=4096, v=128256, t=1.0, ignored=0.05),
        # one row of logits that a model has already produced
        dict(name="logits-1", op="logits", rows=1, v=128256, dtype="fp32", k=8, t=1.0, ignored=0.0, grad=False),
        # a batch of rows, odd vocabulary, with the gradient in the logits
        dict(name="logits-grad-2047", op="logits", rows=2047, v=128255, dtype="bf16", k=0, t=1.0, ignored=0.1, grad=True),
        # a frozen teacher's lm_head in 8 bits, one token
        dict(name="fp8-1", op="fp8", m=1, k=4096, n=128256),
        # the same over a batch of prompts
        dict(name="fp8-4096", op="fp8", m=4096, k=4096, n=128256),
        # the small tensors of a model: norms, biases, adapters
        dict(name="adamw-small", op="adamw", tensors=64, elements=300000, param="fp32", bits=32, master=False),
        # an lm_head and its neighbours, held in bf16
        dict(name="adamw-head", op="adamw", tensors=8, elements=525340672, param="bf16", bits=32, master=False),
        # the same in 8-bit states, with 32-bit master weights
        dict(name="adamw-8bit", op="adamw", tensors=24, elements=131072000, param="bf16", bits=8, master=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["head", "head", "head_grad", "head_grad", "logits", "logits", "fp8", "fp8", "adamw", "adamw"])
    t = rng.choice([0.5, 0.7, 1.0, 1.0, 1.3])
    ignored = rng.choice([0.0, 0.05, 0.3])
    if op in ("head", "head_grad"):
        c = dict(op=op, bt=_log(rng, 1, 4096), h=8 * _log(rng, 16, 512), v=_log(rng, 1000, 128256), t=t, ignored=ignored)
        if op == "head":
            c["k"] = rng.choice([0, 1, 3, 5, 8, 20, 32])
        return c
    if op == "logits":
        dtype = rng.choice(["bf16", "fp32"])
        return dict(op=op, rows=_log(rng, 1, 2047 if dtype == "bf16" else 1023), v=_log(rng, 1000, 128255), dtype=dtype,
                    k=rng.choice([0, 1, 8, 20]), t=t, ignored=ignored, grad=rng.random() < 0.5)
    if op == "fp8":
        return dict(op=op, m=_log(rng, 1, 4096), k=8 * _log(rng, 16, 512), n=_log(rng, 1000, 128256))
    bits = rng.choice([32, 8])
    return dict(op=op, tensors=_log(rng, 1, 300), elements=_log(rng, 20000, 130000000), param=rng.choice(["bf16", "fp32"]), bits=bits,
                master=False) if rng.random() < 0.6 else dict(op=op, tensors=_log(rng, 1, 300), elements=_log(rng, 20000, 130000000),
                                                             param="bf16", bits=bits, master=True)


def _sizes(case):
    """The tensors' sizes: many small ones, few that hold most of the elements, odd ones among them."""
    r = random.Random(case["tensors"] * 1000003 + case["elements"])
    w = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    top = sum(w)
    return [max(1, int(case["elements"] * x / top)) for x in w]


# ---- inputs ------------------------------------------------------------------------------------------------
def _normal(shape, unit, std, most, gen):
    """Normal values on a grid of `unit`, so that the sums of their products are exact in 32 bits in any order: which of
    two alternatives comes first is then a matter of the inputs, not of the order in which a product is summed."""
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return x.div_(unit).round_().clamp_(-most, most).mul_(unit).to(torch.bfloat16)


def _labels(n, v, ignored, gen):
    y = torch.randint(0, v, (n,), device="cuda", generator=gen)
    return torch.where(torch.rand(n, device="cuda", generator=gen) < ignored, torch.full_like(y, IGNORE), y)


def _quantise(x):
    """e4m3 codes and scales of [rows x 128] blocks: amax / 448, the value times 448 / amax rounded to the nearest."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    return (x * (E4M3_MAX / amax)).to(torch.float8_e4m3fn), amax / E4M3_MAX


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("head", "head_grad"):
        bt, h, v = case["bt"], case["h"], case["v"]
        s["x"] = _normal((bt, h), 1 / 16, 1.0, 64, gen)
        unit = 2.0 ** round(math.log2(0.375 / math.sqrt(h)))  # logits of a deviation of about 3, as trained models have
        s["w"] = _normal((v, h), unit, 8 * unit, 32, gen)
        s["y"] = _labels(bt, v, case["ignored"], gen)
        if op == "head_grad":
            s["a"] = torch.randn(bt, device="cuda", generator=gen) / bt  # advantages
            s["b"] = torch.full((bt,), -0.01 / bt, device="cuda")  # an entropy bonus
    elif op == "logits":
        rows, v = case["rows"], case["v"]
        s["z"] = (3 * torch.randn(rows, v, device="cuda", generator=gen)).to(DT[case["dtype"]])
        s["y"] = _labels(rows, v, case["ignored"], gen)
        s["a"] = torch.randn(rows, device="cuda", generator=gen) / rows
        s["b"] = torch.full((rows,), -0.01 / rows, device="cuda")
    elif op == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = torch.randn(m, k, device="cuda", generator=gen).to(torch.bfloat16)
        kb, nb, ld = -(-k // BLOCK), -(-n // BLOCK), -(-k // 16) * 16
        w = torch.zeros(nb * BLOCK, kb * BLOCK, device="cuda")
        w[:n, :k].normal_(0.0, 1 / math.sqrt(k), generator=gen)
        q, sc = _quantise(w.view(nb, BLOCK, kb, BLOCK).transpose(1, 2).reshape(nb, kb, BLOCK * BLOCK))
        q = q.view(nb, kb, BLOCK, BLOCK).transpose(1, 2).reshape(nb * BLOCK, kb * BLOCK)
        s["wq"] = q[:n, :ld].contiguous()[:, :k]  # rows a multiple of 16 bytes apart
        s["ws"] = sc.view(nb, kb).contiguous()
    else:
        sizes, pd = _sizes(case), DT[case["param"]]
        ends = [sum(-(-n // BLOCK) for n in sizes[:i + 1]) for i in range(len(sizes))]  # in blocks, for the tensors start on one
        cut = lambda flat: [flat[(e - -(-n // BLOCK)) * BLOCK:][:n] for e, n in zip(ends, sizes)]  # noqa: E731
        rows = lambda flat: [flat[e - -(-n // BLOCK):e] for e, n in zip(ends, sizes)]  # noqa: E731
        live = torch.zeros(ends[-1] * BLOCK, dtype=torch.bool, device="cuda")
        [x.fill_(True) for x in cut(live)]
        rand = lambda std: torch.empty(live.shape[0], device="cuda").normal_(0.0, std, generator=gen).mul_(live)  # noqa: E731
        flat = {"p": rand(0.02), "g": rand(1e-3).to(pd), "m": rand(3e-4), "v": rand(3e-4).abs_().add_(1e-5).mul_(live)}
        if case["master"]:
            flat["master"] = flat["p"]
        flat["p"] = flat["p"].to(pd)
        if case["bits"] == 32:
            flat["v"].square_()
        else:  # the second moment is held as its root
            for x, sc in (("m", "ms"), ("v", "vs")):
                q, c = _quantise(flat[x].view(-1, BLOCK))
                flat[x], flat[sc] = q.reshape(-1), c.reshape(-1).contiguous()
        s.update(flat=flat, t=10)  # t: steps taken
        s.update({x: (rows if x in ("ms", "vs") else cut)(flat[x]) if x in flat else None for x in ("p", "g", "m", "v", "master", "ms", "vs")})
    return s


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


# ---- plain forms -------------------------------------------------------------------------------------------
def _scores(z, y, t, k):
    """Of logits in 32 bits: what the operators return, and what the gradient needs."""
    s = z * (1.0 / t)
    u = s - s.amax(1, keepdim=True)
    e = u.exp()
    d = e.sum(1, keepdim=True)
    logd = d.log()
    valid = y != IGNORE
    at = torch.where(valid, y, 0)[:, None]
    ent = (logd - (e * u).sum(1, keepdim=True) / d)[:, 0]
    out = {"logp": torch.where(valid, (u.gather(1, at) - logd)[:, 0], 0.0), "entropy": torch.where(valid, ent, 0.0)}
    if k:
        bits = z.contiguous().view(torch.int32).to(torch.int64)
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)  # rises with the value
        ids = torch.arange(z.shape[1], device=z.device)
        top = (order * (1 << 32) + ((1 << 32) - 1 - ids)).topk(k, 1).values  # one key for each, so no ties
        out["top_id"] = ((1 << 32) - 1) - (top & 0xFFFFFFFF)
        out["top_logp"] = u.gather(1, out["top_id"]) - logd
    return out, (u, e, d, logd, ent, at, valid)


def _dz(more, a, b, t):
    u, e, d, logd, ent, at, valid = more
    p = e / d
    g = -p * (a[:, None] + b[:, None] * (u - logd + ent[:, None]))
    g.scatter_add_(1, at, a[:, None])
    return torch.where(valid[:, None], g * (1.0 / t), 0.0)


def _wide(q, scales, k):
    """The values of 128 x 128 blocks in 32 bits."""
    n = q.shape[0]
    return q.float() * scales.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _adamw(p, g, m, r2, t):
    """New parameters and states in 32 bits, one rounding to an operation, in this order."""
    m = m * BETA1 + g * (1 - BETA1)
    v = r2 * BETA2 + g * (1 - BETA2) * g
    den = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    return p * (1 - LR * DECAY) - (m / den) * (LR / (1 - BETA1 ** t)), m, v


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    op = c["op"]
    if op in ("head", "head_grad"):
        x, w = s["x"].float(), s["w"].float()
        out, more = _scores(x @ w.T, s["y"], c["t"], c.get("k", 0))
        if op == "head_grad":
            dz = _dz(more, s["a"], s["b"], c["t"])
            out["grad_x"], out["grad_w"] = (dz @ w).to(s["x"].dtype), (dz.T @ x).to(s["w"].dtype)
        return out
    if op == "logits":
        out, more = _scores(s["z"].float(), s["y"], c["t"], c["k"])
        if c["grad"]:
            out["grad_z"] = _dz(more, s["a"], s["b"], c["t"]).to(s["z"].dtype)
        return out
    if op == "fp8":
        x, k = s["x"].float(), c["k"]
        q, sc = _quantise(torch.nn.functional.pad(x, (0, -k % BLOCK)).view(c["m"], -1, BLOCK))
        x = (q.float() * sc).view(c["m"], -1)[:, :k]
        return (x @ _wide(s["wq"], s["ws"], k).T).to(torch.bfloat16)
    s["t"] += 1
    sizes = [p.numel() for p in s["p"]]
    base = s["p"] if s["master"] is None else s["master"]
    if c["bits"] == 32:
        cat = lambda xs: torch.cat([x.float() for x in xs])  # noqa: E731
        p, m, v = _adamw(cat(base), cat(s["g"]), cat(s["m"]), cat(s["v"]), s["t"])
        parts = [(x.split(sizes), to) for x, to in ((p, base), (m, s["m"]), (v, s["v"]))]
    else:
        cat = lambda xs: torch.cat([_blocks(x) for x in xs])  # noqa: E731
        f32 = lambda xs: cat([x.float() for x in xs])  # noqa: E731
        sm, sv = torch.cat(s["ms"])[:, None], torch.cat(s["vs"])[:, None]
        r = f32(s["v"]) * sv
        p, m, v = _adamw(f32(base), f32(s["g"]), f32(s["m"]) * sm, r * r, s["t"])
        (qm, cm), (qr, cr) = _quantise(m), _quantise(v.sqrt())
        rows = [-(-n // BLOCK) for n in sizes]
        back = lambda x: [y.reshape(-1)[:n] for y, n in zip(x.split(rows), sizes)]  # noqa: E731
        parts = [(back(p), base), (back(qm), s["m"]), (back(qr), s["v"]), (cm[:, 0].split(rows), s["ms"]), (cr[:, 0].split(rows), s["vs"])]
    if s["master"] is not None:
        parts.append((parts[0][0], s["p"]))
    [to.copy_(new) for news, olds in parts for new, to in zip(news, olds)]
    return _updated(s)


def _updated(s):
    """All that a step changes: the tensors lie one after the other, each from a block's start."""
    return {x: s["flat"][x] for x in ("p", "master", "m", "v", "ms", "vs") if x in s["flat"]}


# ---- the framework's calls ---------------------------------------------------------------------------------
def _own(s):
    import lm_head_jsd_gb300 as fl

    c = s["case"]
    op = c["op"]
    if op in ("head", "head_grad"):
        if "plan" not in s:
            s["plan"] = fl.FusedLinearLogprobs(c["bt"], c["h"], c["v"], s["x"].dtype, top_k=c.get("k", 0), temperature=c["t"],
                                               ignore_index=IGNORE, keep_for_backward=op == "head_grad")
        r = s["plan"].forward(s["x"], s["w"], s["y"])
        out = {"logp": r.logp, "entropy": r.entropy}
        if c.get("k", 0):
            out.update(top_id=r.top_id, top_logp=r.top_logp)
        if op == "head_grad":
            out["grad_x"], out["grad_w"] = s["plan"].backward(s["x"], s["w"], s["y"], r, grad_logp=s["a"], grad_entropy=s["b"])
        return out
    if op == "logits":
        r = fl.logits_logprobs(s["z"], s["y"], top_k=c["k"], temperature=c["t"], ignore_index=IGNORE)
        out = {"logp": r.logp, "entropy": r.entropy}
        if c["k"]:
            out.update(top_id=r.top_id, top_logp=r.top_logp)
        if c["grad"]:
            out["grad_z"] = fl.logits_logprobs_backward(s["z"], s["y"], r, grad_logp=s["a"], grad_entropy=s["b"], temperature=c["t"],
                                                        ignore_index=IGNORE)
        return out
    if op == "fp8":
        return fl.fp8_linear(s["x"], s["wq"], s["ws"])
    if "plan" not in s:
        s["plan"] = fl.AdamW(s["p"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=c["bits"], master=s["master"],
                             exp_avg=s["m"], exp_avg_sq=s["v"], exp_avg_scale=s["ms"], exp_avg_sq_scale=s["vs"], step=s["t"])
    s["plan"].step(s["g"])
    return _updated(s)


# ---- the work that cannot be done without ------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("head", "head_grad"):
        bt, h, v = case["bt"], case["h"], case["v"]
        one = 2.0 * (bt * h + v * h)  # x and w, or their gradients
        rows = 16.0 * bt + 12.0 * bt * case.get("k", 0)
        return {"bytes": one + rows, "flops": 2.0 * bt * h * v} if op == "head" else {"bytes": 2 * one + rows + 8.0 * bt, "flops": 6.0 * bt * h * v}
    if op == "logits":
        n = case["rows"] * case["v"]
        return {"bytes": n * (4.0 if case["dtype"] == "fp32" else 2.0) * (2 if case["grad"] else 1) + case["rows"] * (16.0 + 12.0 * case["k"]),
                "flops": (10.0 if case["grad"] else 5.0) * n}
    if op == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2.0 * m * k + n * k + 4.0 * -(-n // BLOCK) * -(-k // BLOCK) + 2.0 * m * n, "flops": 2.0 * m * k * n}
    size = 2.0 if case["param"] == "bf16" else 4.0
    each = size + (size if case["master"] else 2 * size) + (8.0 if case["master"] else 0.0) + (16.0 if case["bits"] == 32 else 4.0 + 16.0 / BLOCK)
    return {"bytes": each * sum(_sizes(case)), "flops": 15.0 * sum(_sizes(case))}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------
def _exact_rows(z, y, t, k, a=None, b=None):
    """(logp, entropy, ids, log probabilities, dz) of logits in 64 bits."""
    logp = torch.log_softmax(z / t, 1)
    p = logp.exp()
    ent = -(p * logp).sum(1)
    live = (y >= 0).double()
    hit = torch.zeros_like(z).scatter_(1, y.clamp_min(0)[:, None], live[:, None])
    lp = (hit * logp).sum(1)
    ids, left, col = [], z.clone(), torch.arange(z.shape[1], device=z.device)
    for _ in range(k):
        first = torch.where(left == left.amax(1, keepdim=True), col, z.shape[1]).amin(1)
        ids.append(first)
        left.scatter_(1, first[:, None], -math.inf)
    ids = torch.stack(ids, 1) if k else None
    dz = None
    if a is not None:
        a, b = a.double()[:, None] * live[:, None], b.double()[:, None] * live[:, None]
        dz = (a * (hit - p) - b * p * (logp + ent[:, None])) / t
    return lp, ent * live, ids, logp.gather(1, ids) if k else None, dz


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("head", "head_grad", "logits"):
        head, grad = op != "logits", op == "head_grad" or case.get("grad", False)
        if head and 2.0 * case["bt"] * case["h"] * case["v"] * (3 if grad else 1) > 1.4e13:
            return None
        k, rows = case.get("k", 0), case["bt"] if head else case["rows"]
        if head:
            w = s["w"].double()
            gw = torch.zeros_like(w) if grad else None
        parts = []
        for r0 in range(0, rows, 512):
            cut = slice(r0, min(rows, r0 + 512))
            z = s["x"][cut].double() @ w.T if head else s["z"][cut].double()
            q = list(_exact_rows(z, s["y"][cut], case["t"], k, s["a"][cut] if grad else None, s["b"][cut] if grad else None))
            if grad and head:
                gw += q[4].T @ s["x"][cut].double()
                q[4] = q[4] @ w
            parts.append(q)
        cat = [torch.cat(v) if v[0] is not None else None for v in zip(*parts)]
        out = {"logp": cat[0], "entropy": cat[1]}
        if k:
            out.update(top_id=cat[2], top_logp=cat[3])
        if grad:
            out.update(dict(grad_x=cat[4], grad_w=gw) if head else dict(grad_z=cat[4]))
        return out
    if op == "fp8":
        m, k, n = case["m"], case["k"], case["n"]
        if 2.0 * m * k * n > 1.4e13:
            return None
        x = torch.zeros(m, -(-k // BLOCK) * BLOCK, device="cuda", dtype=torch.float64)
        x[:, :k] = s["x"].double()
        x = x.view(m, -1, BLOCK)
        amax = x.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR)
        x = ((x / amax * E4M3_MAX).float().to(torch.float8_e4m3fn).double() * (amax / E4M3_MAX)).reshape(m, -1)
        out = torch.empty(m, n, device="cuda", dtype=torch.float64)
        for n0 in range(0, n, 16384):
            w = s["wq"][n0:n0 + 16384].double()
            sc = s["ws"][n0 // BLOCK:(n0 + w.shape[0] + BLOCK - 1) // BLOCK].double()
            for j in range(sc.shape[1]):
                w[:, j * BLOCK:(j + 1) * BLOCK] *= sc[:, j].repeat_interleave(BLOCK)[:w.shape[0], None]
            out[:, n0:n0 + w.shape[0]] = x[:, :k] @ w.T
        return out
    t, flat = s["t"] + 1, s["flat"]
    spread = lambda c: c.double().repeat_interleave(BLOCK)  # noqa: E731
    g, p, m, v = flat["g"].double(), flat["master" if case["master"] else "p"].double(), flat["m"].double(), flat["v"].double()
    if case["bits"] == 8:
        m, v = m * spread(flat["ms"]), (v * spread(flat["vs"])) ** 2
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    out = {"p": p, "m": m, "v": v}
    if case["master"]:
        out["master"] = p
    if case["bits"] == 8:  # which of two codes a value next to their border gets goes by 32 bits; the scales are given
        tops = [x.view(-1, BLOCK).abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX for x in (m, v.sqrt())]
        out.update(m=None, v=None, ms=tops[0], vs=tops[1])
    return out
