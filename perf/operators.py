"""What is measured of the operators over a frozen LM head: token log-probabilities with entropy
and top alternatives, and distillation from a teacher's top logits, each forward alone and as a
training step (forward and the gradient in the hidden states).

``run`` computes them in plain fp32 torch, or (``own``) through the package's layers.  Hidden
states and heads lie on power-of-two grids, so every sum of products X·Wᵀ is exact in fp32 in any
order: the ids of the top alternatives then do not depend on how a product was summed.
"""
import math

import torch

own = False

IGNORE = -100


def _lp(name, M, D, V, n, k, T=1.0, grad=False, went=0.0):
    return {"name": name, "op": "logprob", "M": M, "D": D, "V": V, "n": n, "k": k, "T": T, "grad": grad,
            "went": went, "masked": 0.05}


def _kd(name, M, D, V, n, T=1.0, grad=True, masked=0.05):
    return {"name": name, "op": "distill", "M": M, "D": D, "V": V, "n": n, "k": 0, "T": T, "grad": grad,
            "went": 0.0, "masked": masked}


def listed():
    return [
        # three tokens of a test-sized model: nothing but latency
        _lp("lp_few_small_head", 3, 200, 1000, 1, 5),
        # one decoding step of one sequence, with the alternatives an API returns
        _lp("lp_decode_1", 1, 4096, 128256, 1, 8),
        # one decoding step of a batch
        _lp("lp_decode_48", 48, 4096, 128256, 1, 20),
        # scoring a sequence of the benchmark's head: log-probabilities and entropy only
        _lp("lp_score_2048", 2048, 4096, 128256, 1, 0),
        # four given tokens a row and the longest list of alternatives, a teacher's pass at a smaller head
        _lp("lp_alternatives_777", 777, 2048, 32000, 4, 32, T=0.7),
        # a policy-gradient step with an entropy bonus
        _lp("lp_policy_step_4096", 4096, 4096, 128256, 1, 0, grad=True, went=0.01),
        # the same on odd sizes, two tokens a row, without the bonus
        _lp("lp_pair_step_odd", 1001, 1000, 50008, 2, 0, T=1.3, grad=True),
        # a student checked against a stored teacher while it decodes
        _kd("kd_decode_5", 5, 4096, 128256, 16, grad=False),
        # a distillation step of a test-sized model
        _kd("kd_step_small", 129, 328, 4096, 8),
        # half of the rows are prompt or padding, long lists, softened
        _kd("kd_step_masked", 1500, 1024, 65536, 64, T=2.0, masked=0.5),
        # an ordinary distillation step
        _kd("kd_step_2048", 2048, 4096, 128256, 32),
        # the benchmark's batch (4 x 4096 tokens) over its head
        _kd("kd_step_16384", 16384, 4096, 128256, 32, T=1.5),
    ]


def draw(rng):
    def log(lo, hi):
        return math.exp(rng.uniform(math.log(lo), math.log(hi)))

    most = 2 * 16384 * 4096 * 128256
    while True:
        op = rng.choice(["logprob", "logprob", "distill"])
        grad = rng.random() < 0.5
        M = int(log(1, 16385))
        D = 8 * int(log(8, 1025))
        V = 8 * int(log(32, 16385))
        if (2 if grad else 1) * M * D * V > most:
            continue
        T = rng.choice([1.0, 1.0, round(rng.uniform(0.5, 3.0), 2)])
        if op == "distill":
            n = int(log(1, 129))
            c = _kd("", M, D, V, n, T, grad, rng.choice([0.0, 0.05, 0.5]))
        else:
            k = 0 if grad or M > 2048 or rng.random() < 0.25 else int(log(1, 33))
            c = _lp("", M, D, V, int(log(1, 9)), k, T, grad, 0.02 if grad and rng.random() < 0.5 else 0.0)
        del c["name"]
        return c


def _inputs(case, seed):
    """Hidden states X [M, D] with unit variance and a head W [V, D] with logits of standard
    deviation about 2, rows leaning towards their first token (so some are certain of it and some
    are not); ids [M, n] with a share of ignored rows and, of several, some ignored entries; a
    teacher's logits falling from the first entry on."""
    M, D, V, n = case["M"], case["D"], case["V"], case["n"]
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + M + 7 * D + 13 * V + n)
    std = 2.0 / math.sqrt(D)
    step = 2.0 ** (math.floor(math.log2(std)) - 4)
    W = torch.empty((V, D), device=dev, dtype=torch.bfloat16)
    for r in range(0, V, 16384):
        w = torch.randn((min(16384, V - r), D), generator=g, device=dev)
        W[r:r + 16384] = (w * (std / step)).round_().clamp_(-250, 250).mul_(step)
    ids = torch.randint(0, V, (M, n), generator=g, device=dev)
    lean = torch.rand((M, 1), generator=g, device=dev) * (8.0 / math.sqrt(D))
    X = torch.randn((M, D), generator=g, device=dev) + lean * (1.0 / std) * W[ids[:, 0]].float()
    X = (X * 16).round_().clamp_(-250, 250).div_(16).to(torch.bfloat16)
    if n > 1:
        cut = torch.randint(1, n + 1, (M, 1), generator=g, device=dev)
        short = torch.rand((M, 1), generator=g, device=dev) < 0.2
        ids[short & (torch.arange(n, device=dev) >= cut)] = IGNORE
    ids[torch.rand(M, generator=g, device=dev) < case["masked"]] = IGNORE
    s = {"X": X, "W": W, "ids": ids.to(torch.int32)}
    if case["op"] == "distill":
        t = torch.randn((M, n), generator=g, device=dev) * 2.0
        s["teacher"] = t.sort(1, descending=True)[0] + 10.0
        s["dloss"] = torch.full((M,), 1.0 / max(1, M), device=dev)
    else:
        s["dlogprob"] = torch.randn((M, n), generator=g, device=dev) / M
        s["dentropy"] = torch.full((M,), case["went"] / M, device=dev) if case["went"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    if own:
        import qlora_linear_b200 as q

        head = q.LoraWeight.bf16(s["W"])
        cls = q.LoraDistill if case["op"] == "distill" else q.LoraTokenLogProbs
        s["layer"] = cls(head, ignore_index=IGNORE, temperature=case["T"])
    return s


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return _run_plain(state, c)


def _run_own(s, c):
    layer, X, ids = s["layer"], s["X"], s["ids"]
    if c["op"] == "distill":
        out = layer.forward(X, ids, s["teacher"], save=c["grad"])
        if not c["grad"]:
            return {"loss": out.loss}
        return {"loss": out.loss, "dX": layer.backward(X, ids, s["teacher"], out, s["dloss"])}
    out = layer.forward(X, ids, top_k=c["k"], save=c["grad"])
    res = {"logprob": out.logprob, "entropy": out.entropy}
    if c["k"]:
        res["top_ids"], res["top_logprob"] = out.top_ids, out.top_logprob
    if c["grad"]:
        res["dX"] = layer.backward(X, ids, out, s["dlogprob"], s["dentropy"])
    return res


def _run_plain(s, c):
    """Elementary fp32 operations."""
    W, X, ids = s["W"].float(), s["X"].float(), s["ids"].long()
    z = (X @ W.t()) * (1.0 / c["T"])
    top = z.max(1, keepdim=True)[0]
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    logp = (z - top) - torch.log(total)
    p = e.div_(total)
    there = ids >= 0
    lp = torch.where(there, logp.gather(1, ids.clamp(min=0)), 0.0)
    if c["op"] == "distill":
        t = torch.where(there, s["teacher"] * (1.0 / c["T"]), -math.inf)
        t = t - t.max(1, keepdim=True)[0].clamp(min=-3e38)
        qe = torch.exp(t)
        qs = qe.sum(1, keepdim=True)
        qs = torch.where(qs > 0, qs, 1.0)
        q = qe / qs
        logq = torch.where(there, t, 0.0) - torch.log(qs)
        out = {"loss": (q * (logq - lp)).sum(1)}
        coef, dent = -q * s["dloss"][:, None] if c["grad"] else None, None
    else:
        out = {"logprob": lp, "entropy": -(p * logp).sum(1)}
        if c["k"]:
            val, idx = torch.sort(z, dim=1, descending=True, stable=True)
            out["top_ids"] = idx[:, :c["k"]].to(torch.int32)
            out["top_logprob"] = (val[:, :c["k"]] - top) - torch.log(total)
        coef, dent = torch.where(there, s["dlogprob"], 0.0), s["dentropy"]
    if c["grad"]:
        w = coef.sum(1, keepdim=True)
        if dent is not None:
            w = w + dent[:, None] * (logp + out["entropy"][:, None])
        dz = p.mul_(w).neg_()
        dz.scatter_add_(1, ids.clamp(min=0), coef)
        out["dX"] = ((dz @ W) * (1.0 / c["T"])).to(torch.bfloat16)
    return out


def work(case):
    M, D, V, n, k = (case[x] for x in ("M", "D", "V", "n", "k"))
    b = 2 * M * D + 2 * V * D + 4 * M * n
    f = 2 * M * V * D
    if case["op"] == "distill":
        b += 4 * M * n + 4 * M
    else:
        b += 4 * M * n + 4 * M + 8 * M * k
    if case["grad"]:
        b += 2 * M * D + (4 * M if case["op"] == "distill" else 4 * M * n + (4 * M if case["went"] else 0))
        f *= 2
    return {"bytes": b, "flops": f}


def exact(case, seed):
    """In 64 bits, a block of rows at a time: the definitions by way of the normaliser, and the
    gradient as a difference of two averages of head rows."""
    s = _inputs(case, seed)
    M, D, V, n = case["M"], case["D"], case["V"], case["n"]
    if M * D * V * (2 if case["grad"] else 1) > 2 * 16384 * 4096 * 128256:
        return None
    f64 = torch.float64
    W = s["W"].to(f64)
    block = max(1, min(M, 1 << 27 >> max(0, (V - 1).bit_length())))
    outs = []
    for a in range(0, M, block):
        b = min(M, a + block)
        z = torch.mm(s["X"][a:b].to(f64), W.T) / case["T"]
        lse = torch.logsumexp(z, 1)
        prob = torch.softmax(z, 1)
        o = {}
        ids = s["ids"][a:b]
        keep = ids != IGNORE
        safe = torch.where(keep, ids, torch.zeros_like(ids)).long()
        lp = (torch.gather(z, 1, safe) - lse[:, None]) * keep
        if case["op"] == "distill":
            t = s["teacher"][a:b].to(f64) / case["T"]
            t = t.masked_fill(~keep, -math.inf)
            empty = ~keep.any(1)
            norm = torch.where(empty, torch.zeros_like(lse), torch.logsumexp(t, 1))
            logq = t - norm[:, None]
            q = torch.exp(logq)
            o["loss"] = torch.xlogy(q, q).sum(1) - (q * lp).sum(1)
            pull = s["dloss"][a:b].to(f64)[:, None] * q
            ent_w = None
        else:
            ent = lse - (prob * z).sum(1)
            o["logprob"], o["entropy"] = lp, ent
            if case["k"]:
                order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :case["k"]]
                o["top_ids"] = order.to(torch.int32)
                o["top_logprob"] = torch.gather(z, 1, order) - lse[:, None]
            pull = -s["dlogprob"][a:b].to(f64) * keep
            ent_w = None if s["dentropy"] is None else s["dentropy"][a:b].to(f64)
        if case["grad"]:
            mean = prob * pull.sum(1, keepdim=True)
            if ent_w is not None:
                mean -= ent_w[:, None] * prob * (z - lse[:, None] + ent[:, None])
            grad = mean @ W
            for i in range(n):
                grad -= pull[:, i:i + 1] * W[safe[:, i]] * keep[:, i:i + 1]
            o["dX"] = grad / case["T"]
        outs.append(o)
    return {k: torch.cat([o[k] for o in outs]) for k in outs[0]}
