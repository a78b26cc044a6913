"""Cases that time the token log-probability operators and gradient clipping.

Token log probabilities (from materialised logits, or from hidden states and the
head weight) with the entropy and the top alternatives of every row, their
backward passes, and the global gradient norm with clipping.  ``run`` computes
them from elementary torch operations in 32 bits, or, with ``own`` set, through
the library.
"""
import math

import torch

own = False

IGNORE = -100
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _case(op, **kw):
    base = {"op": op}
    if op in ("logits_fwd", "logits_bwd"):
        base.update(n=1, v=32000, dtype="bf16", k=0, t=1.0, std=4.0, pad=0, ignore=0.0)
    elif op in ("hidden_fwd", "hidden_bwd"):
        base.update(n=1, v=32000, d=2048, k=0, t=1.0, grid=False, ignore=0.0)
    else:
        base.update(layout="head", v=32000, d=2048, layers=1, dtype="bf16", max_norm=1.0)
    base.update(kw)
    return base


def listed():
    return [
        # a decoding step of one sequence: the sampled token's log probability
        # and the 20 best alternatives, from the logits the sampler has
        _case("logits_fwd", name="decode_logits_top20", n=1, v=151936, k=20),
        # a teacher's cache of top-100 log probabilities from materialised logits
        _case("logits_fwd", name="cache_logits_top100", n=4096, v=151936, k=100),
        # scoring in fp32 at a sampling temperature: an odd vocabulary whose
        # last ids are forbidden (-inf), some tokens ignored
        _case("logits_fwd", name="score_fp32_odd", n=333, v=32003, dtype="fp32", k=5, t=0.7,
              pad=61, ignore=0.08),
        # a policy-gradient step with an entropy bonus on materialised logits
        _case("logits_bwd", name="policy_logits_grad", n=8192, v=128256, ignore=0.08),
        # the same in fp32 on a short ragged batch
        _case("logits_bwd", name="policy_fp32_odd_grad", n=77, v=32003, dtype="fp32", t=0.7,
              pad=61, ignore=0.08),
        # a decoding step of one sequence from its hidden state
        _case("hidden_fwd", name="decode_hidden_top20", n=1, v=151936, d=4096, k=20, grid=True),
        # scoring a batch of given tokens in training, no alternatives
        _case("hidden_fwd", name="score_hidden", n=4096, v=32000, d=2048, ignore=0.05),
        # a teacher's cache of top-100 log probabilities from its hidden states
        _case("hidden_fwd", name="cache_hidden_top100", n=2048, v=151936, d=4096, k=100,
              grid=True),
        # the gradients of a policy-gradient step to hidden states and head
        _case("hidden_bwd", name="policy_hidden_grad", n=4096, v=32000, d=2048, ignore=0.05),
        # the same on a short ragged batch of a small model
        _case("hidden_bwd", name="policy_small_grad", n=300, v=5003, d=520, t=0.7, ignore=0.1),
        # clipping the many small gradients of adapters
        _case("clip", name="clip_adapters", layout="adapters", layers=9, d=2048, dtype="fp32"),
        # clipping the gradients of a head and the hidden states' projections
        _case("clip", name="clip_head", layout="head", v=151936, d=4096, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logits_fwd", "logits_fwd", "logits_bwd", "hidden_fwd", "hidden_fwd",
                     "hidden_bwd", "clip"])
    ignore = rng.choice([0.0, 0.05, 0.3])
    t = rng.choice([1.0, 1.0, 0.7, 2.0])
    if op in ("logits_fwd", "logits_bwd"):
        v = _log(rng, 500, 250000)
        n = _log(rng, 1, max(2, min(16384, 600_000_000 // v)))
        k = min(rng.choice([0, 1, 5, 20, 64, 100, 257, 1000]), v // 2)
        return _case(op, n=n, v=v, k=k if op == "logits_fwd" else 0, t=t, ignore=ignore,
                     dtype=rng.choice(["bf16", "bf16", "fp32"]), pad=rng.choice([0, 0, 7, 200]),
                     std=rng.choice([1.5, 3.0, 4.0]))
    if op in ("hidden_fwd", "hidden_bwd"):
        d = 8 * _log(rng, 8, 512)
        v = _log(rng, 500, 152000)
        most = 1_200_000_000_000 if op == "hidden_fwd" else 200_000_000_000
        n = _log(rng, 1, max(2, min(8192, most // (v * d))))
        k = min(rng.choice([0, 0, 1, 5, 20, 100, 300]), v // 2) if op == "hidden_fwd" else 0
        return _case(op, n=n, v=v, d=d, k=k, t=t, ignore=ignore, grid=k > 0)
    if rng.random() < 0.5:
        return _case("clip", layout="adapters", layers=rng.randint(1, 9),
                     d=_log(rng, 100, 4096), dtype=rng.choice(["bf16", "fp32"]),
                     max_norm=rng.choice([0.5, 1.0, 1e6]))
    return _case("clip", layout="head", v=_log(rng, 500, 152000), d=_log(rng, 64, 4096),
                 layers=rng.randint(1, 6), dtype="bf16", max_norm=rng.choice([0.5, 1.0, 1e6]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(case, g):
    """Upstream gradients of the log probabilities (advantages over the batch)
    and of the entropies (a small bonus)."""
    n = case["n"]
    d_lp = torch.randn(n, generator=g, device="cuda") / n
    d_h = 0.01 * torch.rand(n, generator=g, device="cuda") / n
    return d_lp, d_h


def _ignore(case, tokens, g):
    if case["ignore"] > 0:
        drop = torch.rand(case["n"], generator=g, device="cuda") < case["ignore"]
        tokens[drop] = IGNORE
    return tokens


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("logits_fwd", "logits_bwd"):
        n, v = case["n"], case["v"]
        z = (torch.randn(n, v, generator=g, device="cuda") * case["std"]).to(DT[case["dtype"]])
        if case["pad"]:
            z[:, v - case["pad"]:] = float("-inf")
        # tokens as a sampler draws them: an exponential race over exp(z / T)
        race = torch.empty(n, v, device="cuda").exponential_(generator=g).log_()
        tokens = (z.float() / case["t"]).sub_(race).argmax(dim=1)
        return {"logits": z, "tokens": _ignore(case, tokens, g), "up": _rows(case, g)}
    if op in ("hidden_fwd", "hidden_bwd"):
        n, v, d = case["n"], case["v"], case["d"]
        h = torch.randn(n, d, generator=g, device="cuda")
        w = torch.randn(v, d, generator=g, device="cuda") * 0.02
        if case["grid"]:
            # values of a coarsely quantised checkpoint: every partial sum of a
            # logit is exact in fp32, so the order of the alternatives does not
            # depend on the order of summation
            h = (h * 16).round_().clamp_(-64, 64) / 16
            w = (w * 1024).round_().clamp_(-127, 127) / 1024
        tokens = torch.randint(0, v, (n,), generator=g, device="cuda")
        return {"h": h.bfloat16(), "w": w.bfloat16(), "tokens": _ignore(case, tokens, g),
                "up": _rows(case, g)}
    shapes = _shapes(case)
    # gradients differ in size by tensor, as those of different layers do
    return {"grads": [(torch.randn(*s, generator=g, device="cuda") * (0.3 / (1 + i % 7)))
                      .to(DT[case["dtype"]]) for i, s in enumerate(shapes)]}


def _shapes(case):
    d = case["d"]
    if case["layout"] == "adapters":
        # rank-8 pairs on two projections, two norms and a bias of each layer
        return [s for _ in range(case["layers"])
                for s in ((8, d), (d, 8), (8, d), (d + 1, 8), (d,), (d,))]
    return [(case["v"], d)] + [s for _ in range(case["layers"]) for s in ((d, d), (d,), (d + 3,))]


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    s["case"] = case
    if op in ("logits_bwd", "hidden_bwd"):
        # the saved statistics of the forward pass
        z = _logits(s)
        s["stats"] = _stats(z / case["t"] if case["t"] != 1.0 else z, z, case["t"])
        del z
    if op == "clip":
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
    s["kept"] = {}  # the program's problem, workspace and output buffers
    return s


# ---------------------------------------------------------------- plain forms

def _logits(s):
    return s["logits"].float() if "logits" in s else s["h"].float() @ s["w"].float().t()


def _stats(a, z, t):
    """(max z, log sum exp(a - max a), entropy, log sum exp a) per row."""
    m = z.amax(dim=1)
    x = a - (m / t)[:, None]
    e = x.exp()
    total = e.sum(dim=1)
    log_s = total.log()
    ent = log_s - torch.where(e > 0, e * x, torch.zeros_like(e)).sum(dim=1) / total
    return torch.stack([m, log_s, ent, m / t + log_s], dim=1)


def _top(z, k):
    """Ids of the k largest of each row, ties to the lowest id."""
    bits = (z + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    low = 0xFFFFFFFF - torch.arange(z.shape[1], device=z.device)
    key = order * 4294967296 + low
    return (0xFFFFFFFF - (key.topk(k, dim=1).values & 0xFFFFFFFF)).int()


def _plain_fwd(s):
    case = s["case"]
    t, k = case["t"], case["k"]
    z = _logits(s)
    tokens = s["tokens"]
    on = tokens != IGNORE
    st = _stats(z / t, z, t)
    m, log_s = st[:, :1], st[:, 1:2]
    zero = torch.zeros_like(st[:, 0])
    zy = z.gather(1, tokens.clamp(min=0)[:, None])
    out = {"logprob": torch.where(on, ((zy - m) / t - log_s)[:, 0], zero),
           "entropy": torch.where(on, st[:, 2], zero)}
    if k:
        ids = _top(z, k)
        lp = (z.gather(1, ids.long()) - m) / t - log_s
        low = torch.arange(k, device=z.device, dtype=torch.int32).expand_as(ids)
        out["topk_idx"] = torch.where(on[:, None], ids, low)
        out["topk_logprob"] = torch.where(on[:, None], lp, torch.full_like(lp, -math.inf))
    return out


def _plain_grad(s):
    """The gradient of the logits, in 32 bits."""
    t = s["case"]["t"]
    z, st, tokens = _logits(s), s["stats"], s["tokens"]
    on = tokens != IGNORE
    d_lp, d_h = (torch.where(on, u, torch.zeros_like(u))[:, None] for u in s["up"])
    lp = (z - st[:, :1]) / t - st[:, 1:2]
    p = lp.exp()
    g = torch.where(p > 0, p * (d_lp + d_h * (lp + st[:, 2:3])), torch.zeros_like(p)) / -t
    return g.scatter_add_(1, tokens.clamp(min=0)[:, None], d_lp / t)


def _plain(s):
    op = s["case"]["op"]
    if op in ("logits_fwd", "hidden_fwd"):
        return _plain_fwd(s)
    if op == "logits_bwd":
        return {"d_logits": _plain_grad(s).to(s["logits"].dtype)}
    if op == "hidden_bwd":
        g = _plain_grad(s)
        return {"d_h": (g @ s["w"].float()).bfloat16(), "d_w": (g.t() @ s["h"].float()).bfloat16()}
    sq = torch.stack([x.float().square().sum() for x in s["grads"]])
    norm = sq.sum().sqrt()
    coef = (s["case"]["max_norm"] / norm).clamp(max=1.0)
    return {"norm": norm, "grads": [(x.float() * coef).to(x.dtype) for x in s["grads"]]}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from lm_head_cross_vocab_gb300 import kd

    case, kept = s["case"], s["kept"]
    op = case["op"]
    if op == "clip":
        if not kept:
            kept["list"] = kd.GradList(s["grads"], out=s["out"])
            kept["ws"] = kd.Workspace()
        r = kd.clip_grad_norm(kept["list"], case["max_norm"], workspace=kept["ws"], check=False)
        return {"norm": r["norm"], "grads": r["grads"]}
    if not kept:
        hidden = op in ("hidden_fwd", "hidden_bwd")
        kept["ws"] = kd.Workspace()
        kept["problem"] = kd.LogprobProblem(
            n_tokens=case["n"], vocab=case["v"], d_model=case["d"] if hidden else 0,
            topk=case["k"], dtype="bf16" if hidden else case["dtype"],
            source="hidden" if hidden else "logits", temperature=case["t"], ignore_index=IGNORE)
        kept["tensors"] = ({"h": s["h"], "w": s["w"], "tokens": s["tokens"]} if hidden
                           else {"logits": s["logits"], "tokens": s["tokens"]})
    if op in ("logits_fwd", "hidden_fwd"):
        r = kept["out"] = kd.token_logprobs(kept["problem"], kept["tensors"], workspace=kept["ws"],
                                            check=False, out=kept.get("out"))
        names = ("logprob", "entropy") + (("topk_idx", "topk_logprob") if case["k"] else ())
    else:
        d_lp, d_h = s["up"]
        r = kept["out"] = kd.token_logprobs_backward(
            kept["problem"], kept["tensors"], s["stats"], d_logprob=d_lp, d_entropy=d_h,
            workspace=kept["ws"], check=False, out=kept.get("out"))
        names = ("d_logits",) if op == "logits_bwd" else ("d_h", "d_w")
    return {name: r[name] for name in names}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "clip":
        size = sum(math.prod(x) for x in _shapes(case)) * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": 2 * size + 4, "flops": 3 * size // (2 if case["dtype"] == "bf16" else 4)}
    n, v, k = case["n"], case["v"], case["k"]
    if op in ("logits_fwd", "logits_bwd"):
        size = n * v * (2 if case["dtype"] == "bf16" else 4)
        if op == "logits_fwd":
            return {"bytes": size + n * (16 + 8 * k), "flops": 6 * n * v}
        return {"bytes": 2 * size + n * 32, "flops": 6 * n * v}
    d = case["d"]
    if op == "hidden_fwd":
        return {"bytes": 2 * (n + v) * d + n * (16 + 8 * k), "flops": 2 * n * v * d}
    return {"bytes": 4 * (n + v) * d + n * 32, "flops": 6 * n * v * d}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "clip":
        norm = torch.linalg.vector_norm(
            torch.stack([torch.linalg.vector_norm(x.double()) for x in s["grads"]]))
        scale = min(1.0, case["max_norm"] / float(norm))
        return {"norm": norm, "grads": [x.double() * scale for x in s["grads"]]}
    z = s["logits"].double() if "logits" in s else s["h"].double() @ s["w"].double().t()
    tokens = s["tokens"]
    off = (tokens == IGNORE)[:, None]
    lp = torch.log_softmax(z / case["t"], dim=1)
    p = torch.softmax(z / case["t"], dim=1)
    ent = -torch.nan_to_num(p * lp, nan=0.0).sum(dim=1, keepdim=True)
    if op in ("logits_fwd", "hidden_fwd"):
        out = {"logprob": lp.gather(1, tokens.clamp(min=0)[:, None]).masked_fill_(off, 0.0)[:, 0],
               "entropy": ent.masked_fill(off, 0.0)[:, 0]}
        if case["k"]:
            del p
            val, ids = torch.sort(z, dim=1, descending=True, stable=True)
            del val
            ids = ids[:, :case["k"]]
            top = lp.gather(1, ids)
            out["topk_idx"] = None  # whole numbers: equal or not
            out["topk_logprob"] = top.masked_fill_(off, -math.inf)
        return out
    d_lp, d_h = (u.double()[:, None].masked_fill(off, 0.0) for u in s["up"])
    # d log p_y / d z_v = (1[v = y] - p_v) / T and dH / d z_v = -p_v (log p_v + H) / T
    g = -d_lp * p - d_h * torch.nan_to_num(p * lp, nan=0.0) - d_h * ent * p
    del lp, p
    g[torch.arange(case["n"], device=g.device), tokens.clamp(min=0)] += d_lp[:, 0]
    g /= case["t"]
    if op == "logits_bwd":
        return {"d_logits": g}
    return {"d_h": g @ s["w"].double(), "d_w": g.t() @ s["h"].double()}
