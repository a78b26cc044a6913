"""Cases that time what stands around the head: verification of drafted tokens,
the embedding lookup and its gradient, and the norm that makes the hidden states.

``run`` computes them from elementary torch operations in 32 bits (64 where a
decision lies next to a border), or, with ``own`` set, through the library.
"""
import math

import torch

own = False

IGNORE = -100
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _case(op, **kw):
    base = {"op": op, "dtype": "bf16"}
    if op == "verify":
        # t = 0: greedy; draft: the drafter's logits, or none (looked-up drafts)
        base.update(b=1, k=4, v=32000, t=1.0, t_draft=1.0, draft="logits", ragged=False, pad=0)
    elif op in ("embed", "embed_grad"):
        base.update(n=1, v=32000, d=2048, scale=1.0, ignore=0.0)
        if op == "embed_grad":
            base.update(accumulate=False)
    else:
        base.update(n=1, d=2048, residual=True, offset=0.0)
    base.update(kw)
    return base


def listed():
    return [
        # one sequence of a chat: four drafts of a small drafter
        _case("verify", name="verify_one", b=1, k=4, v=151936),
        # a serving batch at a sampling temperature, some sequences with fewer drafts
        _case("verify", name="verify_batch", b=48, k=5, v=128256, t=0.75, t_draft=0.75,
              ragged=True),
        # the largest batch, seven drafts each
        _case("verify", name="verify_large", b=256, k=7, v=151936),
        # fp32 logits of an odd vocabulary whose last ids are forbidden
        _case("verify", name="verify_fp32_odd", b=9, k=3, v=32003, dtype="fp32", pad=61,
              ragged=True),
        # a decoding step of a serving batch: its last tokens' rows of the table
        _case("embed", name="embed_decode", n=48, v=151936, d=4096),
        # a training batch of a model that scales its embeddings
        _case("embed", name="embed_batch", n=16384, v=128256, d=4096, scale=64.0, ignore=0.05),
        # the gradient of a tied table, added to what the head gave it
        _case("embed_grad", name="embed_grad_tied", n=4096, v=32000, d=2048, accumulate=True,
              ignore=0.05),
        # the gradient of a table of its own, written whole
        _case("embed_grad", name="embed_grad_whole", n=16384, v=151936, d=4096),
        # the last norm of a decoding step
        _case("norm", name="norm_decode", n=48, d=4096),
        # the same over a training batch
        _case("norm", name="norm_batch", n=16384, d=4096),
        # the way back through it, from the loss's gradient of the hidden states
        _case("norm_grad", name="norm_grad_batch", n=16384, d=4096, residual=False),
        # inside a small model in fp32, odd width, a gradient of the residual stream
        _case("norm_grad", name="norm_grad_fp32_odd", n=1000, d=1001, dtype="fp32", offset=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    d = _log(rng, 64, hi)
    return d if rng.random() < 0.25 else (d + 7) // 8 * 8


def draw(rng):
    op = rng.choice(["verify", "verify", "verify", "embed", "embed_grad", "embed_grad", "norm",
                     "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "verify":
        k = rng.choice([0, 1, 2, 3, 4, 5, 7, 8])
        v = _log(rng, 500, 152000)
        b = _log(rng, 1, max(2, min(512, 250_000_000 // (v * (2 * k + 1)))))
        t = rng.choice([1.0, 1.0, 0.75, 1.5, 0.0])
        return _case(op, b=b, k=k, v=v, dtype=dtype, t=t, t_draft=t or 1.0,
                     draft=rng.choice(["logits", "logits", "none"]),
                     ragged=rng.random() < 0.5, pad=rng.choice([0, 0, 7, 200]))
    if op in ("embed", "embed_grad"):
        d = _width(rng, 8192)
        v = _log(rng, 500, max(501, min(152000, 300_000_000 // d)))
        n = _log(rng, 1, max(2, min(65536, 33_000_000 // d)))
        kw = dict(n=n, v=v, d=d, dtype=dtype, scale=rng.choice([1.0, 1.0, 45.25]),
                  ignore=rng.choice([0.0, 0.05, 0.3]))
        if op == "embed_grad":
            kw["accumulate"] = rng.random() < 0.5
        return _case(op, **kw)
    d = _width(rng, 8192)
    n = _log(rng, 1, max(2, min(65536, 33_000_000 // d)))
    return _case(op, n=n, d=d, dtype=dtype, residual=rng.random() < 0.5,
                 offset=rng.choice([0.0, 0.0, 1.0]))


# ---------------------------------------------------------------- inputs

def _lengths(case):
    b, k = case["b"], case["k"]
    return [(5 * i + 3) % (k + 1) if case["ragged"] else k for i in range(b)]


def _text(case, g):
    """Tokens as text has them: low ids are the frequent ones, id i's frequency
    about 1 / (i + 3.2)."""
    u = torch.rand(case["n"], generator=g, device="cuda", dtype=torch.float64)
    tokens = (2.7 * (case["v"] / 2.7 + 1.0) ** u - 2.7).long().clamp_(0, case["v"] - 1)
    if case["ignore"] > 0:
        drop = torch.rand(case["n"], generator=g, device="cuda") < case["ignore"]
        tokens[drop] = IGNORE
    return tokens


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "verify":
        b, k, v = case["b"], case["k"], case["v"]
        target = randn(b, k + 1, v).mul_(3.5).to(dt)
        # a distilled drafter's logits lie near the target's
        draft = (target[:, :k].float() + 0.8 * randn(b, k, v)).to(dt)
        if case["pad"]:
            target[..., v - case["pad"]:] = float("-inf")
            draft[..., v - case["pad"]:] = float("-inf")
        race = torch.empty(b, k, v, device="cuda").exponential_(generator=g).log_()
        drafts = (draft.float() / case["t_draft"]).sub_(race).argmax(dim=2)
        del race
        s = {"target": target, "drafts": drafts,
             "uniform": torch.rand(b, k, generator=g, device="cuda"),
             "noise": torch.empty(b, v, device="cuda").exponential_(generator=g),
             "lengths": torch.tensor(_lengths(case), dtype=torch.int32).cuda()}
        if case["draft"] == "logits":
            s["draft"] = draft
        return s
    if op == "embed":
        return {"w": (randn(case["v"], case["d"]) * 0.02).to(dt), "tokens": _text(case, g)}
    if op == "embed_grad":
        s = {"tokens": _text(case, g), "d_h": (randn(case["n"], case["d"]) * 1e-3).to(dt)}
        # what the head's backward gave the table, or whatever the buffer holds
        s["d_w"] = (randn(case["v"], case["d"]) * 1e-4).to(dt)
        return s
    n, d = case["n"], case["d"]
    # a few channels of the residual stream are much larger than the others
    size = torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    s = {"x": (randn(n, d) * size).to(dt),
         "weight": (1.0 - case["offset"] + 0.1 * randn(d)).to(dt)}
    if case["residual"]:
        s["residual"] = (randn(n, d) * (size if op == "norm" else 1e-3)).to(dt)
    if op == "norm_grad":
        s["d_h"] = (randn(n, d) * 1e-3).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["kept"] = {}  # the program's problem, workspace and output buffers
    return s


# ---------------------------------------------------------------- plain forms

def _sums(z, t):
    """(max z, sum exp((z - max z) / t)) of every row, the sum in 64 bits."""
    m = z.amax(dim=-1)
    return m, ((z - m[..., None]) / t).exp().sum(dim=-1, dtype=torch.float64)


def _plain_verify(s):
    case = s["case"]
    b, k, v = case["b"], case["k"], case["v"]
    t = case["t"] or 1.0
    length, x = s["lengths"].long(), s["drafts"]
    z = s["target"].float()
    m, total = _sums(z, t)
    zx = z[:, :k].gather(2, x[..., None])[..., 0].double()
    px = ((zx - m[:, :k]) / t).exp() / total[:, :k]
    if case["t"] == 0.0:
        best = z.argmax(dim=2)
        ok = best[:, :k] == x
    elif "draft" in s:
        zq = s["draft"].float()
        mq, total_q = _sums(zq, case["t_draft"])
        zqx = zq.gather(2, x[..., None])[..., 0].double()
        qx = ((zqx - mq) / case["t_draft"]).exp() / total_q
        ok = s["uniform"].double() * qx < px
    else:
        ok = s["uniform"].double() < px
    step = torch.arange(k + 1, device=z.device)
    ok = ok & (step[:k] < length[:, None])
    n_ok = ok.long().cumprod(dim=1).sum(dim=1)
    seq = torch.arange(b, device=z.device)
    row = z[seq, n_ok].double()
    if case["t"] == 0.0:
        drawn = best[seq, n_ok]
    else:
        # the race over the row behind the last accepted draft, in 64 bits: two
        # ids may lie next to each other
        p = ((row - m[seq, n_ok, None]) / t).exp() / total[seq, n_ok, None]
        if k:
            at = n_ok.clamp(max=k - 1)
            if "draft" in s:
                q = ((zq[seq, at].double() - mq[seq, at, None]) / case["t_draft"]).exp()
                q = q / total_q[seq, at, None]
            else:
                q = torch.zeros_like(p).scatter_(1, x[seq, at, None], 1.0)
            rest = torch.where((n_ok < length)[:, None], (p - q).clamp(min=0.0), p)
            p = torch.where((rest > 0).any(dim=1, keepdim=True), rest, p)
        drawn = (p / s["noise"].double()).argmax(dim=1)
    tokens = torch.where(step < n_ok[:, None],
                         torch.cat([x, torch.zeros_like(x[:, :1]) if k else drawn[:, None]], 1),
                         torch.full((b, k + 1), IGNORE, device=z.device))
    tokens[seq, n_ok] = drawn
    zy = z.gather(2, tokens.clamp(min=0)[..., None])[..., 0].double()
    lp = (zy - m) / t - total.log()
    lp = torch.where(step <= n_ok[:, None], lp, torch.zeros_like(lp))
    return {"tokens": tokens, "accepted": n_ok.int(), "logprob": lp.float()}


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op == "verify":
        return _plain_verify(s)
    if op == "embed":
        on = (s["tokens"] != IGNORE)[:, None]
        h = s["w"][s["tokens"].clamp(min=0)].float() * case["scale"]
        return {"h": torch.where(on, h, torch.zeros_like(h)).to(dt)}
    if op == "embed_grad":
        on = (s["tokens"] != IGNORE)[:, None]
        g = s["d_h"].float() * case["scale"]
        g = torch.where(on, g, torch.zeros_like(g))
        d_w = s["d_w"].float() if case["accumulate"] else torch.zeros(s["d_w"].shape,
                                                                      device=g.device)
        if case["accumulate"] and dt == torch.float32:
            d_w = d_w.clone()
        s["d_w"].copy_(d_w.index_add_(0, s["tokens"].clamp(min=0), g))
        return {"d_w": s["d_w"]}
    x, w = s["x"].float(), s["weight"].float() + case["offset"]
    if op == "norm":
        if "residual" in s:
            x = x + s["residual"].float()
        h = x * (x.square().mean(dim=1, keepdim=True) + EPS).rsqrt() * w
        return {"h": h.to(dt), "sum": x.to(dt)} if "residual" in s else {"h": h.to(dt)}
    r = (x.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
    d_h = s["d_h"].float()
    g = d_h * w
    d_x = r * g - x * (r * r * r * (g * x).mean(dim=1, keepdim=True))
    if "residual" in s:
        d_x = d_x + s["residual"].float()
    return {"d_x": d_x.to(dt), "d_weight": (d_h * x * r).sum(dim=0).to(dt)}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from lm_head_cross_vocab_gb300 import kd

    case, kept = s["case"], s["kept"]
    op = case["op"]
    if op == "verify":
        if not kept:
            kept["ws"] = kd.Workspace()
            kept["problem"] = kd.VerifyProblem(
                n_seqs=case["b"], n_drafts=case["k"], vocab=case["v"], dtype=case["dtype"],
                t_target=case["t"], t_draft=case["t_draft"], ignore_index=IGNORE)
            kept["tensors"] = {"target_logits": s["target"], "draft_logits": s.get("draft"),
                               "drafts": s["drafts"], "lengths": s["lengths"],
                               "uniform": s["uniform"], "noise": s["noise"]}
        r = kept["out"] = kd.verify_drafts(kept["problem"], kept["tensors"], workspace=kept["ws"],
                                           check=False, out=kept.get("out"))
        return {name: r[name] for name in ("tokens", "accepted", "logprob")}
    if op in ("embed", "embed_grad"):
        if not kept:
            kept["ws"] = kd.Workspace()
            kept["problem"] = kd.EmbedProblem(
                n_tokens=case["n"], vocab=case["v"], d_model=case["d"], dtype=case["dtype"],
                scale=case["scale"], ignore_index=IGNORE)
            kept["out"] = {"d_w": s["d_w"]} if op == "embed_grad" else None
        if op == "embed":
            r = kept["out"] = kd.embed_tokens(kept["problem"], s["w"], s["tokens"], check=False,
                                              out=kept["out"])
            return {"h": r["h"]}
        r = kept["out"] = kd.embed_tokens_backward(
            kept["problem"], s["tokens"], s["d_h"], accumulate=case["accumulate"],
            workspace=kept["ws"], check=False, out=kept["out"])
        return {"d_w": r["d_w"]}
    if not kept:
        kept["ws"] = kd.Workspace()
        kept["problem"] = kd.NormProblem(n_tokens=case["n"], d_model=case["d"],
                                         dtype=case["dtype"], eps=EPS,
                                         weight_offset=case["offset"])
    if op == "norm":
        r = kept["out"] = kd.rms_norm(kept["problem"], s["x"], s["weight"],
                                      residual=s.get("residual"), out=kept.get("out"))
        return {name: r[name] for name in (("h", "sum") if "residual" in s else ("h",))}
    r = kept["out"] = kd.rms_norm_backward(kept["problem"], s["x"], s["weight"], s["d_h"],
                                           d_sum=s.get("residual"), workspace=kept["ws"],
                                           out=kept.get("out"))
    return {"d_x": r["d_x"], "d_weight": r["d_weight"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "verify":
        b, k, v = case["b"], case["k"], case["v"]
        drafts = sum(_lengths(case))
        draft_rows = drafts if case["draft"] == "logits" and case["t"] else 0
        rows = drafts + b + draft_rows
        noise = 4 * b * v if case["t"] else 0
        return {"bytes": size * rows * v + noise + 12 * drafts + b * (k + 1) * 12 + 8 * b,
                "flops": 4 * rows * v + 6 * b * v}
    if op == "embed":
        return {"bytes": 2 * case["n"] * case["d"] * size + 8 * case["n"],
                "flops": case["n"] * case["d"]}
    if op == "embed_grad":
        n, v, d = case["n"], case["v"], case["d"]
        # ids that occur, as text has them (an expectation)
        per = n * (1 - case["ignore"]) / math.log(v / 2.7 + 1.0)
        used = sum(1.0 - math.exp(-per * math.log1p(1.0 / (i + 2.7))) for i in range(v))
        rows = 2 * used if case["accumulate"] else v
        return {"bytes": (n * (1 - case["ignore"]) + rows) * d * size + 8 * n,
                "flops": 2 * n * d}
    n, d = case["n"], case["d"]
    if op == "norm":
        return {"bytes": (4 if case["residual"] else 2) * n * d * size + d * size,
                "flops": 6 * n * d}
    return {"bytes": (4 if case["residual"] else 3) * n * d * size + 2 * d * size,
            "flops": 12 * n * d}


# ---------------------------------------------------------------- 64 bits

def _exact_verify(case, s):
    t = case["t"] or 1.0
    logprob = torch.zeros(case["b"], case["k"] + 1, dtype=torch.float64, device="cuda")
    u = s["uniform"].double().cpu().tolist()
    for i, length in enumerate(_lengths(case)):
        lp = torch.log_softmax(s["target"][i, :length + 1].double() / t, dim=1)
        left, j = None, 0
        while j < length:
            x = int(s["drafts"][i, j])
            if case["t"] == 0.0:
                good = int(s["target"][i, j].float().argmax()) == x
            else:
                if "draft" in s:
                    q = torch.softmax(s["draft"][i, j].double() / case["t_draft"], dim=0)
                else:
                    q = torch.zeros(case["v"], dtype=torch.float64, device="cuda")
                    q[x] = 1.0
                p = lp[j].exp()
                good = u[i][j] * float(q[x]) < float(p[x])
                left = torch.relu(p - q)
            if not good:
                break
            logprob[i, j] = lp[j, x]
            j += 1
        if case["t"] == 0.0:
            y = int(s["target"][i, j].float().argmax())
        else:
            weight = left if j < length and float(left.sum()) > 0 else lp[j].exp()
            # the first arrival of exponential clocks of these rates
            y = int((s["noise"][i].double().log() - weight.log()).argmin())
        logprob[i, j] = lp[j, y]
    return {"tokens": None, "accepted": None, "logprob": logprob}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(case, s)
    if op in ("embed", "embed_grad"):
        tokens = s["tokens"]
        live = torch.nonzero(tokens != IGNORE)[:, 0]
        if op == "embed":
            h = torch.zeros(case["n"], case["d"], dtype=torch.float64, device="cuda")
            h[live] = s["w"].index_select(0, tokens[live]).double() * case["scale"]
            return {"h": h}
        d_w = s["d_w"].double() if case["accumulate"] else torch.zeros(
            s["d_w"].shape, dtype=torch.float64, device="cuda")
        d_w.index_put_((tokens[live],), s["d_h"][live].double() * case["scale"], accumulate=True)
        return {"d_w": d_w}
    leaf = s["x"].double()
    if op == "norm" and "residual" in s:
        leaf = leaf + s["residual"].double()
    weight = s["weight"].double() + case["offset"]
    if op == "norm":
        scale = leaf.norm(dim=1, keepdim=True).square() / case["d"] + EPS
        out = {"h": weight * leaf / scale.sqrt()}
        if "residual" in s:
            out["sum"] = leaf
        return out
    leaf.requires_grad_()
    weight.requires_grad_()
    h = weight * leaf / (leaf.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt()
    d_x, d_w = torch.autograd.grad(h, (leaf, weight), s["d_h"].double())
    if "residual" in s:
        d_x = d_x + s["residual"].double()
    return {"d_x": d_x, "d_weight": d_w}
