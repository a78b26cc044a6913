"""Token log-probabilities on the GPU (kd_logprob_*) against the fp64 oracle.

Tolerances, in units of u = 2^-24 (half a step of fp32 near 1), derived from
the sums the kernels form; none is fitted to a run.  With x = (z - max z) / T:
  * each exponential has a relative error of at most (4 |x| + 8) u (rounding of
    z - max z, of the scale, of the product, 2 ulp of ex2); weighted with p the
    |x| average to at most log V + 1 (the entropy bound), and a sum of V terms
    over at least 256 accumulators has at most V/256 + 24 further roundings:
    S, and with it log S, is off by e_S = (V/256 + 32 + 4 (log V + 1)) u.
  * log p = x - log S: e_S + (2 |x| + 2 |log p| + 4) u.
  * entropy = log S - t/S: e_S plus e_S relative on t/S <= log V + 1:
    e_S (log V + 3).
  * dz = p (c0 + c1 log p): p is off by (4 |x| + 16) u + e_S relative, the
    bracket by (e_H |g_H| + 8 u (|g_l| + |g_H| (|log p| + H + log V)));
    plus half a step of the gradient's own type (u for fp32, 2^-8 for bf16),
    and the smallest fp32 / bf16 normal number (results below are flushed).
"""
import math

import numpy as np
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd
from oracle import token_oracle as O
from oracle.kd_oracle import as_f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24
TINY = 2.0 ** -126
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _logits(n, v, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, v, generator=g) * std).to(DT[dtype])


def _tokens(n, v, seed, ignore=0.2):
    g = torch.Generator().manual_seed(seed + 1)
    y = torch.randint(0, v, (n,), generator=g)
    y[torch.rand(n, generator=g) < ignore] = IGN
    return y


def _e_s(v):
    return (v / 256 + 32 + 4 * (math.log(v) + 1)) * U


def _spread(z, t):
    """|z - max z| / T of every finite logit, 0 elsewhere."""
    z = as_f64(z)
    with np.errstate(invalid="ignore"):
        x = np.abs(z - z.max(axis=1, keepdims=True)) / t
    return np.where(np.isfinite(x), x, 0.0)


def _close(got, ref, tol, what):
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape
    with np.errstate(over="ignore"):  # beyond fp32: its infinity
        ref = np.where(np.isinf(ref.astype(np.float32)), np.sign(ref) * math.inf, ref)
    fin = np.isfinite(ref)
    assert (np.isnan(got) == np.isnan(ref)).all(), what
    odd = ~fin & ~np.isnan(ref)
    assert (got[odd] == ref[odd]).all(), what
    tol = np.broadcast_to(tol, ref.shape)
    bad = np.abs(got - ref)[fin] > tol[fin]
    assert not bad.any(), (what, np.abs(got - ref)[fin][bad].max(), tol[fin][bad].min())


def _check_forward(out, z, y, t, k, has_tokens=True):
    """z: the exact logits [N, V] (any dtype, CPU)."""
    ref = O.forward(z, None if not has_tokens else y.tolist(), temperature=t, topk=k,
                    ignore_index=IGN)
    n, v = z.shape
    es, x = _e_s(v), _spread(z, t)
    if has_tokens:
        yy = y.clamp(0, v - 1).numpy()
        tol = es + (2 * x[np.arange(n), yy] + 2 * np.nan_to_num(np.abs(ref["logprob"]), posinf=0)
                    + 4) * U
        _close(out["logprob"].cpu(), ref["logprob"], tol, "logprob")
    _close(out["entropy"].cpu(), ref["entropy"], es * (math.log(v) + 3), "entropy")
    if k:
        assert (out["topk_idx"].cpu().numpy() == ref["topk_idx"]).all()
        xt = np.take_along_axis(x, ref["topk_idx"], axis=1)
        lp = np.nan_to_num(np.abs(ref["topk_logprob"]), posinf=0)
        _close(out["topk_logprob"].cpu(), ref["topk_logprob"], es + (2 * xt + 2 * lp + 4) * U,
               "topk_logprob")
    return ref


def _grad_tol(z, y, gl, gh, t, dtype):
    """(elementwise tolerance, reference) of d_logits."""
    ref = O.grad_logits(z, None if y is None else y.tolist(),
                        None if gl is None else gl.tolist(), None if gh is None else gh.tolist(),
                        temperature=t, ignore_index=IGN)
    n, v = z.shape
    zz = as_f64(z)
    zero = np.zeros(n)
    a_l = np.abs(zero if gl is None else gl.double().numpy())[:, None]
    a_h = np.abs(zero if gh is None else gh.double().numpy())[:, None]
    es, x = _e_s(v), _spread(z, t)
    with np.errstate(invalid="ignore", divide="ignore"):
        a = zz / t
        lp = a - a.max(axis=1, keepdims=True)
        lp = lp - np.log(np.exp(lp).sum(axis=1, keepdims=True))
        p = np.nan_to_num(np.exp(lp))
        lp = np.where(p > 0, np.abs(lp), 0.0)
    lv = math.log(v) + 1
    bracket = a_l + a_h * (lp + lv)
    tol = p * (((4 * x + 16) * U + es) * bracket + a_h * es * (lv + 2) + 8 * U * bracket) / t
    return tol + HALF[dtype] * (np.abs(ref) + tol) + 4 * U * a_l / t + TINY, ref


def _run(z, y, t, k, dtype, **kw):
    n, v = z.shape
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=k, dtype=dtype, temperature=t)
    tens = {"logits": z.cuda(), "tokens": None if y is None else y.cuda()}
    return p, tens, kd.token_logprobs(p, tens, **kw)


# sizes around the vectors, warps and blocks of the kernels; K from none to all
SHAPES = [(1, 1, 1), (3, 1, 0), (5, 7, 7), (4, 31, 5), (2, 256, 256), (7, 257, 20), (3, 1000, 1000),
          (2, 2047, 1024), (33, 4099, 3), (1, 5000, 100), (6, 32003, 64), (2, 40961, 1024),
          (1, 151936, 20), (1, 151937, 1000), (300, 1024, 8), (700, 9000, 1), (2, 600011, 30)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v,k", SHAPES)
def test_logits_forward_and_backward(n, v, k, dtype):
    t = (1.0, 0.7, 2.0)[(n + v) % 3]
    z, y = _logits(n, v, dtype, n + v), _tokens(n, v, n + v)
    p, tens, out = _run(z, y, t, k, dtype)
    if n * v <= 4_000_000:
        _check_forward(out, z, y, t, k)
    g = torch.Generator().manual_seed(v)
    gl, gh = torch.randn(n, generator=g), torch.randn(n, generator=g) * 0.3
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(), d_entropy=gh.cuda())
    if n * v <= 4_000_000:
        tol, ref = _grad_tol(z, y, gl, gh, t, dtype)
        _close(r["d_logits"].float().cpu(), ref, tol, "d_logits")
        assert (r["d_logits"][(y == IGN).cuda()] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_tokens_and_single_upstreams(dtype):
    z, y = _logits(9, 3001, dtype, 3), _tokens(9, 3001, 3)
    p, tens, out = _run(z, None, 1.0, 6, dtype)
    assert out["logprob"] is None
    _check_forward(out, z, y, 1.0, 6, has_tokens=False)
    gh = torch.linspace(-1, 1, 9)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_entropy=gh.cuda())
    tol, ref = _grad_tol(z, None, None, gh, 1.0, dtype)
    _close(r["d_logits"].float().cpu(), ref, tol, "entropy alone")
    p, tens, out = _run(z, y, 1.0, 0, dtype)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gh.cuda())
    tol, ref = _grad_tol(z, y, gh, None, 1.0, dtype)
    _close(r["d_logits"].float().cpu(), ref, tol, "logprob alone")
    r = kd.token_logprobs_backward(p, tens, out["stats"])
    assert (r["d_logits"] == 0).all()


def _special_rows(v, dtype):
    """Rows where a selection or a running maximum goes wrong."""
    inf, lo = math.inf, torch.finfo(DT[dtype]).min
    up = torch.linspace(-20, 20, v)
    rows = [torch.zeros(v), up, up.flip(0), torch.full((v,), lo), torch.full((v,), -inf),
            torch.full((v,), 5.0), -up.abs(), torch.where(torch.arange(v) % 2 == 0, up, -up)]
    few = torch.full((v,), -inf)
    few[v // 2], few[v - 1], few[0] = 1.0, 3.0, -2.0
    rows.append(few)
    few = torch.full((v,), lo)
    few[v // 3] = 2.0
    rows.append(few)
    neg = torch.zeros(v)
    neg[::3] = -0.0
    rows.append(neg)
    big = torch.randn(v, generator=torch.Generator().manual_seed(1)) * 1e4
    rows += [big, big * 1e30, torch.cat([torch.full((v - 1,), lo), torch.full((1,), -lo)])]
    nan = up.clone()
    nan[v // 4] = math.nan
    pinf = up.clone()
    pinf[v // 5] = inf
    one = torch.full((v,), -inf)
    one[v // 7] = math.nan
    rows += [nan, pinf, one, torch.full((v,), math.nan)]
    return torch.stack(rows).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,k", [(64, 64), (1000, 5), (1000, 257), (9001, 1024), (9000, 20)])
@pytest.mark.parametrize("t", [1.0, 0.5])
def test_special_rows(v, k, dtype, t):
    z = _special_rows(v, dtype)
    n = len(z)
    y = torch.arange(n) * 37 % v
    p, tens, out = _run(z, y, t, k, dtype)
    _check_forward(out, z, y, t, k)
    fine = [r for r in range(n) if not (torch.isnan(z[r]).any() or (z[r] == math.inf).any())]
    gl, gh = torch.linspace(-1, 1, n), torch.linspace(0.3, -0.4, n)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(), d_entropy=gh.cuda())
    tol, ref = _grad_tol(z[fine], y[fine], gl[fine], gh[fine], t, dtype)
    _close(r["d_logits"][fine].float().cpu(), ref, tol, "d_logits")
    # the same rows ignored: exact zeros, whatever they hold
    y[:] = IGN
    p, tens, out = _run(z, y, t, k, dtype)
    assert (out["logprob"] == 0).all() and (out["entropy"] == 0).all()
    assert (out["topk_idx"].cpu() == torch.arange(k).expand(n, k)).all()
    assert (out["topk_logprob"] == -math.inf).all()
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda() * math.nan,
                                   d_entropy=gh.cuda())
    assert (r["d_logits"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 6, 400])
@pytest.mark.parametrize("k", [1, 33, 700])
def test_special_rows_of_a_large_vocabulary(n, k, dtype):
    """The same kinds of rows split over the blocks of a cluster (few rows) and
    in one block each, against a stable sort."""
    v = 70001
    kinds = _special_rows(v, dtype)[:14].cuda()  # (no NaN or +infinity)
    z = kinds[torch.arange(n, device="cuda") % len(kinds) if n > 1 else [0]].contiguous()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=k, dtype=dtype)
    out = kd.token_logprobs(p, {"logits": z})
    order = torch.sort(z.double(), dim=1, descending=True, stable=True)[1]
    assert torch.equal(out["topk_idx"], order[:, :k].int())
    lp = torch.log_softmax(z.double(), dim=1).gather(1, order[:, :k])
    dead = (z == -math.inf).all(dim=1)
    lp[dead] = -math.inf
    x = (z.double().amax(dim=1, keepdim=True) - z.double().gather(1, order[:, :k])).nan_to_num(0.0)
    tol = _e_s(v) + (2 * x + 2 * lp.abs().nan_to_num(0.0, posinf=0.0) + 4) * U
    got, fin = out["topk_logprob"].double(), torch.isfinite(lp.float())
    assert torch.equal(torch.isfinite(got), fin)
    assert ((got - lp).abs()[fin] <= tol[fin]).all()
    assert (got[~fin] == -math.inf).all() and (out["entropy"][dead] == 0).all()


def _hard_rows(v, dtype, seed):
    """Rows whose best ids lie together, are many, few, or hard to tell apart."""
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(10, v, generator=g) * 3
    rows[1] = torch.linspace(-8, 8, v)
    rows[2] = torch.linspace(8, -8, v)
    rows[3] = rows[3].round()                       # long runs of equal values
    rows[4] = -1.5
    rows[5] = -math.inf
    rows[5, torch.randint(0, v, (9,), generator=g)] = torch.randn(9, generator=g)
    for i in range(64):                             # 64 bytes in each 16384: one warp's
        rows[6, i * 8192 % max(v - 32, 1):][:32] += 20
    rows[7, -min(v, 1100):] += 30                   # the end of the row
    rows[8] = -rows[8].abs()
    rows[8, ::97] = 0.0                             # the two zeros are equal
    rows[8, ::89] = -0.0
    rows[9] = -rows[9].abs() - 1
    rows[9, ::101] = -0.0
    if dtype == "fp32":                             # just below them
        rows[9, 1::101] = -1e-40
        rows[9, 2::101] = -3e-39
    return rows.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v", [(1, 16411), (3, 151937), (9, 65543), (45, 40001), (170, 33001),
                                 (650, 9001), (650, 33001), (650, 151936), (1300, 1003)])
def test_alternatives_of_hard_rows(n, v, dtype):
    """The ids of one row to several blocks, and of blocks to one row, around the
    numbers of alternatives at which the selection changes: exact, and the same
    in every copy of a row; the statistics do not depend on the alternatives."""
    base = _hard_rows(v, dtype, n + v)
    order = torch.sort(base.float() + 0.0, dim=1, descending=True, stable=True).indices
    pick = torch.arange(n) % 10 if n > 9 else torch.arange(10)
    for start in range(0, len(pick), n):            # few rows: a few at a time
        rows = pick[start:start + n]
        z = base[rows]
        y = order[rows, 0].contiguous()
        ref = None
        for k in (0, 1, 14, 28, 29, 57, 64, 65, 113, 114, 128, 129, 300, 1000):
            if k > v:
                continue
            _, _, out = _run(z, y, 1.0, k, dtype)
            if k:
                assert (out["topk_idx"].cpu() == order[rows, :k]).all(), (k, rows.tolist()[:10])
                fin = torch.isfinite(out["logprob"])
                assert torch.equal(out["topk_logprob"][fin, 0], out["logprob"][fin]), k
            if ref is None:
                ref = out
            _close(out["entropy"].cpu(), ref["entropy"].cpu().double().numpy(),
                   2 * _e_s(v) * (math.log(v) + 3), ("entropy", k))
            _close(out["logprob"].cpu(), ref["logprob"].cpu().double().numpy(),
                   2 * _e_s(v) + 8 * U * 40, ("logprob", k))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,pitch,shift", [(1000, 1000, 1), (1000, 1003, 0), (1001, 1016, 3),
                                           (4096, 4104, 8), (32003, 32100, 5)])
def test_pitches_and_unaligned_rows(v, pitch, shift, dtype):
    n = 5
    store = _logits(1, n * pitch + shift, dtype, v).reshape(-1).cuda()
    z = store[shift:shift + n * pitch].view(n, pitch)[:, :v]
    y = _tokens(n, v, v)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=9, dtype=dtype)
    tens = {"logits": z, "tokens": y.cuda()}
    out = kd.token_logprobs(p, tens)
    _check_forward(out, z.cpu(), y, 1.0, 9)
    gl = torch.linspace(-1, 1, n)
    grad = torch.full_like(store, 7.0)
    dz = grad[shift:shift + n * pitch].view(n, pitch)[:, :v]
    kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(),
                               out={"d_logits": dz, "dev_status": out["dev_status"]})
    tol, ref = _grad_tol(z.cpu(), y, gl, None, 1.0, dtype)
    _close(dz.float().cpu(), ref, tol, "d_logits")
    between = torch.ones_like(grad, dtype=torch.bool)
    between[shift:shift + n * pitch].view(n, pitch)[:, :v] = False
    assert (grad[between] == 7.0).all()
    # into the logits' own memory, and into a dense tensor
    dense = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda())["d_logits"]
    assert torch.equal(dense, dz)
    kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(),
                               out={"d_logits": z, "dev_status": out["dev_status"]})
    assert torch.equal(z, dz)


def test_bad_tokens_are_reported():
    z, y = _logits(4, 100, "fp32", 1), torch.tensor([3, 100, -1, 99])
    with pytest.raises(kd.KDError) as e:
        _run(z, y, 1.0, 2, "fp32")
    assert e.value.status == kd.KD_ERR_BAD_LABEL
    p, tens, out = _run(z, y, 1.0, 2, "fp32", check=False)
    _check_forward(out, z, y, 1.0, 2)
    assert int(out["dev_status"].item()) == kd.KD_DEV_BAD_LABEL
    gl = torch.ones(4)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(), check=False)
    tol, ref = _grad_tol(z, y, gl, None, 1.0, "fp32")
    _close(r["d_logits"].cpu(), ref, tol, "d_logits")
    assert int(r["dev_status"].item()) == kd.KD_DEV_BAD_LABEL


def test_no_tokens_no_rows():
    for kw in (dict(source="logits"), dict(source="hidden", d_model=64)):
        p = kd.LogprobProblem(n_tokens=0, vocab=300, topk=3, **kw)
        bf = torch.bfloat16
        tens = {"logits": torch.empty(0, 300, dtype=bf, device="cuda"),
                "h": torch.empty(0, 64, dtype=bf, device="cuda"),
                "w": torch.ones(300, 64, dtype=bf, device="cuda"),
                "tokens": torch.empty(0, dtype=torch.int64, device="cuda")}
        out = kd.token_logprobs(p, tens)
        assert out["topk_idx"].shape == (0, 3)
        r = kd.token_logprobs_backward(p, tens, out["stats"])
        if kw["source"] == "hidden":
            assert (r["d_w"] == 0).all()


# ------------------------------------------------------------------ hidden states

def _hidden(n, v, d, dtype, seed, grid=True):
    """On the grid every logit is an exact sum (products of multiples of 2^-4
    and 2^-10, fewer than 2^24 units in all), so the logits are known exactly."""
    g = torch.Generator().manual_seed(seed)
    h, w = torch.randn(n, d, generator=g), torch.randn(v, d, generator=g) * 0.05
    if grid:
        h = (h * 16).round().clamp(-64, 64) / 16
        w = (w * 1024).round().clamp(-255, 255) / 1024
    return h.to(DT[dtype]), w.to(DT[dtype])


def _exact(h, w):
    return h.double() @ w.double().t()


HIDDEN = [(1, 1, 8, 1), (1, 700, 64, 7), (5, 33, 8, 33), (3, 257, 72, 20), (70, 1000, 136, 5),
          (130, 2049, 64, 100), (257, 5003, 200, 33), (300, 513, 520, 0), (17, 6000, 1032, 1024),
          (1, 9001, 4096, 300), (1000, 3001, 256, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d,k", HIDDEN)
def test_hidden_forward(n, v, d, k, dtype):
    t = (1.0, 0.7)[v % 2]
    h, w = _hidden(n, v, d, dtype, n + v)
    y = _tokens(n, v, n + v)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, dtype=dtype, source="hidden",
                          temperature=t)
    tens = {"h": h.cuda(), "w": w.cuda(), "tokens": y.cuda()}
    out = kd.token_logprobs(p, tens)
    _check_forward(out, _exact(h, w), y, t, k)
    # the same logits, materialised in fp32 (exact), give the same alternatives
    q = kd.LogprobProblem(n_tokens=n, vocab=v, topk=k, dtype="fp32", temperature=t)
    ref = kd.token_logprobs(q, {"logits": _exact(h, w).float().cuda(), "tokens": y.cuda()})
    if k:
        assert torch.equal(out["topk_idx"], ref["topk_idx"])
    es = _e_s(v)
    assert torch.allclose(out["entropy"], ref["entropy"], rtol=0, atol=2 * es * (math.log(v) + 3))


@pytest.mark.parametrize("n,v", [(1, 40000), (5, 6000), (1100, 20000), (9000, 3000)])
@pytest.mark.parametrize("k", [1, 20, 128])
def test_hidden_alternatives_of_ordered_rows(n, v, k):
    """Rows whose logits rise or fall with the id, have long runs of equal
    values, or are all equal (a zero hidden state), between ordinary ones, over
    several tiles of a part; against a stable sort of the exact logits."""
    d = 64
    h, w = _hidden(n, v, d, "bf16", v)
    ids = torch.arange(v)
    w[:, 0] = (ids // 256 / 8).to(w.dtype)       # exact: at most 8 bits each
    w[:, 1] = (ids % 256 / 2048).to(w.dtype)
    kind = torch.arange(n) % 6
    h[kind > 0] = 0
    h[kind == 1, :2] = 1.0
    h[kind == 2, :2] = -1.0
    h[kind == 3, 0] = 1.0
    h[kind == 4, 1] = -2.0
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, source="hidden")
    out = kd.token_logprobs(p, {"h": h.cuda(), "w": w.cuda()})
    z = (h.cuda().double() @ w.cuda().double().t()).float()  # exact
    best, order = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(out["topk_idx"], order[:, :k].int())
    lp = torch.log_softmax(z.double(), dim=1).gather(1, order[:, :k])
    tol = _e_s(v) + (2 * (best[:, :1] - best[:, :k]).double() + 2 * lp.abs() + 4) * U
    assert ((out["topk_logprob"].double() - lp).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v,d", [(1, 700, 64), (3, 257, 72), (130, 2049, 64), (257, 5003, 200),
                                   (300, 513, 520), (600, 700, 136)])
def test_hidden_backward(n, v, d, dtype):
    """d_h = G W and d_w = G^T H: |error| is at most the product of the matrices
    of absolute values with G's own error (its tolerance: half a step of its
    type, which is bf16 for bf16 problems), K roundings of the fp32 sum, and
    half a step of the result."""
    t = (1.0, 0.7)[v % 2]
    h, w = _hidden(n, v, d, dtype, n + v)
    y = _tokens(n, v, n + v)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, dtype=dtype, source="hidden",
                          temperature=t)
    bad = h.clone()
    bad[y == IGN] = math.nan  # rows that take no part may hold anything
    tens = {"h": bad.cuda(), "w": w.cuda(), "tokens": y.cuda()}
    out = kd.token_logprobs(p, tens)
    z = _exact(h, w)
    _check_forward(out, z, y, t, 0)
    g = torch.Generator().manual_seed(v)
    gl, gh = torch.randn(n, generator=g), torch.randn(n, generator=g) * 0.3
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(), d_entropy=gh.cuda())
    g_tol, g_ref = _grad_tol(z, y, gl, gh, t, dtype)
    hh, ww = as_f64(h), as_f64(w)
    for name, a, at, b in (("d_h", g_ref, g_tol, ww), ("d_w", g_ref.T, g_tol.T, hh)):
        ref = a @ b
        mass = (np.abs(a) + at) @ np.abs(b)
        # twice u: the tensor cores may cut a sum off instead of rounding it
        tol = at @ np.abs(b) + 2 * U * a.shape[1] * mass
        tol = tol + HALF[dtype] * (np.abs(ref) + tol) + TINY
        _close(r[name].float().cpu(), ref, tol, name)
    assert (r["d_h"][(y == IGN).cuda()] == 0).all()
    one = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(),
                                     d_entropy=gh.cuda(), want=("w",))
    assert "d_h" not in one and torch.equal(one["d_w"], r["d_w"])


@pytest.mark.parametrize("n,v,d", [(2100, 9000, 64), (700, 30000, 264), (5000, 5003, 136)])
@pytest.mark.parametrize("want", [("h", "w"), ("h",), ("w",)])
def test_hidden_backward_in_chunks(n, v, d, want):
    """Problems whose gradient is made in several chunks of tokens and columns,
    against the formula in fp64 (torch, on the same device), with the bound of
    test_hidden_backward; three calls in a row give the same bits."""
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", n + v))
    y = _tokens(n, v, n).cuda()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens = {"h": h, "w": w, "tokens": y}
    out = kd.token_logprobs(p, tens)
    g = torch.Generator().manual_seed(v)
    gl, gh = (torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 0.3)
    lp = torch.log_softmax(h.double() @ w.double().t(), dim=1)
    pr, on = lp.exp(), (y != IGN)[:, None]
    ent = -(pr * lp).sum(dim=1, keepdim=True)
    a, b = gl.double()[:, None], gh.double()[:, None]
    gz = -pr * (a + b * (lp + ent))
    tol = pr * ((a.abs() + b.abs() * (lp.abs() + math.log(v) + 1)) * 200 * U
                + b.abs() * _e_s(v) * (math.log(v) + 3))
    gz[torch.arange(n), y.clamp(min=0)] += a[:, 0]
    gz, tol = torch.where(on, gz, 0.0), torch.where(on, tol, 0.0)
    tol = tol + 2.0 ** -8 * (gz.abs() + tol) + 4 * U * a.abs() * on
    ws, kept = kd.Workspace(), []
    for _ in range(3):
        r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl, d_entropy=gh,
                                       want=want, workspace=ws)
        kept.append(r)
    for name, x, xt, m in (("d_h", gz, tol, w.double()), ("d_w", gz.t(), tol.t(), h.double())):
        if name[2:] not in want:
            continue
        ref = x @ m
        off = xt @ m.abs() + 2 * U * x.shape[1] * ((x.abs() + xt) @ m.abs())
        off = off + 2.0 ** -8 * (ref.abs() + off) + TINY
        assert ((kept[0][name].double() - ref).abs() <= off).all(), name
        assert all(torch.equal(kept[0][name], r[name]) for r in kept[1:])


@pytest.mark.parametrize("v,k", [(300, 5), (30000, 128), (30000, 200)])
def test_hidden_rows_that_are_not_finite(v, k):
    """A hidden state with a NaN, and one that overflows the logits: that row is
    NaN (its alternatives by id, a NaN above every number), the others are as
    without it."""
    n, d = 70, 64
    h, w = _hidden(n, v, d, "bf16", 5)
    y = _tokens(n, v, 5, ignore=0.0)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, source="hidden")
    ref = kd.token_logprobs(p, {"h": h.cuda(), "w": w.cuda(), "tokens": y.cuda()})
    bad = h.clone()
    bad[3, 7], bad[40] = math.nan, math.inf
    out = kd.token_logprobs(p, {"h": bad.cuda(), "w": w.cuda(), "tokens": y.cuda()})
    fine = [r for r in range(n) if r not in (3, 40)]
    for name in ("logprob", "entropy", "topk_idx", "topk_logprob"):
        assert torch.equal(out[name][fine], ref[name][fine]), name
    for r in (3, 40):
        assert out["logprob"][r].isnan() and out["entropy"][r].isnan()
        assert out["topk_logprob"][r].isnan().all()
    assert out["topk_idx"][3].tolist() == list(range(k))


def test_single_cta_tiles(monkeypatch):
    """The CTA-pair tiles off (a debug override): the same alternatives, and
    sums and gradients that differ by their order only."""
    n, v, d, k = 300, 5003, 200, 20
    h, w = _hidden(n, v, d, "bf16", 9)
    y = _tokens(n, v, 9)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, source="hidden")
    tens = {"h": h.cuda(), "w": w.cuda(), "tokens": y.cuda()}
    gl = torch.linspace(-1, 1, n).cuda()
    ref = kd.token_logprobs(p, tens)
    grad = kd.token_logprobs_backward(p, tens, ref["stats"], d_logprob=gl)
    monkeypatch.setenv("KD_TC_PAIR", "0")
    out = kd.token_logprobs(p, tens)
    _check_forward(out, _exact(h, w), y, 1.0, k)
    assert torch.equal(out["topk_idx"], ref["topk_idx"])
    one = kd.token_logprobs_backward(p, tens, ref["stats"], d_logprob=gl)
    for name in ("d_h", "d_w"):
        a, b = one[name].double(), grad[name].double()
        # the sums differ by some u, so that a result may round the other way
        assert ((a - b).abs() <= 2 * HALF["bf16"] * b.abs() + 1e-5 * b.abs().max()).all()


def test_chunked_backward_in_a_graph():
    """Several chunks captured into a graph and replayed on changed inputs."""
    n, v, d = 2100, 9000, 64
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", 1))
    y = _tokens(n, v, 1).cuda()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens, gl = {"h": h, "w": w, "tokens": y}, torch.linspace(-1, 1, n).cuda()
    ws, s = kd.Workspace(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = kd.token_logprobs(p, tens, workspace=ws)
        g = kd.token_logprobs_backward(p, tens, o["stats"], d_logprob=gl, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        kd.token_logprobs(p, tens, workspace=ws, check=False, out=o)
        kd.token_logprobs_backward(p, tens, o["stats"], d_logprob=gl, workspace=ws, check=False,
                                   out=g)
    for _ in range(2):
        h.copy_(h.roll(17, 0))
        y.copy_(y.roll(5, 0))
        graph.replay()
        torch.cuda.synchronize()
        o2 = kd.token_logprobs(p, tens)
        g2 = kd.token_logprobs_backward(p, tens, o2["stats"], d_logprob=gl)
        assert torch.equal(o["stats"], o2["stats"])
        assert torch.equal(g["d_h"], g2["d_h"]) and torch.equal(g["d_w"], g2["d_w"])


def test_ignore_index_that_is_an_id_and_repeated_tokens():
    """Padding with an id of the vocabulary, and many tokens of one id: the
    bound of test_hidden_backward, and rows that take no part exactly 0."""
    n, v, d = 400, 900, 72
    h, w = _hidden(n, v, d, "bf16", 3)
    y = _tokens(n, v, 3, ignore=0.0)
    y[::3], y[1::5] = 0, 7
    y[50:53], y[60:64], y[70:75] = 11, 12, 13
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden", ignore_index=0)
    tens = {"h": h.cuda(), "w": w.cuda(), "tokens": y.cuda()}
    out = kd.token_logprobs(p, tens)
    gl = torch.linspace(-1, 1, n)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda())
    z, yy = _exact(h, w), torch.where(y == 0, IGN, y)
    g_tol, g_ref = _grad_tol(z, yy, gl, None, 1.0, "bf16")
    for name, a, at, b in (("d_h", g_ref, g_tol, as_f64(w)), ("d_w", g_ref.T, g_tol.T, as_f64(h))):
        ref = a @ b
        tol = at @ np.abs(b) + 2 * U * a.shape[1] * ((np.abs(a) + at) @ np.abs(b))
        tol = tol + HALF["bf16"] * (np.abs(ref) + tol) + TINY
        _close(r[name].float().cpu(), ref, tol, name)
    assert (r["d_h"][(y == 0).cuda()] == 0).all()


def test_gradients_by_differences():
    """The fp32 backward against central differences of the fp64 definition."""
    n, v, d = 3, 40, 8
    h, w = _hidden(n, v, d, "fp32", 11, grid=False)
    y = torch.tensor([5, IGN, 39])
    gl, gh = torch.tensor([0.7, 0.2, -1.1]), torch.tensor([-0.4, 0.3, 0.6])
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32", source="hidden",
                          temperature=0.8)
    tens = {"h": h.cuda(), "w": w.cuda(), "tokens": y.cuda()}
    out = kd.token_logprobs(p, tens)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl.cuda(), d_entropy=gh.cuda())

    def f(hh, ww):
        o = O.forward(hh @ ww.T, y.tolist(), temperature=0.8, ignore_index=IGN)
        return float(gl.double().numpy() @ o["logprob"] + gh.double().numpy() @ o["entropy"])

    hh, ww = as_f64(h), as_f64(w)
    for name, x in (("d_h", hh), ("d_w", ww)):
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            old = x[i]
            x[i] = old + 1e-4
            up = f(hh, ww)
            x[i] = old - 1e-4
            num[i] = (up - f(hh, ww)) / 2e-4
            x[i] = old
        # truncation 1e-8 |f'''| and fp32 sums: both well below 1e-5 here
        assert np.abs(r[name].cpu().double().numpy() - num).max() <= 1e-5


# ------------------------------------------------------------------ use

def test_streams_and_graphs():
    """On a side stream, and captured twice with a workspace of its own each;
    replays follow the inputs."""
    n, v, d = 40, 3000, 128
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", 5))
    y = _tokens(n, v, 5).cuda()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=12, source="hidden")
    tens = {"h": h, "w": w, "tokens": y}
    gl = torch.linspace(-1, 1, n, device="cuda")

    def call(ws, o, g):
        o = kd.token_logprobs(p, tens, workspace=ws, check=False, out=o)
        return o, kd.token_logprobs_backward(p, tens, o["stats"], d_logprob=gl, workspace=ws,
                                             check=False, out=g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o1, g1 = call(kd.Workspace(), None, None)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        ws, o, g = kd.Workspace(), None, None
        with torch.cuda.stream(s):
            o, g = call(ws, o, g)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=s):
            call(ws, o, g)
        graphs.append((cg, o, g))
    h.copy_(h.flip(0))
    y.copy_(y.flip(0))
    o2, g2 = call(kd.Workspace(), None, None)
    for cg, o, g in graphs:
        cg.replay()
        torch.cuda.synchronize()
        for key in ("logprob", "entropy", "topk_idx", "topk_logprob", "stats"):
            assert torch.equal(o[key], o2[key]), key
        assert torch.equal(g["d_h"], g2["d_h"]) and torch.equal(g["d_w"], g2["d_w"])
    assert torch.equal(o2["logprob"], o1["logprob"].flip(0))


def test_cache_teacher_then_distil_then_clip():
    """The run of calls a distillation program makes: a teacher's hidden states
    to a top-K cache, the cache to the sparse loss and its gradients, and the
    gradients clipped."""
    from oracle import kd_oracle as KO
    n, v, d, k = 96, 1500, 64, 16
    ht, wt = _hidden(n, v, 128, "bf16", 1)
    hs, ws = _hidden(n, v, d, "bf16", 2, grid=False)
    y = _tokens(n, v, 1)
    cache = kd.token_logprobs(
        kd.LogprobProblem(n_tokens=n, vocab=v, d_model=128, topk=k, source="hidden"),
        {"h": ht.cuda(), "w": wt.cuda(), "tokens": y.cuda()}, save_stats=False)
    assert cache["stats"] is None
    t = {"h_s": hs.cuda(), "w_s": ws.cuda(), "labels": y.cuda(), "topk_idx": cache["topk_idx"],
         "topk_p": cache["topk_logprob"].exp()}
    prob = kd.Problem(n_tokens=n, vocab=v, d_student=d, topk=k, teacher="topk", w_student_ce=0.0)
    fwd = kd.forward(prob, t)
    g = kd.backward(prob, t, fwd["stats"], want=("h_s", "w_s"))
    r = kd.clip_grad_norm([g["d_h_s"], g["d_w_s"]], 0.01)
    ref = O.forward(_exact(ht, wt), y.tolist(), topk=k, ignore_index=IGN)
    kw = dict(topk_idx=ref["topk_idx"], topk_p=np.exp(ref["topk_logprob"]), w_student_ce=0.0,
              ignore_index=IGN)
    zs = KO.project(hs, ws)
    loss = KO.forward(zs, None, y.numpy(), **kw)["loss"]
    assert abs(fwd["loss"].item() - loss) <= 2e-3 * abs(loss)
    gs, _ = KO.grad_logits(zs, None, y.numpy(), **kw)
    dh, dw = KO.hidden_grads(hs, ws, gs)
    norm, out = O.clip([dh, dw], 0.01)
    assert norm > 0.01 and abs(r["norm"].item() - norm) <= 1e-2 * norm
    for got, want in zip(r["grads"], out):
        err = np.linalg.norm(as_f64(got) - want) / np.linalg.norm(want)
        assert err <= 2e-2  # 1e-2 of the gradients (the loss's own bound), 1e-2 of the norm


def test_offsets_beyond_32_bits():
    """3.0e9 logits: the last rows, whose offsets pass 2^32 bytes and 2^31
    elements, are as in a call of their own."""
    n, v, tail = 20000, 151936, 40
    z = torch.empty(n, v, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    z[-tail:] = (torch.randn(tail, v, generator=g, device="cuda") * 3).bfloat16()
    z[:-tail] = 0
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    up = torch.linspace(-1, 1, n, device="cuda")
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=3)
    out = kd.token_logprobs(p, {"logits": z, "tokens": y})
    q = kd.LogprobProblem(n_tokens=tail, vocab=v, topk=3)
    last = {"logits": z[-tail:], "tokens": y[-tail:]}
    ref = kd.token_logprobs(q, last)
    assert torch.equal(out["topk_idx"][-tail:], ref["topk_idx"])
    # (a row in one block or in eight: the sums differ by their order)
    assert torch.allclose(out["stats"][-tail:], ref["stats"], rtol=2 * _e_s(v), atol=2 * _e_s(v))
    assert torch.allclose(out["logprob"][:-tail], torch.full((1,), -math.log(v), device="cuda"))
    assert out["topk_idx"][0].tolist() == [0, 1, 2]
    dz = kd.token_logprobs_backward(p, {"logits": z, "tokens": y}, out["stats"], d_logprob=up,
                                    out={"d_logits": z, "dev_status": out["dev_status"]})
    assert torch.equal(dz["d_logits"][0, :5], dz["d_logits"][0, 1000:1005])
    z2 = dz["d_logits"][-tail:].float().sum(dim=1)
    # a row of the gradient sums to 0 but for the roundings of its elements
    assert (z2.abs() <= 2.0 ** -7 * dz["d_logits"][-tail:].float().abs().sum(dim=1)).all()


def test_hidden_gradient_without_tokens():
    n, v, d = 150, 3001, 64
    h, w = _hidden(n, v, d, "bf16", 21)
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens = {"h": h.cuda(), "w": w.cuda()}
    out = kd.token_logprobs(p, tens)
    assert out["logprob"] is None
    gh = torch.linspace(-1, 1, n)
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_entropy=gh.cuda())
    g_tol, g_ref = _grad_tol(_exact(h, w), None, None, gh, 1.0, "bf16")
    for name, a, at, b in (("d_h", g_ref, g_tol, as_f64(w)), ("d_w", g_ref.T, g_tol.T, as_f64(h))):
        ref = a @ b
        tol = at @ np.abs(b) + 2 * U * a.shape[1] * ((np.abs(a) + at) @ np.abs(b))
        _close(r[name].float().cpu(), ref, tol + HALF["bf16"] * (np.abs(ref) + tol) + TINY, name)


@pytest.mark.parametrize("source", ["logits", "hidden"])
def test_outputs_can_be_left_out(source):
    n, v, d, k = 20, 2000, 64, 9
    h, w = _hidden(n, v, d, "bf16", 4)
    tens = {"h": h.cuda(), "w": w.cuda(), "tokens": _tokens(n, v, 4).cuda(),
            "logits": _logits(n, v, "bf16", 4).cuda()}
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, source=source)
    ref = kd.token_logprobs(p, tens)
    for names in (("topk_idx",), ("topk_logprob",), ("logprob",), ("entropy", "stats"), ()):
        out = {x: torch.empty_like(ref[x]) for x in names}
        out["dev_status"] = torch.zeros((), dtype=torch.int32, device="cuda")
        got = kd.token_logprobs(p, tens, out=out)
        for x in names:
            assert torch.equal(got[x], ref[x]) or (
                x != "topk_idx" and torch.allclose(got[x], ref[x], rtol=0, atol=1e-5)), (names, x)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, in flight together."""
    n, v, d, k = 500, 20000, 256, 30
    sides = []
    for i in range(2):
        h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", 30 + i))
        tens = {"h": h, "w": w, "tokens": _tokens(n, v, 30 + i).cuda()}
        p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, topk=k, source="hidden")
        up = torch.linspace(-1, 1, n, device="cuda")
        ref = kd.token_logprobs(p, tens)
        grad = kd.token_logprobs_backward(p, tens, ref["stats"], d_logprob=up)
        sides.append((torch.cuda.Stream(), kd.Workspace(), p, tens, up, ref, grad))
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, ws, p, tens, up, ref, grad in sides:
            with torch.cuda.stream(s):
                o = kd.token_logprobs(p, tens, workspace=ws, check=False)
                g = kd.token_logprobs_backward(p, tens, o["stats"], d_logprob=up, workspace=ws,
                                               check=False)
                got.append((o, g, ref, grad))
    torch.cuda.synchronize()
    for o, g, ref, grad in got:
        for x in ("logprob", "entropy", "topk_idx", "topk_logprob", "stats"):
            assert torch.equal(o[x], ref[x]), x
        assert torch.equal(g["d_h"], grad["d_h"]) and torch.equal(g["d_w"], grad["d_w"])


@pytest.mark.parametrize("n,v,d", [(2100, 9000, 64), (700, 30000, 264), (5000, 5003, 136)])
def test_hidden_backward_by_turns_on_two_sets_of_inputs(n, v, d):
    """Call after call through one workspace, the inputs changing each time: a
    value of the chunk or the call before, read in place of this one's, would
    show.  The same bits as each set's first call."""
    ws, sides = kd.Workspace(), []
    for seed in (1, 2):
        h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", seed))
        tens = {"h": h, "w": w, "tokens": _tokens(n, v, seed).cuda()}
        p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
        stats = kd.token_logprobs(p, tens)["stats"]
        up = torch.linspace(-seed, seed, n, device="cuda")
        ref = kd.token_logprobs_backward(p, tens, stats, d_logprob=up, workspace=ws)
        sides.append((p, tens, stats, up, ref))
    got = []
    for _ in range(8):
        for p, tens, stats, up, ref in sides:
            got.append((ref, kd.token_logprobs_backward(p, tens, stats, d_logprob=up, workspace=ws,
                                                        check=False)))
    for ref, r in got:
        assert torch.equal(r["d_h"], ref["d_h"]) and torch.equal(r["d_w"], ref["d_w"])
        assert int(r["dev_status"].item()) == 0


def _hidden_grads_close(n, v, d, want, seed, calls=1):
    """The bf16 hidden backward against the formula in fp64 (torch, on the same
    device), with the bound of test_hidden_backward; every call the same bits."""
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", seed))
    y = _tokens(n, v, seed).cuda()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens = {"h": h, "w": w, "tokens": y}
    out = kd.token_logprobs(p, tens)
    g = torch.Generator().manual_seed(v)
    gl, gh = (torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 0.3)
    lp = torch.log_softmax(h.double() @ w.double().t(), dim=1)
    pr, on = lp.exp(), (y != IGN)[:, None]
    ent = -(pr * lp).sum(dim=1, keepdim=True)
    a, b = gl.double()[:, None], gh.double()[:, None]
    gz = -pr * (a + b * (lp + ent))
    tol = pr * ((a.abs() + b.abs() * (lp.abs() + math.log(v) + 1)) * 200 * U
                + b.abs() * _e_s(v) * (math.log(v) + 3))
    gz[torch.arange(n), y.clamp(min=0)] += a[:, 0]
    gz, tol = torch.where(on, gz, 0.0), torch.where(on, tol, 0.0)
    tol = tol + 2.0 ** -8 * (gz.abs() + tol) + 4 * U * a.abs() * on
    ws = kd.Workspace()
    kept = [kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl, d_entropy=gh,
                                       want=want, workspace=ws) for _ in range(calls)]
    for name, x, xt, m in (("d_h", gz, tol, w.double()), ("d_w", gz.t(), tol.t(), h.double())):
        if name[2:] not in want:
            continue
        ref = x @ m
        off = xt @ m.abs() + 2 * U * x.shape[1] * ((x.abs() + xt) @ m.abs())
        off = off + 2.0 ** -8 * (ref.abs() + off) + TINY
        assert ((kept[0][name].double() - ref).abs() <= off).all(), name
        assert all(torch.equal(kept[0][name], r[name]) for r in kept[1:])


# On 152 SMs the products of a whole chunk take 2, 12, 2, 2 and 3 parts of K; the
# last chunk has 13, 428, 40, 20 and 17 columns, 1, 7, 1, 1 and 1 blocks of 64.
@pytest.mark.parametrize("n,v,d", [(1813, 5133, 96), (8, 399788, 272), (3439, 5160, 144),
                                   (2629, 5140, 456), (1287, 7697, 680)])
@pytest.mark.parametrize("want", [("h", "w"), ("h",)])
def test_hidden_backward_with_a_narrow_last_chunk(n, v, d, want):
    _hidden_grads_close(n, v, d, want, n + v, calls=2)


def test_a_reused_out_after_a_bad_token():
    """An error that was raised is told: the next call with the same dict of
    outputs and good tokens passes, in both directions."""
    n, v = 6, 500
    z, y = _logits(n, v, "fp32", 2).cuda(), torch.arange(n, device="cuda")
    p = kd.LogprobProblem(n_tokens=n, vocab=v, dtype="fp32")
    good, bad = {"logits": z, "tokens": y}, {"logits": z, "tokens": y + v}
    out = kd.token_logprobs(p, good)
    up = torch.ones(n, device="cuda")
    grad = kd.token_logprobs_backward(p, good, out["stats"], d_logprob=up)
    ref = out["logprob"].clone(), grad["d_logits"].clone()
    with pytest.raises(kd.KDError):
        kd.token_logprobs(p, bad, out=out)
    assert torch.equal(kd.token_logprobs(p, good, out=out)["logprob"], ref[0])
    with pytest.raises(kd.KDError):
        kd.token_logprobs_backward(p, bad, out["stats"], d_logprob=up, out=grad)
    r = kd.token_logprobs_backward(p, good, out["stats"], d_logprob=up, out=grad)
    assert torch.equal(r["d_logits"], ref[1])
    # without a check the bits stay for the caller
    kd.token_logprobs(p, bad, out=out, check=False)
    assert int(kd.token_logprobs(p, good, out=out, check=False)["dev_status"].item()) \
        == kd.KD_DEV_BAD_LABEL


def test_out_with_the_gradients_alone():
    """``out`` may bring the gradients and no status word: over the logits, and
    a head's gradients into a caller's buffers."""
    n, v, d = 30, 700, 64
    z, y = _logits(n, v, "bf16", 8).cuda(), _tokens(n, v, 8).cuda()
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=3)
    out = kd.token_logprobs(p, {"logits": z, "tokens": y})
    up = torch.linspace(-1, 1, n, device="cuda")
    ref = kd.token_logprobs_backward(p, {"logits": z, "tokens": y}, out["stats"], d_logprob=up)
    r = kd.token_logprobs_backward(p, {"logits": z, "tokens": y}, out["stats"], d_logprob=up,
                                   out={"d_logits": z})
    assert torch.equal(z, ref["d_logits"]) and int(r["dev_status"].item()) == 0
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", 8))
    q = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens = {"h": h, "w": w, "tokens": y}
    r = kd.token_logprobs(q, tens, out={"logprob": torch.empty(n, device="cuda"),
                                        "stats": torch.empty(n, 4, device="cuda")})
    assert int(r["dev_status"].item()) == 0
    ref = kd.token_logprobs_backward(q, tens, r["stats"], d_logprob=up)
    g = kd.token_logprobs_backward(q, tens, r["stats"], d_logprob=up,
                                   out={"d_w": torch.empty_like(w)})
    assert torch.equal(g["d_w"], ref["d_w"])


@pytest.mark.parametrize("tokens", ["uniform", "sampled"])
@pytest.mark.parametrize("scale", [1, 16])
@pytest.mark.parametrize("n,v,d", [(500, 2000, 256), (900, 7000, 64), (40, 3001, 128)])
def test_the_tokens_own_element_keeps_more_than_bf16(n, v, d, scale, tokens):
    """G is rounded to bf16, and what that takes from a token's own element goes
    into both products all the same.  Both forms of the products, of G rounded
    and of G rounded but there, are made in fp64 and rounded to bf16; the
    library's has to be as near the exact one as the latter, which lies clearly
    nearer than the former.  (G in fp32 is off by some 1e-6 relative: one element
    in a thousand rounds the other way, from one side of the exact value to the
    other about as far, so that the norm of the error, over n d roundings or v d,
    stays within 2 %.)"""
    h, w = (x.cuda() for x in _hidden(n, v, d, "bf16", n))
    h *= scale  # (exact; 16: the likeliest id has 0.6 to 0.8 on average)
    z = h.double() @ w.double().t()
    lp = torch.log_softmax(z, dim=1)
    g = torch.Generator(device="cuda").manual_seed(n)
    if tokens == "uniform":
        y = torch.randint(0, v, (n,), generator=g, device="cuda")
    else:
        y = torch.multinomial(lp.exp(), 1, generator=g)[:, 0]
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    tens = {"h": h, "w": w, "tokens": y}
    out = kd.token_logprobs(p, tens)
    up = torch.randn(n, generator=g, device="cuda")
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=up)
    gz = -lp.exp() * up.double()[:, None]
    rows = torch.arange(n, device="cuda")
    gz[rows, y] += up.double()
    cut = gz.bfloat16().double()
    own_h = cut.clone()
    own_h[rows, y] = gz[rows, y]
    few = torch.bincount(y, minlength=v)[y] <= 4
    own_w = cut.clone()
    own_w[rows[few], y[few]] = gz[rows[few], y[few]]
    for name, exact, plain, own in (
            ("d_h", gz @ w.double(), cut @ w.double(), own_h @ w.double()),
            ("d_w", gz.t() @ h.double(), cut.t() @ h.double(), own_w.t() @ h.double())):
        err = [float((x.bfloat16().double() - exact).norm() / exact.norm()) for x in (plain, own)]
        got = float((r[name].double() - exact).norm() / exact.norm())
        assert err[0] > 1.1 * err[1], (name, err)  # else this shows nothing
        assert got <= 1.02 * err[1], (name, got, err)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,v,k", [(700, 9000, 1), (1500, 4099, 20), (400, 32003, 64)])
def test_many_rows_forward_and_backward(n, v, k, dtype):
    """More rows than the oracle takes: the definitions in fp64 on the same
    device, with the tolerances above."""
    t = (1.0, 0.7, 2.0)[(n + v) % 3]
    z, y = _logits(n, v, dtype, n + v).cuda(), _tokens(n, v, n + v).cuda()
    on = y != IGN
    p = kd.LogprobProblem(n_tokens=n, vocab=v, topk=k, dtype=dtype, temperature=t)
    tens = {"logits": z, "tokens": y}
    out = kd.token_logprobs(p, tens)
    zz = z.double()
    lp = torch.log_softmax(zz / t, dim=1)
    pr = lp.exp()
    ent = -(pr * lp).sum(dim=1)
    x = (zz.amax(dim=1, keepdim=True) - zz) / t
    es, yy = _e_s(v), y.clamp(min=0)[:, None]
    off = (out["logprob"].double() - lp.gather(1, yy)[:, 0]).abs()
    assert (off <= es + (2 * x + 2 * lp.abs() + 4).gather(1, yy)[:, 0] * U)[on].all()
    assert ((out["entropy"].double() - ent).abs() <= es * (math.log(v) + 3))[on].all()
    assert (out["logprob"][~on] == 0).all() and (out["entropy"][~on] == 0).all()
    ids = torch.sort(zz, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(out["topk_idx"][on], ids[on].int())
    off = (out["topk_logprob"].double() - lp.gather(1, ids)).abs()
    assert (off <= es + (2 * x + 2 * lp.abs() + 4).gather(1, ids) * U)[on].all()
    g = torch.Generator().manual_seed(v)
    gl, gh = torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda() * 0.3
    r = kd.token_logprobs_backward(p, tens, out["stats"], d_logprob=gl, d_entropy=gh)
    a, b = gl.double()[:, None], gh.double()[:, None]
    ref = -pr * (a + b * (lp + ent[:, None]))
    ref[torch.arange(n), yy[:, 0]] += a[:, 0]
    ref = torch.where(on[:, None], ref / t, 0.0)
    bracket = a.abs() + b.abs() * (lp.abs() + math.log(v) + 1)
    tol = pr * (((4 * x + 16) * U + es) * bracket + b.abs() * es * (math.log(v) + 3)
                + 8 * U * bracket) / t
    tol = tol + HALF[dtype] * (ref.abs() + tol) + 4 * U * a.abs() / t + TINY
    assert ((r["d_logits"].double() - ref).abs() <= tol).all()
    assert (r["d_logits"][~on] == 0).all()
