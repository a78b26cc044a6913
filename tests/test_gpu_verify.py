"""Draft verification on the GPU against the fp64 oracle.

Whole numbers are equal: the inputs are made so that no decision lies within
1e-4 of its border (an accepting uniform number is moved away, the winner's
noise made smaller), where the kernels' decisions are off by less than 1e-5:
u = 2^-24, a thread's sum of V / 512 exponentials in sequence at most V / 512 u,
2^x 4 u, the products 4 u, the exponent's roundings made up for.
log p: V / 512 u for the sum, 4 u of log S and (z - m) / T each, and for the
exponents' two roundings, weighted by 2^-x, at most 4 u."""
import math

import numpy as np
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd
from oracle import rows_oracle as R
from oracle.kd_oracle import as_f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
FAR = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _data(b, k, v, dtype, seed=0, std=3.0, near=0.8):
    g = torch.Generator().manual_seed(seed)
    target = (torch.randn(b, k + 1, v, generator=g) * std).to(DT[dtype])
    draft = (target[:, :k].float() + near * torch.randn(b, k, v, generator=g)).to(DT[dtype])
    e = torch.empty(b, k, v).exponential_(generator=g).log_()
    return {"target_logits": target, "draft_logits": draft,
            "drafts": (draft.float() - e).argmax(dim=2) if k else torch.zeros(b, 0).long(),
            "uniform": torch.rand(b, k, generator=g),
            "noise": torch.empty(b, v).exponential_(generator=g).clamp_min(1e-20)}


def _apart(c, t_target, t_draft):
    """Moves the inputs off the borders of their own decisions."""
    args = dict(t_target=t_target, t_draft=t_draft)
    for _ in range(20):
        r = _oracle(c, **args)
        close = np.nonzero(r["margin"] < FAR)[0]
        if not len(close):
            return r
        for s in close:
            n = int(r["accepted"][s])
            c["uniform"][s] = c["uniform"][s] * 0.9
            y = int(r["tokens"][s, n])
            if y >= 0:
                c["noise"][s, y] *= 0.9
    raise AssertionError("no inputs off the borders")


def _oracle(c, t_target=1.0, t_draft=1.0, ignore_index=-100):
    n = lambda x: None if x is None else x.numpy()  # noqa: E731
    return R.verify(c["target_logits"], c.get("draft_logits"), n(c["drafts"]), n(c.get("lengths")),
                    n(c["uniform"]), n(c["noise"]), t_target=t_target, t_draft=t_draft,
                    ignore_index=ignore_index)


def _problem(c, dtype, t_target=1.0, t_draft=1.0, **kw):
    b, rows, v = c["target_logits"].shape
    return kd.VerifyProblem(n_seqs=b, n_drafts=rows - 1, vocab=v, dtype=dtype, t_target=t_target,
                            t_draft=t_draft, **kw)


def _run(c, dtype, t_target=1.0, t_draft=1.0, **kw):
    p = _problem(c, dtype, t_target, t_draft)
    return kd.verify_drafts(p, {k: v.cuda() for k, v in c.items() if v is not None}, **kw)


def _check(r, ref, v, t):
    assert r["tokens"].tolist() == ref["tokens"].tolist()
    assert r["accepted"].tolist() == ref["accepted"].tolist()
    got, want = as_f64(r["logprob"]), ref["logprob"]
    assert (np.isnan(got) == np.isnan(want)).all()
    fine = ~np.isnan(want)
    tol = U * (v / 512 + 12 + 8 * np.abs(want[fine]) + 8 * math.log(v))
    assert (np.abs(got[fine] - want[fine]) <= tol).all()
    bits = ((kd.KD_DEV_BAD_LABEL if ref["bad_label"] else 0)
            | (kd.KD_DEV_NONFINITE if ref["nonfinite"] else 0))
    assert int(r["dev_status"]) == bits


SHAPES = [(1, 4, 151936), (1, 0, 32000), (3, 1, 1), (5, 2, 2), (2, 3, 7), (40, 5, 500),
          (9, 3, 32003), (6, 32, 1000), (300, 1, 130), (17, 7, 8200), (2, 1, 40001)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t_target,t_draft", [(1.0, 1.0), (0.75, 1.5), (0.0, 1.0)])
@pytest.mark.parametrize("b,k,v", SHAPES)
def test_drafter_with_logits(b, k, v, t_target, t_draft, dtype):
    c = _data(b, k, v, dtype, seed=v)
    g = torch.Generator().manual_seed(v + 1)
    c["lengths"] = torch.randint(-1, k + 1, (b,), generator=g, dtype=torch.int32)
    c["lengths"][0] = k
    ref = _apart(c, t_target, t_draft)
    _check(_run(c, dtype, t_target, t_draft), ref, v, t_target or 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t_target", [1.0, 0.75, 0.0])
@pytest.mark.parametrize("b,k,v", SHAPES)
def test_drafts_without_logits(b, k, v, t_target, dtype):
    c = _data(b, k, v, dtype, seed=v + 2, std=1.0 if v > 10 else 0.1)
    c["draft_logits"] = None
    if k:  # some that are likely to stand
        top = c["target_logits"][:, :k].float().argmax(dim=2)
        c["drafts"][::2] = top[::2]
        c["uniform"][::2] *= 0.01
    ref = _apart(c, t_target, 1.0)
    _check(_run(c, dtype, t_target), ref, v, t_target or 1.0)


def test_greedy_ties_go_to_the_lowest_id():
    b, k, v = 6, 2, 9000
    c = _data(b, k, v, "bf16", seed=3)
    z = c["target_logits"]
    ids = torch.tensor([0, 5, 4095, 4096, 8191, 8999])
    for s in range(b):
        z[s, :, :] = z[s].clamp(max=8.0)
        z[s, :, ids[s:]] = 9.0
        c["drafts"][s] = ids[s]
    c["drafts"][1, 0] = ids[2]  # equal, but not the lowest
    ref = _oracle(c, t_target=0.0)
    assert ref["accepted"].tolist() == [2, 0, 2, 2, 2, 2]
    _check(_run(c, "bf16", 0.0), ref, v, 1.0)
    z[:, :, :] = -1.0  # the lowest id of -0 and +0
    z[:, :, 77], z[:, :, 78] = -0.0, 0.0
    c["drafts"][:] = 77
    assert (_run(c, "bf16", 0.0)["tokens"] == 77).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [3, 1000, 20011])
@pytest.mark.parametrize("t_target", [1.0, 0.0])
def test_rows_without_a_distribution(v, t_target, dtype):
    """NaN, +inf and rows of -inf, in the target's and the drafter's rows, in front of
    and behind the row where a sequence ends."""
    c = _data(16, 2, v, dtype, seed=v + 4)
    z, q = c["target_logits"], c["draft_logits"]
    c["uniform"][:] = 0.0  # drafts stand wherever they can
    if t_target == 0.0:
        c["drafts"] = z[:, :2].float().argmax(dim=2)
    z[0, 0, v // 2] = float("nan")
    z[1, 1, 0] = float("inf")
    z[2, 2, :] = -float("inf")
    z[3, 0, :] = -float("inf")
    q[4, 0, v - 1] = float("nan")
    q[5, 1, 1] = float("inf")
    q[6, 0, :] = -float("inf")
    for s in range(7):
        one = {k: x[s:s + 1] for k, x in c.items()}
        ref = _apart(one, t_target, 1.0)
        assert ref["nonfinite"] == (t_target > 0 or s < 4)
        _check(_run(one, dtype, t_target, check=False), ref, v, 1.0)
        if ref["nonfinite"]:
            with pytest.raises(kd.KDError):
                _run(one, dtype, t_target)
    # behind the first draft that does not stand nothing is looked at
    c["drafts"][7:] = 0
    z[7:, 0, 0] = -float("inf")
    z[7:, 1:] = float("nan")
    q[7:, 1] = float("nan")
    one = {k: x[7:] for k, x in c.items()}
    ref = _apart(one, t_target, 1.0)
    assert not ref["nonfinite"] and (ref["accepted"] == 0).all()
    _check(_run(one, dtype, t_target), ref, v, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forbidden_ids(dtype):
    """-inf and the type's lowest value: no probability; a row that holds nothing but
    the lowest value is uniform."""
    b, k, v = 12, 3, 5003
    c = _data(b, k, v, dtype, seed=6)
    low = torch.finfo(DT[dtype]).min
    c["target_logits"][:6, :, 7:] = -float("inf")
    c["target_logits"][6:, :, 7:] = low
    c["draft_logits"][:6, :, 9:] = low
    c["target_logits"][11] = low
    c["draft_logits"][10] = low
    c["drafts"] = torch.randint(0, 12, (b, k), generator=torch.Generator().manual_seed(7))
    ref = _apart(c, 1.0, 1.0)
    assert (ref["tokens"][:11] < 7).all()
    _check(_run(c, dtype), ref, v, 1.0)


def test_logits_of_any_size():
    """A hundred equal logits of 1e30, the others -3e38: only differences count."""
    b, k, v = 4, 2, 300
    c = _data(b, k, v, "fp32", seed=8)
    c["target_logits"] = 1e30 + torch.zeros(b, k + 1, v)
    c["target_logits"][:, :, 100:] = -3e38
    ref = _apart(c, 1.0, 1.0)
    _check(_run(c, "fp32"), ref, v, 1.0)


def test_equal_rows_always_stand():
    b, k, v = 50, 4, 1000
    c = _data(b, k, v, "bf16", seed=9, near=0.0)
    c["uniform"][:] = 1.0 - 2.0 ** -24
    r = _run(c, "bf16")
    assert (r["accepted"] == k).all() and torch.equal(r["tokens"][:, :k].cpu(), c["drafts"])
    # u = 1 is outside the range, and rejects: there is no residual, p is drawn from
    c["uniform"][:] = 1.0
    r = _run(c, "bf16")
    assert (r["accepted"] == 0).all()
    p = torch.softmax(c["target_logits"][:, 0].double(), 1)
    first = (c["noise"].double() / p).argsort(dim=1)[:, :2]
    near = (c["noise"].double() / p).gather(1, first)
    sure = near[:, 1] / near[:, 0] > 1 + FAR
    assert (r["tokens"][:, 0].cpu() == first[:, 0])[sure].all() and sure.sum() > 40


@pytest.mark.parametrize("v", [900, 20011, 60000])
@pytest.mark.parametrize("near", [0.05, 0.5])
def test_rejected_drafts_of_a_near_drafter(near, v):
    """The id that the drafter overrates most, rejected: what is left to draw from is
    small beside p, and many ids' p pass what the residual's scores hold.  A weight
    p - q is off by some 2^-21 p; the smallest share that wins is above 2^-7 here."""
    b, k = 12, 1
    c = _data(b, k, v, "fp32", seed=v + 17, std=1.0, near=near)
    p = torch.softmax(c["target_logits"][:, :1].double(), -1)
    q = torch.softmax(c["draft_logits"].double(), -1)
    c["drafts"] = (q - p).argmax(-1)
    c["uniform"][:] = 1.0 - 2.0 ** -24
    ref = _apart(c, 1.0, 1.0)
    c["uniform"][:] = 1.0 - 2.0 ** -24  # (q is above p by far more than FAR)
    ref = _oracle(c)
    assert (ref["accepted"] == 0).all() and (ref["margin"] >= FAR).all()
    y = torch.from_numpy(ref["tokens"][:, :1])
    won = 1 - q[:, 0].gather(1, y) / p[:, 0].gather(1, y)
    assert won.min() > 2.0 ** -7
    _check(_run(c, "fp32"), ref, v, 1.0)


def test_equal_rows_that_are_rejected_draw_from_p():
    """u = 1, outside the range: no residual, and more ids than are looked at closely.
    The rows are whole 16-byte vectors, so that both sums are formed in the same
    order and are the same; of rows that begin elsewhere in their vectors they may
    differ in their last bit, and u q < p may hold at u = 1."""
    b, k, v = 9, 2, 30000
    c = _data(b, k, v, "bf16", seed=19, near=0.0)
    c["uniform"][:] = 1.0
    time = c["noise"].double() / torch.softmax(c["target_logits"][:, 0].double(), 1)
    first = time.topk(2, dim=1, largest=False)
    sure = first.values[:, 1] / first.values[:, 0] > 1 + FAR
    r = _run(c, "bf16")
    assert (r["accepted"] == 0).all() and sure.sum() >= b - 1
    assert (r["tokens"][:, 0].cpu() == first.indices[:, 0])[sure].all()


def test_bad_drafts_and_lengths():
    b, k, v = 5, 3, 600
    c = _data(b, k, v, "bf16", seed=10)
    c["uniform"][:] = 0.0
    for i, bad in enumerate((v, -1, -100, 2 ** 40)):
        one = {n: x.clone() for n, x in c.items()}
        one["drafts"][i, i % k] = bad
        ref = _apart(one, 1.0, 1.0)
        assert ref["bad_label"] and ref["accepted"][i] == i % k
        _check(_run(one, "bf16", check=False), ref, v, 1.0)
        with pytest.raises(kd.KDError) as e:
            _run(one, "bf16")
        assert e.value.status == kd.KD_ERR_BAD_LABEL
        one["draft_logits"] = None
        one["uniform"] = torch.full_like(one["uniform"], 1e-30)
        _check(_run(one, "bf16", check=False), _apart(one, 1.0, 1.0), v, 1.0)
    # a bad draft behind the sequence's length is not looked at
    c["drafts"][2, 2] = -7
    c["lengths"] = torch.tensor([3, 0, 2, -9, 1], dtype=torch.int32)
    ref = _apart(c, 1.0, 1.0)
    assert not ref["bad_label"] and (ref["tokens"][3] == -100).all()
    _check(_run(c, "bf16"), ref, v, 1.0)
    c["lengths"][0] = 4
    ref = _apart(c, 1.0, 1.0)
    assert ref["bad_label"]
    _check(_run(c, "bf16", check=False), ref, v, 1.0)


def test_noise_out_of_range_takes_no_part():
    b, k, v = 6, 1, 400
    c = _data(b, k, v, "fp32", seed=11)
    c["uniform"][:] = 0.0
    for x in (0.0, -1.0, float("nan"), float("inf"), 1e-38, 1e38):
        c["noise"][:, ::2] = x
        ref = _apart(c, 1.0, 1.0)
        assert (ref["tokens"][:, 1] % 2 == 1).all()
        _check(_run(c, "fp32"), ref, v, 1.0)
    c["noise"][:] = 0.0
    ref = _oracle(c)
    assert ref["nonfinite"] and (ref["tokens"][:, 1] == -100).all()
    _check(_run(c, "fp32", check=False), ref, v, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pitches_and_views(dtype):
    """Rows at a pitch, at odd offsets, and outputs one by one."""
    b, k, v = 7, 2, 1003
    c = _data(b, k, v, dtype, seed=12)
    ref = _apart(c, 1.0, 1.0)
    for pitch, shift in ((1003, 0), (1024, 0), (1017, 3)):
        t = {n: x.cuda() for n, x in c.items()}
        for n, rows in (("target_logits", b * (k + 1)), ("draft_logits", b * k)):
            store = torch.full((rows * pitch + shift,), float("nan"), dtype=DT[dtype], device="cuda")
            view = store[shift:].view(b, rows // b, pitch)[:, :, :v]
            view.copy_(t[n])
            t[n] = view
        _check(kd.verify_drafts(_problem(c, dtype), t), ref, v, 1.0)
    for n in ("tokens", "accepted", "logprob"):
        full = kd.verify_drafts(_problem(c, dtype), t)
        out = {n: torch.zeros_like(full[n])}
        kd.verify_drafts(_problem(c, dtype), t, out=out)
        assert torch.equal(out[n], full[n])


def test_no_sequences():
    p = kd.VerifyProblem(n_seqs=0, vocab=10, n_drafts=2)
    z = torch.empty(0, 3, 10, dtype=torch.bfloat16, device="cuda")
    t = {"target_logits": z, "drafts": torch.empty(0, 2, dtype=torch.int64, device="cuda"),
         "uniform": torch.empty(0, 2, device="cuda"), "noise": torch.empty(0, 10, device="cuda")}
    assert kd.verify_drafts(p, t)["tokens"].shape == (0, 3)


def test_logits_beyond_32_bit_offsets():
    """The last sequences' rows begin past 2^31 elements."""
    b, k, v = 2100, 7, 131072
    free, _ = torch.cuda.mem_get_info()
    if free < 16e9:
        pytest.skip("needs 16 GB")
    c = _data(2, k, v, "bf16", seed=13)
    ref = _apart(c, 1.0, 1.0)
    t = {n: torch.empty((b,) + x.shape[1:], dtype=x.dtype, device="cuda") for n, x in c.items()}
    for n, x in c.items():
        t[n][b - 2:] = x.cuda()
    t["lengths"] = torch.full((b,), -1, dtype=torch.int32, device="cuda")
    t["lengths"][b - 2:] = k
    p = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v)
    r = kd.verify_drafts(p, t)
    assert (r["tokens"][:b - 2] == -100).all() and (r["accepted"][:b - 2] == 0).all()
    last = {n: r[n][b - 2:] for n in ("tokens", "accepted", "logprob")}
    _check({**last, "dev_status": r["dev_status"]}, ref, v, 1.0)


def test_repeats_exactly_and_in_graphs_that_share_a_workspace():
    b, k, v = 20, 4, 9001
    ws = kd.Workspace()
    jobs = []
    for seed in (14, 15):
        c = {n: x.cuda() for n, x in _data(b, k, v, "bf16", seed=seed).items()}
        p = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v)
        ref = kd.verify_drafts(p, c)
        out = {n: torch.zeros_like(x) for n, x in ref.items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            kd.verify_drafts(p, c, workspace=ws, out=out, check=False)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kd.verify_drafts(p, c, workspace=ws, out=out, check=False)
        jobs.append((graph, out, ref, c))
    for _, out, _, _ in jobs:
        for x in out.values():
            x.zero_()
    for _ in range(3):
        for graph, _, _, _ in jobs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out, ref, _ in jobs:
        assert all(torch.equal(out[n], ref[n]) for n in ref)


def test_emitted_tokens_follow_the_targets_distribution():
    """As the oracle's own test: frequencies within five standard deviations."""
    b, v = 60000, 12
    g = torch.Generator().manual_seed(16)
    zt, zd = torch.randn(1, 2, v, generator=g) * 1.5, torch.randn(1, 1, v, generator=g) * 1.5
    p, q = torch.softmax(zt[0, 0].double(), 0), torch.softmax(zd[0, 0].double(), 0)
    c = {"target_logits": zt.expand(b, 2, v).contiguous(),
         "draft_logits": zd.expand(b, 1, v).contiguous(),
         "drafts": torch.multinomial(q.expand(b, v), 1, generator=g),
         "uniform": torch.rand(b, 1, generator=g),
         "noise": torch.empty(b, v).exponential_(generator=g)}
    r = _run(c, "fp32")
    freq = torch.bincount(r["tokens"][:, 0].cpu(), minlength=v).double() / b
    assert ((freq - p).abs() <= 5 * (p * (1 - p) / b).sqrt()).all()
