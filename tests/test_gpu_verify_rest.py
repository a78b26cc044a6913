"""Draft verification behind a rejected draft, where no id with p > q has usable
noise, and weights and noise at the ends of their ranges, against the
fp64 oracle.

Whole numbers are equal: decisions are kept 1e-4 off their borders, the kernels'
are off by less than 1e-5.  log p, u = 2^-24: a thread adds the exponentials of its
share of a part in sequence, two sums at a time.  A part of up to 4 KB has 32
threads, of up to 32 KB 128, else 256: at most max(64, V / 512) terms a sum, then
some 20 levels of joins.  An exponential is off by 4 u and by its exponent's two
roundings, which its own smallness outweighs (4 u at most), a moved offset's factor
by 4 u: S within (max(64, V / 512) + 32) u.  log S adds 2 u log V, (z - m) / T two
roundings of at most |log p| + log V, the last sum one."""
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


def _both(c, dtype):
    """(the kernel's outputs, the oracle's), and how far the sequences are from a border."""
    b, rows, v = c["target_logits"].shape
    p = kd.VerifyProblem(n_seqs=b, n_drafts=rows - 1, vocab=v, dtype=dtype)
    r = kd.verify_drafts(p, {k: t.cuda() for k, t in c.items() if t is not None}, check=False)
    ref = R.verify(c["target_logits"], c.get("draft_logits"), c["drafts"].numpy(), None,
                   c["uniform"].numpy(), c["noise"].numpy())
    return r, ref


def _check(r, ref, v):
    assert (ref["margin"] >= FAR).all()
    assert r["accepted"].tolist() == ref["accepted"].tolist()
    assert r["tokens"].tolist() == ref["tokens"].tolist()
    got, want = as_f64(r["logprob"]), ref["logprob"]
    assert (np.isnan(got) == np.isnan(want)).all()
    fine = ~np.isnan(want)
    tol = U * (max(64, v / 512) + 36 + 4 * np.abs(want[fine]) + 4 * math.log(v))
    assert (np.abs(got[fine] - want[fine]) <= tol).all()
    assert int(r["dev_status"]) == (kd.KD_DEV_NONFINITE if ref["nonfinite"] else 0)


def _far_noise(b, v, p, g):
    """Exponential noise whose first arrival is clear of the second."""
    noise = torch.empty(b, v).exponential_(generator=g).clamp_min(1e-20)
    for s in range(b):
        noise[s, (noise[s].double() / p[s]).argmin()] *= 0.9
    return noise


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [40, 1003, 60000])
@pytest.mark.parametrize("logits", [True, False])
@pytest.mark.parametrize("bad", [0.0, math.inf, -math.inf, math.nan, -1.0, 1e-30, 1e30])
def test_a_rest_without_usable_noise_draws_nothing(bad, logits, v, dtype):
    """Every second sequence: the ids with p > q have noise that takes no part, the
    others' is fine.  Nothing is drawn, although p itself could be drawn from."""
    b, k = 6, 2
    g = torch.Generator().manual_seed(v)
    target = (torch.randn(b, k + 1, v, generator=g) * 1.5).to(DT[dtype])
    draft = (target[:, :k].float() + torch.randn(b, k, v, generator=g)).to(DT[dtype])
    p = torch.softmax(target[:, 0].double(), -1)
    q = torch.softmax(draft[:, 0].double(), -1)
    # rejected: the id that the drafter overrates most, or one that is no sure thing
    first = (q - p).argmax(-1) if logits else torch.full((b,), 3)
    c = {"target_logits": target, "draft_logits": draft if logits else None,
         "drafts": torch.stack([first, first], 1), "uniform": torch.full((b, k), 1 - 2.0 ** -24)}
    if logits:
        rest = p > q * (1 - 1e-4)  # (also those too close to tell)
    else:
        rest = torch.ones(b, v, dtype=torch.bool)
        rest[:, 3] = False
    weight = (p - q).clamp_min(0) if logits else torch.where(rest, p, 0.0)
    c["noise"] = _far_noise(b, v, weight, g)
    c["noise"][::2][rest[::2]] = bad
    r, ref = _both(c, dtype)
    assert (ref["accepted"] == 0).all() and ref["nonfinite"]
    assert (ref["tokens"][::2] == -100).all() and (ref["tokens"][1::2, 0] >= 0).all()
    _check(r, ref, v)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [40, 8200, 60000])
def test_without_a_rest_the_target_itself_is_drawn_from(v, dtype):
    """Equal rows whose draft has no probability: p <= q everywhere.  Ids whose noise
    takes no part are not drawn; where all of them are, nothing is."""
    b, k = 5, 1
    g = torch.Generator().manual_seed(v + 1)
    target = (torch.randn(b, k + 1, v, generator=g) * 1.5).to(DT[dtype])
    target[:, 0, 7] = -math.inf
    p = torch.softmax(target[:, 0].double(), -1)
    c = {"target_logits": target, "draft_logits": target[:, :1].contiguous(),
         "drafts": torch.full((b, k), 7), "uniform": torch.full((b, k), 0.5)}
    p[:, ::2] = 0.0
    c["noise"] = _far_noise(b, v, p, g)
    c["noise"][:, ::2] = math.nan
    c["noise"][3] = 0.0
    r, ref = _both(c, dtype)
    assert (ref["accepted"] == 0).all() and ref["tokens"][3, 0] == -100
    assert all(ref["tokens"][s, 0] % 2 == 1 for s in (0, 1, 2, 4))
    _check(r, ref, v)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v", [40, 9000, 60001])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** -59, 1.0])
def test_weights_and_noise_at_the_ends_of_their_ranges(size, v, dtype):
    """Only ids of p = 2^-94 and less have noise that takes part, 2^60 or 2^-60 among it."""
    z = torch.full((3, 1, v), -65.0)
    z[:, :, 0], z[:, :, 11] = 0.0, -80.0
    c = {"target_logits": z.to(DT[dtype]), "drafts": torch.zeros(3, 0, dtype=torch.int64),
         "uniform": torch.zeros(3, 0), "noise": torch.full((3, v), size)}
    c["noise"][:, 0] = 0.0
    c["noise"][0, 5] *= 0.5
    c["noise"][1, v // 2] *= 0.5
    c["noise"][2] = -1.0
    c["noise"][2, 11] = size  # the least likely one alone is left
    r, ref = _both(c, dtype)
    assert ref["tokens"][:, 0].tolist() == [5, v // 2, 11]
    _check(r, ref, v)


@pytest.mark.parametrize("b,k,v", [(19, 12, 32000), (8, 5, 40000), (16, 4, 33000), (3, 32, 20000),
                                   (1, 1, 151936), (50, 1, 900)])
@pytest.mark.parametrize("form", ["greedy", "without", "logits"])
def test_the_workspace_is_what_was_asked_for(form, b, k, v):
    """Rows are read in parts by how many there are, the drafter's among them or not:
    every form of the call keeps to one problem's workspace."""
    g = torch.Generator(device="cuda").manual_seed(b)
    target = torch.randn(b, k + 1, v, generator=g, device="cuda").bfloat16()
    t = {"target_logits": target, "drafts": target[:, :k].float().argmax(-1),
         "uniform": torch.zeros(b, k, device="cuda"),
         "noise": torch.rand(b, v, generator=g, device="cuda") + 0.5}
    t["drafts"][:, -1] = 3  # (mostly not the largest: greedy ends there)
    if form == "logits":
        t["draft_logits"] = target[:, :k].contiguous()
    p = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v, t_target=0.0 if form == "greedy" else 1.0)
    size = kd.kd_verify_workspace_size(p.to_c())
    buf = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0

    class Exact:
        def get(self, nbytes, device):
            assert nbytes == size
            return buf.data_ptr(), nbytes

    r = kd.verify_drafts(p, t, workspace=Exact())
    assert (buf[size:] == 77).all()
    if form == "greedy":
        best = target.float().argmax(-1)
        stood = (best[:, :k] == t["drafts"]).long().cumprod(1).sum(1)
        assert torch.equal(r["accepted"].long(), stood)
        assert torch.equal(r["tokens"].gather(1, stood[:, None]), best.gather(1, stood[:, None]))
    else:
        assert (r["accepted"] == k).all()
