"""The operators around the head as a model uses them together.

Training: a tied student h = norm(embed(tokens) + residual) against a teacher's
logits; its table's gradient is the head's share (kd_bwd) and the embedding's,
added into one buffer, then clipped with the others.  Serving: the student
drafts, the target's logits of a tied model verify, and the emitted tokens are
looked up again.  All in fp32 against fp64 compositions of the oracles: each
step's tolerance is that of its own test, and the compositions are compared at
1e-4 of the largest element, some hundred times the sum of their errors
(sums of up to 1500 terms of fp32, 1500 u = 1e-4 at the very worst)."""
import ctypes
import functools
import sys
import threading

import numpy as np
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd
from oracle import kd_oracle as O
from oracle import rows_oracle as R
from oracle.kd_oracle import as_f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _near(got, want, rel=1e-4):
    return np.abs(as_f64(got) - want).max() <= rel * np.abs(want).max()


def test_a_training_step_of_a_tied_student():
    n, v, d = 96, 1500, 72
    g = torch.Generator().manual_seed(21)
    w, weight = torch.randn(v, d, generator=g) * 0.2, 1 + 0.1 * torch.randn(d, generator=g)
    res, z_t = torch.randn(n, d, generator=g) * 0.3, torch.randn(n, v, generator=g) * 2
    tokens = torch.randint(0, 40, (n,), generator=g)  # each occurs some times
    labels = torch.randint(0, v, (n,), generator=g)
    tokens[5], labels[5], labels[50] = -100, -100, -100
    ep = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32", scale=d ** 0.5)
    np_ = kd.NormProblem(n_tokens=n, d_model=d, dtype="fp32", eps=EPS)
    kp = kd.Problem(n_tokens=n, vocab=v, d_student=d, dtype="fp32", teacher="logits",
                    variant="forward", t_student=2.0, w_student_ce=0.5, w_kl=0.5)
    dev = [x.cuda() for x in (w, weight, res, z_t, tokens, labels)]
    x = kd.embed_tokens(ep, dev[0], dev[4])["h"]
    r = kd.rms_norm(np_, x, dev[1], residual=dev[2])
    t = {"h_s": r["h"], "w_s": dev[0], "logits_t": dev[3], "labels": dev[5]}
    f = kd.forward(kp, t)
    b = kd.backward(kp, t, f["stats"], want=("h_s", "w_s"))
    nb = kd.rms_norm_backward(np_, r["sum"], dev[1], b["d_h_s"])
    head_only = b["d_w_s"].clone()
    table = kd.embed_tokens_backward(ep, dev[4], nb["d_x"], accumulate=True,
                                     out={"d_w": b["d_w_s"]})["d_w"]
    assert table is b["d_w_s"] and not torch.equal(table, head_only)
    clip = kd.clip_grad_norm([table, nb["d_weight"]], 0.5)

    scale = float(np.float32(d ** 0.5))
    x64 = R.embed(w, tokens.tolist(), scale)
    h64, s64 = R.rms_norm(x64, weight, res, eps=EPS)
    z64 = h64 @ as_f64(w).T
    kw = dict(variant="forward", t_student=2.0, t_teacher=2.0, w_student_ce=0.5, w_teacher_ce=0.0,
              w_kl=0.5)
    ref = O.forward(z64, as_f64(z_t), labels.numpy(), **kw)
    g_s, _ = O.grad_logits(z64, as_f64(z_t), labels.numpy(), **kw)
    d_h, d_w = g_s @ as_f64(w), g_s.T @ h64
    gn = R.rms_norm_grad(s64, weight, d_h, eps=EPS)
    d_e, _, _ = R.embed_grad(gn["d_x"], tokens.tolist(), v, scale)
    d_table = d_w + d_e
    norm = np.sqrt((d_table ** 2).sum() + (gn["d_weight"] ** 2).sum())
    assert abs(f["loss"].item() - ref["loss"]) <= 1e-4 * abs(ref["loss"])
    assert _near(r["h"], h64) and _near(nb["d_x"], gn["d_x"])
    assert abs(clip["norm"].item() - norm) <= 1e-4 * norm
    factor = min(1.0, 0.5 / norm)
    assert _near(table, d_table * factor) and _near(nb["d_weight"], gn["d_weight"] * factor)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_drafting_and_verification_in_a_loop(dtype):
    """Greedy, so that the emitted text is the target's own whatever the drafter
    drafts: a target whose next token depends on the last one alone."""
    b, k, v, d, steps = 5, 3, 400, 64, 6
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(22)
    w = torch.randn(v, d, generator=g).to(dt).cuda()
    mix = torch.randn(d, d, generator=g).to(dt).cuda()  # the rest of the model
    weight = torch.ones(d, dtype=dt, device="cuda")

    def logits(tokens, noise=0.0):
        flat = tokens.reshape(-1)
        ep = kd.EmbedProblem(n_tokens=flat.numel(), vocab=v, d_model=d, dtype=dtype)
        np_ = kd.NormProblem(n_tokens=flat.numel(), d_model=d, dtype=dtype)
        h = kd.rms_norm(np_, kd.embed_tokens(ep, w, flat)["h"] @ mix, weight)["h"]
        z = h @ w.t()
        if noise:
            z = z + noise * torch.randn(z.shape, device="cuda", dtype=z.dtype)
        return z.view(*tokens.shape, v)

    torch.manual_seed(23)
    last = torch.arange(b, device="cuda")
    text = [[] for _ in range(b)]
    p = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v, dtype=dtype, t_target=0.0)
    accepted = 0
    for _ in range(steps):
        drafts, x = [], last
        for _ in range(k):  # the drafter: the target with noise on its logits
            x = logits(x, 8.0).argmax(-1)
            drafts.append(x)
        drafts = torch.stack(drafts, 1)
        seen = torch.cat([last[:, None], drafts], 1)
        r = kd.verify_drafts(p, {"target_logits": logits(seen), "drafts": drafts})
        n = r["accepted"]
        accepted += int(n.sum())
        last = r["tokens"].gather(1, n.long()[:, None])[:, 0]
        for s in range(b):
            text[s] += [t for t in r["tokens"][s].tolist() if t != -100]
        assert ((r["tokens"] != -100).sum(1) == n + 1).all()
    assert 0 < accepted < steps * b * k
    want = torch.arange(b, device="cuda")
    for i in range(min(len(t) for t in text)):
        # one row at a time and several: the product's rows do not depend on it here
        want = logits(want[:, None].expand(b, k + 1).contiguous())[:, 0].argmax(-1)
        assert [t[i] for t in text] == want.tolist()


def test_a_drafter_over_another_vocabulary():
    """Its logits moved onto the target's ids by the token map, then verified."""
    b, k, v, vd = 30, 2, 500, 120
    g = torch.Generator().manual_seed(24)
    tmap = torch.randperm(v, generator=g)[:vd].int()
    target = torch.randn(b, k + 1, v, generator=g) * 2
    draft = target[:, :k][:, :, tmap.long()] + 0.5 * torch.randn(b, k, vd, generator=g)
    q = torch.softmax(draft, -1).reshape(-1, vd)
    drafts = tmap[torch.multinomial(q, 1, generator=g)[:, 0]].long().view(b, k)
    moved = kd.project_teacher_logits(tmap.cuda(), draft.reshape(-1, vd).cuda(), v).view(b, k, v)
    u, e = torch.rand(b, k, generator=g), torch.empty(b, v).exponential_(generator=g)
    p = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v, dtype="fp32")
    r = kd.verify_drafts(p, {"target_logits": target.cuda(), "draft_logits": moved,
                             "drafts": drafts.cuda(), "uniform": u.cuda(), "noise": e.cuda()})
    full = np.full((b, k, v), -np.inf)
    full[:, :, tmap.numpy()] = as_f64(draft)
    ref = R.verify(target, full, drafts.numpy(), None, u.numpy(), e.numpy())
    sure = ref["margin"] > 1e-3
    assert sure.sum() >= b - 2
    assert (r["tokens"].cpu().numpy() == ref["tokens"])[sure].all()


def test_calls_on_two_streams_at_once():
    """Each with its own workspace and outputs, their inputs shared, over and over."""
    g = torch.Generator().manual_seed(25)
    n, v, d, b, k = 3000, 9000, 520, 6, 3
    w = torch.randn(v, d, generator=g).bfloat16().cuda()
    tokens = (torch.rand(n, generator=g) ** 4 * v).long().cuda()
    d_h = torch.randn(n, d, generator=g).bfloat16().cuda()
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    target = torch.randn(b, k + 1, v, generator=g).bfloat16().cuda()
    drafts = torch.randint(0, v, (b, k), generator=g).cuda()
    u, e = torch.rand(b, k, generator=g).cuda(), torch.rand(b, v, generator=g).cuda() + 0.01
    ep = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d)
    np_ = kd.NormProblem(n_tokens=n, d_model=d)
    vp = kd.VerifyProblem(n_seqs=b, n_drafts=k, vocab=v)
    ins = {"target_logits": target, "draft_logits": target[:, 1:].contiguous(), "drafts": drafts,
           "uniform": u, "noise": e}

    def step(ws, out):
        out["x"] = kd.embed_tokens(ep, w, tokens, check=False, out=out.get("x"))
        out["h"] = kd.rms_norm(np_, out["x"]["h"], gain, out=out.get("h"))
        out["n"] = kd.rms_norm_backward(np_, out["x"]["h"], gain, d_h, workspace=ws[0],
                                        out=out.get("n"))
        out["t"] = kd.embed_tokens_backward(ep, tokens, out["n"]["d_x"], workspace=ws[1],
                                            check=False, out=out.get("t"))
        out["v"] = kd.verify_drafts(vp, ins, workspace=ws[2], check=False, out=out.get("v"))
        return out

    ref = step([kd.Workspace() for _ in range(3)], {})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [([kd.Workspace() for _ in range(3)], {}) for _ in streams]
    for _ in range(8):
        for s, (ws, out) in zip(streams, held):
            with torch.cuda.stream(s):
                step(ws, out)
    torch.cuda.synchronize()
    for _, out in held:
        for op, r in ref.items():
            for name, t in r.items():
                if t is not None:
                    assert torch.equal(out[op][name], t), (op, name)


@pytest.mark.parametrize("op", ["norm", "embed"])
def test_calls_from_two_threads_at_once(op):
    """Two threads whose calls need different amounts of a kernel's shared memory
    (the norm's backward with and without d_sum, tables of 32000 and 151936 ids),
    each on its own stream, through the C ABI, where they do run at once: neither's
    call is refused, and the results are those of one thread."""
    g, lib = torch.Generator().manual_seed(26), kd.load_library()
    n, d = 8, 4096
    s, d_h, up = (torch.randn(n, d, generator=g).bfloat16().cuda() for _ in range(3))
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(n, 8, generator=g).bfloat16().cuda()
    held = [s, d_h, up, gain, rows]

    def prepared(which, stream):
        """(call, its outputs)"""
        if op == "norm":
            cp = kd.NormProblem(n_tokens=n, d_model=d).to_c()
            size = kd.kd_rmsnorm_workspace_size(cp)
            outs = [torch.zeros_like(s), torch.zeros_like(gain)]
        else:
            vocab = (32000, 151936)[which]
            cp = kd.EmbedProblem(n_tokens=n, vocab=vocab, d_model=8).to_c()
            size = kd.kd_embed_workspace_size(cp)
            outs = [torch.zeros(vocab, 8, dtype=torch.bfloat16, device="cuda")]
        # (memory of the allocator is 512-byte aligned)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        tokens = torch.arange(n, device="cuda") * 797
        held.extend([cp, ws, tokens, *outs])
        if op == "norm":
            args = (ctypes.byref(cp), s.data_ptr(), gain.data_ptr(), d_h.data_ptr(),
                    up.data_ptr() if which else None, outs[0].data_ptr(), outs[1].data_ptr(),
                    ws.data_ptr(), size, stream.cuda_stream)
            return functools.partial(lib.kd_rmsnorm_bwd, *args), outs
        args = (ctypes.byref(cp), tokens.data_ptr(), rows.data_ptr(), outs[0].data_ptr(), 1, None,
                ws.data_ptr(), size, stream.cuda_stream)
        return functools.partial(lib.kd_embed_bwd, *args), outs

    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = [prepared(i, stream) for i, stream in enumerate(streams)]
    torch.cuda.synchronize()
    want = []
    for call, outs in jobs:
        assert call() == kd.KD_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    told = [[], []]

    def work(i):
        call = jobs[i][0]
        for _ in range(100):
            told[i].extend(call() for _ in range(100))
            streams[i].synchronize()

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert [len(t) for t in told] == [10000, 10000]
    assert set(told[0] + told[1]) == {kd.KD_OK}
    for (call, outs), ref in zip(jobs, want):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        assert call() == kd.KD_OK
        torch.cuda.synchronize()
        for got, t in zip(outs, ref):
            assert torch.equal(got, t)
