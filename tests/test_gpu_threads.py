"""Two host threads whose calls need different amounts of one kernel's shared memory,
each on its own stream, through the C ABI, where they do run at once: neither's call
is refused, and the results are those of one thread."""
import ctypes
import functools
import sys
import threading

import pytest
import torch

from lm_head_cross_vocab_gb300 import kd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _space(nbytes, held):
    ws = kd.Workspace()
    held.append(ws)
    return ws.get(nbytes, torch.device("cuda:0"))


def _logprob(which, stream, held):
    """Alternatives of one long row, 128 or 1024 of them: a cluster of eight blocks."""
    k, v = (128, 1024)[which], 151936
    z = torch.randn(1, v, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    tokens = torch.zeros(1, dtype=torch.int64, device="cuda")
    cp = kd.LogprobProblem(n_tokens=1, vocab=v, topk=k).to_c()
    ins = kd.kd_logprob_inputs(z.data_ptr(), None, None, tokens.data_ptr())
    outs = [torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"),
            torch.zeros(1, k, dtype=torch.int32, device="cuda"), torch.zeros(1, k, device="cuda"),
            torch.zeros(1, kd.KD_LOGPROB_STATS, device="cuda"),
            torch.zeros((), dtype=torch.int32, device="cuda")]
    held += [z, tokens, cp, ins]
    return functools.partial(kd.load_library().kd_logprob_fwd, ctypes.byref(cp), ctypes.byref(ins),
                             *[t.data_ptr() for t in outs], None, 0, stream.cuda_stream), outs


def _mix(which, stream, held):
    v = (400, 20000)[which]
    g = torch.Generator().manual_seed(2)
    z = [torch.randn(1, v, generator=g).bfloat16().cuda() for _ in range(2)]
    ptrs = (ctypes.c_void_p * 2)(*[t.data_ptr() for t in z])
    outs = [torch.zeros(1, v, device="cuda"), torch.zeros((), dtype=torch.int32, device="cuda")]
    held += [*z, ptrs]
    return functools.partial(kd.load_library().kd_mix_teacher_logits, ptrs, 2, None, 1, v,
                             kd.KD_BF16, kd.KD_MIX_ARITHMETIC, outs[0].data_ptr(), kd.KD_FP32,
                             outs[1].data_ptr(), stream.cuda_stream), outs


def _project(sizes, which, stream, held):
    vt, vs = sizes[which]
    g = torch.Generator().manual_seed(3)
    z = torch.randn(1, vt, generator=g).bfloat16().cuda()
    tmap = torch.randint(0, vs, (vt,), generator=g, dtype=torch.int32).cuda()
    nbytes, lib = ctypes.c_size_t(0), kd.load_library()
    assert lib.kd_project_workspace_size(vt, vs, ctypes.byref(nbytes)) == kd.KD_OK
    outs = [torch.zeros(1, vs, device="cuda"), torch.zeros((), dtype=torch.int32, device="cuda")]
    held += [z, tmap]
    return functools.partial(lib.kd_project_teacher_logits, tmap.data_ptr(), vt, vs, z.data_ptr(),
                             1, kd.KD_BF16, 1.0, outs[0].data_ptr(), kd.KD_FP32,
                             outs[1].data_ptr(), *_space(nbytes.value, held),
                             stream.cuda_stream), outs


def _projected_loss(which, stream, held):
    n, vt, vs = 2, (200, 50000)[which], 700
    g = torch.Generator().manual_seed(4)
    t = {"logits_s": torch.randn(n, vs, generator=g).bfloat16().cuda(),
         "logits_t": torch.randn(n, vt, generator=g).bfloat16().cuda(),
         "labels": torch.zeros(n, dtype=torch.int64, device="cuda"),
         "token_map": torch.randint(0, vs, (vt,), generator=g, dtype=torch.int32).cuda()}
    cp = kd.Problem(n_tokens=n, vocab=vs, dtype="bf16", student="logits", teacher="projected",
                    variant="forward", t_student=1.0, t_teacher=1.0, w_student_ce=0.5,
                    w_teacher_ce=0.0, w_kl=1.0, ignore_index=-100, vocab_teacher=vt).to_c()
    ins = kd.make_inputs(t)
    outs = [*(torch.zeros(n, device="cuda") for _ in range(3)),
            torch.zeros(n, kd.KD_STATS_PER_TOKEN, device="cuda"), torch.zeros((), device="cuda"),
            torch.zeros((), dtype=torch.int32, device="cuda")]
    held += [t, cp, ins]
    return functools.partial(kd.load_library().kd_fwd, ctypes.byref(cp), ctypes.byref(ins),
                             *[o.data_ptr() for o in outs],
                             *_space(kd.kd_workspace_size(cp)[0], held), stream.cuda_stream), outs


JOBS = {
    "logprob": _logprob,
    "mix": _mix,
    # the staged slices of short and long teacher rows (and an exchange of two blocks an SM)
    "project": functools.partial(_project, ((1000, 500), (38000, 500))),
    # an exchange of one block an SM, by the student ids it serves
    "project_wide": functools.partial(_project, ((8, 20000), (15000, 20000))),
    "projected_loss": _projected_loss,
}
CALLS = {"project": 12000, "projected_loss": 12000}  # (a limit and its launch are a small part)


@pytest.mark.parametrize("op", list(JOBS))
def test_two_threads_at_once(op):
    held, streams = [], [torch.cuda.Stream() for _ in range(2)]
    jobs = [JOBS[op](i, s, held) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    want = []
    for call, outs in jobs:
        assert call() == kd.KD_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    told, times = [[], []], CALLS.get(op, 3000)

    def work(i):
        call = jobs[i][0]
        for _ in range(times // 50):
            told[i].extend(call() for _ in range(50))
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
    assert [len(t) for t in told] == [times, times]
    refused = [sum(s != kd.KD_OK for s in t) for t in told]
    assert refused == [0, 0]
    for (call, outs), ref in zip(jobs, want):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        assert call() == kd.KD_OK
        torch.cuda.synchronize()
        for got, t in zip(outs, ref):
            assert torch.equal(got, t)
