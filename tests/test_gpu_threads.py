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


JOBS = {
    "logprob": _logprob,
    "mix": _mix,
}


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
    told, times = [[], []], 3000

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
