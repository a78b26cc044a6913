"""Host-side rules of kd_logprob_* and kd_clip_grad_norm: struct layout, refused
arguments, workspace sizes.  No kernel is launched on this machine, and the GPU
is never reached by a refused call."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a pointer that is never followed


@pytest.fixture(scope="module")
def kd():
    from lm_head_cross_vocab_gb300 import build, kd as K
    build.build()
    K.load_library()
    return K


@pytest.mark.parametrize("name", ["kd_logprob_problem", "kd_logprob_inputs"])
def test_struct_layout_matches_c(kd, tmp_path, name):
    struct = getattr(kd, name)
    fields = [f for f, _ in struct._fields_]
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "kd.h"', "int main(void){",
            f'printf("%zu\\n", sizeof({name}));']
    prog += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["return 0;}"]
    c, exe = tmp_path / "probe.c", tmp_path / "probe"
    c.write_text("\n".join(prog))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o",
                    str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                           check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(struct)
    assert vals[1:] == [getattr(struct, f).offset for f in fields]


def _prob(kd, ld=0, ldg=0, **kw):
    base = dict(n_tokens=8, vocab=100, d_model=64, topk=4, dtype="bf16", source="logits")
    base.update(kw)
    return kd.LogprobProblem(**base).to_c(ld, ldg)


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1),
    dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
    dict(temperature=float("inf")), dict(temperature=1e-45), dict(topk=-1), dict(topk=101),
    dict(topk=1025, vocab=5000), dict(ld=99), dict(ldg=99), dict(source="hidden", d_model=0),
])
def test_bad_problems_are_refused(kd, bad):
    p = _prob(kd, **bad)
    f, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = kd.load_library().kd_logprob_workspace_size(ctypes.byref(p), ctypes.byref(f),
                                                     ctypes.byref(b))
    assert st == kd.KD_ERR_INVALID_ARG


def test_unknown_types_and_null_problem(kd):
    lib = kd.load_library()
    assert lib.kd_logprob_workspace_size(None, None, None) == kd.KD_ERR_INVALID_ARG
    for field in ("dtype", "source"):
        p = _prob(kd)
        setattr(p, field, 7)
        assert lib.kd_logprob_workspace_size(ctypes.byref(p), None, None) == kd.KD_ERR_INVALID_ARG
    # a bf16 head is read by TMA: rows of a multiple of 16 bytes
    p = _prob(kd, source="hidden", d_model=60)
    assert lib.kd_logprob_workspace_size(ctypes.byref(p), None, None) == kd.KD_ERR_UNSUPPORTED
    p = _prob(kd, source="hidden", d_model=60, dtype="fp32")
    assert lib.kd_logprob_workspace_size(ctypes.byref(p), None, None) == kd.KD_OK


def _fwd(kd, p, ins, **out):
    o = {k: out.get(k) for k in ("logprob", "entropy", "topk_idx", "topk_logprob", "stats")}
    return kd.load_library().kd_logprob_fwd(ctypes.byref(p), ctypes.byref(ins), *o.values(), None,
                                            out.get("ws"), out.get("bytes", 0), None)


def test_forward_argument_rules(kd):
    logits = kd.kd_logprob_inputs(logits=FAKE, tokens=FAKE)
    assert _fwd(kd, _prob(kd), kd.kd_logprob_inputs(), entropy=FAKE) == kd.KD_ERR_INVALID_ARG
    assert _fwd(kd, _prob(kd), kd.kd_logprob_inputs(logits=FAKE), logprob=FAKE) \
        == kd.KD_ERR_INVALID_ARG  # a log-probability of which token
    assert _fwd(kd, _prob(kd), logits, stats=FAKE + 4) == kd.KD_ERR_INVALID_ARG
    hidden = _prob(kd, source="hidden")
    assert _fwd(kd, hidden, logits, entropy=FAKE) == kd.KD_ERR_INVALID_ARG
    odd = kd.kd_logprob_inputs(h=FAKE + 8, w=FAKE)
    assert _fwd(kd, hidden, odd, entropy=FAKE) == kd.KD_ERR_UNSUPPORTED
    ok = kd.kd_logprob_inputs(h=FAKE, w=FAKE)
    assert _fwd(kd, hidden, ok, entropy=FAKE) == kd.KD_ERR_WORKSPACE
    f, _ = kd.kd_logprob_workspace_size(hidden)
    assert _fwd(kd, hidden, ok, entropy=FAKE, ws=FAKE + 16, bytes=f) == kd.KD_ERR_WORKSPACE
    assert _fwd(kd, hidden, ok, entropy=FAKE, ws=FAKE, bytes=f - 1) == kd.KD_ERR_WORKSPACE


def test_backward_argument_rules(kd):
    lib = kd.load_library()

    def bwd(p, ins, stats=FAKE, dlp=None, dh=None, dw=None, dz=None, ws=None, nbytes=0):
        return lib.kd_logprob_bwd(ctypes.byref(p), ctypes.byref(ins), stats, dlp, None, dh, dw,
                                  dz, None, ws, nbytes, None)

    logits = kd.kd_logprob_inputs(logits=FAKE)
    hidden = kd.kd_logprob_inputs(h=FAKE, w=FAKE, tokens=FAKE)
    assert bwd(_prob(kd), logits, dh=FAKE) == kd.KD_ERR_INVALID_ARG
    assert bwd(_prob(kd), logits, stats=None, dz=FAKE) == kd.KD_ERR_INVALID_ARG
    assert bwd(_prob(kd), logits, dlp=FAKE, dz=FAKE) == kd.KD_ERR_INVALID_ARG  # no tokens
    assert bwd(_prob(kd, source="hidden"), hidden, dz=FAKE) == kd.KD_ERR_INVALID_ARG
    assert bwd(_prob(kd, source="hidden"), hidden, dw=FAKE) == kd.KD_ERR_WORKSPACE


def test_no_scratch_buffer_spans_tokens_by_vocab(kd):
    """Large hidden problems: neither pass holds the logits, nor half of them in bf16."""
    for n, v, d in ((4096, 32000, 2048), (32768, 151936, 4096)):
        f, b = kd.kd_logprob_workspace_size(_prob(kd, n_tokens=n, vocab=v, d_model=d, topk=100,
                                                  source="hidden"))
        assert f < n * v * 2
        assert b - 4 * (n + v) * d - 2 * n * d < n * v * 2


def _clip(kd, grads, outs, numel, n=None, dtype=None, max_norm=1.0, ws=FAKE, nbytes=1 << 20):
    arr = (ctypes.c_void_p * max(1, len(grads)))(*grads)
    oarr = None if outs is None else (ctypes.c_void_p * max(1, len(outs)))(*outs)
    cnt = (ctypes.c_int64 * max(1, len(numel)))(*numel)
    return kd.load_library().kd_clip_grad_norm(
        arr, oarr, cnt, len(numel) if n is None else n, kd.KD_BF16 if dtype is None else dtype,
        ctypes.c_float(max_norm), None, None, ws, nbytes, None)


def test_clip_argument_rules(kd):
    import torch
    a, b = FAKE, 2 * FAKE
    bad = [dict(n=-1), dict(dtype=5), dict(max_norm=-1.0), dict(max_norm=float("nan")),
           dict(max_norm=float("inf"))]
    for kw in bad:
        assert _clip(kd, [a, b], [a, b], [10, 10], **kw) == kd.KD_ERR_INVALID_ARG, kw
    refused = [
        ([a, None], [a, b], [10, 10]), ([a, b], [a, None], [10, 10]), ([a, b], [a, b], [10, -1]),
        ([a + 1, b], [a + 1, b], [10, 10]),            # odd address of a bf16 tensor
        ([a, a], [a, a], [10, 10]),                     # the same tensor twice
        ([a, b], [a, a + 18], [10, 10]),                # an out inside another tensor
        ([a, b], [a + 2, b], [10, 10]),                 # an out that overlaps its own gradient
        ([a, b], [4 * FAKE, 4 * FAKE + 19], [10, 10]),  # two outs one element apart
    ]
    for g, o, cnt in refused:
        assert _clip(kd, g, o, cnt) == kd.KD_ERR_INVALID_ARG, (g, o, cnt)
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(nbytes=0)):
        assert _clip(kd, [a], [a], [10], **kw) == kd.KD_ERR_WORKSPACE, kw
    if torch.cuda.is_available():
        return  # well-formed calls would launch
    for g, o, cnt in (([a, b], [a, b], [10, 10]), ([a, b], None, [10, 10]),
                      ([a, a], None, [10, 10]), ([None, b], [None, b], [0, 10]),
                      ([a, b], [a + 20, b + 20], [10, 10])):
        assert _clip(kd, g, o, cnt) == kd.KD_ERR_NO_DEVICE, (g, o, cnt)


def test_binding_refuses_wrong_tensors(kd):
    import torch
    p = kd.LogprobProblem(n_tokens=2, vocab=8)
    with pytest.raises(ValueError):
        kd.token_logprobs(p, {"logits": torch.zeros(2, 8, dtype=torch.bfloat16)})
    with pytest.raises(ValueError):
        kd.token_logprobs(p, {})
    with pytest.raises(ValueError):
        kd.GradList([])
    with pytest.raises(ValueError):
        kd.GradList([torch.zeros(3)])


def test_unaligned_hidden_gradients_are_refused(kd):
    """bf16 gradients are stored in 16-byte vectors: a buffer at another address,
    a view behind a tensor of odd length for example, is refused before anything
    is launched.  fp32 ones take any element's address, and without tokens d_w is
    only cleared."""
    lib = kd.load_library()
    ins = kd.kd_logprob_inputs(h=FAKE, w=FAKE, tokens=FAKE)

    def bwd(p, dh, dw):
        return lib.kd_logprob_bwd(ctypes.byref(p), ctypes.byref(ins), FAKE, None, None, dh, dw,
                                  None, None, None, 0, None)

    p = _prob(kd, source="hidden")
    for off in (2, 4, 8, 14):
        assert bwd(p, 2 * FAKE + off, None) == kd.KD_ERR_UNSUPPORTED
        assert bwd(p, None, 3 * FAKE + off) == kd.KD_ERR_UNSUPPORTED
        assert bwd(p, 2 * FAKE, 3 * FAKE + off) == kd.KD_ERR_UNSUPPORTED
    assert bwd(p, 2 * FAKE + 16, 3 * FAKE + 32) == kd.KD_ERR_WORKSPACE  # and no further
    for kw in (dict(dtype="fp32"), dict(n_tokens=0)):
        p = _prob(kd, source="hidden", **kw)
        assert bwd(p, 2 * FAKE + 4, 3 * FAKE + 8) == kd.KD_ERR_WORKSPACE


class _Fake:
    """Stands in for the library: no kernel runs, what a call is given is kept."""

    def __init__(self, kd, monkeypatch):
        import contextlib
        import weakref
        self.alive, self.status, self.seen = [], 0, []
        made = []

        class Tracked(kd.Workspace):
            def __init__(self):
                super().__init__()
                made.append(weakref.ref(self))

        def call(*args):
            self.alive.append(bool(made) and made[-1]() is not None)
            word = next(a for a in args if isinstance(a, int) and a in self.words)
            self.seen.append(word)
            if self.status:
                ctypes.c_int32.from_address(word).value |= self.status
            return kd.KD_OK

        self.words = set()
        zeros = kd.torch.zeros

        def status_word(*a, **kw):
            t = zeros(*a, **kw)
            if t.dtype == kd.torch.int32 and t.dim() == 0:
                self.words.add(t.data_ptr())
            return t

        monkeypatch.setattr(kd, "Workspace", Tracked)
        monkeypatch.setattr(kd, "load_library", lambda: self)
        monkeypatch.setattr(kd, "kd_logprob_workspace_size", lambda p: (1000, 1000))
        monkeypatch.setattr(kd, "_on", lambda dev: contextlib.nullcontext(0))
        monkeypatch.setattr(kd.torch, "zeros", status_word)
        self.kd_logprob_fwd = self.kd_logprob_bwd = self.kd_clip_grad_norm = call
        self.kd_clip_grad_norm_workspace_size = lambda *a: kd.KD_OK
        self.kd_status_string = lambda s: b"status"


def _as_cuda(t):
    """A tensor here that says it is on a GPU."""
    import torch

    class Device(torch.Tensor):
        is_cuda = True

    return t.as_subclass(Device)


def _hidden_call(kd, n=4, v=50, d=8):
    import torch
    p = kd.LogprobProblem(n_tokens=n, vocab=v, d_model=d, source="hidden")
    bf = torch.bfloat16
    return p, {"h": _as_cuda(torch.zeros(n, d, dtype=bf)), "w": torch.zeros(v, d, dtype=bf),
               "tokens": torch.zeros(n, dtype=torch.int64)}


def test_a_calls_own_workspace_lives_until_it_returns(kd, monkeypatch):
    """Without a workspace of the caller's: the one made for the call is still
    held while the library enqueues its kernels."""
    import torch
    fake = _Fake(kd, monkeypatch)
    p, tens = _hidden_call(kd)
    out = kd.token_logprobs(p, tens)
    kd.token_logprobs_backward(p, tens, out["stats"])
    kd.clip_grad_norm([_as_cuda(torch.zeros(5))], 1.0)
    assert fake.alive == [True, True, True]


def test_an_error_is_told_once(kd, monkeypatch):
    """A dict of outputs that is used again: the status of a call that raised is
    told, and the next call without an error passes."""
    fake = _Fake(kd, monkeypatch)
    p, tens = _hidden_call(kd)
    out = kd.token_logprobs(p, tens)
    grad = kd.token_logprobs_backward(p, tens, out["stats"])
    for call in (lambda **kw: kd.token_logprobs(p, tens, out=out, **kw),
                 lambda **kw: kd.token_logprobs_backward(p, tens, out["stats"], out=grad, **kw)):
        fake.status = kd.KD_DEV_BAD_LABEL
        with pytest.raises(kd.KDError) as e:
            call()
        assert e.value.status == kd.KD_ERR_BAD_LABEL
        fake.status = 0
        call()
        # without a check the bits stay, for the caller to read and to clear
        fake.status = kd.KD_DEV_BAD_LABEL
        call(check=False)
        fake.status = 0
        assert int(call(check=False)["dev_status"]) == kd.KD_DEV_BAD_LABEL
        with pytest.raises(kd.KDError):
            call()
        call()


def test_out_needs_no_status_word_and_refuses_a_wrong_one(kd, monkeypatch):
    """``out`` may bring the gradients alone; a status word that a kernel could
    not write to is refused before the library is called."""
    import torch
    fake = _Fake(kd, monkeypatch)
    p, tens = _hidden_call(kd)
    stats = torch.zeros(4, 4)
    d_w = torch.zeros(50, 8, dtype=torch.bfloat16)
    r = kd.token_logprobs_backward(p, tens, stats, out={"d_w": d_w})
    assert r["d_w"] is d_w and int(r["dev_status"]) == 0
    assert int(kd.token_logprobs(p, tens, out={"logprob": torch.zeros(4)})["dev_status"]) == 0
    calls = len(fake.seen)
    assert calls == 2
    for word in (torch.zeros((), dtype=torch.int64), torch.zeros(2, dtype=torch.int32),
                 torch.zeros((), dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError):
            kd.token_logprobs_backward(p, tens, stats, out={"d_w": d_w, "dev_status": word})
        with pytest.raises(ValueError):
            kd.token_logprobs(p, tens, out={"logprob": torch.zeros(4), "dev_status": word})
    assert len(fake.seen) == calls


def test_gradients_that_overlap_what_is_read_are_refused(kd):
    """d_logits may be the logits, or lie between their rows; any other overlap,
    and any of the hidden gradients', would be read after it was written."""
    lib = kd.load_library()

    def bwd(p, ins, dh=None, dw=None, dz=None):
        return lib.kd_logprob_bwd(ctypes.byref(p), ctypes.byref(ins), FAKE, None, None, dh, dw,
                                  dz, None, FAKE, 1 << 24, None)

    z = 1 << 30
    ins = kd.kd_logprob_inputs(logits=z, tokens=FAKE)
    tight, wide = _prob(kd), _prob(kd, ld=250, ldg=250)  # 8 rows of 100
    for p, off in ((tight, 2), (tight, -2), (tight, 200), (tight, -1598), (wide, 2), (wide, 198),
                   (wide, -302), (wide, 502), (wide, 302), (_prob(kd, ld=100, ldg=250), 0),
                   (_prob(kd, ld=250, ldg=100), 1000)):
        assert bwd(p, ins, dz=z + off) == kd.KD_ERR_INVALID_ARG, off
    import torch
    here = not torch.cuda.is_available()  # (well-formed calls would launch)
    if here:
        for p, off in ((tight, 0), (tight, 1600), (tight, -1600), (wide, 0), (wide, 200),
                       (wide, 300), (wide, -200), (wide, 700), (wide, 3700), (wide, -3700)):
            assert bwd(p, ins, dz=z + off) == kd.KD_ERR_NO_DEVICE, off
    p, h, w = _prob(kd, source="hidden"), 1 << 30, 1 << 31  # 1024 and 12800 bytes
    ins = kd.kd_logprob_inputs(h=h, w=w, tokens=FAKE)
    far = 1 << 32
    for dh, dw in ((h, None), (None, w), (h + 1008, None), (None, h + 16), (w + 12784, None),
                   (None, w - 12784), (far, far + 1008), (far + 12784, far)):
        assert bwd(p, ins, dh, dw) == kd.KD_ERR_INVALID_ARG, (dh, dw)
    if here:
        for dh, dw in ((h + 1024, w + 12800), (far, far + 1024), (far + 12800, far),
                       (h - 1024, None)):
            assert bwd(p, ins, dh, dw) == kd.KD_ERR_NO_DEVICE, (dh, dw)


def test_arrays_off_their_elements_boundaries_are_refused(kd):
    """An address that is no multiple of its elements' size, by name; the same
    call with every address in order gets as far as the workspace."""
    lib = kd.load_library()

    def fwd(p, ins, **o):
        names = ("logprob", "entropy", "topk_idx", "topk_logprob", "stats", "dev_status")
        return lib.kd_logprob_fwd(ctypes.byref(p), ctypes.byref(ins),
                                  *[o.get(x, 3 * FAKE) for x in names], None, 0, None)

    def bwd(p, ins, **o):
        names = ("d_logprob", "d_entropy", "d_h", "d_w", "d_logits", "dev_status")
        return lib.kd_logprob_bwd(ctypes.byref(p), ctypes.byref(ins), FAKE,
                                  *[o.get(x) for x in names], None, 0, None)

    for dtype, size in (("bf16", 2), ("fp32", 4)):
        p = _prob(kd, source="hidden", dtype=dtype)
        base = dict(h=FAKE, w=2 * FAKE, tokens=FAKE)
        ins = kd.kd_logprob_inputs(**base)
        assert fwd(p, ins) == bwd(p, ins, d_h=FAKE) == kd.KD_ERR_WORKSPACE
        for name in ("logprob", "entropy", "topk_idx", "topk_logprob", "stats", "dev_status"):
            assert fwd(p, ins, **{name: 3 * FAKE + 2}) == kd.KD_ERR_INVALID_ARG, name
        for name in ("d_logprob", "d_entropy", "dev_status"):
            assert bwd(p, ins, d_h=FAKE, **{name: FAKE + 2}) == kd.KD_ERR_INVALID_ARG, name
        for name in ("d_h", "d_w"):
            assert bwd(p, ins, **{name: FAKE + size // 2}) == kd.KD_ERR_INVALID_ARG, name
        for name, off in (("tokens", 4),) + ((("h", 2), ("w", 2)) if dtype == "fp32" else ()):
            bad = kd.kd_logprob_inputs(**{**base, name: base[name] + off})
            assert fwd(p, bad) == bwd(p, bad, d_h=FAKE) == kd.KD_ERR_INVALID_ARG, name
        p = _prob(kd, dtype=dtype)
        bad = kd.kd_logprob_inputs(logits=FAKE + size // 2, tokens=FAKE)
        assert fwd(p, bad) == kd.KD_ERR_INVALID_ARG
        assert bwd(p, kd.kd_logprob_inputs(logits=FAKE, tokens=FAKE), d_logits=3 * FAKE + size // 2) \
            == kd.KD_ERR_INVALID_ARG
    arr, cnt = (ctypes.c_void_p * 1)(FAKE), (ctypes.c_int64 * 1)(10)
    for norm, status in ((FAKE + 2, None), (None, FAKE + 1)):
        assert lib.kd_clip_grad_norm(arr, arr, cnt, 1, kd.KD_FP32, 1.0, norm, status, FAKE,
                                     1 << 20, None) == kd.KD_ERR_INVALID_ARG
