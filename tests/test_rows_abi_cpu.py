"""Host-side rules of kd_verify_*, kd_embed_* and kd_rmsnorm_*: struct layout,
refused arguments, workspace sizes.  No kernel is launched on this machine, and
the GPU is never reached by a refused call."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40  # pointers that are never followed, far apart
A, B, C, D, E, F, G, H, I = (FAKE + (i << 32) for i in range(9))


@pytest.fixture(scope="module")
def kd():
    from lm_head_cross_vocab_gb300 import build, kd as K
    build.build()
    K.load_library()
    return K


def _gpu():
    import torch
    return torch.cuda.is_available()


@pytest.mark.parametrize("name", ["kd_verify_problem", "kd_verify_inputs", "kd_embed_problem",
                                  "kd_rmsnorm_problem"])
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


# ---------------------------------------------------------------- verification

def _vp(kd, ldt=0, ldd=0, **kw):
    base = dict(n_seqs=4, vocab=100, n_drafts=3)
    base.update(kw)
    return kd.VerifyProblem(**base).to_c(ldt, ldd)


def _verify(kd, p, ws=I, nbytes=1 << 30, tokens=G, accepted=H, logprob=H + 4096, status=None,
            **ins):
    base = dict(target_logits=A, draft_logits=B, drafts=C, lengths=D, uniform=E, noise=F)
    base.update(ins)
    return kd.load_library().kd_verify_drafts(
        ctypes.byref(p), ctypes.byref(kd.kd_verify_inputs(**base)), tokens, accepted, logprob,
        status, ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(n_seqs=-1), dict(n_seqs=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1),
    dict(n_drafts=-1), dict(n_drafts=33), dict(t_target=-1.0), dict(t_target=float("nan")),
    dict(t_target=float("inf")), dict(t_target=1e-45), dict(t_draft=0.0), dict(t_draft=-1.0),
    dict(t_draft=float("inf")), dict(ldt=99), dict(ldd=99)])
def test_verify_bad_problems_are_refused(kd, bad):
    p, n = _vp(kd, **bad), ctypes.c_size_t(0)
    assert kd.load_library().kd_verify_workspace_size(ctypes.byref(p), ctypes.byref(n)) \
        == kd.KD_ERR_INVALID_ARG
    assert _verify(kd, p) == kd.KD_ERR_INVALID_ARG


def test_verify_argument_rules(kd):
    p = _vp(kd)
    lib = kd.load_library()
    assert lib.kd_verify_workspace_size(None, None) == kd.KD_ERR_INVALID_ARG
    odd = _vp(kd)
    odd.dtype = 7
    assert _verify(kd, odd) == kd.KD_ERR_INVALID_ARG
    assert lib.kd_verify_drafts(ctypes.byref(p), None, G, H, H, None, I, 1 << 30, None) \
        == kd.KD_ERR_INVALID_ARG
    for name in ("target_logits", "drafts", "uniform", "noise"):
        assert _verify(kd, p, **{name: None}) == kd.KD_ERR_INVALID_ARG, name
    for name in ("target_logits", "draft_logits", "drafts", "lengths", "uniform", "noise"):
        assert _verify(kd, p, **{name: A + 1}) == kd.KD_ERR_INVALID_ARG, name
    for kw in (dict(tokens=G + 4), dict(accepted=H + 2), dict(logprob=H + 2), dict(status=I + 1)):
        assert _verify(kd, p, **kw) == kd.KD_ERR_INVALID_ARG, kw
    # outputs over inputs, or over one another
    for kw in (dict(tokens=C), dict(tokens=A + 800), dict(logprob=F + 1596), dict(accepted=D),
               dict(logprob=E), dict(accepted=G), dict(logprob=G + 120), dict(logprob=B + 2396)):
        assert _verify(kd, p, **kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=I + 16), dict(nbytes=kd.kd_verify_workspace_size(p) - 1)):
        assert _verify(kd, p, **kw) == kd.KD_ERR_WORKSPACE, kw
    if _gpu():
        return  # well-formed calls would launch
    greedy = _vp(kd, t_target=0.0)
    for q, kw in ((p, {}), (p, dict(draft_logits=None, lengths=None)),
                  (p, dict(logprob=G + 128)), (p, dict(tokens=None, accepted=None, logprob=None)),
                  (greedy, dict(uniform=None, noise=None)),
                  (_vp(kd, n_drafts=0), dict(drafts=None, uniform=None))):
        assert _verify(kd, q, **kw) == kd.KD_ERR_NO_DEVICE, kw


def test_verify_workspace_does_not_grow_with_the_vocabulary(kd):
    small = kd.kd_verify_workspace_size(_vp(kd, n_seqs=256, n_drafts=7, vocab=32000))
    assert kd.kd_verify_workspace_size(_vp(kd, n_seqs=256, n_drafts=7, vocab=256000)) < 16 * small
    assert small < 4 << 20


# ---------------------------------------------------------------- embedding

def _ep(kd, **kw):
    base = dict(n_tokens=10, vocab=100, d_model=64)
    base.update(kw)
    return kd.EmbedProblem(**base).to_c()


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_tokens=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1),
    dict(d_model=0), dict(d_model=(1 << 30) + 1), dict(scale=float("nan")),
    dict(scale=float("inf"))])
def test_embed_bad_problems_are_refused(kd, bad):
    p = _ep(kd, **bad)
    lib = kd.load_library()
    assert lib.kd_embed_workspace_size(ctypes.byref(p), None) == kd.KD_ERR_INVALID_ARG
    assert lib.kd_embed_fwd(ctypes.byref(p), A, B, C, None, None) == kd.KD_ERR_INVALID_ARG
    assert lib.kd_embed_bwd(ctypes.byref(p), A, B, C, 0, None, I, 1 << 40, None) \
        == kd.KD_ERR_INVALID_ARG


def test_embed_argument_rules(kd):
    lib, p = kd.load_library(), _ep(kd)

    def fwd(tokens=A, w=B, h=C, status=None, p=p):
        return lib.kd_embed_fwd(ctypes.byref(p), tokens, w, h, status, None)

    def bwd(tokens=A, d_h=B, d_w=C, acc=0, status=None, ws=I, nbytes=1 << 30, p=p):
        return lib.kd_embed_bwd(ctypes.byref(p), tokens, d_h, d_w, acc, status, ws, nbytes, None)

    table, rows = 100 * 64 * 2, 10 * 64 * 2
    for kw in (dict(tokens=None), dict(w=None), dict(h=None), dict(tokens=A + 4), dict(w=B + 1),
               dict(h=C + 1), dict(status=I + 2), dict(h=B), dict(h=B + table - 2),
               dict(h=B - rows + 2), dict(h=A + 64)):
        assert fwd(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(tokens=None), dict(d_h=None), dict(d_w=None), dict(tokens=A + 4),
               dict(d_h=B + 1), dict(d_w=C + 1), dict(status=I + 2), dict(acc=2), dict(acc=-1),
               dict(d_w=B), dict(d_w=B + rows - 2), dict(d_w=B - table + 2), dict(d_w=A + 8)):
        assert bwd(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=I + 8), dict(nbytes=kd.kd_embed_workspace_size(p) - 1)):
        assert bwd(**kw) == kd.KD_ERR_WORKSPACE, kw
    # more blocks than a launch takes
    huge = _ep(kd, n_tokens=1 << 30, d_model=1 << 12)
    assert fwd(p=huge) == kd.KD_ERR_UNSUPPORTED
    huge = _ep(kd, n_tokens=1 << 30, d_model=1 << 16, vocab=100)
    assert bwd(p=huge, nbytes=1 << 62, tokens=1 << 50, d_h=1 << 60) == kd.KD_ERR_UNSUPPORTED
    if _gpu():
        return
    assert fwd() == kd.KD_ERR_NO_DEVICE and fwd(h=B + table) == kd.KD_ERR_NO_DEVICE
    assert bwd() == kd.KD_ERR_NO_DEVICE and bwd(acc=1) == kd.KD_ERR_NO_DEVICE


# ---------------------------------------------------------------- norm

def _np(kd, **kw):
    base = dict(n_tokens=10, d_model=64)
    base.update(kw)
    return kd.NormProblem(**base).to_c()


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(d_model=0), dict(d_model=32769),
    dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight_offset=float("inf")), dict(weight_offset=float("nan"))])
def test_norm_bad_problems_are_refused(kd, bad):
    p = _np(kd, **bad)
    lib = kd.load_library()
    assert lib.kd_rmsnorm_workspace_size(ctypes.byref(p), None) == kd.KD_ERR_INVALID_ARG
    assert lib.kd_rmsnorm_fwd(ctypes.byref(p), A, B, C, D, E, None) == kd.KD_ERR_INVALID_ARG
    assert lib.kd_rmsnorm_bwd(ctypes.byref(p), A, B, C, D, E, F, I, 1 << 40, None) \
        == kd.KD_ERR_INVALID_ARG


def test_norm_argument_rules(kd):
    lib, p = kd.load_library(), _np(kd)

    def fwd(x=A, res=B, w=C, sum=D, h=E):
        return lib.kd_rmsnorm_fwd(ctypes.byref(p), x, res, w, sum, h, None)

    def bwd(s=A, w=B, d_h=C, d_sum=D, d_x=E, d_w=F, ws=I, nbytes=1 << 30):
        return lib.kd_rmsnorm_bwd(ctypes.byref(p), s, w, d_h, d_sum, d_x, d_w, ws, nbytes, None)

    for kw in (dict(x=None), dict(w=None), dict(h=None), dict(x=A + 1), dict(res=B + 1),
               dict(w=C + 1), dict(sum=D + 1), dict(h=E + 1), dict(h=A + 2), dict(sum=A - 2),
               dict(h=B + 128), dict(h=D), dict(sum=C), dict(h=C + 126), dict(sum=E + 128),
               dict(h=A, sum=A)):
        assert fwd(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(s=None), dict(w=None), dict(d_h=None), dict(s=A + 1), dict(d_sum=D + 1),
               dict(d_x=E + 1), dict(d_w=F + 1), dict(d_x=A + 2), dict(d_x=C + 128),
               dict(d_x=D - 2), dict(d_x=B), dict(d_w=B), dict(d_w=A + 2), dict(d_w=C),
               dict(d_w=D), dict(d_w=E + 1278)):
        assert bwd(**kw) == kd.KD_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=I + 8), dict(nbytes=kd.kd_rmsnorm_workspace_size(p) - 1)):
        assert bwd(**kw) == kd.KD_ERR_WORKSPACE, kw
    if _gpu():
        return
    for kw in ({}, dict(res=None), dict(sum=None), dict(h=A, sum=B), dict(h=A + 1280)):
        assert fwd(**kw) == kd.KD_ERR_NO_DEVICE, kw
    for kw in ({}, dict(d_sum=None), dict(d_x=A), dict(d_x=C), dict(d_x=D), dict(d_x=None),
               dict(d_w=None, ws=None)):
        assert bwd(**kw) == kd.KD_ERR_NO_DEVICE, kw


# ---------------------------------------------------------------- binding

def test_binding_refuses_wrong_tensors(kd):
    import torch
    z = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kd.verify_drafts(kd.VerifyProblem(n_seqs=2, vocab=8, n_drafts=2), {"target_logits": z})
    with pytest.raises(ValueError):
        kd.verify_drafts(kd.VerifyProblem(n_seqs=2, vocab=8, n_drafts=2), {})
    p = kd.EmbedProblem(n_tokens=2, vocab=8, d_model=8)
    w, t = torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        kd.embed_tokens(p, w, t)
    with pytest.raises(ValueError):
        kd.embed_tokens_backward(p, t, w[:2])
    with pytest.raises(ValueError):
        kd.rms_norm(kd.NormProblem(n_tokens=8, d_model=8), w, w[0])
    with pytest.raises(ValueError):
        kd.rms_norm_backward(kd.NormProblem(n_tokens=8, d_model=8), w, w[0], w)


@pytest.mark.parametrize("strides,shape,pitch", [
    ((24, 8, 1), (2, 3, 8), 0), ((30, 10, 1), (2, 3, 8), 10), ((10, 99, 1), (4, 1, 8), 10),
    ((999, 10, 1), (1, 3, 8), 10)])
def test_pitches_of_sequences_of_rows(kd, strides, shape, pitch):
    import torch
    z = torch.zeros(4096).as_strided(shape, strides)
    assert kd._seq_rows_pitch("z", z, shape, torch.float32, z.device) == pitch


@pytest.mark.parametrize("strides,shape", [
    ((31, 10, 1), (2, 3, 8)), ((24, 8, 2), (2, 3, 8)), ((21, 7, 1), (2, 3, 8)),
    ((0, 8, 1), (2, 3, 8)), ((8, 16, 1), (2, 3, 8))])
def test_other_strides_are_refused(kd, strides, shape):
    import torch
    z = torch.zeros(4096).as_strided(shape, strides)
    with pytest.raises(ValueError):
        kd._seq_rows_pitch("z", z, shape, torch.float32, z.device)
