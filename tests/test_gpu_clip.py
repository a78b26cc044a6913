"""Gradient norm and clipping on the GPU against the fp64 oracle.

The norm: each square has a relative error of at most u = 2^-24 (an fma into
the sum), a thread's fp32 sum of at most 64 squares 64 u more, fp64 beyond; the
square root halves it, and storing adds u: 40 u.  A clipped element: that, u
for the coefficient, u for the product, and half a step of its type."""
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _grads(sizes, dtype, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale * (1 + i % 5)).to(DT[dtype])
            for i, s in enumerate(sizes)]


def _check(r, cpu, max_norm, dtype, tiny=0.0):
    norm, ref = O.clip(cpu, max_norm)
    assert abs(r["norm"].item() - norm) <= 40 * U * norm
    for got, want, g in zip(r["grads"], ref, cpu):
        if norm <= max_norm:
            assert torch.equal(got.cpu(), g)
            continue
        want = np.asarray(want)
        tol = (42 * U + HALF[dtype] * (1 + 42 * U)) * np.abs(want) + tiny
        assert (np.abs(as_f64(got) - want) <= tol).all()


SIZES = [[1], [7, 1, 3], [16384], [16383, 16385, 5], [100003, 0, 64, 8, 9], [65536] * 3,
         [3_000_001, 17], [33] * 700]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e9])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_clip_in_place_and_out(sizes, max_norm, dtype):
    cpu = _grads(sizes, dtype)
    gpu = [g.cuda() for g in cpu]
    out = [torch.full_like(g, 9.0) for g in gpu]
    r = kd.clip_grad_norm(gpu, max_norm, out=out)
    _check(r, cpu, max_norm, dtype)
    assert all(torch.equal(g.cpu(), c) for g, c in zip(gpu, cpu))
    again = kd.clip_grad_norm(gpu, max_norm)
    assert again["grads"][0] is gpu[0] and torch.equal(again["norm"], r["norm"])
    assert all(torch.equal(a, b) for a, b in zip(gpu, out))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_unaligned_tensors(shift, dtype):
    """Views at any element: each of the two sides at its own offset."""
    cpu = _grads([20000, 40001], dtype, seed=shift)
    store = [torch.zeros(c.numel() + 8, dtype=c.dtype, device="cuda") for c in cpu]
    gpu = [s[shift:shift + c.numel()] for s, c in zip(store, cpu)]
    for g, c in zip(gpu, cpu):
        g.copy_(c)
    out_store = [torch.full_like(s, 3.0) for s in store]
    out = [s[i:i + c.numel()] for i, (s, c) in enumerate(zip(out_store, cpu))]
    _check(kd.clip_grad_norm(gpu, 1.0, out=out), cpu, 1.0, dtype)
    for i, (s, c) in enumerate(zip(out_store, cpu)):
        assert (s[:i] == 3.0).all() and (s[i + c.numel():] == 3.0).all()
    _check(kd.clip_grad_norm(gpu, 1.0), cpu, 1.0, dtype)
    for s, c in zip(store, cpu):
        assert (s[:shift] == 0).all() and (s[shift + c.numel():] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e30, 1e-25, 1e25, 1e-18])
def test_squares_outside_the_range(scale, dtype):
    """Squares far above and below fp32's range, beside ordinary ones; clipped
    elements below 2^-126 may be flushed to 0."""
    cpu = _grads([30000, 3], dtype, scale) + [torch.zeros(5, dtype=DT[dtype])]
    norm, _ = O.clip(cpu, 1.0)
    r = kd.clip_grad_norm([g.cuda() for g in cpu], norm / 3 if norm / 3 < 3e38 else 1.0)
    _check(r, cpu, norm / 3 if norm / 3 < 3e38 else 1.0, dtype, tiny=2.0 ** -126)


def test_zero_and_nonfinite():
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert kd.clip_grad_norm(z, 0.0)["norm"].item() == 0.0
    for bad in (math.inf, math.nan, -math.inf):
        cpu = torch.arange(5000.0)
        cpu[777] = bad
        g = cpu.cuda()
        with pytest.raises(kd.KDError):
            kd.clip_grad_norm([g], 1.0)
        out = torch.zeros_like(g)
        r = kd.clip_grad_norm([g], 1.0, out=[out], check=False)
        assert int(r["dev_status"].item()) == kd.KD_DEV_NONFINITE
        assert not math.isfinite(r["norm"].item())
        assert torch.equal(g.cpu().nan_to_num(1.5), cpu.nan_to_num(1.5))
        assert torch.equal(out.cpu().nan_to_num(1.5), cpu.nan_to_num(1.5))


def test_repeats_give_the_same_bits_and_graphs_replay():
    cpu = _grads([500_000, 40_001, 3], "bf16")
    src = [g.cuda() for g in cpu]
    out = [torch.empty_like(g) for g in src]
    gl, ws = kd.GradList(src, out), kd.Workspace()
    first = kd.clip_grad_norm(gl, 1.0, workspace=ws)
    kept = [o.clone() for o in out]
    for _ in range(3):
        r = kd.clip_grad_norm(gl, 1.0, workspace=ws)
        assert torch.equal(r["norm"], first["norm"])
        assert all(torch.equal(a, b) for a, b in zip(out, kept))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r = kd.clip_grad_norm(gl, 1.0, workspace=ws, check=False)
    for g in src:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(r["norm"].item() - 2 * first["norm"].item()) <= 2 * U * 2 * first["norm"].item()
    # twice the gradients, half the coefficient: the same clipped values
    assert all(torch.equal(a, b) for a, b in zip(out, kept))


def test_norm_alone():
    cpu = _grads([1000, 50], "fp32")
    gpu = [g.cuda() for g in cpu]
    gl = kd.GradList(gpu)
    norm = torch.zeros(1, device="cuda")
    ws = kd.Workspace().get(gl._bytes, gl.device)
    st = kd.load_library().kd_clip_grad_norm(gl._grads, None, gl._numel, 2, kd.KD_FP32, 0.5,
                                             norm.data_ptr(), None, ws[0], ws[1],
                                             torch.cuda.current_stream().cuda_stream)
    assert st == kd.KD_OK
    want, _ = O.clip(cpu, 1.0)
    assert abs(norm.item() - want) <= 40 * U * want
    assert all(torch.equal(g.cpu(), c) for g, c in zip(gpu, cpu))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale,max_norm", [(1e30, 1e-8), (1e34, 1e-3), (1e30, 1e-15),
                                            (1e34, 1e-36), (1e34, 1e34)])
def test_coefficients_below_the_normal_range(scale, max_norm, dtype):
    """A large norm over a small bound: max_norm / norm has few bits or none in
    fp32, the clipped elements have all of theirs."""
    cpu = _grads([30000, 3], dtype, scale)
    r = kd.clip_grad_norm([g.cuda() for g in cpu], max_norm)
    _check(r, cpu, max_norm, dtype, tiny=2.0 ** -126)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value,count", [(2.0 ** -133, 50000), (2.0 ** -130, 40000)])
def test_norm_of_subnormal_gradients(value, count, dtype):
    """Equal elements far below 2^-126: the norm is value sqrt(count), itself a
    subnormal number, to half a step of those."""
    g = [torch.full((count,), value, device="cuda").to(DT[dtype])]
    norm = kd.clip_grad_norm(g, 1.0)["norm"].item()
    want = value * math.sqrt(count)
    assert abs(norm - want) <= 40 * U * want + 2.0 ** -150
    g = [torch.full((count,), 2.0 ** -133 if dtype == "bf16" else 2.0 ** -149, device="cuda")
         .to(DT[dtype])]
    want = float(g[0][0].double()) * math.sqrt(count)
    assert abs(kd.clip_grad_norm(g, 1.0)["norm"].item() - want) <= 40 * U * want + 2.0 ** -150


def test_norm_beyond_fp32():
    """Finite elements whose norm fp32 cannot hold: stored as infinity, clipped
    by the norm that it is."""
    cpu = [torch.full((4,), 3e38), torch.tensor([1e38, -2.0])]
    r = kd.clip_grad_norm([g.cuda() for g in cpu], 1e30)
    assert r["norm"].item() == math.inf and int(r["dev_status"].item()) == 0
    _, ref = O.clip(cpu, 1e30)
    for got, want in zip(r["grads"], ref):
        tol = (42 * U + U * (1 + 42 * U)) * np.abs(want) + 2.0 ** -126
        assert (np.abs(as_f64(got) - want) <= tol).all()
