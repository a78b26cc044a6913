"""The norm and its backward on the GPU against the fp64 oracle.

u = 2^-24.  A row's sum of squares: a thread adds at most E = 64 products, then
10 levels of shuffles; its relative error (all terms positive) is at most
(E + 12) u, the root halves it; mean, root, reciprocal and the three products
of h add 8 u: (E / 2 + 14) u, plus half a step of the type.  The backward's sum
of g s is off by (E + 14) u of the sum of absolute values, r^3 by three times
r's error: each term of d_x is within (4 E) u of its absolute value.  d_weight
adds up to N rows in fp32: (N + E) u of the sum of absolute values."""
import numpy as np
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd
from oracle import rows_oracle as R
from oracle.kd_oracle import as_f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
U, E = 2.0 ** -24, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _data(n, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    size = torch.where(torch.rand(d, generator=g) < 0.05, 20.0, 1.0)
    mk = lambda scale: (torch.randn(n, d, generator=g) * scale).to(DT[dtype])  # noqa: E731
    return {"x": mk(size), "residual": mk(size), "d_h": mk(1e-3), "d_sum": mk(1e-3),
            "weight": (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype])}


def _check_fwd(r, c, dtype, residual, **kw):
    h, s = R.rms_norm(c["x"], c["weight"], c["residual"] if residual else None, **kw)
    rel = (E / 2 + 14) * U
    assert (np.abs(as_f64(r["h"]) - h) <= (rel + HALF[dtype] * (1 + rel)) * np.abs(h) + 1e-40).all()
    if residual:
        tol = U * (np.abs(as_f64(c["x"])) + np.abs(as_f64(c["residual"]))) + HALF[dtype] * np.abs(s)
        assert (np.abs(as_f64(r["sum"]) - s) <= tol).all()


def _check_bwd(r, s, c, dtype, d_sum, n, **kw):
    ref = R.rms_norm_grad(s, c["weight"], c["d_h"], c["d_sum"] if d_sum else None, **kw)
    for name, size, adds in (("d_x", ref["x_size"], 4 * E), ("d_weight", ref["w_size"], n + E)):
        if r.get(name) is not None:
            err = np.abs(as_f64(r[name]) - ref[name])
            fp32 = adds * U * size
            assert (err <= fp32 + HALF[dtype] * (np.abs(ref[name]) + fp32) + 1e-40).all(), name


SHAPES = [(1, 1), (3, 7), (5, 64), (17, 72), (33, 256), (9, 264), (700, 520), (50, 1000),
          (40, 1001), (1300, 1024), (7, 2048), (300, 4096), (48, 4104), (5, 8192), (6, 12288),
          (3, 16384), (2, 16389), (2, 32768), (11, 32767), (100, 129), (70, 513), (2000, 61)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_norm_and_gradients(n, d, dtype):
    c = _data(n, d, dtype)
    t = {k: v.cuda() for k, v in c.items()}
    for residual, offset, eps in ((True, 0.0, 1e-6), (False, 1.0, 1e-2)):
        p = kd.NormProblem(n_tokens=n, d_model=d, dtype=dtype, eps=eps, weight_offset=offset)
        kw = dict(eps=eps, weight_offset=offset)
        r = kd.rms_norm(p, t["x"], t["weight"], residual=t["residual"] if residual else None)
        _check_fwd(r, c, dtype, residual, **kw)
        s = r["sum"] if residual else t["x"]
        g = kd.rms_norm_backward(p, s, t["weight"], t["d_h"],
                                 d_sum=t["d_sum"] if residual else None)
        _check_bwd(g, s, c, dtype, residual, n, **kw)
        for want in (("x",), ("weight",)):
            one = kd.rms_norm_backward(p, s, t["weight"], t["d_h"], want=want,
                                       d_sum=t["d_sum"] if residual else None)
            name = "d_" + want[0]
            assert set(one) == {name} and torch.equal(one[name], g[name])
    assert all(torch.equal(t[k].cpu(), c[k]) for k in c)


def test_gradient_of_differences_on_the_device():
    """fp32, a step of 2^-7 along one direction: the loss differs by the step times
    the gradient's share, up to the third derivative (step^2) and rounding."""
    n, d, step = 4, 96, 2.0 ** -7
    c = _data(n, d, "fp32", seed=5)
    c["x"] = c["x"].clamp(-3, 3)
    t = {k: v.cuda() for k, v in c.items()}
    p = kd.NormProblem(n_tokens=n, d_model=d, dtype="fp32", eps=1e-3)
    way = torch.randn(n, d, generator=torch.Generator().manual_seed(6)).cuda()
    up = torch.randn(n, d, generator=torch.Generator().manual_seed(7)).cuda()
    g = kd.rms_norm_backward(p, t["x"], t["weight"], up)

    def loss(x):
        return (kd.rms_norm(p, x, t["weight"])["h"].double() * up.double()).sum().item()

    num = (loss(t["x"] + step * way) - loss(t["x"] - step * way)) / (2 * step)
    want = (g["d_x"].double() * way.double()).sum().item()
    # rounding: 2 n d terms of size 1 off by 2^-21 each, over 2 step; third derivative
    # of a norm of unit rows along a unit-variance direction: below 50 a row
    assert abs(num - want) <= n * d * 2.0 ** -21 / step + 50 * n * step ** 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 1000, 4096])
def test_in_place(d, dtype):
    n = 37
    c = _data(n, d, dtype, seed=1)
    p = kd.NormProblem(n_tokens=n, d_model=d, dtype=dtype)
    t = {k: v.cuda() for k, v in c.items()}
    ref = kd.rms_norm(p, t["x"], t["weight"], residual=t["residual"])
    x, res = t["x"].clone(), t["residual"].clone()
    r = kd.rms_norm(p, x, t["weight"], residual=res, out={"h": x, "sum": res})
    assert r["h"] is x and torch.equal(x, ref["h"]) and torch.equal(res, ref["sum"])
    g = kd.rms_norm_backward(p, ref["sum"], t["weight"], t["d_h"], d_sum=t["d_sum"])
    for over in ("sum", "d_h", "d_sum"):
        b = {"sum": ref["sum"].clone(), "d_h": t["d_h"].clone(), "d_sum": t["d_sum"].clone()}
        o = kd.rms_norm_backward(p, b["sum"], t["weight"], b["d_h"], d_sum=b["d_sum"],
                                 out={"d_x": b[over], "d_weight": torch.empty_like(t["weight"])})
        assert torch.equal(b[over], g["d_x"]) and torch.equal(o["d_weight"], g["d_weight"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [512, 517])
@pytest.mark.parametrize("shifts", [(1, 2, 3, 4, 5, 3), (3, 3, 3, 3, 3, 3), (0, 0, 0, 0, 1, 0)])
def test_views_at_odd_elements(shifts, d, dtype):
    """Contiguous views whose first element is not at 16 bytes: all alike, or not."""
    n = 21
    c = _data(n, d, dtype, seed=2)

    def view(shift, like, value=None):
        store = torch.full((like.numel() + 16,), 3.0, dtype=like.dtype, device="cuda")
        v = store[shift:shift + like.numel()].view(like.shape)
        if value is not None:
            v.copy_(value)
        return v, store

    t = {k: view(s, v, v)[0] for s, (k, v) in zip(shifts, c.items())}
    p = kd.NormProblem(n_tokens=n, d_model=d, dtype=dtype)
    stores = [view(shifts[5], c["x"]) for _ in range(3)]
    out = {"h": stores[0][0], "sum": stores[1][0]}
    r = kd.rms_norm(p, t["x"], t["weight"], residual=t["residual"], out=out)
    _check_fwd(r, c, dtype, True)
    g = kd.rms_norm_backward(p, r["sum"], t["weight"], t["d_h"], d_sum=t["d_sum"], out={
        "d_x": stores[2][0], "d_weight": torch.empty_like(t["weight"])})
    _check_bwd(g, r["sum"], c, dtype, True, n)
    for _, store in stores:  # nothing beside the rows
        assert (store[:shifts[5]] == 3.0).all() and (store[shifts[5] + n * d:] == 3.0).all()


def test_special_rows():
    """A row of zeros is zero (gradient r g); a NaN or an infinity stays in its row."""
    n, d = 5, 520
    c = _data(n, d, "bf16", seed=3)
    c["x"][1] = 0
    c["x"][2, 3] = float("nan")
    c["x"][3, 500] = float("inf")
    t = {k: v.cuda() for k, v in c.items()}
    p = kd.NormProblem(n_tokens=n, d_model=d, eps=1e-2)
    h = kd.rms_norm(p, t["x"], t["weight"])["h"]
    assert (h[1] == 0).all() and torch.isnan(h[2]).all() and torch.isnan(h[3, 500])
    d_x = kd.rms_norm_backward(p, t["x"], t["weight"], t["d_h"], want=("x",))["d_x"]
    want = 10.0 * as_f64(c["d_h"][1]) * as_f64(c["weight"])
    assert (np.abs(as_f64(d_x[1]) - want) <= (2.0 ** -8 + 4 * E * U) * np.abs(want)).all()
    for i in (0, 4):
        assert torch.isfinite(h[i]).all() and torch.isfinite(d_x[i]).all()


def test_rows_beyond_32_bit_offsets():
    """The last rows begin past 2^31 elements."""
    n, d = 530000, 4096
    free, _ = torch.cuda.mem_get_info()
    if free < 24e9:
        pytest.skip("needs 24 GB")
    c = _data(64, d, "bf16", seed=8)
    x, d_h = (torch.zeros(n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-64:], d_h[-64:] = c["x"].cuda(), c["d_h"].cuda()
    w = c["weight"].cuda()
    p = kd.NormProblem(n_tokens=n, d_model=d)
    r = kd.rms_norm(p, x, w)
    _check_fwd({"h": r["h"][-64:]}, c, "bf16", False)
    assert int(torch.count_nonzero(r["h"][:-64])) == 0
    g = kd.rms_norm_backward(p, x, w, d_h)
    _check_bwd({"d_x": g["d_x"][-64:], "d_weight": g["d_weight"]}, c["x"], c, "bf16", False, 64)
    assert int(torch.count_nonzero(g["d_x"][:-64])) == 0


def test_no_rows():
    p = kd.NormProblem(n_tokens=0, d_model=64)
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64).bfloat16().cuda()
    assert kd.rms_norm(p, x, w)["h"].shape == (0, 64)
    g = kd.rms_norm_backward(p, x, w, x)
    assert g["d_x"].shape == (0, 64) and (g["d_weight"] == 0).all()


def test_repeats_exactly_and_in_a_graph_on_another_stream():
    n, d = 777, 1536
    t = {k: v.cuda() for k, v in _data(n, d, "bf16", seed=4).items()}
    p = kd.NormProblem(n_tokens=n, d_model=d)
    ref = kd.rms_norm(p, t["x"], t["weight"], residual=t["residual"])
    gref = kd.rms_norm_backward(p, ref["sum"], t["weight"], t["d_h"])
    ws = kd.Workspace()
    out = {k: torch.zeros_like(v) for k, v in ref.items()}
    gout = {k: torch.zeros_like(v) for k, v in gref.items()}

    def both():
        kd.rms_norm(p, t["x"], t["weight"], residual=t["residual"], out=out)
        kd.rms_norm_backward(p, out["sum"], t["weight"], t["d_h"], workspace=ws, out=gout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for o in (*out.values(), *gout.values()):
        o.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], ref[k]) for k in ref)
    assert all(torch.equal(gout[k], gref[k]) for k in gref)
