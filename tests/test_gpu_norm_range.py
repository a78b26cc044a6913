"""The norm and its backward over rows of large and of tiny magnitude, up to the
limits that the header states, against the fp64 oracle.

Tolerances as tests/test_gpu_norm.py derives them (E = 64 elements a thread at most,
u = 2^-24): r within (E / 2 + 10) u; the sum of g s within (E + 14) u of the sum of
absolute values.  d_x = r g - (s r) (r m), m = r mean(g s): each term holds r up to
three times, so that it is off by at most 4 E u of its absolute value.  All factors
are normal fp32 numbers within the stated range: nothing is lost below it."""
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


def _near(got, want, fp32, dtype):
    err = np.abs(as_f64(got) - want)
    return np.isfinite(err).all() and (err <= fp32 + HALF[dtype] * (np.abs(want) + fp32)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 100, 520, 1001, 4096, 16384, 32767])
@pytest.mark.parametrize("power", [-55, -44, -40, 40, 48, 51, 55])
def test_rows_of_large_and_tiny_magnitude(power, d, dtype):
    """d_sum is of r g's size, so that it hides nothing."""
    n = 5
    g = torch.Generator().manual_seed(d)
    mk = lambda scale: (torch.randn(n, d, generator=g) * scale).to(DT[dtype])  # noqa: E731
    x, res, d_h = mk(2.0 ** power), mk(2.0 ** power), mk(0.5)
    d_sum = mk(2.0 ** -power)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype])
    # a gradient along the rows: the projection takes half of it away
    d_h = (d_h.float() + 0.5 * (x.double() * 2.0 ** -power).float()).to(DT[dtype])
    for eps, up in ((0.0, None), (1e-6, d_sum)):
        p = kd.NormProblem(n_tokens=n, d_model=d, dtype=dtype, eps=eps)
        r = kd.rms_norm(p, x.cuda(), w.cuda(), residual=res.cuda())
        h, s = R.rms_norm(x, w, res, eps=eps)
        lost = U * np.abs(s)  # x + residual in fp32
        scale = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
        assert _near(r["sum"], s, lost, dtype)
        assert _near(r["h"], h, (E / 2 + 14) * U * np.abs(h) + 2 * lost * scale * np.abs(as_f64(w)),
                     dtype)
        b = kd.rms_norm_backward(p, r["sum"], w.cuda(), d_h.cuda(),
                                 d_sum=None if up is None else up.cuda())
        ref = R.rms_norm_grad(r["sum"], w, d_h, up, eps=eps)
        assert _near(b["d_x"], ref["d_x"], 4 * E * U * ref["x_size"], dtype)
        assert _near(b["d_weight"], ref["d_weight"], (n + E) * U * ref["w_size"], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 32767, 32768])
def test_rows_just_inside_the_stated_limits(d, dtype):
    """Sums of squares of 2^127 at most, and of a mean square of 2^-126 at least."""
    up = int((127 - np.log2(d)) // 2)
    n = 4
    g = torch.Generator().manual_seed(d + 1)
    sign = torch.where(torch.rand(n, d, generator=g) < 0.5, -1.0, 1.0)
    size = torch.tensor([2.0 ** up, 2.0 ** (up - 1), 2.0 ** -62, 2.0 ** -63])[:, None]
    x = (sign * size).to(DT[dtype])
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype])
    d_h = (0.5 * torch.randn(n, d, generator=g) + 0.5 * sign).to(DT[dtype])
    p = kd.NormProblem(n_tokens=n, d_model=d, dtype=dtype, eps=0.0)
    h, _ = R.rms_norm(x, w, eps=0.0)
    assert _near(kd.rms_norm(p, x.cuda(), w.cuda())["h"], h, (E / 2 + 14) * U * np.abs(h), dtype)
    b = kd.rms_norm_backward(p, x.cuda(), w.cuda(), d_h.cuda())
    ref = R.rms_norm_grad(x, w, d_h, eps=0.0)
    assert _near(b["d_x"], ref["d_x"], 4 * E * U * ref["x_size"], dtype)
    assert _near(b["d_weight"], ref["d_weight"], (n + E) * U * ref["w_size"], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_beyond_the_stated_limits(dtype):
    """As stated: a sum of squares beyond fp32 makes a row of zeros, and a row of zeros
    has no norm without eps; other rows are not touched by either."""
    x = torch.ones(3, 32768, dtype=DT[dtype])
    x[0], x[2] = 2.0 ** 57, 0.0
    w = torch.ones(32768, dtype=DT[dtype]).cuda()
    h = kd.rms_norm(kd.NormProblem(n_tokens=3, d_model=32768, dtype=dtype, eps=0.0), x.cuda(),
                    w)["h"]
    assert (h[0] == 0).all() and (h[1] == 1).all() and torch.isnan(h[2]).all()
    h = kd.rms_norm(kd.NormProblem(n_tokens=3, d_model=32768, dtype=dtype, eps=1e-30), x.cuda(),
                    w)["h"]
    assert (h[0] == 0).all() and (h[1] == 1).all() and (h[2] == 0).all()
