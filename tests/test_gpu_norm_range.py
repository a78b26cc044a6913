"""The norm and its backward over rows of large and of tiny magnitude, against the
fp64 oracle.

Tolerances as tests/test_gpu_norm.py derives them (E = 64 elements a thread at most,
u = 2^-24): r within (E / 2 + 10) u; the sum of g s within (E + 14) u of the sum of
absolute values.  d_x = r (g - (s r) m), m = r mean(g s): each term holds r up to
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
