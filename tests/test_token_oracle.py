"""Pins of oracle/token_oracle.py (CPU): closed forms, library routines, finite
differences and limits, none of which uses the oracle's own formulas."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as O


def test_two_ids_by_hand():
    # logits (ln 3, 0): p = (3/4, 1/4)
    o = O.forward(np.array([[math.log(3.0), 0.0]]), [1], topk=2)
    assert o["logprob"][0] == pytest.approx(math.log(0.25))
    assert o["entropy"][0] == pytest.approx(-0.75 * math.log(0.75) - 0.25 * math.log(0.25))
    assert o["topk_idx"].tolist() == [[0, 1]]
    # T = 2: p = sqrt(3) / (1 + sqrt(3)), ...
    o = O.forward(np.array([[math.log(3.0), 0.0]]), [0], temperature=2.0)
    assert o["logprob"][0] == pytest.approx(math.log(math.sqrt(3) / (1 + math.sqrt(3))))


def test_against_torch():
    g = torch.Generator().manual_seed(3)
    z = torch.randn(6, 50, generator=g, dtype=torch.float64) * 3
    y = torch.randint(0, 50, (6,), generator=g)
    for t in (1.0, 0.7, 3.0):
        o = O.forward(z, y, temperature=t, topk=50)
        d = torch.distributions.Categorical(logits=z / t)
        assert np.allclose(o["logprob"], d.log_prob(y).numpy(), rtol=1e-12)
        assert np.allclose(o["entropy"], d.entropy().numpy(), rtol=1e-12)
        assert (o["topk_idx"] == torch.argsort(z, dim=1, descending=True).numpy()).all()
        assert np.allclose(np.exp(o["topk_logprob"]).sum(axis=1), 1.0)


def test_uniform_rows_masks_and_ties():
    lo = float(np.finfo(np.float32).min)
    z = np.array([[lo] * 5, [-math.inf] * 5, [0.0, -math.inf, 0.0, -math.inf, -1e9],
                  [1.0, math.nan, 2.0, 0.0, 0.0]])
    o = O.forward(z, [0, 0, 2, 0], topk=5)
    assert o["logprob"][0] == pytest.approx(-math.log(5))
    assert o["entropy"][0] == pytest.approx(math.log(5))
    assert o["logprob"][1] == -math.inf and o["entropy"][1] == 0.0
    assert o["logprob"][2] == pytest.approx(-math.log(2))
    assert o["topk_idx"].tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 2, 4, 1, 3],
                                      [1, 2, 0, 3, 4]]
    assert math.isnan(o["logprob"][3]) and math.isnan(o["entropy"][3])
    o = O.forward(z, [-100, -1, 7, -100], topk=2)
    assert o["logprob"][0] == 0 and o["entropy"][0] == 0 and math.isnan(o["logprob"][2])
    assert o["topk_idx"][3].tolist() == [0, 1] and (o["topk_logprob"][3] == -math.inf).all()


@pytest.mark.parametrize("t", [1.0, 0.6])
def test_gradient_by_differences(t):
    rng = np.random.default_rng(5)
    z = rng.normal(size=(3, 7)) * 2
    z[1, 2] = -math.inf
    y, gl, gh = [4, -100, 0], rng.normal(size=3), rng.normal(size=3)
    g = O.grad_logits(z, y, gl, gh, temperature=t)

    def f(zz):
        o = O.forward(zz, y, temperature=t)
        return float(gl @ o["logprob"] + gh @ o["entropy"])

    for r in range(3):
        for c in range(7):
            if not math.isfinite(z[r, c]):
                assert g[r, c] == 0
                continue
            up, dn = z.copy(), z.copy()
            up[r, c] += 1e-5
            dn[r, c] -= 1e-5
            assert g[r, c] == pytest.approx((f(up) - f(dn)) / 2e-5, rel=1e-6, abs=1e-9)
    assert (g[1] == 0).all()
    # each row of the gradient sums to 0: adding a constant changes nothing
    assert np.allclose(g.sum(axis=1), 0.0, atol=1e-14)


def test_clip_by_hand():
    norm, out = O.clip([np.array([3.0, 0.0]), np.array([4.0])], 2.5)
    assert norm == 5.0 and out[0].tolist() == [1.5, 0.0] and out[1].tolist() == [2.0]
    norm, out = O.clip([np.array([3.0, 0.0]), np.array([4.0])], 5.0)
    assert out[1].tolist() == [4.0]
    norm, _ = O.clip([np.full(4, 1e300)], 1.0)
    assert norm == pytest.approx(2e300)
