"""The fp64 oracle of the row operators, pinned by closed forms, sampling
frequencies and differences."""
import numpy as np
import pytest

from oracle import rows_oracle as R


def test_verify_emits_the_targets_distribution():
    """Whatever the drafter's distribution is, the first emitted token's is the
    target's: frequencies over 20000 sequences within five standard deviations."""
    rng = np.random.default_rng(1)
    b, v = 20000, 6
    zt, zd = rng.normal(size=(1, 1, v)) * 1.5, rng.normal(size=(1, 1, v)) * 1.5
    p, q = np.exp(zt[0, 0]) / np.exp(zt).sum(), np.exp(zd[0, 0]) / np.exp(zd).sum()
    drafts = rng.choice(v, size=(b, 1), p=q)
    target = np.repeat(np.concatenate([zt, rng.normal(size=(1, 1, v))], 1), b, 0)
    r = R.verify(target, np.repeat(zd, b, 0), drafts, None, rng.random((b, 1)),
                 rng.exponential(size=(b, v)))
    freq = np.bincount(r["tokens"][:, 0], minlength=v) / b
    assert (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / b)).all()
    share = np.minimum(p, q).sum()  # accepted drafts
    assert abs(r["accepted"].mean() - share) <= 5 * np.sqrt(share * (1 - share) / b)


def test_verify_closed_forms():
    z = np.log(np.array([[[0.5, 0.3, 0.2], [0.2, 0.2, 0.6]]]))
    same = z[:, :1]
    noise = np.ones((1, 3))
    r = R.verify(z, same, [[1]], None, [[0.999]], noise)  # p = q: stands, then the likeliest
    assert r["tokens"].tolist() == [[1, 2]] and r["accepted"].tolist() == [1]
    assert np.allclose(r["logprob"], np.log([[0.3, 0.6]]))
    r = R.verify(z, None, [[1]], None, [[0.29]], noise)
    assert r["tokens"].tolist() == [[1, 2]]
    r = R.verify(z, None, [[0]], None, [[0.51]], noise)  # the rejected id is not drawn again
    assert r["tokens"].tolist() == [[1, -100]] and r["accepted"].tolist() == [0]
    r = R.verify(z, None, [[2]], [0], None, noise)
    assert r["tokens"].tolist() == [[0, -100]]
    r = R.verify(z, None, [[0]], None, None, None, t_target=0.0)
    assert r["tokens"].tolist() == [[0, 2]]


@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradient_is_that_of_differences(offset):
    rng = np.random.default_rng(2)
    s, w, d_h = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7))
    g = R.rms_norm_grad(s, w, d_h, eps=0.1, weight_offset=offset)

    def loss(s, w):
        return (R.rms_norm(s, w, eps=0.1, weight_offset=offset)[0] * d_h).sum()

    step = 1e-6
    for arr, grad, of in ((s, g["d_x"], 0), (w, g["d_weight"], 1)):
        num = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += step
            dn[i] -= step
            num[i] = (loss(*((up, w), (s, up))[of]) - loss(*((dn, w), (s, dn))[of])) / (2 * step)
        # central differences: step^2 of the third derivative, and 1e-16 / step
        assert np.allclose(num, grad, atol=1e-8, rtol=1e-7)


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    rng = np.random.default_rng(3)
    w, d_h = rng.normal(size=(5, 4)), rng.normal(size=(6, 4))
    tokens = [1, 3, 1, -100, 7, 0]
    h = R.embed(w, tokens, 2.0)
    d_w, size, count = R.embed_grad(d_h, tokens, 5, 2.0)
    assert np.isclose((h * d_h).sum(), (w * d_w).sum())
    assert (h[3:5] == 0).all() and count.tolist() == [1, 2, 0, 1, 0]
    assert (size >= np.abs(d_w) - 1e-12).all()
