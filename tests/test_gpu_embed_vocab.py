"""The embedding gradient over vocabularies around those where the number of sorting
blocks changes (128 blocks of up to 1628 ids, then 256 and so on), against sums in
fp64 on the device.  u = 2^-24: each of an id's `count` additions is off by at most u
of the sum of absolute values, the scale by u, the rounding by half a step."""
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _case(n, v, d, crowd):
    g = torch.Generator(device="cuda").manual_seed(n)
    tokens = torch.randint(0, v, (n,), generator=g, device="cuda")
    tokens[::3] = torch.randint(v - 140, v, (n + 2,), generator=g, device="cuda")[::3][:(n + 2) // 3]
    if crowd:  # ids of one block and of one id: most of its warps' tokens are its own
        tokens[n // 2:] = (tokens[n // 2:] // 4096 * 4096 + 5).clamp(max=v - 1)
        tokens[n // 4:n // 2] = v - 1
    tokens[7::50] = -100
    return tokens, torch.randn(n, d, generator=g, device="cuda")


@pytest.mark.parametrize("crowd", [False, True])
@pytest.mark.parametrize("n", [900, 60000])
@pytest.mark.parametrize("v", [155648, 155649, 200019, 208383, 208384, 208385, 262144, 416769])
def test_vocabularies_where_the_blocks_change(v, n, crowd):
    d = 8
    tokens, d_h = _case(n, v, d, crowd)
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32", scale=2.0)
    got = kd.embed_tokens_backward(p, tokens, d_h)["d_w"]
    live = tokens >= 0
    want = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    size, count = torch.zeros_like(want), torch.zeros(v, 1, dtype=torch.float64, device="cuda")
    want.index_add_(0, tokens[live], 2.0 * d_h[live].double())
    size.index_add_(0, tokens[live], 2.0 * d_h[live].double().abs())
    count.index_add_(0, tokens[live], torch.ones(int(live.sum()), 1, dtype=torch.float64,
                                                 device="cuda"))
    assert ((got.double() - want).abs() <= U * (count + 2) * size).all()
    # the order of an id's sum depends on the tokens alone, not on how the ids are dealt
    wide = kd.EmbedProblem(n_tokens=n, vocab=2 * v, d_model=d, dtype="fp32", scale=2.0)
    more = kd.embed_tokens_backward(wide, tokens, d_h)["d_w"]
    assert torch.equal(more[:v], got) and int(torch.count_nonzero(more[v:])) == 0
