"""The embedding lookup and its gradient on the GPU against the fp64 oracle.

u = 2^-24.  A looked-up value: one product (u) and half a step of the type.  A
gradient row: each of its `count` additions in fp32 is off by at most u of the
sum of absolute values, the scale and the value added to by 2 u, and half a
step of the type."""
import numpy as np
import pytest
import torch

from lm_head_cross_vocab_gb300 import kd
from oracle import rows_oracle as R
from oracle.kd_oracle import as_f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kd.load_library()
    assert kd.kd_device_supported(0), "tests need an sm_103 GPU"


def _tokens(kind, n, v, g):
    if kind == "same":
        return torch.full((n,), v - 1)
    if kind == "text":
        return (2.7 * (v / 2.7 + 1.0) ** torch.rand(n, generator=g, dtype=torch.float64)
                - 2.7).long().clamp(0, v - 1)
    if kind == "distinct":
        return torch.randperm(max(n, v), generator=g)[:n] % v
    t = torch.randint(0, v, (n,), generator=g)
    t[torch.rand(n, generator=g) < 0.3] = -100
    return t


SHAPES = [(1, 1, 1), (1, 500, 64), (7, 3, 5), (64, 1000, 520), (63, 90, 1001), (257, 5003, 24),
          (1000, 32003, 128), (2048, 700, 1024), (4100, 151936, 72), (5000, 11, 40),
          (40, 130, 2056)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1.0, 45.25])
@pytest.mark.parametrize("n,v,d", SHAPES)
def test_lookup(n, v, d, scale, dtype):
    g = torch.Generator().manual_seed(n)
    w = torch.randn(v, d, generator=g).to(DT[dtype])
    for kind in ("text", "ignored"):
        tokens = _tokens(kind, n, v, g)
        p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype=dtype, scale=scale)
        out = {"h": torch.full((n, d), 9.0, dtype=DT[dtype], device="cuda")}
        h = kd.embed_tokens(p, w.cuda(), tokens.cuda(), out=out)["h"]
        ref = R.embed(w, tokens.tolist(), scale)
        if scale == 1.0:
            assert (as_f64(h) == ref).all()
        assert (np.abs(as_f64(h) - ref) <= (HALF[dtype] + 2 * U) * np.abs(ref)).all()


def _check_grad(d_w, before, d_h, tokens, v, scale, dtype, accumulate):
    ref, size, count = R.embed_grad(d_h, tokens.tolist(), v, scale)
    got, touched = as_f64(d_w), count > 0
    if accumulate:
        assert torch.equal(d_w.cpu()[~torch.from_numpy(touched)], before[~torch.from_numpy(touched)])
        ref, size = ref + as_f64(before), size + np.abs(as_f64(before))
    else:
        assert (got[~touched] == 0).all()
    fp32 = (count[:, None] + 2) * U * size
    err = np.abs(got - ref)
    assert (err <= fp32 + HALF[dtype] * (np.abs(ref) + fp32))[touched].all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["text", "same", "distinct", "ignored"])
@pytest.mark.parametrize("n,v,d", SHAPES)
def test_gradient(n, v, d, kind, accumulate, dtype):
    g = torch.Generator().manual_seed(n)
    tokens = _tokens(kind, n, v, g)
    d_h = torch.randn(n, d, generator=g).to(DT[dtype])
    dev = d_h.cuda()
    dev[(tokens == -100).cuda()] = float("nan")  # rows that take no part may hold anything
    before = torch.randn(v, d, generator=g).to(DT[dtype])
    buf = before.cuda() if accumulate else torch.full((v, d), float("nan"), dtype=DT[dtype],
                                                      device="cuda")
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype=dtype, scale=1.5)
    r = kd.embed_tokens_backward(p, tokens.cuda(), dev, accumulate=accumulate, out={"d_w": buf})
    _check_grad(r["d_w"], before, d_h, tokens, v, 1.5, dtype, accumulate)
    if not accumulate:
        again = kd.embed_tokens_backward(p, tokens.cuda(), dev)
        assert torch.equal(again["d_w"], buf)


@pytest.mark.parametrize("count", [31, 32, 33, 63, 64, 65, 95, 96, 127, 128, 129, 1000])
def test_counts_next_to_a_piece(count):
    """An id between others, at every phase of the pieces its rows are cut into."""
    v, d = 9, 16
    g = torch.Generator().manual_seed(count)
    for before in (0, 1, 17, 31, 32):
        tokens = torch.cat([torch.full((before,), 2), torch.full((count,), 3), torch.full((70,), 4)])
        tokens = tokens[torch.randperm(len(tokens), generator=g)]
        d_h = torch.randn(len(tokens), d, generator=g)
        p = kd.EmbedProblem(n_tokens=len(tokens), vocab=v, d_model=d, dtype="fp32")
        r = kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda())
        _check_grad(r["d_w"], None, d_h, tokens, v, 1.0, "fp32", False)


def test_many_places_of_many_frequent_ids():
    """Several times the places one joining block looks through."""
    n, v, d = 40000, 150, 8
    g = torch.Generator().manual_seed(8)
    tokens = torch.randint(0, v, (n,), generator=g)
    tokens[:9000] = 77
    d_h = torch.randn(n, d, generator=g)
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32")
    r = kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda())
    _check_grad(r["d_w"], None, d_h, tokens, v, 1.0, "fp32", False)


@pytest.mark.parametrize("share", [0.02, 0.1, 0.4, 1.0])
@pytest.mark.parametrize("n,v", [(700, 900), (9000, 300), (20000, 151936), (50000, 40000)])
def test_a_padding_id_that_is_not_ignored(n, v, share):
    """One id is a large part of all tokens: more than a warp, or a block, keeps."""
    d = 8
    g = torch.Generator().manual_seed(n)
    tokens = _tokens("text", n, v, g)
    tokens[torch.rand(n, generator=g) < share] = 5
    tokens[::97] = -100
    d_h = torch.randn(n, d, generator=g)
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32")
    r = kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda())
    _check_grad(r["d_w"], None, d_h, tokens, v, 1.0, "fp32", False)


def test_bad_tokens_are_told_and_take_no_part():
    n, v, d = 50, 20, 24
    g = torch.Generator().manual_seed(9)
    tokens = torch.randint(0, v, (n,), generator=g)
    tokens[3], tokens[40], tokens[41] = v, -5, 2 ** 40
    w, d_h = torch.randn(v, d, generator=g), torch.randn(n, d, generator=g)
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32")
    with pytest.raises(kd.KDError) as e:
        kd.embed_tokens(p, w.cuda(), tokens.cuda())
    assert e.value.status == kd.KD_ERR_BAD_LABEL
    with pytest.raises(kd.KDError) as e:
        kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda())
    assert e.value.status == kd.KD_ERR_BAD_LABEL
    r = kd.embed_tokens(p, w.cuda(), tokens.cuda(), check=False)
    assert (as_f64(r["h"]) == R.embed(w, tokens.tolist())).all()
    r = kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda(), check=False)
    assert int(r["dev_status"]) == kd.KD_DEV_BAD_LABEL
    _check_grad(r["d_w"], None, d_h, tokens, v, 1.0, "fp32", False)


@pytest.mark.parametrize("d", [24, 1000, 1001])
@pytest.mark.parametrize("ignore", [0, 7, 41, 2 ** 40])
def test_an_ignored_id_of_the_vocabulary(ignore, d):
    """Padding by an id that the table has, or by one far outside it."""
    n, v = 300, 42
    g = torch.Generator().manual_seed(13)
    tokens = torch.randint(0, v, (n,), generator=g)
    tokens[::5] = ignore
    w, d_h = torch.randn(v, d, generator=g), torch.randn(n, d, generator=g)
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d, dtype="fp32", ignore_index=ignore)
    h = kd.embed_tokens(p, w.cuda(), tokens.cuda())["h"]
    assert (as_f64(h) == R.embed(w, tokens.tolist(), ignore_index=ignore)).all()
    assert (h[::5] == 0).all()
    r = kd.embed_tokens_backward(p, tokens.cuda(), d_h.cuda())
    plain = torch.where(tokens == ignore, -100, tokens)
    _check_grad(r["d_w"], None, d_h, plain, v, 1.0, "fp32", False)
    if ignore < v:
        assert (r["d_w"][ignore] == 0).all()


def test_no_tokens():
    p = kd.EmbedProblem(n_tokens=0, vocab=5, d_model=8)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    h = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(5, 8, dtype=torch.bfloat16, device="cuda")
    assert kd.embed_tokens(p, w, t)["h"].shape == (0, 8)
    assert (kd.embed_tokens_backward(p, t, h)["d_w"] == 0).all()
    kept = w.clone()
    kd.embed_tokens_backward(p, t, h, accumulate=True, out={"d_w": w})
    assert torch.equal(w, kept)


def test_views_at_odd_elements():
    n, v, d = 90, 40, 64
    g = torch.Generator().manual_seed(10)
    tokens = _tokens("text", n, v, g)
    w, d_h = torch.randn(v, d, generator=g).bfloat16(), torch.randn(n, d, generator=g).bfloat16()

    def odd(x, shift):
        store = torch.full((x.numel() + 8,), 3.0, dtype=x.dtype, device="cuda")
        view = store[shift:shift + x.numel()].view(x.shape)
        view.copy_(x)
        return store, view

    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d)
    hs, h = odd(torch.zeros(n, d).bfloat16(), 5)
    kd.embed_tokens(p, odd(w, 1)[1], tokens.cuda(), out={"h": h})
    assert (as_f64(h) == R.embed(w, tokens.tolist())).all()
    ws, d_w = odd(w, 3)
    kd.embed_tokens_backward(p, tokens.cuda(), odd(d_h, 2)[1], accumulate=True, out={"d_w": d_w})
    _check_grad(d_w, w, d_h, tokens, v, 1.0, "bf16", True)
    for s, m, i in ((hs, n * d, 5), (ws, v * d, 3)):
        assert (s[:i] == 3.0).all() and (s[i + m:] == 3.0).all()


def test_a_table_beyond_32_bit_offsets():
    """Rows whose first element lies past 2^31."""
    v, d, n = 530000, 4096, 200
    free, _ = torch.cuda.mem_get_info()
    if free < 12e9:
        pytest.skip("needs 12 GB")
    w = torch.zeros(v, d, dtype=torch.bfloat16, device="cuda")
    tokens = torch.arange(v - n, v)
    rows = torch.randn(n, d, generator=torch.Generator().manual_seed(11)).bfloat16()
    w[v - n:] = rows.cuda()
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d)
    assert torch.equal(kd.embed_tokens(p, w, tokens.cuda())["h"].cpu(), rows)
    tokens[1::2] = v - 1  # frequent: more than one piece
    kd.embed_tokens_backward(p, tokens.cuda(), rows.cuda(), out={"d_w": w}, accumulate=True)
    ref, size, count = R.embed_grad(rows, (tokens - (v - n)).tolist(), n)
    ref, size = ref + as_f64(rows), size + np.abs(as_f64(rows))
    fp32 = (count[:, None] + 2) * U * size
    assert (np.abs(as_f64(w[v - n:]) - ref) <= fp32 + HALF["bf16"] * (np.abs(ref) + fp32)).all()
    assert int(torch.count_nonzero(w[:v - n])) == 0


def test_repeats_exactly_and_in_graphs_that_share_a_workspace():
    n, v, d = 3000, 4000, 264
    g = torch.Generator().manual_seed(12)
    ws = kd.Workspace()
    p = kd.EmbedProblem(n_tokens=n, vocab=v, d_model=d)
    jobs = []
    for _ in range(2):
        tokens = _tokens("text", n, v, g).cuda()
        d_h = torch.randn(n, d, generator=g).bfloat16().cuda()
        ref = kd.embed_tokens_backward(p, tokens, d_h)["d_w"]
        out = {"d_w": torch.zeros_like(ref)}
        kd.embed_tokens_backward(p, tokens, d_h, workspace=ws, out=out, check=False)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kd.embed_tokens_backward(p, tokens, d_h, workspace=ws, out=out, check=False)
        jobs.append((graph, out["d_w"], ref, tokens, d_h))  # (a graph reads its inputs' memory)
    for job in jobs:
        job[1].zero_()
    for _ in range(3):
        for job in jobs:
            job[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for _, o, ref, _, _ in jobs)
