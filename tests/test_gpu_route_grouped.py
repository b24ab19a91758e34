"""moe_route_grouped against the definition in 64 bits: equal ids, weights to a few fp32 ulp."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def scores(x, score):
    if score == "sigmoid":
        return np.where(x >= 0, 1.0, np.exp(-np.abs(x))) / (1.0 + np.exp(-np.abs(x)))
    top = x.max(1, keepdims=True)
    p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    z = p.sum(1, keepdims=True)
    return p / np.where(z > 0, z, 1.0)


def definition(logits, K, bias, score, G, chosen, top, renorm=True, scale=1.0):
    """ids and weights of fp32 logits [T, E], by sorting in 64 bits."""
    x = logits.astype(np.float64)
    T, E = x.shape
    s = scores(x, score)
    c = x.copy() if bias is None else s + bias.astype(np.float64)
    worth = s if bias is None and top == 2 else c
    if chosen < G:
        value = np.sort(worth.reshape(T, G, E // G), axis=2)[:, :, -top:].sum(2)
        order = np.argsort(-value, axis=1, kind="stable")
        out = np.ones((T, G), dtype=bool)
        np.put_along_axis(out, order[:, :chosen], False, axis=1)
        gone = np.repeat(out, E // G, axis=1)
    else:
        gone = np.zeros((T, E), dtype=bool)
    # experts that are gone come last, whatever their c
    ids = np.stack([np.lexsort((np.arange(E), -c[t], gone[t]))[:K] for t in range(T)])
    if renorm and score == "sigmoid":  # in logarithms: the scores themselves may underflow
        lt = np.take_along_axis(x, ids, 1)
        ls = np.minimum(lt, 0) - np.log1p(np.exp(-np.abs(lt)))
        w = np.exp(ls - ls.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
    else:
        w = np.take_along_axis(s, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
    return ids, w * scale


def check(m, logits, K, bias=None, score="sigmoid", G=1, chosen=1, top=2, **kw):
    dev = torch.from_numpy(logits).cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = m.moe_route_grouped(dev, K, b, score, G, chosen, top, with_shared=False, **kw)
    kw = {"renorm" if k == "renormalize" else k: v for k, v in kw.items()}
    want, ww = definition(logits, K, bias, score, G, chosen, top, **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    # an exponential's argument rounds to 2^-24 of itself, twice where it is a difference (at most D
    # here, numerator and sum alike); exponentials to 2^-23, sums and quotients (16 of them) to 2^-24
    D = min(2.0 * float(np.abs(logits[np.isfinite(logits)]).max()), 104.0)
    tol = (2 * D + 24) * 2.0 ** -24 * np.abs(ww) + 2.0 ** -140
    assert (np.abs(w.double().cpu().numpy() - ww) <= tol).all()


CASES = [  # T, E, K, groups, chosen, top
    (1, 256, 8, 8, 4, 2), (5, 1, 1, 1, 1, 1), (7, 60, 5, 6, 3, 1), (33, 1024, 32, 1, 1, 1), (19, 1023, 31, 3, 2, 2),
    (64, 512, 10, 1, 1, 2), (40, 992, 12, 31, 17, 2), (40, 1020, 8, 17, 5, 1), (9, 32, 4, 32, 6, 1), (300, 160, 6, 8, 3, 1),
    (17, 64, 12, 16, 6, 2), (3, 12, 12, 3, 3, 2), (11, 40, 32, 5, 4, 2), (1000, 128, 8, 4, 2, 2), (10, 64, 1, 2, 1, 2),
    (20, 1024, 32, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,K,G,chosen,top", CASES)
def test_against_the_definition(m, score, biased, T, E, K, G, chosen, top):
    rng = np.random.default_rng(T * E + K)
    logits = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (rng.standard_normal(E) * (0.2 if score == "sigmoid" else 0.5 / E)).astype(np.float32) if biased else None
    check(m, logits, K, bias, score, G, chosen, top)
    check(m, logits, K, bias, score, G, chosen, top, renormalize=False, scale=2.5)


MANY = [  # long batches, several tokens a warp where K, E and the groups allow it
    (4096, 256, 8, 8, 4, 2), (4099, 512, 10, 1, 1, 1), (5001, 64, 6, 1, 1, 1), (4097, 128, 16, 16, 9, 2), (4200, 96, 4, 3, 2, 1),
    (6002, 16, 8, 2, 1, 2), (4111, 512, 16, 8, 2, 2), (4098, 256, 8, 1, 1, 2), (4100, 60, 3, 5, 2, 1), (4101, 128, 8, 2, 1, 1),
    (4103, 1024, 8, 1, 1, 1), (4105, 64, 12, 32, 20, 1), (4104, 36, 8, 1, 1, 1), (4106, 32, 1, 8, 1, 2), (4107, 500, 16, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,K,G,chosen,top", MANY)
def test_long_batches(m, score, biased, T, E, K, G, chosen, top):
    test_against_the_definition(m, score, biased, T, E, K, G, chosen, top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,chosen,top", [(1, 1, 1), (8, 4, 2), (8, 3, 1)])
@pytest.mark.parametrize("T", [200, 4200])
def test_equal_and_nearly_equal_values(m, score, G, chosen, top, T):
    """Values that round to one another in fp32, and exact ties."""
    rng = np.random.default_rng(3)
    E, K = 64, 8
    for bias in (None, np.zeros(E, np.float32), np.full(E, 0.37, np.float32)):
        check(m, np.zeros((T, E), np.float32), K, bias, score, G, chosen, top)
        # few different logits: ties everywhere
        check(m, rng.integers(-2, 3, (T, E)).astype(np.float32), K, bias, score, G, chosen, top)
        # neighbours: steps of an ulp of the logit
        near = (np.float32(1.5) + rng.integers(0, 64, (T, E)).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
        check(m, near, K, bias, score, G, chosen, top)
    # biases that nearly undo the logits' differences
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:] = logits[:1]
    s = scores(logits.astype(np.float64), score)[0]
    for ulps in (0.0, 1e-9, 1e-8, 1e-7):
        bias = (0.9 - s + ulps * rng.standard_normal(E)).astype(np.float32)
        check(m, logits, K, bias, score, G, chosen, top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [50, 4100])
def test_masked_experts_and_wide_ranges(m, score, T):
    rng = np.random.default_rng(4)
    E, K = 128, 6
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    logits = (20.0 * rng.standard_normal((T, E))).astype(np.float32)
    logits[:, ::3] = -np.inf
    logits[:, 1::7] = -3.4e38
    for b, G, chosen, top in ((None, 1, 1, 1), (None, 8, 4, 1), (bias, 1, 1, 1), (bias, 8, 5, 2)):
        check(m, logits, K, b, score, G, chosen, top)
    # a token with no expert at all: lowest ids, weights 0
    logits[3] = -np.inf
    ids, w = m.moe_route_grouped(torch.from_numpy(logits).cuda(), K, None, score, with_shared=False)
    assert ids[3].tolist() == list(range(K)) and not w[3].any() and torch.isfinite(w).all()
    # scores that underflow fp32 keep their proportions
    low = np.full((1, 16), -300.0, np.float32)
    low[0, 5], low[0, 9] = -200.0, -201.0
    check(m, low, 2, None, score)


@pytest.mark.parametrize("T", [40, 4100])
def test_what_is_not_a_number(m, T):
    """NaN counts as -inf; ids stay distinct and in range whatever the values are."""
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((T, 64)).astype(np.float32)
    plain = logits.copy()
    logits[rng.random((T, 64)) < 0.3] = np.nan
    plain[np.isnan(logits)] = -np.inf
    for score in ("sigmoid", "softmax"):
        a = m.moe_route_grouped(torch.from_numpy(logits).cuda(), 8, None, score, 8, 4, 2)
        b = m.moe_route_grouped(torch.from_numpy(plain).cuda(), 8, None, score, 8, 4, 2)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        wild = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, 3e38, -3e38], np.float32), (160 + T, 64))
        bias = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, 1.0], np.float32), 64)
        for bb in (None, bias):
            for G, chosen, top in ((1, 1, 1), (8, 4, 2), (16, 9, 1)):
                ids, _ = m.moe_route_grouped(torch.from_numpy(wild).cuda(), 8, None if bb is None else torch.from_numpy(bb).cuda(),
                                             score, G, chosen, top, with_shared=False)
                s = ids.sort(1)[0]
                assert (s[:, 0] >= 0).all() and (s[:, -1] < 64).all() and (s[:, 1:] > s[:, :-1]).all()


@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("T", [70, 4200])
def test_bf16_rows_and_slices(m, pad, T):
    rng = np.random.default_rng(6)
    wide = torch.from_numpy(rng.standard_normal((T, 96 + pad)).astype(np.float32)).cuda()
    bias = torch.from_numpy((0.1 * rng.standard_normal(96)).astype(np.float32)).cuda()
    for rows in (wide[:, pad:], wide.bfloat16()[:, pad:], wide[:1].expand(T, -1)[:, :96], wide.bfloat16()[3:4, pad // 2:]):
        rows = rows[:, :96]
        ids, w = m.moe_route_grouped(rows, 6, bias, "sigmoid", 8, 4, 2, with_shared=False)
        want, ww = definition(rows.float().cpu().numpy(), 6, bias.cpu().numpy(), "sigmoid", 8, 4, 2)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert np.abs(w.double().cpu().numpy() - ww).max() <= (2 * 12 + 24) * 2.0 ** -24


def test_shared_slot_and_no_tokens(m):
    logits = torch.randn((5, 16), device="cuda")
    sw = torch.rand(5, device="cuda")
    ids, w = m.moe_route_grouped(logits, 3, shared_w=sw, scale=2.0)
    a, b = m.moe_route_grouped(logits, 3, with_shared=False, scale=2.0)
    assert torch.equal(ids[:, :3], a) and torch.equal(w[:, :3], b) and (ids[:, 3] == 16).all() and torch.equal(w[:, 3], sw)
    assert (m.moe_route_grouped(logits, 3)[1][:, 3] == 1).all()
    ids, w = m.moe_route_grouped(logits[:0], 3)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_agrees_with_moe_route(m):
    logits = torch.randn((64, 512), device="cuda") * 2
    a, b = m.moe_route(logits, 10), m.moe_route_grouped(logits, 10, None, "softmax")
    assert torch.equal(a[0], b[0])
    assert torch.allclose(a[1], b[1], rtol=32 * 2.0 ** -24, atol=0)


def test_rows_past_32_bits(m):
    """Logits of more than 2^31 elements: the last rows are their own."""
    T, E = (1 << 31) // 1024 + 77, 1024
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((80, E), device="cuda").bfloat16()
    logits[-80:] = tail
    ids, w = m.moe_route_grouped(logits, 4, None, "sigmoid", with_shared=False)
    a, b = m.moe_route_grouped(tail, 4, None, "sigmoid", with_shared=False)
    assert torch.equal(ids[-80:], a) and torch.equal(w[-80:], b)
    assert (ids[:-80] == torch.arange(4, device="cuda", dtype=torch.int32)).all()


def test_graph_replay(m):
    logits, bias = torch.randn((37, 256), device="cuda"), torch.randn(256, device="cuda") * 0.1
    ids = torch.empty((37, 8), dtype=torch.int32, device="cuda")
    w = torch.empty((37, 8), device="cuda")
    run = lambda: m.moe_route_grouped(logits, 8, bias, "sigmoid", 8, 4, 2, with_shared=False, topk_ids=ids, topk_w=w)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        logits.normal_()
        g.replay()
        got = ids.clone(), w.clone()
        run()
        assert torch.equal(got[0], ids) and torch.equal(got[1], w)
