"""moe_layer_few against its definition in 64 bits.

Against exact sums the result differs by its rounding to bf16 (at most 2^-8 of
the value next to a power of two, 1.7e-3 in the mean square) and by h's
rounding to 11 bits (2^-11 per term, far less in a sum of many): per element
2^-8 * (|ref| + rms of the token's row), and the parity bar's relative L2 error of 2e-3
(2^-8 where there are too few values for a mean).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def make(T, H, I, E, K, shared=True, gate=False, seed=0, lo=119, hi=124):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Et = E + int(shared)

    def mx(n, k):
        return (torch.randint(0, 256, (Et, n, k // 2), dtype=torch.uint8, device="cuda", generator=g),
                torch.randint(lo, hi, (Et, n, k // 32), dtype=torch.uint8, device="cuda", generator=g))

    def normal(*n):
        return torch.randn(n, device="cuda", generator=g)
    w13, s13 = mx(2 * I, H)
    w2, s2 = mx(H, I)
    return dict(x=normal(T, H).bfloat16(), w_router=(normal(E, H) * 1.5 / H ** 0.5).bfloat16(), w13=w13, s13=s13,
                w2=w2, s2=s2, K=K, with_shared=shared,
                w_shared_gate=(normal(H) / H ** 0.5).bfloat16() if gate else None)


def decode64(codes, scales):
    mag = torch.tensor(MAGS, dtype=torch.float64, device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.where(nib >= 8, -1.0, 1.0) * mag[nib & 7]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def reference(d, renormalize=True):
    x, K = d["x"].double(), d["K"]
    T, E = x.shape[0], d["w_router"].shape[0]
    I = d["w13"].shape[1] // 2
    logits = (x @ d["w_router"].double().T).cpu().numpy()
    ids = np.stack([np.lexsort((np.arange(E), -logits[t]))[:K] for t in range(T)])
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    if d["with_shared"]:
        sw = np.ones((T, 1))
        if d["w_shared_gate"] is not None:
            sw = 1 / (1 + np.exp(-(x @ d["w_shared_gate"].double()).cpu().numpy()))[:, None]
        ids = np.concatenate([ids, np.full((T, 1), E)], 1)
        w = np.concatenate([w, sw], 1)
    out = torch.zeros_like(x)
    for e in np.unique(ids):
        w13, w2 = decode64(d["w13"][e], d["s13"][e]), decode64(d["w2"][e], d["s2"][e])
        for t, j in zip(*np.nonzero(ids == e)):
            g, u = w13[:I] @ x[t], w13[I:] @ x[t]
            out[t] += w[t, j] * (w2 @ (g / (1 + torch.exp(-g)) * u))
    return out.cpu().numpy(), ids, w


def check(got, d, renormalize=True):
    out, ids, w = got
    ref, ref_ids, ref_w = reference(d, renormalize)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    assert np.allclose(w.cpu().numpy(), ref_w, rtol=2e-5, atol=1e-7)
    o = out.double().cpu().numpy()
    rms = np.sqrt(np.mean(ref ** 2, 1, keepdims=True))
    err = np.abs(o - ref)
    assert (err <= 2.0 ** -8 * (np.abs(ref) + rms)).all(), f"{np.max(err / (np.abs(ref) + rms)) * 256:.3g} x the bound"
    rel = np.linalg.norm(o - ref) / np.linalg.norm(ref)
    assert rel <= (2e-3 if o.size >= 2048 else 2.0 ** -8), rel


SHAPES = [
    # T, H, I, E, K, shared, gate
    (1, 32, 32, 1, 1, False, False), (1, 32, 32, 1, 1, True, True), (2, 64, 32, 3, 3, True, False),
    (1, 256, 128, 8, 2, True, False), (7, 256, 128, 8, 2, True, True), (16, 256, 128, 8, 2, True, False),
    (9, 288, 96, 5, 5, False, False), (3, 2080, 608, 60, 6, False, False), (8, 544, 1056, 130, 7, True, True),
    (13, 1024, 512, 1024, 32, True, False), (16, 4096, 256, 40, 4, True, True), (8, 8192, 96, 6, 2, False, False),
    (7, 6144, 512, 16, 4, True, False), (5, 4128, 64, 9, 3, True, True), (4, 128, 8192, 4, 2, True, False),
    (16, 96, 4096, 700, 10, False, False), (5, 1024, 1024, 512, 10, True, True), (1, 4096, 1024, 64, 10, True, False),
    (16, 2048, 1024, 256, 8, True, False), (10, 32, 64, 300, 2, False, False),
    (3, 8160, 4640, 3, 2, False, False), (8, 4384, 8160, 2, 1, False, False), (12, 4064, 6176, 2, 1, True, False),
    (16, 8192, 512, 3, 2, True, True), (11, 6688, 160, 12, 3, False, False),
]


@pytest.mark.parametrize("T,H,I,E,K,shared,gate", SHAPES)
def test_matches_the_definition(m, T, H, I, E, K, shared, gate):
    d = make(T, H, I, E, K, shared, gate, seed=T + H)
    check(m.moe_layer_few(**d), d)
    check(m.moe_layer_few(**d, renormalize=False), d, False)


@pytest.mark.parametrize("T", range(1, 17))
def test_every_batch_size(m, T):
    d = make(T, 512, 256, 16, 3, True, False, seed=T)
    check(m.moe_layer_few(**d), d)


def test_agrees_with_the_layer_in_separate_calls(m):
    """moe_layer on the same logits rounds h to bf16 (relative 2^-9 per term); otherwise the same."""
    d = make(8, 1024, 512, 32, 4, True, False, seed=11)
    out, ids, w = m.moe_layer_few(**d)
    logits = d["x"].float() @ d["w_router"].float().T
    ref = m.moe_layer(logits, d["x"], d["w13"], d["s13"], d["w2"], d["s2"], 4)
    ref_ids, ref_w = m.moe_route(logits, 4)
    assert torch.equal(ids, ref_ids) and torch.allclose(w, ref_w, rtol=1e-5)
    a, b = out.double(), ref.double()
    assert ((a - b).norm() / b.norm()).item() <= 4e-3
    assert ((a - b).abs() <= 1e-2 * (b.abs() + b.pow(2).mean().sqrt())).all()


def test_equal_rows_go_to_the_lower_expert(m):
    d = make(6, 512, 64, 400, 5, False, False, seed=3)
    d["w_router"][1::2] = d["w_router"][0::2]  # pairs of equal logits
    check(m.moe_layer_few(**d), d)
    d["w_router"][:] = d["w_router"][:1]  # all equal
    out, ids, w = m.moe_layer_few(**d)
    assert (ids.cpu().numpy() == np.arange(5)).all() and torch.allclose(w, torch.full_like(w, 0.2))


def test_same_expert_for_all_and_zero_rows(m):
    d = make(16, 256, 128, 8, 2, False, False, seed=5)
    d["x"][:] = d["x"][:1]
    check(m.moe_layer_few(**d), d)
    d["x"][3] = 0  # all logits zero: the first experts, and an output of zeros
    out, ids, _ = m.moe_layer_few(**d)
    assert (out[3] == 0).all() and ids[3].tolist() == [0, 1]


@pytest.mark.parametrize("lo,hi,xs", [(100, 104, 1.0), (119, 124, 2.0 ** 40), (119, 124, 2.0 ** -60), (60, 90, 1.0),
                                      (119, 121, 1e-3)])
def test_scales_far_from_one(m, lo, hi, xs):
    """Small and large weights and activations (h carried by a power of two per row); scale bytes
    across thirty powers of two."""
    d = make(4, 512, 256, 8, 2, True, False, seed=6, lo=lo, hi=hi)
    d["x"] = (d["x"].float() * xs).bfloat16()
    if xs > 1:
        d["w_router"] = (d["w_router"].float() / xs).bfloat16()
    ref = reference(d)[0]
    assert np.abs(ref).max() < 3e38
    if np.abs(ref).max() < 1e-36:
        pytest.skip("outputs below bf16's normal range")
    check(m.moe_layer_few(**d), d)


@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_stays_with_its_token(m, T, bad):
    d = make(T, 512, 128, 16, 3, True, True, seed=7)
    good, good_ids, _ = m.moe_layer_few(**d)
    d["x"] = d["x"].clone()
    d["x"][T // 2, 300] = bad
    out, ids, _ = m.moe_layer_few(**d)
    assert torch.isnan(out[T // 2]).all()
    assert ((ids >= 0) & (ids <= 16)).all()
    rest = [t for t in range(T) if t != T // 2]
    assert torch.equal(ids[rest], good_ids[rest])
    a, b = out[rest].double(), good[rest].double()  # other experts are touched: another order of sums
    assert torch.allclose(a, b, rtol=2.0 ** -7, atol=float(good.double().abs().max()) * 2.0 ** -12)


@pytest.mark.parametrize("T,H,I,E,K", [(1, 4096, 1024, 64, 10), (16, 512, 256, 64, 8), (7, 6144, 512, 16, 4)])
def test_the_same_bits_every_time(m, T, H, I, E, K):
    d = make(T, H, I, E, K, True, True, seed=2)
    ws = m.alloc_workspace_few(T, H, I, E, K, True)
    first = [t.clone() for t in m.moe_layer_few(**d, workspace=ws)]
    for _ in range(20):
        assert int(ws[:256].sum()) == 0  # the barriers are ready for the next call
        ws[256:].random_(0, 256)         # the rest needs no care
        assert all(torch.equal(a, b) for a, b in zip(m.moe_layer_few(**d, workspace=ws), first))


def test_back_to_back_calls_share_a_workspace(m):
    """Calls of different sizes one after another on a workspace made for the largest; the output may
    replace x; ids and weights may be left out (C entry)."""
    sizes = [(16, 512, 256, 64, 8), (1, 512, 256, 64, 8), (5, 256, 64, 8, 2), (8, 512, 256, 64, 8)]
    ws = torch.empty(max(m.moe_layer_few_workspace_size(*s, True) for s in sizes), dtype=torch.uint8, device="cuda")
    ws.random_(0, 256)
    m.moe_layer_few_workspace_init(ws)
    ds = [make(*s, True, False, seed=i) for i, s in enumerate(sizes)]
    xs = [d["x"].clone() for d in ds]
    outs = [m.moe_layer_few(**{**d, "x": x}, out=x, workspace=ws) for d, x in zip(ds, xs)]
    for d, o in zip(ds, outs):
        check(o, d)
    d = ds[1]
    out = torch.empty_like(d["x"])
    p = lambda t: t.data_ptr()  # noqa: E731
    st = m.load().moe_layer_few(p(d["x"]), p(d["w_router"]), None, p(d["w13"]), p(d["s13"]), p(d["w2"]), p(d["s2"]),
                                1, 512, 256, 64, 8, 1, 1, p(out), None, None, p(ws), ws.numel(),
                                torch.cuda.current_stream().cuda_stream)
    assert st == m.MOE_OK and torch.equal(out, outs[1][0])


def test_another_stream_and_a_graph(m):
    d = make(3, 1024, 256, 32, 4, True, False, seed=4)
    ref = m.moe_layer_few(**d)
    ws = m.alloc_workspace_few(3, 1024, 256, 32, 4, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = m.moe_layer_few(**d, workspace=ws)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    out = torch.empty_like(d["x"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_layer_few(**d, out=out, topk_ids=got[1], topk_w=got[2], workspace=ws)
    d["x"].mul_(-1.5)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, m.moe_layer_few(**d)[0])
    check((out, got[1], got[2]), d)
