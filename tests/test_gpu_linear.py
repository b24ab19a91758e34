"""moe_linear_mxfp4act against its definition in 64 bits.

The quantisation is exact in both (a power of two per block, a table of eight
magnitudes), so the only differences are the order of the fp32 sums and the
one rounding to the output type.  With n = K / 32 blocks the MMA's fp32
accumulation errs by at most K * 2^-23 of sum |w| |xq| per element (each
addition by at most 2^-23 of a partial sum, which that sum bounds), the residual's addition by 2^-24 of
the result, and a bf16 output by 2^-8 of it (half an ulp is at most 2^-9,
doubled for a sum that lies next to a rounding boundary).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def decode64(codes, scales):
    c = codes.cpu().numpy()
    nib = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    v = np.where(nib & 8, -1.0, 1.0) * MAGS[nib & 7]
    return v * np.repeat(np.exp2(scales.cpu().numpy().astype(np.float64) - 127), 32, 1)


def quantised64(x):
    """MXFP4 values of float64 rows, block by block."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = np.abs(b).max(-1, keepdims=True)
    e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2, -127.0)
    e = np.maximum(e, -127.0)
    a = np.abs(b) / np.exp2(e)
    # nearest magnitude, ties to the even code: the index whose distance is least, even codes first
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    near = np.abs(a[..., None] - MAGS[order]).argmin(-1)
    return (np.sign(b) * MAGS[order][near] * np.exp2(e)).reshape(x.shape)


def make(T, N, K, xt="bf16", pad=0, seed=0, lo=119, hi=124):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, K + pad), device="cuda", generator=g).to(TYPES[xt])[:, :K]
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(lo, hi, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    return x, codes, scales


def check(out, x, codes, scales, residual=None):
    w, xq = decode64(codes, scales), quantised64(x.double().cpu().numpy())
    ref = xq @ w.T
    size = np.abs(xq) @ np.abs(w).T
    K = x.shape[1]
    if residual is not None:
        ref = ref + residual.double().cpu().numpy()
    bound = K * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(ref)
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    got = out.double().cpu().numpy()
    assert got.shape == ref.shape
    # no partial sum can leave fp32's range where sum |w| |xq| does not; a result outside it is not finite
    inside = size < 2.0 ** 127
    assert np.isfinite(got[inside]).all() and not np.isfinite(got[np.abs(ref) > 2.0 ** 128]).any()
    worst = np.max((np.abs(got - ref) / np.maximum(bound, 1e-300))[inside], initial=0.0)
    assert (np.abs(got - ref) <= bound)[inside].all(), f"{worst:.3g} x the bound"


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


SHAPES = [
    (1, 1, 32), (1, 16, 32), (1, 128, 64), (2, 129, 96), (1, 4096, 4096), (5, 2048, 1024), (8, 640, 8192),
    (15, 127, 288), (16, 1000, 512), (17, 384, 1056), (31, 256, 2048), (33, 257, 2080), (64, 512, 4096),
    (65, 200, 544), (100, 1, 256), (128, 768, 768), (129, 130, 1280), (250, 300, 2048), (256, 1024, 512),
    (300, 520, 800), (513, 1100, 1024), (1030, 640, 352), (2049, 384, 256),
]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matches_the_definition(m, T, N, K):
    x, codes, scales = make(T, N, K, seed=T + N)
    check(m.moe_linear_mxfp4act(x, codes, scales), x, codes, scales)


@pytest.mark.parametrize("T,N,K", [(1, 200, 512), (9, 1000, 1056), (40, 300, 288), (140, 260, 1024),
                                   (700, 1000, 544), (1500, 770, 1024)])
@pytest.mark.parametrize("xt,ot,pad", [("bf16", "bf16", 24), ("bf16", "f32", 5), ("f32", "bf16", 3),
                                       ("f32", "f32", 4)])
def test_types_strides_and_residual(m, T, N, K, xt, ot, pad):
    """Slices of wider rows (aligned and not) for x, residual and out, in both types; what
    lies between out's rows keeps its value."""
    x, codes, scales = make(T, N, K, xt, pad, seed=3 * T + pad)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    res = torch.randn((T, N + pad), device="cuda", generator=g).to(TYPES[ot])[:, :N]
    wide = torch.full((T, N + 7), 123.0, dtype=TYPES[ot], device="cuda")
    out = wide[:, :N]
    assert m.moe_linear_mxfp4act(x, codes, scales, residual=res, out=out) is out
    check(out, x, codes, scales, res)
    assert (wide[:, N:] == 123.0).all()


@pytest.mark.parametrize("T,N,K", [(65, 129, 96), (130, 777, 512), (300, 1003, 288), (800, 518, 1024)])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("with_res", [False, True])
def test_rows_on_16_bytes_that_end_inside_one(m, T, N, K, ot, with_res):
    """out and residual as aligned slices of aligned rows whose width is no multiple of 16 bytes."""
    x, codes, scales = make(T, N, K, seed=T + K)
    width = (N + 15) // 8 * 8 + 8
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    res = torch.randn((T, width), device="cuda", generator=g).to(TYPES[ot])[:, :N] if with_res else None
    wide = torch.full((T, width), 123.0, dtype=TYPES[ot], device="cuda")
    out = wide[:, :N]
    assert m.moe_linear_mxfp4act(x, codes, scales, residual=res, out=out) is out
    check(out, x, codes, scales, res)
    assert (wide[:, N:] == 123.0).all()


@pytest.mark.parametrize("T,N,K", [(3, 300, 512), (600, 512, 512), (1300, 520, 256)])
def test_residual_may_be_the_output(m, T, N, K):
    x, codes, scales = make(T, N, K, seed=8)
    out = torch.randn((T, N), device="cuda").bfloat16()
    res = out.clone()
    m.moe_linear_mxfp4act(x, codes, scales, residual=out, out=out)
    check(out, x, codes, scales, res)


@pytest.mark.parametrize("T", [5, 700])
def test_one_row_for_every_token(m, T):
    x, codes, scales = make(1, 260, 512, seed=9)
    out = m.moe_linear_mxfp4act(x.expand(T, -1), codes, scales)
    check(out, x.expand(T, -1), codes, scales)
    assert (out == out[:1]).all()


@pytest.mark.parametrize("T", [2, 40, 1200])
def test_extreme_scales_and_values(m, T):
    """Zero rows, subnormal and very large inputs, weight scales over 130 powers of two: outputs
    from below 1e-30 to infinite ones."""
    x, codes, scales = make(T, 260, 512, seed=4, lo=60, hi=190)
    x = x.clone()
    x[0] = 0
    x[-1, :32] = torch.finfo(torch.bfloat16).tiny
    x[-1, 32:64] = 1e-40
    x[-1, 64:96] = 3e30
    check(m.moe_linear_mxfp4act(x, codes, scales, out_dtype=torch.float32), x, codes, scales)


@pytest.mark.parametrize("T", [1, 4, 70, 1100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_stays_with_its_token(m, T, bad):
    x, codes, scales = make(T, 300, 512, seed=6)
    good = m.moe_linear_mxfp4act(x, codes, scales)
    y = x.clone()
    y[T // 2, 77] = bad
    out = m.moe_linear_mxfp4act(y, codes, scales)
    assert torch.isnan(out[T // 2]).all()
    rest = [t for t in range(T) if t != T // 2]
    assert torch.equal(out[rest], good[rest])


@pytest.mark.parametrize("T,N,K", [(1, 4096, 4096), (16, 1000, 8192), (64, 512, 4096), (1536, 1024, 1024)])
def test_the_same_bits_every_time(m, T, N, K):
    x, codes, scales = make(T, N, K, seed=5)
    ws = m.alloc_workspace_linear(T, N, K)
    first = m.moe_linear_mxfp4act(x, codes, scales, workspace=ws).clone()
    for _ in range(5):
        ws.random_(0, 256)  # what an earlier call left in the workspace does not matter
        assert torch.equal(m.moe_linear_mxfp4act(x, codes, scales, workspace=ws), first)


def test_another_stream_and_a_graph(m):
    x, codes, scales = make(3, 512, 1024, seed=2)
    ref = m.moe_linear_mxfp4act(x, codes, scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws, out = m.alloc_workspace_linear(3, 512, 1024), torch.empty_like(ref)
    with torch.cuda.stream(s):
        m.moe_linear_mxfp4act(x, codes, scales, out=out, workspace=ws)
    s.synchronize()
    assert torch.equal(out, ref)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_linear_mxfp4act(x, codes, scales, out=out, workspace=ws)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, m.moe_linear_mxfp4act(x, codes, scales))
