"""moe_linear_mxfp4act where its kernels take more than one tile, turn or ring length: both widths of the
CTA-pair kernel over several turns in every form of output, the token tiles and long K ranges of the
streaming kernel, the wide output head.

tile_rule restates launch_linear_mxfp4's choice, and every case says what it is meant to reach: a case
that no longer does fails (tests/test_linear_tile_rule.py holds the rule's text).

Bounds: products and encodings are exact; an MMA adds its products to an fp32 accumulator with every
term cut at 2^-23 of the largest at most.  The K cuts are independent and of either sign: together
sqrt(K) 2^-23 of sum |w| |xq| in the mean square, eight times that for the largest of 10^8 outputs,
and never more than K 2^-23.  Then 2^-24 of the result for the residual, and a bf16
output's 2^-8.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def up(a, b):
    return -(-a // b)


def tile_rule(T, N, K):
    """("pair", width, turns) or ("stream", token tile, splits, most stages of a CTA)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if T > 64 and N >= 128:
        turns = {w: up(up(T, 256) * up(N, w), sms // 2) for w in (128, 256)}
        width = 128 if 4 * turns[128] <= 5 * turns[256] else 256
        return "pair", width, turns[width]
    nt = next(n for n in (16, 32, 64, 128) if T <= n or n == 128)
    tiles, nk, splits = up(N, 128) * up(T, nt), up(K, 256), 1
    while splits < 8 and 2 * splits <= nk and tiles * 2 * splits <= 2 * sms:
        splits *= 2
    return "stream", nt, splits, up(nk, splits)


def values(codes, scales):
    mag = torch.tensor(MAGS + [-v for v in MAGS], dtype=torch.float64, device="cuda")
    v = mag[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def quantised(x):
    """The MXFP4 values of float64 rows."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax)[1].double() - 3
    a = b.abs() / torch.exp2(e)
    # halfway points between neighbours go to the even code
    q = (0.5 * ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0))
    return torch.where(amax > 0, torch.sign(b) * q * torch.exp2(e), 0.0).reshape(x.shape)


def make(T, N, K, xt, ot, residual, pad, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, K), device="cuda", generator=g).to(TYPES[xt])
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(115, 128, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    res = (torch.randn((T, N + pad), device="cuda", generator=g) * 8).to(TYPES[ot])[:, :N] if residual else None
    return x, codes, scales, res


def check(out, x, codes, scales, res):
    xq, K = quantised(x.double()), x.shape[1]
    for n0 in range(0, codes.shape[0], 8192):
        w = values(codes[n0:n0 + 8192], scales[n0:n0 + 8192])
        ref, size = xq @ w.T, xq.abs() @ w.abs().T
        if res is not None:
            ref += res[:, n0:n0 + 8192].double()
        bound = min(K, 8 * math.sqrt(K)) * 2.0 ** -23 * size + 2.0 ** -24 * ref.abs()
        if out.dtype == torch.bfloat16:
            bound += 2.0 ** -8 * (ref.abs() + bound)
        err = (out[:, n0:n0 + 8192].double() - ref).abs()
        assert bool((err <= bound).all()), f"columns from {n0}: {float((err > bound).double().mean()):.3g} of them off"


def run(m, T, N, K, xt="bf16", ot="bf16", residual=False, pad=0):
    """out (and the residual) as a slice of rows `pad` wider, whose rest keeps its value."""
    x, codes, scales, res = make(T, N, K, xt, ot, residual, pad, T + N + K)
    wide = torch.full((T, N + pad), 123.0, dtype=TYPES[ot], device="cuda")
    out = wide[:, :N]
    m.moe_linear_mxfp4act(x, codes, scales, residual=res, out=out)
    check(out, x, codes, scales, res)
    assert bool((wide[:, N:] == 123.0).all())


PAIRS = [
    # T, N, K, width, turns: full and part tiles at both ends, K of 1 to 16 stages (a ring holds 5 or 6)
    (1536, 4096, 4096, 256, 2), (1500, 4090, 1056, 256, 2), (2200, 5100, 288, 256, 3), (1409, 3969, 224, 256, 2),
    (1400, 3150, 1056, 128, 2), (2048, 2400, 2080, 128, 2), (32000, 300, 320, 128, 5), (1321, 3073, 1600, 128, 2),
]


@pytest.mark.parametrize("T,N,K,width,turns", PAIRS)
@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("aligned", [True, False])
def test_pairs_over_several_turns(m, T, N, K, width, turns, ot, residual, aligned):
    assert tile_rule(T, N, K) == ("pair", width, turns)
    pad = 8 + -N % 8 if aligned else 1 + N % 2  # an odd pitch: no row but the first on 16 bytes
    assert ((N + pad) * TYPES[ot].itemsize % 16 == 0) == aligned
    run(m, T, N, K, "f32" if turns == 3 else "bf16", ot, residual, pad)


@pytest.mark.parametrize("T,N,K,width", [(70, 200, 65536, 128), (300, 129, 16384, 128), (4900, 4864, 8224, 256)])
def test_pairs_over_long_rows(m, T, N, K, width):
    assert tile_rule(T, N, K)[:2] == ("pair", width)
    run(m, T, N, K, ot="f32")


@pytest.mark.parametrize("T,N,K,nt,splits,stages", [
    (300, 100, 8192, 128, 8, 4), (65, 127, 65536, 128, 8, 32), (200, 1, 2080, 128, 8, 2), (19700, 100, 1056, 128, 1, 5),
    (16, 40003, 4096, 16, 1, 16), (7, 40003, 1056, 16, 1, 5), (24, 40003, 1056, 32, 1, 5), (40, 40003, 2080, 64, 1, 9),
    (64, 20100, 4096, 64, 1, 16), (5, 300, 65536, 16, 8, 32), (16, 8200, 16384, 16, 4, 16), (33, 520, 32768, 64, 8, 16),
])
@pytest.mark.parametrize("ot,residual", [("f32", False), ("bf16", True)])
def test_streaming_over_a_full_ring(m, T, N, K, nt, splits, stages, ot, residual):
    assert tile_rule(T, N, K) == ("stream", nt, splits, stages)
    run(m, T, N, K, ot=ot, residual=residual)


@pytest.mark.parametrize("T,N,K", [(1536, 4096, 1024), (1400, 3150, 512), (2200, 5100, 288)])
def test_the_same_bits_and_an_aliased_residual(m, T, N, K):
    x, codes, scales, res = make(T, N, K, "bf16", "bf16", True, 0, 3)
    first = m.moe_linear_mxfp4act(x, codes, scales, residual=res)
    ws = m.alloc_workspace_linear(T, N, K)
    for _ in range(3):
        ws.random_(0, 256)
        out = res.clone()
        m.moe_linear_mxfp4act(x, codes, scales, residual=out, out=out, workspace=ws)
        assert torch.equal(out, first)


def test_a_bad_value_in_a_later_turn_stays_with_its_token(m):
    x, codes, scales, _ = make(2200, 5100, 288, "bf16", "bf16", False, 0, 5)
    good = m.moe_linear_mxfp4act(x, codes, scales)
    for t in (0, 1100, 2199):
        x[t, 200] = float("nan")
    out = m.moe_linear_mxfp4act(x, codes, scales)
    bad = torch.zeros(2200, dtype=torch.bool, device="cuda")
    bad[[0, 1100, 2199]] = True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], good[~bad])
