"""moe_lora where nothing is summed but one product's bf16 terms, so that each of them shows: an fp32 x is exact, and
A x enters the second product to 2^-24 of itself for fp32 outputs and 2^-16 for bf16 ones.  Also residual rows that
overlap, in tiles of 128."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import test_gpu_lora as lora  # noqa: E402
from test_gpu_lora import BF16, F32  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def one_product(T, N, K, R, dtype):
    """x with one value a row and adapters with one rank, whose values have all their bits, or many of them, set."""
    n = 2
    full = 2.0 - 2.0 ** -23 if dtype == F32 else 2.0 - 2.0 ** -7
    x = torch.zeros((T, K), dtype=F32, device="cuda")
    t = torch.arange(T, device="cuda")
    x[t, (7 * t) % K] = torch.where(t % 3 == 0, full, torch.randn(T, device="cuda") + 3.0) * torch.where(t % 2 == 0, 1.0, -1.0)
    a = torch.zeros((n, R, K), device="cuda")
    b = torch.randn((n, N, R), device="cuda")
    at = torch.tensor([R - 1, R // 2], device="cuda")
    a[torch.arange(n), at] = torch.where(torch.rand((n, K), device="cuda") < 0.5, 1.0 + 2.0 ** -7, 2.0 - 2.0 ** -7)
    return x.to(dtype), a.bfloat16(), b.bfloat16(), torch.tensor([1.0 / 3.0, 2.0 - 2.0 ** -23], device="cuda"), at


@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("x,out", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("tile", [16, 128])
@pytest.mark.parametrize("N", [136, 133])
def test_every_term_counts(m, x, out, R, tile, N):
    torch.manual_seed(R)
    T, K = 200, 96
    xv, a, b, scale, at = one_product(T, N, K, R, x)
    for ids in (lora.ids_of(T, 2), lora.ids_of(T, 2).sort()[0]):
        e = ids.long()
        v = (xv.double() * a[e, at[e]].double()).sum(1) * scale[e].double()
        want = v[:, None] * b[e, :, at[e]].double()
        plan = m.moe_lora_plan(ids, 2, tile)
        if out == F32:
            got = m.moe_lora(xv, a, b, plan, scale=scale, out_dtype=F32)
            # an accumulator takes three terms of x and three of v, each addition good to 2^-22 of the sum (twice 2^-23, for what
            # an MMA adds at once); v's terms to 2^-24, and roundings of scale's product and of the sum with nothing
            tol = (6 * 4 + 3) * 2.0 ** -24 * want.abs()
        else:
            # all but a 256th of the output is taken away again, so that its own rounding does not cover v's
            res = -want.bfloat16()
            got = m.moe_lora(xv, a, b, plan, scale=scale, residual=res)
            want = want + res.double()
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -16 + (5 * 4 + 3) * 2.0 ** -24) * res.double().abs() * (1 + 2.0 ** -8)
        err = (got.double() - want).abs()
        assert (err <= tol).all(), (err / tol.clamp(min=1e-38)).max()


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,n,N,K,R", [(300, 2, 264, 128, 16), (700, 3, 136, 520, 64), (129, 1, 1032, 64, 128)])
def test_residual_rows_that_overlap(m, T, n, N, K, R, out):
    """One row for every token, and rows that start within one another: not as boxes of rows that lie apart."""
    torch.manual_seed(T)
    a, b, scale = lora.adapters(n, N, K, R)
    x = lora.rows(T, K, BF16)
    base = torch.randn(8 * T + N, device="cuda").to(out)
    for ids in (lora.ids_of(T, n, 0.1), lora.ids_of(T, n).sort()[0]):
        lora.check(m, x, a, b, ids, 128, scale, residual=lora.rows(1, N, out).expand(T, -1), out_dtype=out)
        lora.check(m, x, a, b, ids, 128, scale, residual=base.as_strided((T, N), (8, 1)), out_dtype=out)
