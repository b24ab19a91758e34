"""moe_layer_few keeps h = silu(gate) * up to fp32's accuracy on its way into the down product: the
output is the exact value's bf16 but for what fp32 sums leave.

Before the rounding to bf16 the result errs, in units of its row's rms (rounding errors taken as
independent, each at most half an ulp of a partial sum): the gate and up sums, up to 256 blocks of 32
added one after another, by about 2e-7 each (the tensor core cuts a block's sum at 2^-23 of it, the
running sum is rounded at 2^-24), their product by 3e-7, h's two f16 terms by 2^-24 of each
element, the down sums by 2e-7, the weights and their sum by 1e-7: 5e-7 in all, and 3e-6 for the
largest of a million elements (six times that).  The bound is half an ulp of bf16 next to the exact
value plus 2^-17 = 7.6e-6 of the row's rms.  With h in 11 bits the error is 2.5e-4 of the rms.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_layer_few import make, reference  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def check(out, ref):
    o = out.double().cpu().numpy()
    half_ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(ref), 1e-38))) - 8)
    bound = half_ulp + 2.0 ** -17 * np.sqrt(np.mean(ref ** 2, 1, keepdims=True))
    err = np.abs(o - ref)
    assert (err <= bound).all(), f"{np.mean(err > bound):.3g} of the elements, up to {np.max(err / bound):.3g} x the bound"


SHAPES = [
    # T, H, I, E, K, shared, gate; experts with every number of tokens from 1 to 16
    (1, 4096, 1024, 16, 4, True, False), (5, 2080, 608, 12, 3, False, False), (16, 1024, 512, 8, 2, True, True),
    (12, 512, 256, 4, 4, False, False), (7, 6144, 512, 8, 3, True, False), (16, 512, 8192, 3, 2, True, False),
    (9, 256, 4640, 5, 4, False, False), (13, 96, 64, 7, 5, True, True), (16, 2048, 1024, 64, 8, True, False),
]


@pytest.mark.parametrize("T,H,I,E,K,shared,gate", SHAPES)
def test_outputs_are_the_exact_values_rounded(m, T, H, I, E, K, shared, gate):
    d = make(T, H, I, E, K, shared, gate, seed=31 * T + I)
    check(m.moe_layer_few(**d)[0], reference(d)[0])


@pytest.mark.parametrize("spread", [4, 14])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_elements_far_below_the_largest(m, T, spread):
    """32 elements of h 2^spread above the others, their down weights as far below: both parts count
    alike in the output."""
    d = make(T, 512, 96, 6, 2, True, False, seed=T + spread)
    d["s13"][:, 96:128] += spread
    d["s2"][:, :, 0] -= spread
    check(m.moe_layer_few(**d)[0], reference(d)[0])


@pytest.mark.parametrize("T", [2, 11])
def test_an_infinite_element_of_h(m, T):
    """One element of h that leaves fp32's range: the outputs of its token are infinite with the sign
    of their down weight, or NaN where that is zero, as in the formula; other tokens keep their values."""
    d = make(T, 256, 64, 4, 1, False, False, seed=T)
    d["x"][1] = 0
    d["x"][1, 5] = 1e19
    d["w_router"][:, 5] = 0
    d["s13"][:] = 127
    d["w13"][:, :, 2] &= 0x0F             # the weights of x[5]: 0,
    d["w13"][:, [0, 64], 2] |= 0x60       # but 4 for the first gate and up rows
    out, ids, _ = m.moe_layer_few(**d)
    code = (d["w2"][int(ids[1, 0]), :, 0] & 15).cpu().numpy()
    want = np.where(code & 7, np.where(code & 8, -np.inf, np.inf), np.nan)
    assert np.array_equal(out[1].double().cpu().numpy(), want, equal_nan=True)
    rest = [t for t in range(T) if t != 1]
    check(out[rest], reference(d)[0][rest])


@pytest.mark.parametrize("gate,up,down", [(224, 30, 224), (1, 224, 224), (224, 1, 127), (30, 224, 1), (127, 127, 224)])
@pytest.mark.parametrize("T", [1, 9])
def test_scale_bytes_at_the_ends_of_their_range(m, T, gate, up, down):
    """Weights of 2^-126 and of 2^97 next to each other.  The outputs lie inside bf16's normal range, or
    are skipped below it."""
    d = make(T, 512, 96, 6, 2, True, False, seed=gate + up + T)
    d["s13"][:, :96], d["s13"][:, 96:], d["s2"][:] = gate, up, down
    ref = reference(d)[0]
    assert np.abs(ref).max() < 2.0 ** 126
    if np.abs(ref).max() < 2.0 ** -100:
        assert np.isfinite(m.moe_layer_few(**d)[0].double().cpu().numpy()).all()
    else:
        check(m.moe_layer_few(**d)[0], ref)
