"""moe_route_grouped where fp32 says nothing about the order of up to 32 candidates, against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import test_gpu_route_grouped as route  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K", [(32, 32), (32, 31), (31, 31), (32, 8), (20, 16), (2, 2), (2, 1), (8, 8)])
@pytest.mark.parametrize("T", [3, 4100])
def test_an_order_that_is_wrong_from_end_to_end(m, T, E, K, score):
    """Equal fp32 values, which the lower experts lead, while the exact ones rise with the expert's number."""
    logits = np.zeros((T, E), np.float32)
    rising = (np.arange(E) * 1e-10).astype(np.float32)
    for bias in (rising, rising[::-1].copy(), np.roll(rising, E // 2)):
        route.check(m, logits, K, bias, score)
    # scores that differ too, and biases that take all of the difference but that
    rng = np.random.default_rng(E)
    logits = np.repeat((0.5 * rng.standard_normal((1, E))).astype(np.float32), T, axis=0)
    s = route.scores(logits.astype(np.float64), score)[0]
    for step in (0.0, 1e-10, -1e-10, 3e-9):
        route.check(m, logits, K, (0.25 - s + step * np.arange(E)).astype(np.float32), score)


@pytest.mark.parametrize("E,G,chosen", [(1020, 17, 9), (1023, 31, 20), (1020, 20, 20), (992, 8, 4), (256, 8, 4)])
@pytest.mark.parametrize("T", [20, 4100])
def test_sums_of_many_small_terms(m, T, E, G, chosen):
    """Softmax with a bias: a denominator whose small terms are lost in fp32, all the same way, and biases that take the
    scores' differences to within that error."""
    size, K = E // G, 8
    logits = np.full((1, E), np.float32(-24 * np.log(2) - 0.01), np.float32)  # a little under 2^-24 of the largest
    logits[0, ::size] = 0.0
    rng = np.random.default_rng(E)
    picked = np.arange(K) * size + 1
    logits[0, picked] = -rng.random(K).astype(np.float32) - 0.1
    s = route.scores(logits.astype(np.float64), "softmax")[0]
    for ulps in (0, 16, 48, 60, 64, 68, 80):
        bias = np.zeros(E, np.float32)
        # the picked experts level with one another but for so many parts of 2^24 of their scores
        bias[picked] = (0.5 - s[picked] * (1.0 - ulps * 2.0 ** -24)).astype(np.float32)
        route.check(m, np.repeat(logits, T, axis=0), K, bias, "softmax", G, chosen, 2)
