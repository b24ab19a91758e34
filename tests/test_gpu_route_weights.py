"""moe_route_grouped's weights, each against the formula in 64 bits relative to itself, over logits that lie far apart."""
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


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,K", [(64, 30), (64, 16), (64, 8), (33, 8)])
@pytest.mark.parametrize("shift", [0.0, -70.0])
@pytest.mark.parametrize("T", [300, 4200])
def test_to_a_few_ulp_whatever_the_distance(m, T, shift, E, K, score, renorm):
    rng = np.random.default_rng(E + K)
    logits = (25.0 * rng.standard_normal((T, E)) + shift).astype(np.float32)
    ids, w = m.moe_route_grouped(torch.from_numpy(logits).cuda(), K, None, score, with_shared=False, renormalize=renorm)
    want, ww = route.definition(logits, K, None, score, 1, 1, 1, renorm=renorm)
    assert np.array_equal(ids.cpu().numpy(), want)
    normal = ww > 2.0 ** -125
    # in parts of 2^24: an exponential 2, the rest of its argument's difference 1 (its product and sum), 1 + e 3 (sigmoid), two
    # quotients and a scale 3; the sum: its terms 4, and its additions: 5 levels, and softmax's over all experts up to 16 a lane
    tol = (2 + 1 + 3 + 3 + 4 + 5 + (16 if score == "softmax" and not renorm else 0)) * 2.0 ** -24
    err = np.abs(w.double().cpu().numpy() - ww)[normal] / ww[normal]
    assert err.max() <= tol, err.max() * 2.0 ** 24
