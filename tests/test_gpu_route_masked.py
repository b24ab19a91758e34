"""moe_route_grouped with most experts masked (-inf, or NaN, which counts as -inf): groups with none, one or two
experts left, in batches of either kernel, against the definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import test_gpu_route_grouped as route  # noqa: E402

E, K = 128, 6


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def masked(T, dtype, nan, seed, share):
    """Logits of which this share is masked, one at least of each token's not."""
    rng = np.random.default_rng(seed)
    logits = torch.from_numpy((2.0 * rng.standard_normal((T, E))).astype(np.float32)).to(dtype).float().numpy()
    gone = rng.random((T, E)) < share
    gone[np.arange(T), rng.integers(0, E, T)] = False
    plain = np.where(gone, np.float32(-np.inf), logits)
    given = np.where(gone & (rng.random((T, E)) < 0.5), np.float32(np.nan), plain) if nan else plain
    return plain, torch.from_numpy(given).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("G", [2, 4, 8, 16])
@pytest.mark.parametrize("share", [0.85, 0.98])  # (at 0.98 most tokens keep groups that have nothing left)
@pytest.mark.parametrize("T", [50, 4100])
def test_groups_with_few_experts_left(m, T, share, G, top, biased, score, dtype):
    nan = G in (4, 8)
    plain, given = masked(T, dtype, nan, G + top, share)
    bias = (0.1 * np.random.default_rng(9).standard_normal(E)).astype(np.float32) if biased else None
    b = None if bias is None else torch.from_numpy(bias).cuda()
    for renorm in (True, False):
        ids, w = m.moe_route_grouped(given, K, b, score, G, G // 2, top, with_shared=False, renormalize=renorm)
        # (a chosen expert that is masked has a score of 0: no quotient of infinities in the definition)
        with np.errstate(invalid="ignore"):
            want, ww = route.definition(plain, K, bias, score, G, G // 2, top, renorm=renorm)
        got = ids.cpu().numpy()
        assert not (got != want).any(), f"{(got != want).any(1).sum()} of {T} tokens differ"
        some = np.isfinite(np.take_along_axis(plain, want, 1)).any(1)
        assert some.any()
        # arguments of exponentials to 2^-24 of themselves, twice for a difference of two up to 12; 24 further roundings
        err = np.abs(w.double().cpu().numpy() - ww)[some]
        assert (err <= (2 * 24 + 24) * 2.0 ** -24 * ww[some] + 2.0 ** -140).all()
        assert not w.cpu().numpy()[~some].any()


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("G", [2, 4, 8, 16])
def test_a_long_batch_is_its_pieces(m, G, top):
    for score in ("sigmoid", "softmax"):
        given = masked(8200, torch.float32, True, G, 0.9)[1]
        ids, w = m.moe_route_grouped(given, K, None, score, G, G // 2, top)
        for t0 in range(0, 8200, 2050):
            a, b = m.moe_route_grouped(given[t0:t0 + 2050], K, None, score, G, G // 2, top)
            assert torch.equal(ids[t0:t0 + 2050], a)
            assert torch.allclose(w[t0:t0 + 2050], b, rtol=16 * 2.0 ** -24, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,chosen,K", [(16, 2, 16), (8, 1, 16), (8, 2, 16), (32, 3, 12), (4, 1, 8)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T", [50, 4100])
def test_more_chosen_than_are_left(m, T, top, G, chosen, K, score):
    """Which of the groups with nothing left stay shows where their experts are chosen too."""
    plain, given = masked(T, torch.float32, False, G, 0.98)
    ids, _ = m.moe_route_grouped(given, K, None, score, G, chosen, top, with_shared=False)
    with np.errstate(invalid="ignore"):
        want, _ = route.definition(plain, K, None, score, G, chosen, top)
    got = ids.cpu().numpy()
    assert not (got != want).any(), f"{(got != want).any(1).sum()} of {T} tokens differ"


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [50, 4100])
def test_masks_of_the_lowest_value(m, T, dtype, score):
    """Masked by the type's lowest value instead of -inf: an expert like any other, whose score rounds to 0."""
    plain, given = masked(T, dtype, False, 3, 0.85)
    low = torch.finfo(dtype).min
    given = given.clamp(min=low)
    plain = np.where(np.isfinite(plain), plain, np.float32(low))
    for G, chosen, top in ((8, 4, 2), (8, 4, 1), (4, 1, 2), (1, 1, 1)):
        ids, w = m.moe_route_grouped(given, K, None, score, G, chosen, top, with_shared=False)
        with np.errstate(invalid="ignore"):
            want, _ = route.definition(plain, K, None, score, G, chosen, top)
        assert np.array_equal(ids.cpu().numpy(), want) and torch.isfinite(w).all()
