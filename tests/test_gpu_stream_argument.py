"""Calls that are given a stream and allocate for themselves, while the current stream is busy: nothing
of theirs waits for it, and memory that they give back is not handed to it early."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def mx(g, *shape):
    return (torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device="cuda", generator=g),
            torch.randint(119, 124, (*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device="cuda", generator=g))


def beside_a_busy_stream(call, scribble):
    """The results of call(stream), issued while the current stream sleeps (about 10 ms), then
    overwrites `scribble` bytes of whatever memory it is given."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    results = []
    for _ in range(4):
        torch.cuda._sleep(20_000_000)
        results.append(call(s))
        done = torch.cuda.Event()
        done.record(s)
        junk = torch.full((scribble,), 0xFF, dtype=torch.uint8, device="cuda")
        done.synchronize()
        del junk
    torch.cuda.synchronize()
    return results


def test_layer_few(m):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, H, I, E, K = 6, 1024, 512, 32, 4
    w13, s13 = mx(g, E + 1, 2 * I, H)
    w2, s2 = mx(g, E + 1, H, I)
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    router = (torch.randn((E, H), device="cuda", generator=g) / 32).bfloat16()
    want = m.moe_layer_few(x, router, w13, s13, w2, s2, K)
    size = m.moe_layer_few_workspace_size(T, H, I, E, K, True)
    for got in beside_a_busy_stream(lambda s: m.moe_layer_few(x, router, w13, s13, w2, s2, K, stream=s), size):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [3, 48, 200])
def test_linear(m, T):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    N, K = 1024, 2048
    codes, scales = mx(g, N, K)
    x = torch.randn((T, K), device="cuda", generator=g).bfloat16()
    want = m.moe_linear_mxfp4act(x, codes, scales)
    size = m.moe_linear_mxfp4act_workspace_size(T, N, K)
    for got in beside_a_busy_stream(lambda s: m.moe_linear_mxfp4act(x, codes, scales, stream=s), size):
        assert torch.equal(got, want)
