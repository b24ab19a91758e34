"""moe_combine_norm in its kernels for many rows, and slots in rows of every width: the formula in 64 bits, use in place,
rows that hold no numbers, captured calls."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_combine_norm import BF16, F32, check, rows  # noqa: E402


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def enough(H, turns=1.0):
    """An odd number of rows of H values from which the kernels for many rows run: 32768 values an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return int(turns * 2 * 16 * 1024 * sms / H + 1) | 1


@pytest.mark.parametrize("H", [8, 24, 64, 128, 136, 264, 504, 512])
@pytest.mark.parametrize("ydt,hdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_many_short_rows(m, H, ydt, hdt):
    torch.manual_seed(H)
    T = enough(H, 1.3)
    y, h, pre, post = rows(T, H, ydt), rows(T, H, hdt, 8), rows(1, H, BF16)[0], rows(1, H, BF16)[0]
    check(m, y, h=h, pre_w=pre)
    check(m, y, h=h, post_w=post, pre_w=pre, gate=rows(1, H, BF16), gate_act="silu", alpha=0.5, beta=0.25, w_offset=1.0)
    check(m, y, h=h, post_w=post, gate=rows(T, H, F32), gate_act="sigmoid")
    check(m, y, post_w=post, pre_w=pre, gate=rows(T, 1, BF16), h_out=False)
    check(m, y, h=h, gate=rows(1, 1, BF16), n_out=False)


@pytest.mark.parametrize("H", [387, 388, 1001, 4099, 4100, 8200, 12289, 16384])
@pytest.mark.parametrize("slots", [2, 3, 9])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slots_in_rows_of_any_width(m, H, slots, dtype):
    torch.manual_seed(H + slots)
    T = 5
    check(m, rows(T * slots, H, dtype), slots=slots, h=rows(T, H, BF16), pre_w=rows(1, H, BF16)[0])
    check(m, rows(T * slots, H, dtype, 3, 1), slots=slots, h=rows(T, H, F32, 5), post_w=rows(1, H, F32)[0],
          pre_w=rows(1, H, F32)[0], gate=rows(T, H, BF16), gate_act="silu")


@pytest.mark.parametrize("H", [77, 84, 384, 4100])
def test_all_slots(m, H):
    torch.manual_seed(H)
    check(m, rows(3 * 64, H, F32), slots=64, h=rows(3, H, F32), pre_w=rows(1, H, F32)[0])


LONG = [(64, 2.2), (128, 1.0), (264, 1.5), (512, 1.0), (520, 1.2), (2088, 3.0), (4096, 1.0), (8192, 1.7)]


@pytest.mark.parametrize("H,turns", LONG)
@pytest.mark.parametrize("hdt", [BF16, F32])
def test_in_place(m, H, turns, hdt):
    """The stream in place, the norm over the block's output: the bits of a call that writes elsewhere."""
    torch.manual_seed(H)
    T = enough(H, turns)
    y, h, w, post = rows(T, H, BF16), rows(T, H, hdt), rows(1, H, BF16)[0], rows(1, H, BF16)[0]
    for gate in (None, rows(1, H, BF16), rows(T, H, BF16), rows(T, 1, BF16)):
        kw = dict(pre_w=w, post_w=post, gate=gate, alpha=0.5, beta=0.75)
        want = m.moe_combine_norm(y, h=h, **kw)
        a, b = y.clone(), h.clone()
        m.moe_combine_norm(a, h=b, **kw, h_out=b, n_out=a)
        assert torch.equal(b, want[0]) and torch.equal(a, want[1])


@pytest.mark.parametrize("H,turns", LONG)
def test_rows_do_not_mix(m, H, turns):
    torch.manual_seed(H)
    T = enough(H, turns)
    y, h, w = rows(T, H, BF16), rows(T, H, BF16), rows(1, H, BF16)[0]
    want = m.moe_combine_norm(y, h=h, pre_w=w, post_w=w)
    # of the first turns and of later ones, and the very last
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    for t in (0, 2, T // 3, T // 2, T // 2 + 1, T - 2, T - 1):
        bad[t] = True
        if t % 2:
            y[t, H // 2] = float("nan")
        else:
            h[t] = float("inf")
    got = m.moe_combine_norm(y, h=h, pre_w=w, post_w=w)
    for a, b in zip(got, want):
        assert torch.equal(a[~bad], b[~bad]) and not torch.isfinite(a[bad]).all(1).any()


@pytest.mark.parametrize("H,turns", [(128, 1.5), (2088, 1.5)])
def test_captured_in_place(m, H, turns):
    """A stream that captured calls update in place, replay after replay, and the same calls one by one elsewhere."""
    torch.manual_seed(H)
    T = enough(H, turns)
    y, start, w = rows(T, H, BF16), rows(T, H, F32), rows(1, H, BF16)[0]
    h, n = start.clone(), torch.empty_like(y)

    def step():
        m.moe_combine_norm(y, h=h, pre_w=w, beta=0.5, h_out=h, n_out=n)
        m.moe_combine_norm(n, h=h, pre_w=w, alpha=0.25, h_out=h, n_out=n)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    h.copy_(start)
    for _ in range(4):
        g.replay()
    a, b = start.clone(), None
    for _ in range(4):
        a, b = m.moe_combine_norm(y, h=a, pre_w=w, beta=0.5)
        a, b = m.moe_combine_norm(b, h=a, pre_w=w, alpha=0.25)
    assert torch.equal(h, a) and torch.equal(n, b)


@pytest.mark.parametrize("T,H", [(3, 4096), (3, 77), (None, 128), (None, 2088)])
def test_squares_beyond_fp32(m, T, H):
    """A norm whose sum of squares leaves fp32's range is 0; the other rows are as ever."""
    T = T or enough(H)
    y, w = rows(T, H, F32), rows(1, H, BF16)[0]
    want = m.moe_combine_norm(y, pre_w=w, h_dtype=F32)
    y[1] = 1e20
    h, n = m.moe_combine_norm(y, pre_w=w, h_dtype=F32)
    assert (h[1] == y[1]).all() and not n[1].any()
    keep = [t for t in range(T) if t != 1] if T < 9 else slice(2, None)
    assert torch.equal(h[keep], want[0][keep]) and torch.equal(n[keep], want[1][keep])
