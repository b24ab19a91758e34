"""moe_combine_norm against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # a rounding, relative


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def rows(T, H, dtype, pad=0, shift=0, scale=1.0):
    """[T, H] rows of a wider tensor, `shift` elements into it."""
    return (torch.randn((T, H + pad + shift), device="cuda") * scale).to(dtype)[:, shift:shift + H]


def formula(y, h=None, slots=1, post_w=None, gate=None, gate_act="none", alpha=1.0, beta=1.0, pre_w=None, w_offset=0.0,
            eps=1e-6, **_):
    """h' and n in 64 bits, and for each what its fp32 errors are relative to."""
    T, H = y.shape[0] // slots, y.shape[1]
    y3 = y.double().view(T, slots, H) if y.is_contiguous() else y.double().reshape(T, slots, H)
    u, mag = y3.sum(1), y3.abs().sum(1)
    if post_w is not None:
        f = (post_w.double() + w_offset) / (u.pow(2).mean(1, keepdim=True) + eps).sqrt()
        # an error of the sum moves the norm too: by at most that of the row's largest share
        mag = mag * f.abs() + u.abs() * f.abs() * (mag.norm(dim=1) / u.norm(dim=1).clamp(min=1e-30))[:, None]
        u = u * f
    if gate is not None:
        z = gate.double()
        a = {"none": z, "sigmoid": torch.sigmoid(z), "silu": z * torch.sigmoid(z)}[gate_act]
        u, mag = u * a, mag * a.abs()
    u, mag = alpha * u, abs(alpha) * mag
    if h is not None:
        u, mag = u + beta * h.double(), mag + abs(beta) * h.double().abs()
    r = 1.0 / (u.pow(2).mean(1, keepdim=True) + eps).sqrt()
    f = r * (1.0 if pre_w is None else pre_w.double() + w_offset)
    n = u * f
    nmag = mag * f.abs() + n.abs() * (mag.norm(dim=1) / u.norm(dim=1).clamp(min=1e-30))[:, None]
    return u, mag, n, nmag


def check(m, y, **kw):
    got_h, got_n = m.moe_combine_norm(y, **kw)
    h, mag, n, nmag = formula(y, **kw)
    # sums of squares: 16 a thread, 10 levels, all of one sign; the slots one by one; about 20 further roundings
    ulps = (kw.get("slots", 1) + 50) * 2.0 ** -24
    for got, want, size in ((got_h, h, mag), (got_n, n, nmag)):
        if got is not False:
            err = (got.double() - want).abs()
            assert (err <= HALF[got.dtype] * want.abs() + ulps * size + 1e-38).all(), (err / (size + 1e-30)).max()
    return got_h, got_n


@pytest.mark.parametrize("T,H", [(1, 4096), (1, 1), (3, 7), (5, 64), (64, 2080), (33, 2084), (7, 4099), (130, 128), (4, 8192),
                                 (3, 16384), (2, 16383), (2, 16380), (9, 1000), (600, 96)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_residual_and_norm(m, T, H, dtype):
    torch.manual_seed(T * H)
    check(m, rows(T, H, dtype), h=rows(T, H, dtype, scale=3.0), pre_w=rows(1, H, BF16)[0], n_dtype=dtype)


@pytest.mark.parametrize("gate", [(1, 1), (1, 0), (0, 1), (0, 0), None])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("H", [512, 1025])
def test_norms_on_both_sides_and_gates(m, gate, act, H):
    torch.manual_seed(H)
    T = 21
    g = None if gate is None else 4.0 * rows(T if gate[0] else 1, H if gate[1] else 1, BF16 if H == 512 else F32)
    check(m, rows(T, H, BF16), h=rows(T, H, F32), post_w=rows(1, H, F32)[0], pre_w=rows(1, H, F32)[0], gate=g, gate_act=act,
          alpha=0.3, beta=0.7, w_offset=1.0, eps=1e-3)


@pytest.mark.parametrize("T,H", [(1300, 4096), (2600, 2088), (700, 8192), (20000, 128), (9001, 264), (40003, 64), (700, 8200)])
@pytest.mark.parametrize("ydt,hdt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_many_rows(m, T, H, ydt, hdt):
    torch.manual_seed(T)
    y, h, pre, post = rows(T, H, ydt), rows(T, H, hdt, 8), rows(1, H, BF16)[0], rows(1, H, BF16)[0]
    check(m, y, h=h, pre_w=pre)
    check(m, y, h=h, post_w=post, pre_w=pre, gate=rows(1, H, BF16), gate_act="silu", alpha=0.5, beta=0.25, w_offset=1.0)
    check(m, y, h=h, post_w=post, gate=rows(T, H, F32), gate_act="sigmoid")
    check(m, y, post_w=post, pre_w=pre, gate=rows(T, 1, BF16), h_out=False)
    check(m, y, h=h, gate=rows(1, 1, BF16), n_out=False)


@pytest.mark.parametrize("slots", [1, 2, 9, 11, 64])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slots(m, slots, dtype):
    torch.manual_seed(slots)
    check(m, rows(13 * slots, 384, dtype), slots=slots, h=rows(13, 384, BF16), pre_w=rows(1, 384, BF16)[0])


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (4, 4), (3, 0), (0, 1), (5, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_wider_tensors(m, pad, shift, dtype):
    torch.manual_seed(pad)
    T, H = 19, 320
    h_out, n_out = rows(T, H, dtype, pad, shift), rows(T, H, BF16, pad, shift)
    wide_h, wide_n = h_out._base.clone(), n_out._base.clone()
    check(m, rows(T, H, dtype, pad, shift), h=rows(T, H, dtype, pad, shift), gate=rows(T, H, dtype, pad, shift),
          pre_w=rows(1, H + shift, BF16)[0, shift:].clone(), h_out=h_out, n_out=n_out)
    # what lies beside the rows is as it was
    for out, was in ((h_out, wide_h), (n_out, wide_n)):
        base = out._base
        assert torch.equal(base[:, :shift], was[:, :shift]) and torch.equal(base[:, shift + H:], was[:, shift + H:])


def test_outputs_left_out_and_weights_of_one(m):
    y, h = rows(6, 256, BF16), rows(6, 256, F32)
    a = check(m, y, h=h, n_out=False)[0]
    b = check(m, y, h=h, h_out=False)[1]
    both = check(m, y, h=h)
    assert torch.equal(a, both[0]) and torch.equal(b, both[1])
    check(m, y, h_dtype=F32, n_dtype=F32)  # no residual
    check(m, y, alpha=-2.0, beta=float("nan"))  # which is not used without one


def test_in_place(m):
    y, h, w = rows(9, 640, BF16), rows(9, 640, F32), rows(1, 640, BF16)[0]
    want = m.moe_combine_norm(y, h=h, pre_w=w, post_w=w)
    m.moe_combine_norm(y, h=h, pre_w=w, post_w=w, h_out=h, n_out=y)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


def test_rows_do_not_mix(m):
    y, h, w = rows(8, 512, BF16), rows(8, 512, BF16), rows(1, 512, BF16)[0]
    want = m.moe_combine_norm(y, h=h, pre_w=w, post_w=w)
    y[2, 5], y[4] = float("nan"), float("inf")
    got = m.moe_combine_norm(y, h=h, pre_w=w, post_w=w)
    for a, b in zip(got, want):
        assert torch.isnan(a[2]).all() and torch.isnan(a[4]).all()
        keep = [0, 1, 3, 5, 6, 7]
        assert torch.equal(a[keep], b[keep])
    # zeros have a norm of zero
    z = torch.zeros((2, 512), dtype=BF16, device="cuda")
    assert not m.moe_combine_norm(z, post_w=w, pre_w=w)[1].any()


def test_no_tokens(m):
    h, n = m.moe_combine_norm(rows(0, 64, BF16), pre_w=rows(1, 64, BF16)[0])
    assert h.shape == n.shape == (0, 64)


def test_rows_past_32_bits(m):
    T, H = (1 << 31) // 8192 + 40, 8192
    y = torch.zeros((T, H), dtype=BF16, device="cuda")
    tail = rows(50, H, BF16)
    y[-50:] = tail
    h, n = m.moe_combine_norm(y)
    a, b = m.moe_combine_norm(tail)
    assert torch.equal(h[-50:], a) and torch.equal(n[-50:], b) and not n[:-50].any()


def test_graph_replay(m):
    y, h, w = rows(7 * 3, 768, F32), rows(7, 768, BF16), rows(1, 768, BF16)[0]
    ho, no = torch.empty_like(h), torch.empty_like(h)
    run = lambda: m.moe_combine_norm(y, h=h, slots=3, pre_w=w, h_out=ho, n_out=no)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        y.normal_()
        g.replay()
        got = ho.clone(), no.clone()
        run()
        assert torch.equal(got[0], ho) and torch.equal(got[1], no)
