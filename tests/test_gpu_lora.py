"""moe_lora against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def rows(T, n, dtype, pad=0, shift=0):
    return torch.randn((T, n + pad + shift), device="cuda").to(dtype)[:, shift:shift + n]


def adapters(n, N, K, R):
    a = (torch.randn((n, R, K), device="cuda") / K ** 0.5).bfloat16()
    b = (torch.randn((n, N, R), device="cuda") / R ** 0.5).bfloat16()
    return a, b, 0.25 + torch.rand(n, device="cuda")


def check(m, x, a, b, ids, tile=None, scale=None, ranks=None, residual=None, out=None, out_dtype=None):
    n, N, R = b.shape
    T, K = x.shape
    if out is not None and residual is out:  # in place: the formula needs what was there
        base = out.clone()
    else:
        base = residual
    plan = m.moe_lora_plan(ids, n, tile)
    got = m.moe_lora(x, a, b, plan, scale=scale, ranks=ranks, residual=residual, out=out, out_dtype=out_dtype)
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda") if base is None else base.double().clone()
    size = want.abs()
    inner = torch.zeros_like(want)
    for e in range(n):
        mine = (ids == e).nonzero()[:, 0]
        if not len(mine):
            continue
        r = R if ranks is None else int(ranks[e])
        A, B, s = a[e, :r].double(), b[e, :, :r].double(), 1.0 if scale is None else float(scale[e])
        v, vmag = x[mine].double() @ A.T, x[mine].double().abs() @ A.abs().T
        want[mine] += s * (v @ B.T)
        size[mine] += abs(s) * (vmag @ B.abs().T)
        inner[mine] = abs(s) * (v.abs() @ B.abs().T)
    # an accumulator takes two steps for 32 of K, three times that for an fp32 x, 16 joins, and two for 32 of R and
    # each of three terms, each good to 2^-23 of what is summed, twice that for what an MMA adds at once
    steps = (6 if x.dtype == F32 else 2) * ((K + 31) // 32) + 16 + 6 * ((R + 31) // 32) + 4
    half, term = (2.0 ** -8, 2.0 ** -16) if got.dtype == BF16 else (2.0 ** -24, 2.0 ** -24)
    err = (got.double() - want).abs()
    assert (err <= half * want.abs() + term * inner + steps * 2.0 ** -22 * size + 1e-38).all(), (err / (size + 1e-30)).max()
    return got, plan


def ids_of(T, n, without=0.0, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    ids = torch.randint(0, n, (T,), generator=g, dtype=torch.int32)
    ids[torch.rand(T, generator=g) < without] = -1
    return ids.cuda()


@pytest.mark.parametrize("T,n,N,K,R", [
    (1, 1, 4096, 4096, 16), (1, 5, 8, 8, 8), (2, 3, 33, 40, 8), (16, 1, 100, 64, 16), (17, 2, 1000, 1056, 24), (64, 64, 256, 512, 16),
    (100, 7, 31, 2048, 32), (33, 4, 640, 136, 40), (257, 3, 96, 264, 64), (70, 70, 128, 128, 128), (300, 2, 72, 8192, 104),
    (1, 1, 1, 8, 8), (1100, 3, 264, 512, 16), (4200, 5, 136, 96, 64),
])
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
def test_against_the_formula(m, T, n, N, K, R, tile):
    torch.manual_seed(T + N)
    a, b, scale = adapters(n, N, K, R)
    check(m, rows(T, K, BF16), a, b, ids_of(T, n), tile, scale, residual=rows(T, N, BF16))


@pytest.mark.parametrize("x,out", [(BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
def test_types_and_ranks(m, x, out, R, tile):
    torch.manual_seed(R)
    a, b, scale = adapters(3, 200, 320, R)
    check(m, rows(90, 320, x), a, b, ids_of(90, 3), tile, scale, residual=rows(90, 200, out), out_dtype=out)
    check(m, rows(90, 320, x), a, b, ids_of(90, 3), tile, out_dtype=out)


@pytest.mark.parametrize("T,n,N,K,R", [
    (128, 1, 128, 64, 16), (1, 1, 8, 8, 8), (129, 1, 64, 128, 64), (300, 3, 1032, 1032, 8), (500, 2, 4096, 4096, 64),
    (1000, 5, 136, 2048, 128), (2100, 3, 2048, 520, 40), (777, 40, 320, 256, 24), (256, 2, 8192, 16, 96), (640, 1, 16, 8192, 104),
    (3000, 2, 72, 72, 120), (130, 2, 1024, 4104, 48),
])
@pytest.mark.parametrize("out", [BF16, F32])
def test_prompts(m, T, n, N, K, R, out):
    """Tiles of 128 tokens, with tokens of one adapter together and apart, and without one."""
    torch.manual_seed(T)
    a, b, scale = adapters(n, N, K, R)
    x, res = rows(T, K, BF16, 8), rows(T, N, out, 8, 8)
    for ids in (ids_of(T, n, 0.1), ids_of(T, n).sort()[0]):
        got, plan = check(m, x, a, b, ids, 128, scale, residual=res, out_dtype=out)
        assert torch.equal(m.moe_lora(x, a, b, plan, scale=scale, residual=res, out_dtype=out), got)
    check(m, x, a, b, ids, 128, out_dtype=out)
    check(m, x, a, b, ids, 128, scale, residual=res, out=res)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 0), (0, 1), (4, 4), (2, 2), (6, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_wider_tensors(m, pad, shift, dtype):
    torch.manual_seed(pad)
    T, N, K = 45, 120 - pad, 96
    a, b, scale = adapters(4, N, K, 16)
    out = rows(T, N, dtype, pad, shift)
    was = out._base.clone()
    check(m, rows(T, K, dtype, pad, shift), a, b, ids_of(T, 4, 0.3), scale=scale, residual=rows(T, N, dtype, pad, shift), out=out)
    base = out._base
    assert torch.equal(base[:, :shift], was[:, :shift]) and torch.equal(base[:, shift + N:], was[:, shift + N:])
    # one row for every token
    check(m, rows(1, K, dtype, pad, shift).expand(T, -1), a, b, ids_of(T, 4), residual=rows(1, N, dtype, pad).expand(T, -1),
          out_dtype=dtype)


@pytest.mark.parametrize("T", [5, 700])
def test_tokens_without_an_adapter(m, T):
    a, b, scale = adapters(6, 150, 64, 8)
    x, res, ids = rows(T, 64, BF16), rows(T, 150, BF16), ids_of(T, 6, 0.5, 7)
    ids[0], ids[1], ids[2] = -1, 6, 1 << 30  # outside the range either way
    none = (ids < 0) | (ids >= 6)
    got, plan = check(m, x, a, b, ids, scale=scale, residual=res)
    assert torch.equal(got[none], res[none])
    assert not check(m, x, a, b, ids, scale=scale)[0][none].any()
    check(m, x, a, b, ids, scale=scale, residual=res, out=res)  # in place
    assert torch.equal(res, got)
    # nobody has one
    nobody = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(check(m, x, a, b, nobody, scale=scale, residual=res)[0], res)


def test_ranks_of_their_own(m):
    """What lies behind an adapter's rank plays no part, not even as NaN."""
    for R in (16, 40, 128):
        a, b, scale = adapters(5, 100, 72, R)
        ranks = torch.tensor([R, 1, 7, 0, R - 1], dtype=torch.int32, device="cuda")
        for e, r in enumerate(ranks.tolist()):
            a[e, r:] = float("nan")
            b[e, :, r:] = float("inf")
        check(m, rows(80, 72, BF16), a, b, ids_of(80, 5), scale=scale, ranks=ranks, residual=rows(80, 100, BF16))
        check(m, rows(80, 72, F32), a, b, ids_of(80, 5), 64, ranks=ranks, out_dtype=F32)
        # out of range: clamped
        wild = torch.tensor([R + 5, 1, 7, -3, R - 1], dtype=torch.int32, device="cuda")
        check_same = [m.moe_lora(rows(1, 72, BF16).expand(5, -1) * 0 + 1, a, b, m.moe_lora_plan(ids_of(5, 5), 5), ranks=q)
                      for q in (ranks, wild)]
        assert torch.equal(*check_same)


def test_tokens_do_not_mix(m):
    """Another token's infinities and NaN, and which tokens share a tile, change nothing."""
    for dtype, tile in ((BF16, 16), (F32, 16), (BF16, 128)):
        a, b, scale = adapters(2, 96, 128, 16)
        x, ids = rows(50, 128, dtype), ids_of(50, 2)
        want, plan = check(m, x, a, b, ids, tile, scale=scale)
        x[7, 3], x[8], x[9] = float("nan"), float("inf"), -3e38
        got = m.moe_lora(x, a, b, plan, scale=scale)
        keep = [t for t in range(50) if t not in (7, 8, 9)]
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[7]).all() and not torch.isfinite(got[8]).any()
        order = torch.randperm(50, device="cuda")
        assert torch.equal(m.moe_lora(x[order].contiguous(), a, b, m.moe_lora_plan(ids[order].contiguous(), 2, tile), scale=scale)[
            order.argsort()][keep], want[keep])


def test_a_plan_serves_several_projections(m):
    ids = ids_of(40, 3, 0.2)
    plan = m.moe_lora_plan(ids, 3)
    for N, K, R in ((64, 128, 8), (300, 256, 32)):
        a, b, scale = adapters(3, N, K, R)
        x = rows(40, K, BF16)
        assert torch.equal(m.moe_lora(x, a, b, plan, scale=scale), check(m, x, a, b, ids, scale=scale)[0])
    assert m.moe_lora(rows(0, 256, BF16), a, b, m.moe_lora_plan(ids[:0], 3)).shape == (0, 300)


def test_a_bad_plan_is_reported(m):
    """Entries that moe_permute never makes: the work is skipped and the flag raised.  (The kernel
    compares each with its range before it uses it.)"""
    a, b, _ = adapters(3, 64, 64, 8)
    x, res = rows(20, 64, BF16), rows(20, 64, BF16)
    for tile in (16, 128):
        for key, value in (("tile_expert", 3), ("tile_expert", -1), ("sorted_pairs", 20), ("num_tiles", 1 << 20), ("num_tiles", -1)):
            plan = m.moe_lora_plan(ids_of(20, 3), 3, tile)
            plan[key][0] = value
            m.moe_lora(x, a, b, plan, residual=res)
            assert m.moe_device_error() == 2, key
            assert m.moe_device_error() == 0


def test_offsets_past_32_bits(m):
    """An adapter pool of more than 2^31 elements, and rows further apart than that in all."""
    n, N, K, R = 300, 65536 + 8, 65536, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.zeros((n, R, K), dtype=BF16, device="cuda")
    b = torch.zeros((n, N, R), dtype=BF16, device="cuda")
    a[-1] = torch.randn((R, K), device="cuda", generator=g) / 256
    b[-1] = torch.randn((N, R), device="cuda", generator=g) / 11
    ids = torch.tensor([n - 1, 0, n - 1], dtype=torch.int32, device="cuda")
    x = rows(3, K, BF16)
    want = m.moe_lora(x, a[-1:].contiguous(), b[-1:].contiguous(), m.moe_lora_plan(ids - (n - 1), 1, 16))
    got = m.moe_lora(x, a, b, m.moe_lora_plan(ids, n, 16))
    assert torch.equal(got, want) and not got[1].any() and got[0].any()
    del a, b
    T, N, K = 70000, 32768, 64
    a, b, _ = adapters(2, N, K, 8)
    x = rows(T, K, BF16)
    ids = torch.full((T,), 0, dtype=torch.int32, device="cuda")
    ids[-40:] = 1
    got = m.moe_lora(x, a, b, m.moe_lora_plan(ids, 2, 16))
    assert torch.equal(got[-40:], m.moe_lora(x[-40:], a, b, m.moe_lora_plan(ids[-40:].clone(), 2, 16)))


def test_graphs_and_streams_side_by_side(m):
    """A captured call follows its inputs, the grouping among them; two streams run at once."""
    T, n, N, K, R = 48, 6, 512, 768, 16
    a, b, scale = adapters(n, N, K, R)
    x, res, out, ids = rows(T, K, BF16), rows(T, N, BF16), rows(T, N, BF16), ids_of(T, n)
    plan = m.moe_lora_plan(ids, n)

    def step():
        m.moe_lora_plan(ids, n, out=plan)
        m.moe_lora(x, a, b, plan, scale=scale, residual=res, out=out)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        x.normal_()
        ids.copy_(ids_of(T, n, 0.2, i))
        g.replay()
        got = out.clone()
        assert torch.equal(got, m.moe_lora(x, a, b, m.moe_lora_plan(ids, n), scale=scale, residual=res))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        outs[0].append(m.moe_lora(x, a, b, plan, scale=scale, residual=res))
        outs[1].append(m.moe_lora(x, a, b, plan, scale=scale, residual=res, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(o, got) for both in outs for o in both)
