"""What moe_route_grouped, moe_lora and moe_combine_norm refuse.  CPU only: no call here reaches a
CUDA kernel."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_stream_argument import SIDE, gpu, rand, recorded  # noqa: E402,F401

NUL, FAKE, ODD = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    return libmoe


def test_route_grouped(m):
    def call(l=FAKE, lt=1, ld=None, b=NUL, sw=NUL, T=4, E=64, K=8, score=1, G=8, Gk=4, top=2, shared=0, ids=FAKE, w=FAKE):
        return m.load().moe_route_grouped(l, lt, E if ld is None else ld, b, sw, T, E, K, score, G, Gk, top, shared, 1, 1.0,
                                          ids, w, NUL)
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=0) == m.MOE_OK
    assert call(T=-1) == bad and call(E=0) == bad and call(K=0) == bad and call(G=0) == bad and call(Gk=0) == bad
    assert call(lt=2) == bad and call(score=2) == bad and call(score=-1) == bad and call(top=0) == bad and call(top=3) == bad
    assert call(ld=-1) == bad
    assert call(E=1032) == shape and call(K=33, G=1, Gk=1) == shape and call(E=60) == shape  # 60 % 8
    assert call(E=66, G=33) == shape and call(Gk=9) == shape and call(K=33) == shape
    assert call(E=8, K=4) == shape  # groups of one expert have no second largest
    assert call(E=64, G=16, Gk=1, K=5) == shape  # four experts stay
    for name in ("l", "ids", "w"):
        assert call(**{name: NUL}) == bad and call(**{name: ctypes.c_void_p(0x1002)}) == bad, name
    assert call(l=ODD, lt=0) == bad and call(b=ODD) == bad and call(sw=ODD, shared=1) == bad
    assert call(sw=FAKE) == bad  # a weight for a slot that is not there


def test_lora(m):
    def call(x=FAKE, xt=0, ldx=None, a=FAKE, b=FAKE, sc=NUL, rk=NUL, sp=FAKE, iv=FAKE, te=FAKE, nt=FAKE, tile=16, n=4,
             res=NUL, ldr=0, out=FAKE, ot=0, ldo=None, T=4, N=100, K=64, R=16):
        return m.load().moe_lora(x, xt, K if ldx is None else ldx, a, b, sc, rk, sp, iv, te, nt, tile, n, res, ldr, out, ot,
                                 N if ldo is None else ldo, T, N, K, R, NUL)
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=0) == m.MOE_OK
    for name in ("N", "K", "R", "n"):
        assert call(**{name: 0}) == bad, name
    assert call(T=-1) == bad and call(xt=2) == bad and call(ot=-1) == bad
    assert call(K=60) == shape and call(K=65544) == shape and call(R=12) == shape and call(R=136) == shape
    assert call(N=(1 << 24) + 1) == shape and call(T=(1 << 20) + 1) == shape and call(n=1026) == shape
    for tile in (0, 8, 24, 96, 256):
        assert call(tile=tile) == shape
    for name in ("x", "a", "b", "sp", "iv", "te", "nt", "out"):
        assert call(**{name: NUL}) == bad and call(**{name: ODD}) == bad, name
    assert call(a=ctypes.c_void_p(0x1008)) == bad and call(b=ctypes.c_void_p(0x1008)) == bad
    assert call(sc=ODD) == bad and call(rk=ODD) == bad and call(res=ODD, ldr=100) == bad
    assert call(x=ctypes.c_void_p(0x1002), xt=1) == bad and call(out=ctypes.c_void_p(0x1002), ot=1) == bad
    assert call(ldx=-1) == bad and call(ldo=99) == bad and call(res=FAKE, ldr=-1) == bad


def test_lora_tile_heights(m):
    for T in (0, 1, 16, 100, 1000, 5000, 1 << 20):
        for n in (1, 7, 64, 1025):
            assert m.moe_lora_tile_m(T, n) in (16, 32, 64, 128)
    assert m.load().moe_lora_tile_m(-1, 4) == 0 and m.load().moe_lora_tile_m(4, 0) == 0


def test_combine_norm(m):
    def call(y=FAKE, yt=0, ldy=64, slots=1, post=0, pw=NUL, w=FAKE, wt=0, g=NUL, gt=0, ldg=0, cols=64, act=0, h=FAKE, ldh=64,
             ho=FAKE, ht=0, ldho=64, no=FAKE, nt=0, ldn=64, T=4, H=64):
        return m.load().moe_combine_norm(y, yt, ldy, slots, post, pw, w, wt, 0.0, 1e-6, g, gt, ldg, cols, act, h, ldh, 1.0, 1.0,
                                         ho, ht, ldho, no, nt, ldn, T, H, NUL)
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=0) == m.MOE_OK
    assert call(T=-1) == bad and call(H=0) == bad and call(slots=0) == bad
    for name in ("yt", "wt", "gt", "ht", "nt"):
        assert call(**{name: 2}) == bad and call(**{name: -1}) == bad, name
    assert call(act=3) == bad and call(act=-1) == bad
    assert call(H=16385, ldho=16385, ldn=16385) == shape and call(slots=65) == shape
    assert call(y=NUL) == bad and call(ho=NUL, no=NUL) == bad
    for name in ("y", "pw", "w", "g", "h", "ho", "no"):
        assert call(**{name: ODD}) == bad, name
    assert call(post=1) == bad  # a norm without its weights
    assert call(g=FAKE, cols=2) == bad
    assert call(ldy=-1) == bad and call(ldh=-1) == bad and call(g=FAKE, ldg=-1) == bad
    assert call(ldho=63) == bad and call(ldn=63) == bad


# ------------------------------------------------------------ the bindings

def route_args():
    return dict(logits=rand(3, 16, dtype=torch.float32), K=2, n_groups=4, topk_groups=2)


def lora_args(m, out=False):
    plan = dict(m.alloc_permute(3, 1, 2, 16))
    return dict(x=rand(3, 64), a=rand(2, 8, 64), b=rand(2, 32, 8), plan=plan, **({"out": rand(3, 32)} if out else {}))


def norm_args():
    return dict(y=rand(3, 64), h=rand(3, 64), pre_w=rand(64))


def test_own_buffers_are_made_in_the_calls_stream(recorded):  # noqa: F811
    m, made = recorded
    for name, args, n in (("moe_route_grouped", route_args(), 2), ("moe_lora", lora_args(m), 1),
                          ("moe_combine_norm", norm_args(), 2),
                          ("moe_lora_plan", dict(adapter_ids=rand(3, dtype=torch.int32), adapters=2), 5)):
        made.clear()
        getattr(m, name)(**args, stream=SIDE)
        assert len(made) == n and all(s is SIDE for _, s in made), (name, made)


def test_no_stream_switch_when_everything_is_given(recorded, monkeypatch):  # noqa: F811
    m, made = recorded
    cases = [("moe_route_grouped", dict(route_args(), with_shared=False, topk_ids=rand(3, 2, dtype=torch.int32),
                                        topk_w=rand(3, 2, dtype=torch.float32))),
             ("moe_lora", lora_args(m, True)), ("moe_combine_norm", dict(norm_args(), h_out=rand(3, 64), n_out=False))]
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("switched"))
    made.clear()
    for name, args in cases:
        getattr(m, name)(**args, stream=SIDE)
    assert not made


def test_bindings_refuse(recorded):  # noqa: F811
    m, _ = recorded
    r, lo, n = route_args(), lora_args(m, True), norm_args()
    f32, i32 = torch.float32, torch.int32
    for name, args in (
            ("moe_route_grouped", dict(r, logits=rand(3, 16, dtype=torch.float16))),
            ("moe_route_grouped", dict(r, logits=torch.ones(3, 16))),  # on the host
            ("moe_route_grouped", dict(r, logits=gpu(torch.zeros(16, 3).t()))),
            ("moe_route_grouped", dict(r, bias=rand(15, dtype=f32))),
            ("moe_route_grouped", dict(r, bias=rand(16))),
            ("moe_route_grouped", dict(r, shared_w=rand(4, dtype=f32))),
            ("moe_route_grouped", dict(r, topk_ids=rand(3, 2, dtype=i32))),  # the shared slot is missing
            ("moe_route_grouped", dict(r, topk_ids=rand(3, 3, dtype=f32))),
            ("moe_lora", dict(lo, x=rand(4, 64))), ("moe_lora", dict(lo, x=rand(3, 64, dtype=torch.float16))),
            ("moe_lora", dict(lo, a=rand(2, 8, 32))), ("moe_lora", dict(lo, a=rand(2, 8, 64, dtype=f32))),
            ("moe_lora", dict(lo, b=rand(3, 32, 8))), ("moe_lora", dict(lo, scale=rand(3, dtype=f32))),
            ("moe_lora", dict(lo, ranks=rand(2, dtype=torch.int64))), ("moe_lora", dict(lo, out=rand(3, 33))),
            ("moe_lora", dict(lo, residual=rand(3, 32, dtype=f32))), ("moe_lora", dict(lo, out=torch.ones(3, 32).bfloat16())),
            ("moe_combine_norm", dict(n, slots=2)), ("moe_combine_norm", dict(n, h=rand(2, 64))),
            ("moe_combine_norm", dict(n, h_out=rand(3, 64, dtype=f32))), ("moe_combine_norm", dict(n, pre_w=rand(63))),
            ("moe_combine_norm", dict(n, post_w=rand(64, dtype=f32))), ("moe_combine_norm", dict(n, gate=rand(2, 64))),
            ("moe_combine_norm", dict(n, gate=rand(3, 2))), ("moe_combine_norm", dict(n, y=torch.ones(3, 64))),
    ):
        try:
            getattr(m, name)(**args, stream=SIDE)
        except AssertionError:
            continue
        pytest.fail(f"{name} took {[(k, getattr(v, 'shape', v)) for k, v in args.items()]}")
    ids = rand(3, dtype=i32)
    plan = m.moe_lora_plan(ids, 2, 32, stream=SIDE)
    assert m.moe_lora_plan(ids, 2, out=plan, stream=SIDE) is plan  # keeps its height
    for args in (dict(adapter_ids=rand(4, dtype=i32)), dict(adapters=3), dict(tile_m=16), dict(adapter_ids=rand(3, dtype=torch.int64))):
        with pytest.raises(AssertionError):
            m.moe_lora_plan(**{**dict(adapter_ids=ids, adapters=2, out=plan), **args}, stream=SIDE)
    with pytest.raises(KeyError):
        m.moe_route_grouped(**dict(r, score="relu"), stream=SIDE)
    with pytest.raises(KeyError):
        m.moe_combine_norm(**n, gate_act="relu", stream=SIDE)


def test_direct_calls_are_those_of_the_library(m):
    """The wrappers that skip ctypes pass every argument on: the same refusals, in the same places."""
    lib = m.load()
    p, bad, shape = 0x1000, m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    route = [p, 1, 64, None, None, 4, 64, 8, 1, 8, 4, 2, 0, 1, 1.0, p, p, None]
    lora = [p, 0, 64, p, p, None, None, p, p, p, p, 16, 4, None, 0, p, 0, 100, 4, 100, 64, 16, None]
    norm = [p, 0, 64, 1, 0, None, p, 0, 0.0, 1e-6, None, 0, 0, 64, 0, p, 64, 1.0, 1.0, p, 0, 64, p, 0, 64, 4, 64, None]
    for name, good, changes in (
            ("moe_route_grouped", route, {0: None, 1: 2, 2: -1, 3: 2, 4: p, 5: -1, 6: 0, 7: 0, 8: 2, 9: 7, 10: 9, 11: 3,
                                          15: None, 16: None}),
            ("moe_lora", lora, {0: 1, 1: 2, 2: -1, 3: 8, 4: 8, 5: 1, 6: 1, 7: 1, 8: 1, 9: 1, 10: 1, 11: 8, 12: 1026, 13: 1,
                                15: 1, 16: 2, 17: 99, 18: -1, 19: 0, 20: 60, 21: 12}),
            ("moe_combine_norm", norm, {0: 1, 1: 2, 2: -1, 3: 65, 4: 1, 6: 1, 7: 2, 10: 1, 11: 2, 14: 3, 15: 1, 16: -1, 19: 1,
                                        20: 2, 21: 63, 22: 1, 23: 2, 24: 63, 25: -1, 26: 0})):
        direct, plain = getattr(lib, "direct_" + name), getattr(lib, name)
        for i, v in changes.items():
            args = list(good)
            args[i] = v
            want = plain(*args)
            assert want in (bad, shape) and direct(*args) == want, (name, i)
        with pytest.raises(TypeError):
            direct(*good[:-1])
        with pytest.raises((TypeError, OverflowError)):
            direct(*[1 << 40 if isinstance(v, int) and v == 4 else v for v in good])
        with pytest.raises(TypeError):
            direct("x", *good[1:])
