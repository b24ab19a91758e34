"""What a call allocates for itself belongs to the stream that it runs on.  CPU only: the library and
the stream switch are stand-ins, the tensors live on the host and only say that they are on a GPU."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def recorded(monkeypatch):
    """libmoe with a library whose calls do nothing, and the list of (allocator, stream that was
    current) of every allocation."""
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    real = libmoe.load()
    current, made = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "zeros", "empty_like", "full"):
        def allocate(*args, _name=name, _real=getattr(torch, name), **kw):
            made.append((_name, current[0]))
            kw.pop("device", None)
            return gpu(_real(*args, **kw))
        monkeypatch.setattr(torch, name, allocate)

    class Library:
        def __getattr__(self, name):
            # sizes are asked of the library itself, everything else would launch
            return getattr(real, name) if name.endswith(("_size", "_capacity", "_max_tiles")) else lambda *a: 0
    monkeypatch.setattr(libmoe, "_lib", Library())
    return libmoe, made


SIDE = types.SimpleNamespace(cuda_stream=0x1234)


def rand(*shape, dtype=torch.bfloat16):
    return gpu(torch.zeros(shape).to(dtype))


def few(E=8, T=2, H=64, I=32):
    u8 = torch.uint8
    return dict(x=rand(T, H), w_router=rand(E, H), w13=rand(E + 1, 2 * I, H // 2, dtype=u8),
                s13=rand(E + 1, 2 * I, H // 32, dtype=u8), w2=rand(E + 1, H, I // 2, dtype=u8),
                s2=rand(E + 1, H, I // 32, dtype=u8), K=2)


def linear(T=2, N=16, K=64):
    return dict(x=rand(T, K), codes=rand(N, K // 2, dtype=torch.uint8), scales=rand(N, K // 32, dtype=torch.uint8))


@pytest.mark.parametrize("name,args,allocations", [("moe_layer_few", few, 4), ("moe_linear_mxfp4act", linear, 2)])
def test_the_calls_own_buffers(recorded, name, args, allocations):
    libmoe, made = recorded
    args = args()
    made.clear()
    getattr(libmoe, name)(**args, stream=SIDE)
    assert len(made) == allocations and all(s is SIDE for _, s in made), made
    if name == "moe_layer_few":  # its workspace is zeroed in the kernel's stream too
        assert ("zeros", SIDE) in made


T, H, I, E, K = 2, 64, 32, 8, 2


def layer():
    f = few(E, T, H, I)
    del f["w_router"]
    return dict(f, logits=rand(T, E, dtype=torch.float32))


def ffn(libmoe):
    f = layer()
    del f["logits"], f["K"]
    return dict(f, topk_w=rand(T, K + 1, dtype=torch.float32), perm=libmoe.alloc_permute(T, K + 1, E + 1, 8))


def dense(libmoe):
    f = ffn(libmoe)
    return dict(f, **{n + "s": f[n][0] for n in ("w13", "s13", "w2", "s2")})


@pytest.mark.parametrize("name,args", [
    ("moe_route", lambda m: dict(logits=rand(T, E, dtype=torch.float32), K=K)),
    ("moe_route_permute", lambda m: dict(logits=rand(T, E, dtype=torch.float32), K=K, tile_m=8)),
    ("moe_permute", lambda m: dict(topk_ids=rand(T, K, dtype=torch.int32), Et=E, tile_m=8)),
    ("moe_ffn", ffn), ("moe_ffn_noalloc", ffn), ("moe_ffn_mxfp4act", ffn), ("moe_ffn_dense_shared", dense),
    ("moe_layer", lambda m: layer()),
    ("moe_split_e4m3x2", lambda m: dict(x=rand(T, H))), ("moe_quantize_mxfp4", lambda m: dict(x=rand(T, H))),
    ("moe_selftest_wait_split", lambda m: {}),
])
def test_the_other_calls_own_buffers(recorded, name, args):
    libmoe, made = recorded
    args = args(libmoe)
    made.clear()
    getattr(libmoe, name)(**args, stream=SIDE)
    assert made and all(s is SIDE for _, s in made), made


def given(libmoe, name):
    """Arguments with every buffer among them."""
    u8, bf16 = torch.uint8, torch.bfloat16
    ids, w = rand(T, K + 1, dtype=torch.int32), rand(T, K + 1, dtype=torch.float32)
    perm, ws, out = libmoe.alloc_permute(T, K + 1, E + 1, 8), rand(1 << 20, dtype=u8), rand(T, H)
    return {
        "moe_route": dict(logits=rand(T, E, dtype=torch.float32), K=K, topk_ids=ids, topk_w=w),
        "moe_route_permute": dict(logits=rand(T, E, dtype=torch.float32), K=K, tile_m=8, topk_ids=ids, topk_w=w, perm=perm),
        "moe_ffn": dict(ffn(libmoe), out=out, workspace=ws), "moe_ffn_mxfp4act": dict(ffn(libmoe), out=out, workspace=ws),
        "moe_ffn_dense_shared": dict(dense(libmoe), out=out, workspace=ws),
        "moe_quantize_mxfp4": dict(x=rand(T, H), codes=rand(T, H // 2, dtype=u8), scales=rand(T, H // 32, dtype=u8)),
        "moe_layer_few": dict(few(E, T, H, I), out=out, topk_ids=ids, topk_w=w, workspace=ws),
        "moe_linear_mxfp4act": dict(linear(T, 16, H), out=rand(T, 16, dtype=bf16), workspace=ws),
    }[name]


@pytest.mark.parametrize("name", ["moe_route", "moe_route_permute", "moe_ffn", "moe_ffn_mxfp4act", "moe_ffn_dense_shared",
                                  "moe_quantize_mxfp4", "moe_layer_few", "moe_linear_mxfp4act"])
def test_no_stream_switch_when_everything_is_given(recorded, monkeypatch, name):
    """A call that allocates nothing does not pay for a switch."""
    libmoe, made = recorded
    args = given(libmoe, name)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: pytest.fail("switched"))
    made.clear()
    getattr(libmoe, name)(**args, stream=SIDE)
    assert not made
