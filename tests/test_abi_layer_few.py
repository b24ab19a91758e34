"""moe_layer_few's checks of its arguments.  CPU only: no call here reaches a
CUDA kernel."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    return libmoe


def test_refusals(m):
    lib, nul, fake = m.load(), ctypes.c_void_p(0), ctypes.c_void_p(0x1000)

    def call(x=fake, wr=fake, gate=nul, w13=fake, s13=fake, w2=fake, s2=fake, T=4, H=256, I=128, E=8, K=2,
             shared=1, out=fake, ids=fake, w=fake, ws=fake, n=1 << 30):
        return lib.moe_layer_few(x, wr, gate, w13, s13, w2, s2, T, H, I, E, K, shared, 1, out, ids, w, ws, n, nul)
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=0) == m.MOE_OK
    assert call(T=-1) == bad and call(H=0) == bad and call(I=0) == bad and call(E=0) == bad and call(K=0) == bad
    assert call(T=17) == shape and call(H=48) == shape and call(I=80) == shape
    assert call(H=8224) == shape and call(I=8224) == shape
    assert call(E=1025) == shape and call(K=9) == shape and call(E=64, K=33) == shape
    for name in ("x", "wr", "w13", "s13", "w2", "s2", "out", "ws"):
        assert call(**{name: nul}) == bad, name
    for name in ("x", "wr", "w13", "w2", "out", "ws", "gate"):
        assert call(**{name: ctypes.c_void_p(0x1008)}) == bad, name
    for name in ("s13", "s2", "ids", "w"):
        assert call(**{name: ctypes.c_void_p(0x1002)}) == bad, name
    assert call(gate=fake, shared=0) == bad  # a gate without a shared expert
    need = m.moe_layer_few_workspace_size(4, 256, 128, 8, 2, True)
    assert call(n=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib.moe_layer_few_workspace_init(nul, 1 << 20, nul) == bad
    assert lib.moe_layer_few_workspace_init(ctypes.c_void_p(0x1008), 1 << 20, nul) == bad
    assert lib.moe_layer_few_workspace_init(fake, 128, nul) == m.MOE_ERR_WORKSPACE_TOO_SMALL


def test_workspace_sizes(m):
    size = m.moe_layer_few_workspace_size
    # logits, h of every pair in fp32
    assert size(16, 4096, 1024, 512, 10, True) >= 16 * 513 * 4 + 16 * 11 * 1024 * 4
    assert size(16, 4096, 1024, 512, 10, True) > size(16, 4096, 1024, 512, 10, False)
    assert size(17, 4096, 1024, 512, 10, True) == 0 and size(4, 250, 128, 8, 2, True) == 0
