"""moe_linear_mxfp4act's checks of its arguments.  CPU only: no call here
reaches a CUDA kernel."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    return libmoe


def test_refusals(m):
    lib, nul, fake = m.load(), ctypes.c_void_p(0), ctypes.c_void_p(0x1000)

    def call(x=fake, xt=0, ldx=None, w=fake, s=fake, res=nul, ldr=0, out=fake, ot=0, ldo=None, T=4, N=100,
             K=256, ws=fake, n=1 << 30):
        return lib.moe_linear_mxfp4act(x, xt, K if ldx is None else ldx, w, s, res, ldr, out, ot,
                                       N if ldo is None else ldo, T, N, K, ws, n, nul)
    bad, shape = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=0) == m.MOE_OK  # nothing to do
    assert call(T=-1) == bad and call(N=0) == bad and call(K=0) == bad
    assert call(xt=2) == bad and call(ot=-1) == bad
    assert call(K=48) == shape and call(K=65568) == shape
    assert call(N=(1 << 24) + 1) == shape and call(T=(1 << 20) + 1) == shape
    for name in ("x", "w", "s", "out", "ws"):
        assert call(**{name: nul}) == bad, name
    assert call(w=ctypes.c_void_p(0x1008)) == bad and call(ws=ctypes.c_void_p(0x1008)) == bad
    assert call(s=ctypes.c_void_p(0x1002)) == bad
    assert call(x=ctypes.c_void_p(0x1001)) == bad and call(x=ctypes.c_void_p(0x1002), xt=1) == bad
    assert call(out=ctypes.c_void_p(0x1002), ot=1) == bad
    assert call(res=ctypes.c_void_p(0x1001), ldr=100) == bad
    assert call(ldx=-1) == bad and call(ldo=99) == bad and call(res=fake, ldr=-1) == bad
    assert call(n=64) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    need = m.moe_linear_mxfp4act_workspace_size(4, 100, 256)
    assert call(n=need - 1) == m.MOE_ERR_WORKSPACE_TOO_SMALL


def test_workspace_sizes(m):
    size = m.moe_linear_mxfp4act_workspace_size
    for T, N, K in ((1, 4096, 4096), (16, 100003, 4096), (1536, 4096, 4096), (8192, 8192, 4096)):
        assert size(T, N, K) >= T * K // 2 + T * K // 32  # x's codes and scales
    assert size(0, 8, 32) == 0
    for T, N, K in ((-1, 8, 32), (1, 0, 32), (1, 8, 40), (1, 8, 0), (1, 8, 65568)):
        assert size(T, N, K) == 0
