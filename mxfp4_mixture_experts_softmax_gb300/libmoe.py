"""Thin Python binding of the libmoe C ABI (include/moe.h), same entry-point names.

Argument marshalling only: every step runs in libmoe's CUDA kernels.  Torch
is used for device memory and the current stream.  If the shared library is
missing it is compiled with nvcc; if that is impossible the import fails --
there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
import threading

from . import build_lib

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_CUDA = 4
MOE_ERR_INTERNAL = 5

MOE_PATH_AUTO = 0
MOE_PATH_DECODE = 1
MOE_PATH_PREFILL = 2
MOE_PATH_PREFILL_FP8X2 = 3

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F32 = 1

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

MOE_GATE_NONE = 0
MOE_GATE_SIGMOID = 1
MOE_GATE_SILU = 2

EXPORTS = ("moe_status_string", "moe_version", "moe_route", "moe_route_ex", "moe_permute_capacity",
           "moe_permute_max_tiles", "moe_permute", "moe_route_permute", "moe_ffn_workspace_size",
           "moe_ffn",
           "moe_ffn_path", "moe_ffn_auto_path", "moe_ffn_gate_up", "moe_ffn_down", "moe_combine",
           "moe_ffn_y_offset", "moe_device_error", "moe_ffn_noalloc", "moe_combine_ex",
           "moe_ffn_dense_shared_workspace_size", "moe_ffn_dense_shared",
           "moe_selftest_wait_timeout", "moe_selftest_wait_split", "moe_set_gemm_events",
           "moe_quantize_mxfp4", "moe_ffn_mxfp4act_workspace_size",
           "moe_ffn_mxfp4act", "moe_ffn_mxfp4act_gate_up", "moe_ffn_mxfp4act_down",
           "moe_ffn_mxfp4act_h_offsets", "moe_ffn_down_combine", "moe_split_e4m3x2", "moe_ffn_auto_path_shape",
           "moe_linear_mxfp4act_workspace_size", "moe_linear_mxfp4act",
           "moe_layer_few_workspace_size", "moe_layer_few_workspace_init", "moe_layer_few",
           "moe_route_grouped", "moe_lora_tile_m", "moe_lora", "moe_combine_norm")

# bytes of the fixed device scratch behind moe_ffn_noalloc (include/moe.h)
MOE_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
# most tokens of moe_layer_few (include/moe.h)
MOE_LAYER_FEW_MAX_T = 16
# most ranks of an adapter of moe_lora (include/moe.h)
MOE_LORA_MAX_RANK = 128
# batches up to this many tokens route and permute in one launch (include/moe.h)
MOE_ROUTE_PERMUTE_FUSED_MAX_T = 32

_lock = threading.Lock()
_lib = None
_as_is = contextlib.nullcontext()


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib_path() -> str:
    return build_lib.LIB


def load(build: bool = True):
    """Load libmoe.so (building it first if needed) and declare the signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = build_lib.build() if build else build_lib.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libmoe is not built ({path}); run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_status_string.argtypes = [ci]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_version.restype = ci
        L.moe_route.argtypes = [vp, ci, ci, ci, ci, ci, vp, vp, vp]
        L.moe_route.restype = ci
        L.moe_route_ex.argtypes = [vp, vp, ci, ci, ci, ci, ci, vp, vp, vp]
        L.moe_route_ex.restype = ci
        L.moe_route_permute.argtypes = [vp, vp, ci, ci, ci, ci, ci, ci, vp, vp, vp, vp, vp, vp, vp,
                                        vp]
        L.moe_route_permute.restype = ci
        L.moe_permute_capacity.argtypes = [ci, ci, ci, ci]
        L.moe_permute_capacity.restype = sz
        L.moe_permute_max_tiles.argtypes = [ci, ci, ci, ci]
        L.moe_permute_max_tiles.restype = sz
        L.moe_permute.argtypes = [vp, ci, ci, ci, ci, vp, vp, vp, vp, vp, vp]
        L.moe_permute.restype = ci
        L.moe_ffn_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci]
        L.moe_ffn_workspace_size.restype = sz
        ffn_args = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, vp, sz]
        L.moe_ffn.argtypes = ffn_args + [vp]
        L.moe_ffn.restype = ci
        L.moe_ffn_path.argtypes = ffn_args + [ci, vp]
        L.moe_ffn_path.restype = ci
        L.moe_ffn_auto_path.argtypes = [ci, ci, ci, ci]
        L.moe_ffn_auto_path.restype = ci
        L.moe_ffn_auto_path_shape.argtypes = [ci, ci, ci, ci, ci, ci]
        L.moe_ffn_auto_path_shape.restype = ci
        L.moe_ffn_gate_up.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, sz, ci, vp]
        L.moe_ffn_gate_up.restype = ci
        L.moe_ffn_down.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, sz, ci, vp]
        L.moe_ffn_down.restype = ci
        L.moe_combine.argtypes = [vp, ci, ci, ci, vp, vp]
        L.moe_combine.restype = ci
        L.moe_ffn_y_offset.argtypes = [ci, ci, ci, ci, ci]
        L.moe_ffn_y_offset.restype = sz
        L.moe_ffn_noalloc.argtypes = ffn_args[:-2] + [vp]
        L.moe_ffn_noalloc.restype = ci
        L.moe_combine_ex.argtypes = [vp, vp, ci, ci, ci, vp, vp]
        L.moe_combine_ex.restype = ci
        L.moe_ffn_dense_shared_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci]
        L.moe_ffn_dense_shared_workspace_size.restype = sz
        L.moe_ffn_dense_shared.argtypes = (ffn_args[:17] + [vp, vp, vp, vp, ci, vp, vp, vp, sz, vp])
        L.moe_ffn_dense_shared.restype = ci
        L.moe_selftest_wait_timeout.argtypes = [ci, vp]
        L.moe_selftest_wait_timeout.restype = ci
        L.moe_selftest_wait_split.argtypes = [ci, vp, vp]
        L.moe_selftest_wait_split.restype = ci
        L.moe_set_gemm_events.argtypes = [vp, vp]
        L.moe_set_gemm_events.restype = ci
        L.moe_ffn_down_combine.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, vp,
                                           sz, ci, vp]
        L.moe_ffn_down_combine.restype = ci
        L.moe_quantize_mxfp4.argtypes = [vp, ci, ci, vp, vp, vp]
        L.moe_quantize_mxfp4.restype = ci
        L.moe_split_e4m3x2.argtypes = [vp, ci, ci, vp, vp, vp, vp, vp]
        L.moe_split_e4m3x2.restype = ci
        L.moe_ffn_mxfp4act_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci]
        L.moe_ffn_mxfp4act_workspace_size.restype = sz
        L.moe_ffn_mxfp4act.argtypes = ffn_args + [vp]
        L.moe_ffn_mxfp4act.restype = ci
        L.moe_ffn_mxfp4act_gate_up.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp, sz,
                                               vp]
        L.moe_ffn_mxfp4act_gate_up.restype = ci
        L.moe_ffn_mxfp4act_down.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp,
                                            vp, sz, vp]
        L.moe_ffn_mxfp4act_down.restype = ci
        L.moe_ffn_mxfp4act_h_offsets.argtypes = [ci, ci, ci, ci, ci, ci, vp, vp]
        L.moe_ffn_mxfp4act_h_offsets.restype = ci
        i64 = ctypes.c_int64
        L.moe_linear_mxfp4act_workspace_size.argtypes = [ci, ci, ci]
        L.moe_linear_mxfp4act_workspace_size.restype = sz
        L.moe_linear_mxfp4act.argtypes = [vp, ci, i64, vp, vp, vp, i64, vp, ci, i64, ci, ci, ci, vp, sz,
                                          vp]
        L.moe_linear_mxfp4act.restype = ci
        L.moe_layer_few_workspace_size.argtypes = [ci] * 6
        L.moe_layer_few_workspace_size.restype = sz
        L.moe_layer_few_workspace_init.argtypes = [vp, sz, vp]
        L.moe_layer_few_workspace_init.restype = ci
        L.moe_layer_few.argtypes = [vp] * 7 + [ci] * 7 + [vp, vp, vp, vp, sz, vp]
        L.moe_layer_few.restype = ci
        cf = ctypes.c_float
        L.moe_route_grouped.argtypes = [vp, ci, i64, vp, vp] + [ci] * 9 + [cf, vp, vp, vp]
        L.moe_route_grouped.restype = ci
        L.moe_lora_tile_m.argtypes = [ci, ci]
        L.moe_lora_tile_m.restype = ci
        L.moe_lora.argtypes = [vp, ci, i64, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, vp, i64, vp, ci, i64, ci, ci, ci, ci, vp]
        L.moe_lora.restype = ci
        L.moe_combine_norm.argtypes = [vp, ci, i64, ci, ci, vp, vp, ci, cf, cf, vp, ci, i64, ci, ci, vp, i64, cf, cf,
                                       vp, ci, i64, vp, ci, i64, ci, ci, vp]
        L.moe_combine_norm.restype = ci
        L.moe_device_error.argtypes = [vp, ci]
        L.moe_device_error.restype = ci
        # the same functions without ctypes' conversion of every argument (csrc/pycall.c), or with it
        # where there is no such module for this interpreter
        try:
            spec = importlib.util.spec_from_file_location("_pycall", build_lib.PYCALL)
            direct = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(direct)
        except ImportError:
            direct = None
        for name in ("moe_route_grouped", "moe_lora", "moe_combine_norm"):
            if direct is not None:
                direct.bind(name, ctypes.cast(getattr(L, name), vp).value)
            setattr(L, "direct_" + name, getattr(direct or L, name))
        _lib = L
        return L


def status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t):
    if t is None:
        return None
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream, *buffers):
    """Makes `stream` current for what a call allocates itself (the `buffers` that are None): fills
    then come before the call's kernels, and memory that is freed goes to work that comes after
    them."""
    if stream is None or (buffers and all(b is not None for b in buffers)):
        return _as_is
    import torch
    return torch.cuda.stream(stream)


def _dev(t, dtype_name: str):
    import torch
    assert t.is_cuda and t.is_contiguous(), f"{dtype_name} must be a contiguous CUDA tensor"
    return t


def _route_outputs(logits, K, with_shared, topk_ids, topk_w, shared_w, stream):
    import torch
    _dev(logits, "logits")
    assert logits.dtype == torch.float32
    T, E = logits.shape
    Kt = K + (1 if with_shared else 0)
    with _on(stream, topk_ids, topk_w):
        if topk_ids is None:
            topk_ids = torch.empty((T, Kt), dtype=torch.int32, device=logits.device)
        if topk_w is None:
            topk_w = torch.empty((T, Kt), dtype=torch.float32, device=logits.device)
    if shared_w is not None:
        _dev(shared_w, "shared_w")
        assert shared_w.dtype == torch.float32 and shared_w.shape == (T,)
    return T, E, Kt, topk_ids, topk_w


def moe_route(logits, K: int, with_shared: bool = True, renormalize: bool = True,
              topk_ids=None, topk_w=None, stream=None, shared_w=None):
    """fp32 logits [T, E] -> (int32 ids [T, Kt], fp32 weights [T, Kt]).  shared_w (fp32 [T],
    optional): per-token weight of the shared slot (moe_route_ex)."""
    T, E, Kt, topk_ids, topk_w = _route_outputs(logits, K, with_shared, topk_ids, topk_w, shared_w, stream)
    if shared_w is None:
        _check(load().moe_route(_ptr(logits), T, E, K, int(with_shared), int(renormalize),
                                _ptr(topk_ids), _ptr(topk_w), _stream(stream)), "moe_route")
    else:
        _check(load().moe_route_ex(_ptr(logits), _ptr(shared_w), T, E, K, int(with_shared),
                                   int(renormalize), _ptr(topk_ids), _ptr(topk_w),
                                   _stream(stream)), "moe_route_ex")
    return topk_ids, topk_w


def moe_route_permute(logits, K: int, tile_m: int, with_shared: bool = True,
                      renormalize: bool = True, topk_ids=None, topk_w=None,
                      perm: dict | None = None, shared_w=None, stream=None):
    """moe_route_ex + moe_permute in one call (one launch for small batches):
    returns (ids, weights, perm dict as from moe_permute)."""
    T, E, Kt, topk_ids, topk_w = _route_outputs(logits, K, with_shared, topk_ids, topk_w, shared_w, stream)
    Et = E + (1 if with_shared else 0)
    if perm is None:
        with _on(stream):
            perm = alloc_permute(T, Kt, Et, tile_m, logits.device)
    _check(load().moe_route_permute(_ptr(logits), _ptr(shared_w), T, E, K, int(with_shared),
                                    int(renormalize), tile_m, _ptr(topk_ids), _ptr(topk_w),
                                    _ptr(perm["sorted_pairs"]), _ptr(perm["expert_offsets"]),
                                    _ptr(perm["inv_pairs"]), _ptr(perm["tile_expert"]),
                                    _ptr(perm["num_tiles"]), _stream(stream)), "moe_route_permute")
    return topk_ids, topk_w, perm


def moe_permute_capacity(T: int, Kt: int, Et: int, tile_m: int) -> int:
    return int(load().moe_permute_capacity(T, Kt, Et, tile_m))


def moe_permute_max_tiles(T: int, Kt: int, Et: int, tile_m: int) -> int:
    return int(load().moe_permute_max_tiles(T, Kt, Et, tile_m))


def alloc_permute(T: int, Kt: int, Et: int, tile_m: int, device="cuda") -> dict:
    import torch
    cap = moe_permute_capacity(T, Kt, Et, tile_m)
    mt = moe_permute_max_tiles(T, Kt, Et, tile_m)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(sorted_pairs=torch.empty(max(cap, 1), **i32)[:cap],
                expert_offsets=torch.empty(Et + 1, **i32),
                inv_pairs=torch.empty(max(T * Kt, 1), **i32)[:T * Kt],
                tile_expert=torch.empty(max(mt, 1), **i32)[:mt],
                num_tiles=torch.empty(1, **i32), T=T, Kt=Kt, Et=Et, tile_m=tile_m)


def moe_permute(topk_ids, Et: int, tile_m: int, out: dict | None = None, stream=None) -> dict:
    """int32 ids [T, Kt] -> dict of sorted_pairs, expert_offsets, inv_pairs,
    tile_expert, num_tiles (device tensors) plus the sizes."""
    T, Kt = topk_ids.shape
    _dev(topk_ids, "topk_ids")
    if out is None:
        with _on(stream):
            out = alloc_permute(T, Kt, Et, tile_m, topk_ids.device)
    _check(load().moe_permute(_ptr(topk_ids), T, Kt, Et, tile_m, _ptr(out["sorted_pairs"]),
                              _ptr(out["expert_offsets"]), _ptr(out["inv_pairs"]),
                              _ptr(out["tile_expert"]), _ptr(out["num_tiles"]), _stream(stream)),
           "moe_permute")
    return out


def moe_ffn_workspace_size(T: int, H: int, I: int, Et: int, Kt: int, tile_m: int) -> int:
    return int(load().moe_ffn_workspace_size(T, H, I, Et, Kt, tile_m))


def moe_ffn_auto_path(T: int, Kt: int, Et: int, tile_m: int) -> int:
    return int(load().moe_ffn_auto_path(T, Kt, Et, tile_m))


def moe_ffn_auto_path_shape(T: int, H: int, I: int, Et: int, Kt: int, tile_m: int) -> int:
    return int(load().moe_ffn_auto_path_shape(T, H, I, Et, Kt, tile_m))


def alloc_workspace(T: int, H: int, I: int, Et: int, Kt: int, tile_m: int, device="cuda"):
    import torch
    n = moe_ffn_workspace_size(T, H, I, Et, Kt, tile_m)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def moe_ffn(x, w13, s13, w2, s2, topk_w, perm: dict, out=None, workspace=None,
            path: int = MOE_PATH_AUTO, stream=None):
    """bf16 x [T, H] -> bf16 out [T, H] through the grouped MXFP4 expert MLPs."""
    import torch
    T, H = x.shape
    Et, twoI, _ = w13.shape
    I = twoI // 2
    Kt, tile_m = perm["Kt"], perm["tile_m"]
    for t in (x, w13, s13, w2, s2, topk_w):
        _dev(t, "ffn input")
    with _on(stream, out, workspace):
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = alloc_workspace(T, H, I, Et, Kt, tile_m, x.device)
    _check(load().moe_ffn_path(_ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(topk_w),
                               _ptr(perm["sorted_pairs"]), _ptr(perm["expert_offsets"]),
                               _ptr(perm["inv_pairs"]), _ptr(perm["tile_expert"]),
                               _ptr(perm["num_tiles"]), T, H, I, Et, Kt, tile_m, _ptr(out),
                               _ptr(workspace), workspace.numel(), int(path), _stream(stream)),
           "moe_ffn")
    return out


def moe_device_error(clear: bool = True) -> int:
    """The device error bits: 1 = a bounded wait inside a kernel gave up, 2 = an index out of
    range was met and that work skipped (include/moe.h)."""
    flag = ctypes.c_int(0)
    _check(load().moe_device_error(ctypes.byref(flag), int(clear)), "moe_device_error")
    return flag.value


def moe_selftest_wait_timeout(limit_us: int = 2000, stream=None):
    """Diagnostic: a bounded wait that runs out (include/moe.h)."""
    _check(load().moe_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "moe_selftest_wait_timeout")


def moe_set_gemm_events(before=None, after=None):
    """Profiling hook (include/moe.h): record the torch.cuda.Event pair around
    the grouped GEMM kernel of each following FFN call; None, None switches it
    off.  The events are created here if they have not been recorded yet."""
    import torch
    handles = []
    for ev in (before, after):
        if ev is None:
            handles.append(None)
            continue
        if ev.cuda_event == 0:  # torch creates an event lazily, on its first record
            ev.record(torch.cuda.current_stream())
        handles.append(ctypes.c_void_p(ev.cuda_event))
    _check(load().moe_set_gemm_events(*handles), "moe_set_gemm_events")


def moe_selftest_wait_split(limit_us: int = 2000, stream=None):
    """Diagnostic: two warps whose bounded waits end differently must stop
    together (include/moe.h).  Returns the device tensor of the two warps'
    outcomes (int32 [2]; 0 = stopped)."""
    import torch
    with _on(stream):
        out = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    _check(load().moe_selftest_wait_split(int(limit_us), _ptr(out), _stream(stream)),
           "moe_selftest_wait_split")
    return out


def moe_ffn_noalloc(x, w13, s13, w2, s2, topk_w, perm: dict, out=None, stream=None):
    """moe_ffn without a workspace argument: the scratch is the library's fixed
    device array (for callers that cannot allocate device memory).  Calls on
    one device share that array: do not overlap them on the GPU."""
    import torch
    T, H = x.shape
    Et, twoI, _ = w13.shape
    if out is None:
        with _on(stream):
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(load().moe_ffn_noalloc(_ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(topk_w),
                                  _ptr(perm["sorted_pairs"]), _ptr(perm["expert_offsets"]),
                                  _ptr(perm["inv_pairs"]), _ptr(perm["tile_expert"]),
                                  _ptr(perm["num_tiles"]), T, H, twoI // 2, Et, perm["Kt"],
                                  perm["tile_m"], _ptr(out), _stream(stream)), "moe_ffn_noalloc")
    return out


def moe_ffn_y_offset(T: int, I: int, Et: int, Kt: int, tile_m: int) -> int:
    return int(load().moe_ffn_y_offset(T, I, Et, Kt, tile_m))


def ffn_views(workspace, T: int, H: int, I: int, Et: int, Kt: int, tile_m: int):
    """(h [cap, I] 16-bit, y fp32 [T*Kt, H]) views of a moe_ffn workspace (after the gate_up
    step h holds scaled f16 rows: see moe_ffn_gate_up in include/moe.h)."""
    import torch
    cap = moe_permute_capacity(T, Kt, Et, tile_m)
    off = moe_ffn_y_offset(T, I, Et, Kt, tile_m)
    h = workspace[:cap * I * 2].view(torch.bfloat16).view(cap, I)
    y = workspace[off:off + T * Kt * H * 4].view(torch.float32).view(T * Kt, H)
    return h, y


def moe_ffn_gate_up(x, w13, s13, perm: dict, workspace, path: int = MOE_PATH_AUTO, stream=None):
    """gate_up + SwiGLU into the workspace's h (see ffn_views)."""
    T, H = x.shape
    Et, twoI, _ = w13.shape
    _check(load().moe_ffn_gate_up(_ptr(x), _ptr(w13), _ptr(s13), _ptr(perm["sorted_pairs"]),
                                  _ptr(perm["tile_expert"]), _ptr(perm["num_tiles"]), T, H,
                                  twoI // 2, Et, perm["Kt"], perm["tile_m"], _ptr(workspace),
                                  workspace.numel(), int(path), _stream(stream)), "moe_ffn_gate_up")
    return workspace


def moe_ffn_down(w2, s2, topk_w, perm: dict, workspace, T: int, path: int = MOE_PATH_AUTO,
                 stream=None):
    """down x routing weight from the workspace's h into its y (see ffn_views)."""
    Et, H, halfI = w2.shape
    _check(load().moe_ffn_down(_ptr(w2), _ptr(s2), _ptr(topk_w), _ptr(perm["sorted_pairs"]),
                               _ptr(perm["tile_expert"]), _ptr(perm["num_tiles"]), T, H, 2 * halfI,
                               Et, perm["Kt"], perm["tile_m"], _ptr(workspace), workspace.numel(),
                               int(path), _stream(stream)), "moe_ffn_down")
    return workspace


def moe_ffn_down_combine(w2, s2, topk_w, perm: dict, workspace, T: int, out,
                         path: int = MOE_PATH_AUTO, stream=None):
    """down x routing weight and the combine into out (include/moe.h)."""
    Et, H, halfI = w2.shape
    _check(load().moe_ffn_down_combine(
        _ptr(w2), _ptr(s2), _ptr(topk_w), _ptr(perm["sorted_pairs"]), _ptr(perm["inv_pairs"]),
        _ptr(perm["tile_expert"]), _ptr(perm["num_tiles"]), T, H, 2 * halfI, Et, perm["Kt"],
        perm["tile_m"], _ptr(out), _ptr(workspace), workspace.numel(), int(path),
        _stream(stream)), "moe_ffn_down_combine")
    return out


def moe_combine(y, T: int, H: int, Kt: int, out, stream=None):
    _check(load().moe_combine(_ptr(y), T, H, Kt, _ptr(out), _stream(stream)), "moe_combine")
    return out


def moe_layer(logits, x, w13, s13, w2, s2, K: int, with_shared: bool = True,
              renormalize: bool = True, tile_m: int = 8, path: int = MOE_PATH_AUTO,
              bufs: dict | None = None, stream=None, router: dict | None = None):
    """The whole layer: route -> permute -> ffn, all on one stream.  `bufs`
    (from alloc_layer) reuses preallocated device buffers.  `router`: arguments of
    moe_route_grouped (bias, score, n_groups, topk_groups, group_top, scale, shared_w), which then
    routes instead of moe_route."""
    T, E = logits.shape
    Et = w13.shape[0]
    if bufs is None:
        with _on(stream):
            bufs = alloc_layer(T, E, K, with_shared, x.shape[1], w13.shape[1] // 2, Et, tile_m,
                               x.device)
    if Et != E + (1 if with_shared else 0):
        raise ValueError("weights must hold E experts plus the shared one when with_shared")
    if router is None:
        ids, w, perm = moe_route_permute(logits, K, tile_m, with_shared, renormalize, bufs["topk_ids"],
                                         bufs["topk_w"], bufs["perm"], stream=stream)
    else:
        ids, w = moe_route_grouped(logits, K, with_shared=with_shared, renormalize=renormalize, topk_ids=bufs["topk_ids"],
                                   topk_w=bufs["topk_w"], stream=stream, **router)
        perm = moe_permute(ids, Et, tile_m, bufs["perm"], stream)
    return moe_ffn(x, w13, s13, w2, s2, w, perm, bufs["out"], bufs["workspace"], path, stream)


def alloc_layer(T, E, K, with_shared, H, I, Et, tile_m, device="cuda") -> dict:
    import torch
    Kt = K + (1 if with_shared else 0)
    return dict(topk_ids=torch.empty((T, Kt), dtype=torch.int32, device=device),
                topk_w=torch.empty((T, Kt), dtype=torch.float32, device=device),
                perm=alloc_permute(T, Kt, Et, tile_m, device),
                workspace=alloc_workspace(T, H, I, Et, Kt, tile_m, device),
                out=torch.empty((T, H), dtype=torch.bfloat16, device=device))


def moe_ffn_dense_shared(x, w13, s13, w2, s2, topk_w, perm: dict, w13s, s13s, w2s, s2s,
                         shared_w=None, out=None, workspace=None, stream=None):
    """Routed layer + a shared expert of another width run as a dense MLP over all tokens
    (include/moe.h, moe_ffn_dense_shared)."""
    import torch
    T, H = x.shape
    Et, twoI, _ = w13.shape
    Is = w13s.shape[1] // 2
    Kt, tm = perm["Kt"], perm["tile_m"]
    n = int(load().moe_ffn_dense_shared_workspace_size(T, H, twoI // 2, Et, Kt, Is, tm))
    with _on(stream, workspace, out):
        if workspace is None:
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=x.device)
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(load().moe_ffn_dense_shared(
        _ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(topk_w),
        _ptr(perm["sorted_pairs"]), _ptr(perm["expert_offsets"]), _ptr(perm["inv_pairs"]),
        _ptr(perm["tile_expert"]), _ptr(perm["num_tiles"]), T, H, twoI // 2, Et, Kt, tm,
        _ptr(w13s), _ptr(s13s), _ptr(w2s), _ptr(s2s), Is, _ptr(shared_w), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(stream)), "moe_ffn_dense_shared")
    return out


# ------------------------------------------------ MXFP4-quantised activations

def moe_split_e4m3x2(x, stream=None):
    """bf16 [rows, cols] -> (q_hi, q_lo uint8 [rows, cols], s_hi, s_lo uint8
    [rows, cols/32]): the two-term E4M3 encoding of MOE_PATH_PREFILL_FP8X2
    (include/moe.h)."""
    import torch
    _dev(x, "x")
    rows, cols = x.shape
    with _on(stream):
        q_hi = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        q_lo = torch.empty_like(q_hi)
        s_hi = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
        s_lo = torch.empty_like(s_hi)
    _check(load().moe_split_e4m3x2(_ptr(x), rows, cols, _ptr(q_hi), _ptr(q_lo), _ptr(s_hi), _ptr(s_lo),
                                   _stream(stream)), "moe_split_e4m3x2")
    return q_hi, q_lo, s_hi, s_lo


def moe_quantize_mxfp4(x, codes=None, scales=None, stream=None):
    """bf16 [rows, cols] -> (codes uint8 [rows, cols/2], scales uint8 [rows, cols/32]),
    OCP MX rounding (include/moe.h)."""
    import torch
    _dev(x, "x")
    rows, cols = x.shape
    with _on(stream, codes, scales):
        if codes is None:
            codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        if scales is None:
            scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    _check(load().moe_quantize_mxfp4(_ptr(x), rows, cols, _ptr(codes), _ptr(scales),
                                     _stream(stream)), "moe_quantize_mxfp4")
    return codes, scales


def moe_ffn_mxfp4act_workspace_size(T: int, H: int, I: int, Et: int, Kt: int, tile_m: int) -> int:
    return int(load().moe_ffn_mxfp4act_workspace_size(T, H, I, Et, Kt, tile_m))


def alloc_workspace_mxfp4act(T: int, H: int, I: int, Et: int, Kt: int, tile_m: int,
                             device="cuda"):
    import torch
    n = moe_ffn_mxfp4act_workspace_size(T, H, I, Et, Kt, tile_m)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def moe_ffn_mxfp4act(x, w13, s13, w2, s2, topk_w, perm: dict, out=None, workspace=None,
                     stream=None):
    """The expert FFN with MXFP4-quantised activations (both GEMMs block-scaled MXFP4 x MXFP4)."""
    import torch
    T, H = x.shape
    Et, twoI, _ = w13.shape
    Kt, tile_m = perm["Kt"], perm["tile_m"]
    for t in (x, w13, s13, w2, s2, topk_w):
        _dev(t, "ffn input")
    with _on(stream, out, workspace):
        if out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = alloc_workspace_mxfp4act(T, H, twoI // 2, Et, Kt, tile_m, x.device)
    _check(load().moe_ffn_mxfp4act(_ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), _ptr(topk_w),
                                   _ptr(perm["sorted_pairs"]), _ptr(perm["expert_offsets"]),
                                   _ptr(perm["inv_pairs"]), _ptr(perm["tile_expert"]),
                                   _ptr(perm["num_tiles"]), T, H, twoI // 2, Et, Kt, tile_m,
                                   _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_ffn_mxfp4act")
    return out


def moe_ffn_mxfp4act_gate_up(x, w13, s13, perm: dict, workspace, stream=None):
    T, H = x.shape
    Et, twoI, _ = w13.shape
    _check(load().moe_ffn_mxfp4act_gate_up(
        _ptr(x), _ptr(w13), _ptr(s13), _ptr(perm["sorted_pairs"]), _ptr(perm["tile_expert"]),
        _ptr(perm["num_tiles"]), T, H, twoI // 2, Et, perm["Kt"], perm["tile_m"], _ptr(workspace),
        workspace.numel(), _stream(stream)), "moe_ffn_mxfp4act_gate_up")
    return workspace


def moe_ffn_mxfp4act_down(w2, s2, topk_w, perm: dict, workspace, T: int, out, stream=None):
    Et, H, halfI = w2.shape
    _check(load().moe_ffn_mxfp4act_down(
        _ptr(w2), _ptr(s2), _ptr(topk_w), _ptr(perm["sorted_pairs"]), _ptr(perm["inv_pairs"]),
        _ptr(perm["tile_expert"]),
        _ptr(perm["num_tiles"]), T, H, 2 * halfI, Et, perm["Kt"], perm["tile_m"], _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(stream)), "moe_ffn_mxfp4act_down")
    return out


def mxfp4act_h_views(workspace, T: int, H: int, I: int, Et: int, Kt: int, tile_m: int):
    """(h codes uint8 [cap, I/2], h scales uint8 [cap, I/32]) views of a moe_ffn_mxfp4act
    workspace, rows by sorted position."""
    co, so = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load().moe_ffn_mxfp4act_h_offsets(T, H, I, Et, Kt, tile_m, ctypes.byref(co),
                                             ctypes.byref(so)), "moe_ffn_mxfp4act_h_offsets")
    cap = moe_permute_capacity(T, Kt, Et, tile_m)
    codes = workspace[co.value:co.value + cap * (I // 2)].view(cap, I // 2)
    scales = workspace[so.value:so.value + cap * (I // 32)].view(cap, I // 32)
    return codes, scales


def _workspace_bytes(workspace) -> int:
    """The size of a workspace that the caller passed, in bytes whatever its type."""
    assert workspace.is_cuda and workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor"
    return workspace.numel() * workspace.element_size()


# ------------------------------------------------- the layer for a few tokens

def moe_layer_few_workspace_size(T: int, H: int, I: int, E: int, K: int, with_shared: bool) -> int:
    return int(load().moe_layer_few_workspace_size(T, H, I, E, K, int(with_shared)))


def alloc_workspace_few(T: int, H: int, I: int, E: int, K: int, with_shared: bool = True,
                        device="cuda"):
    """An initialised workspace for moe_layer_few, to be kept from call to call (one for each
    stream that calls may overlap on)."""
    import torch
    n = moe_layer_few_workspace_size(T, H, I, E, K, with_shared)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def moe_layer_few_workspace_init(workspace, stream=None):
    """Zero the barrier counters of a workspace that did not come from alloc_workspace_few
    (include/moe.h)."""
    _check(load().moe_layer_few_workspace_init(_ptr(workspace), _workspace_bytes(workspace), _stream(stream)),
           "moe_layer_few_workspace_init")


def moe_layer_few(x, w_router, w13, s13, w2, s2, K: int, with_shared: bool = True,
                  renormalize: bool = True, w_shared_gate=None, out=None, topk_ids=None, topk_w=None,
                  workspace=None, stream=None):
    """The whole layer for up to 16 tokens in one launch: bf16 x [T, H], router weights bf16
    [E, H], expert weights as for moe_ffn -> (bf16 out [T, H], int32 ids [T, Kt], fp32 weights
    [T, Kt]).  w_shared_gate (bf16 [H], optional): the shared expert's weight is
    sigmoid(w_shared_gate . x).  workspace: from alloc_workspace_few (include/moe.h)."""
    import torch
    T, H = x.shape
    E = w_router.shape[0]
    Et, twoI, _ = w13.shape
    I, shared = twoI // 2, 1 if with_shared else 0
    bf16, u8 = torch.bfloat16, torch.uint8
    if Et != E + shared or w2.shape != (Et, H, I // 2) or w13.shape[2] != H // 2:
        raise ValueError("weights must hold E experts plus the shared one when with_shared")
    assert x.dtype == bf16 and w_router.dtype == bf16 and w_router.shape[1] == H, "x and w_router are bfloat16"
    assert w13.dtype == s13.dtype == w2.dtype == s2.dtype == u8, "weights are uint8"
    assert s13.shape == (Et, twoI, H // 32) and s2.shape == (Et, H, I // 32), "scales do not match the weights"
    for t in (x, w_router, w13, s13, w2, s2):
        _dev(t, "layer input")
    if w_shared_gate is not None:
        _dev(w_shared_gate, "w_shared_gate")
        assert w_shared_gate.dtype == bf16 and w_shared_gate.shape == (H,)
    if out is not None and not (out.is_cuda and out.is_contiguous() and out.dtype == bf16 and out.shape == x.shape):
        raise ValueError("out must be a contiguous CUDA bfloat16 tensor like x")
    with _on(stream, out, topk_ids, topk_w, workspace):
        if out is None:
            out = torch.empty_like(x)
        if topk_ids is None:
            topk_ids = torch.empty((T, K + shared), dtype=torch.int32, device=x.device)
        if topk_w is None:
            topk_w = torch.empty((T, K + shared), dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = alloc_workspace_few(T, H, I, E, K, with_shared, x.device)
    for t, dt in ((topk_ids, torch.int32), (topk_w, torch.float32)):
        assert t.is_cuda and t.is_contiguous() and t.dtype == dt and t.numel() == T * (K + shared)
    status = (_lib or load()).moe_layer_few(
        x.data_ptr(), w_router.data_ptr(), None if w_shared_gate is None else w_shared_gate.data_ptr(),
        w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(), T, H, I, E, K, shared,
        1 if renormalize else 0, out.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(), workspace.data_ptr(),
        _workspace_bytes(workspace), _raw_stream(stream, x))
    if status:
        raise MoeError(status, "moe_layer_few")
    return out, topk_ids, topk_w


# ------------------------------------------------------------- dense projections

def moe_linear_mxfp4act_workspace_size(T: int, N: int, K: int) -> int:
    return int(load().moe_linear_mxfp4act_workspace_size(T, N, K))


def alloc_workspace_linear(T: int, N: int, K: int, device="cuda"):
    import torch
    n = moe_linear_mxfp4act_workspace_size(T, N, K)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _raw_stream(stream, t):
    """The handle of `stream`, or of the current stream of t's device (without the Stream object
    that torch.cuda.current_stream makes: 3 us of a call that takes 10)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _row_stride(t, rows: int, width: int, what: str) -> int:
    """The row stride of a 2D CUDA tensor whose rows are contiguous."""
    ld, inner = t.stride()
    assert t.is_cuda and (inner == 1 or width <= 1), f"{what} must be a CUDA tensor with contiguous rows"
    # a single row has no neighbour: its stride means nothing
    return ld if rows > 1 else width


def moe_linear_mxfp4act(x, codes, scales, residual=None, out=None, out_dtype=None, workspace=None,
                        stream=None):
    """bf16 or fp32 x [T, K] times MXFP4 weights (codes [N, K/2], scales [N, K/32]), x quantised
    to MXFP4 inside the call, plus residual [T, N] (include/moe.h).  x, residual and out may be
    row slices of wider tensors; out_dtype: torch.bfloat16 (default) or torch.float32."""
    import torch
    f32, bf16 = torch.float32, torch.bfloat16
    T, K = x.shape
    N = codes.shape[0]
    _dev(codes, "codes")
    _dev(scales, "scales")
    assert codes.shape == (N, K // 2) and scales.shape == (N, K // 32), "weights do not match x"
    assert codes.dtype == torch.uint8 and scales.dtype == torch.uint8, "weights are uint8"
    if out is None:
        out_dtype = out_dtype or bf16
        with _on(stream):
            out = torch.empty((T, N), dtype=out_dtype, device=x.device)
        ldo = N
    else:
        assert out.shape == (T, N) and out_dtype in (None, out.dtype), "out must be [T, N]"
        out_dtype = out.dtype
        ldo = _row_stride(out, T, N, "out")
    xt = x.dtype
    assert (xt == bf16 or xt == f32) and (out_dtype == bf16 or out_dtype == f32), \
        "x and out must be bfloat16 or float32"
    res, ldr = None, 0
    if residual is not None:
        assert residual.shape == (T, N) and residual.dtype == out_dtype, "residual must match out"
        res, ldr = residual.data_ptr(), _row_stride(residual, T, N, "residual")
    if workspace is None:
        with _on(stream):
            workspace = alloc_workspace_linear(T, N, K, x.device)
    status = (_lib or load()).moe_linear_mxfp4act(
        x.data_ptr(), MOE_DTYPE_F32 if xt == f32 else MOE_DTYPE_BF16, _row_stride(x, T, K, "x"),
        codes.data_ptr(), scales.data_ptr(), res, ldr, out.data_ptr(),
        MOE_DTYPE_F32 if out_dtype == f32 else MOE_DTYPE_BF16, ldo, T, N, K, workspace.data_ptr(),
        _workspace_bytes(workspace), _raw_stream(stream, x))
    if status:
        raise MoeError(status, "moe_linear_mxfp4act")
    return out


# ------------------------------------------------- what lies between the products

_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GATES = {"none": MOE_GATE_NONE, "sigmoid": MOE_GATE_SIGMOID, "silu": MOE_GATE_SILU}


_codes: dict = {}


def _code(t):
    """MOE_DTYPE_... of a tensor, -1 for int32, None for other types.  (A dict of torch's types made at the
    first call: importing torch in every call and function took a fourth of a small call's time.)"""
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32, torch.int32: -1})
    return _codes.get(t.dtype)


def _dtype_code(t, what: str) -> int:
    """MOE_DTYPE_... of a tensor."""
    code = _code(t)
    assert code is not None and code >= 0, f"{what} must be bfloat16 or float32"
    return code


def _vector(t, n: int, code: int, what: str) -> int:
    """The address of a contiguous CUDA tensor [n] of the type with this code."""
    assert t.is_cuda and t.is_contiguous() and _code(t) == code and t.shape == (n,), \
        f"{what} must be a contiguous CUDA tensor [{n}] of its type"
    return t.data_ptr()


_current_stream = None


def _stream_handle(stream, t):
    """The handle of `stream`, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream
    global _current_stream
    if _current_stream is None:
        import torch
        _current_stream = torch._C._cuda_getCurrentRawStream
    return _current_stream(t.get_device())


def moe_route_grouped(logits, K: int, bias=None, score: str = "sigmoid", n_groups: int = 1, topk_groups: int = 1,
                      group_top: int = 2, with_shared: bool = True, renormalize: bool = True, scale: float = 1.0,
                      topk_ids=None, topk_w=None, shared_w=None, stream=None):
    """fp32 or bf16 logits [T, E] (rows may be slices of wider ones) -> (int32 ids [T, Kt], fp32
    weights [T, Kt]), by softmax or sigmoid scores plus bias (fp32 [E]), within the topk_groups best
    of n_groups groups of experts, each worth the sum of its group_top largest (include/moe.h)."""
    T, E = logits.shape
    Kt = K + 1 if with_shared else K
    if topk_ids is None or topk_w is None:
        import torch
        with _on(stream):
            if topk_ids is None:
                topk_ids = torch.empty((T, Kt), dtype=torch.int32, device=logits.device)
            if topk_w is None:
                topk_w = torch.empty((T, Kt), dtype=torch.float32, device=logits.device)
    assert topk_ids.is_cuda and topk_ids.is_contiguous() and _code(topk_ids) == -1 and topk_ids.numel() == T * Kt \
        and topk_w.is_cuda and topk_w.is_contiguous() and _code(topk_w) == MOE_DTYPE_F32 and topk_w.numel() == T * Kt, \
        "topk_ids and topk_w must be contiguous CUDA tensors of int32 and float32 [T, Kt]"
    status = (_lib or load()).direct_moe_route_grouped(
        logits.data_ptr(), _dtype_code(logits, "logits"), _row_stride(logits, T, E, "logits"),
        None if bias is None else _vector(bias, E, MOE_DTYPE_F32, "bias"),
        None if shared_w is None else _vector(shared_w, T, MOE_DTYPE_F32, "shared_w"), T, E, K,
        _SCORES[score], n_groups, topk_groups, group_top, 1 if with_shared else 0, 1 if renormalize else 0, scale,
        topk_ids.data_ptr(), topk_w.data_ptr(), _stream_handle(stream, logits))
    if status:
        raise MoeError(status, "moe_route_grouped")
    return topk_ids, topk_w


def moe_lora_tile_m(T: int, adapters: int) -> int:
    return int(load().moe_lora_tile_m(T, adapters))


def moe_lora_plan(adapter_ids, adapters: int, tile_m: int | None = None, out: dict | None = None, stream=None) -> dict:
    """The grouping of tokens by adapter that moe_lora takes: int32 adapter_ids [T] (-1: none) ->
    moe_permute's dict.  One serves every projection of a step.  `out`: a plan of the same sizes to
    write to, whose tile height it keeps (15 us instead of 47 for five new tensors, 3 to 5 in a graph).  tile_m
    goes by `adapters` if it is None; with a pool of which few are used, moe_lora_tile_m(T, those in use) suits prompts
    better."""
    T, = adapter_ids.shape
    assert _code(adapter_ids) == -1, "adapter_ids must be int32"
    if out is not None:
        assert out["T"] == T and out["Kt"] == 1 and out["Et"] == adapters and tile_m in (None, out["tile_m"]), \
            "out is a plan of other sizes"
        tile_m = out["tile_m"]
    return moe_permute(adapter_ids.view(T, 1), adapters, tile_m or moe_lora_tile_m(T, adapters), out=out, stream=stream)


def moe_lora(x, a, b, plan: dict, scale=None, ranks=None, residual=None, out=None, out_dtype=None, stream=None):
    """residual + scale * B (A x) with each token's own adapter: x [T, K] bf16 or fp32, a bf16
    [adapters, R, K], b bf16 [adapters, N, R], plan from moe_lora_plan, scale fp32 and ranks int32
    [adapters], residual [T, N] (may be out) (include/moe.h).  x, residual and out may be row slices of
    wider tensors; out_dtype: torch.bfloat16 (default) or torch.float32."""
    T, K = x.shape
    n, N, R = b.shape
    assert plan["T"] == T and plan["Kt"] == 1 and plan["Et"] == n, "plan does not match x and the adapters"
    assert a.shape == (n, R, K) and _code(a) == MOE_DTYPE_BF16 and _code(b) == MOE_DTYPE_BF16, "a and b must be bfloat16 [n, R, K] and [n, N, R]"
    assert a.is_cuda and a.is_contiguous() and b.is_cuda and b.is_contiguous(), "a and b must be contiguous CUDA tensors"
    if out is None:
        import torch
        with _on(stream):
            out = torch.empty((T, N), dtype=out_dtype or torch.bfloat16, device=x.device)
        ldo = N
    else:
        assert out.shape == (T, N) and out_dtype in (None, out.dtype), "out must be [T, N]"
        ldo = _row_stride(out, T, N, "out")
    res, ldr = None, 0
    if residual is not None:
        assert residual.shape == (T, N) and residual.dtype is out.dtype, "residual must match out"
        res, ldr = residual.data_ptr(), _row_stride(residual, T, N, "residual")
    status = (_lib or load()).direct_moe_lora(
        x.data_ptr(), _dtype_code(x, "x"), _row_stride(x, T, K, "x"), a.data_ptr(), b.data_ptr(),
        None if scale is None else _vector(scale, n, MOE_DTYPE_F32, "scale"),
        None if ranks is None else _vector(ranks, n, -1, "ranks"),
        plan["sorted_pairs"].data_ptr(), plan["inv_pairs"].data_ptr(), plan["tile_expert"].data_ptr(),
        plan["num_tiles"].data_ptr(), plan["tile_m"], n, res, ldr, out.data_ptr(), _dtype_code(out, "out"), ldo, T, N, K, R,
        _stream_handle(stream, x))
    if status:
        raise MoeError(status, "moe_lora")
    return out


def moe_combine_norm(y, h=None, slots: int = 1, post_w=None, gate=None, gate_act: str = "none", alpha: float = 1.0,
                     beta: float = 1.0, pre_w=None, w_offset: float = 0.0, eps: float = 1e-6, h_out=None, n_out=None,
                     h_dtype=None, n_dtype=None, stream=None):
    """From a block's output to the next block's input: y [T * slots, H] summed over a token's slots,
    its norm with post_w, times act(gate) (gate [T or 1, H or 1]), h' = beta h + alpha u, and the norm of
    h' with pre_w -> (h' [T, H], n [T, H]) (include/moe.h).  h_out may be h, n_out may be y.  Without h, h'
    has h_dtype (default bfloat16) and is not written if h_out is False; n has n_dtype (default
    bfloat16) and is not written if n_out is False."""
    rows, H = y.shape
    T = rows // slots
    assert T * slots == rows, "y must hold slots rows a token"
    if h_out is None or n_out is None:
        import torch
        with _on(stream):
            if h_out is None:
                h_out = torch.empty((T, H), dtype=h.dtype if h is not None else h_dtype or torch.bfloat16, device=y.device)
            if n_out is None:
                n_out = torch.empty((T, H), dtype=n_dtype or torch.bfloat16, device=y.device)
    shape = (T, H)
    hp, ht, ldh, hop, ldho, np_, nt, ldn = None, 0, 0, None, 0, None, 0, 0
    if h is not None:
        assert h.shape == shape, "h must be [T, H]"
        hp, ht, ldh = h.data_ptr(), _dtype_code(h, "h"), _row_stride(h, T, H, "h")
    if h_out is not False:
        assert h_out.shape == shape and (h is None or h_out.dtype is h.dtype), "h_out must be [T, H] of h's type"
        hop, ht, ldho = h_out.data_ptr(), _dtype_code(h_out, "h_out"), _row_stride(h_out, T, H, "h_out")
    if n_out is not False:
        assert n_out.shape == shape, "n_out must be [T, H]"
        np_, nt, ldn = n_out.data_ptr(), _dtype_code(n_out, "n_out"), _row_stride(n_out, T, H, "n_out")
    w_type, pw, w = 0, None, None
    if pre_w is not None:
        w_type = _dtype_code(pre_w, "pre_w")
        w = _vector(pre_w, H, w_type, "pre_w")
    if post_w is not None:
        assert pre_w is None or pre_w.dtype is post_w.dtype, "post_w and pre_w must have one type"
        w_type = _dtype_code(post_w, "post_w")
        pw = _vector(post_w, H, w_type, "post_w")
    gp, gt, ldg, cols = None, 0, 0, 1
    if gate is not None:
        grows, cols = gate.shape
        assert grows in (1, T) and cols in (1, H), "gate must be [T or 1, H or 1]"
        gp, gt, ldg = gate.data_ptr(), _dtype_code(gate, "gate"), _row_stride(gate, grows, cols, "gate")
        ldg = ldg if grows > 1 else 0
    status = (_lib or load()).direct_moe_combine_norm(
        y.data_ptr(), _dtype_code(y, "y"), _row_stride(y, rows, H, "y"), slots, 0 if pw is None else 1, pw, w, w_type, w_offset,
        eps, gp, gt, ldg, cols, _GATES[gate_act], hp, ldh, alpha, beta, hop, ht, ldho, np_, nt, ldn, T, H,
        _stream_handle(stream, y))
    if status:
        raise MoeError(status, "moe_combine_norm")
    return h_out, n_out
