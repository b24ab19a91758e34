"""Cases, plain forms and 64-bit values of two operators of an MXFP4 decoder block.

layer   The whole mixture-of-experts layer for a few tokens (``libmoe.moe_layer_few``): router product, softmax
        top-K with ties to the lower expert, gate_up, SwiGLU, down, weighted sum over the chosen experts and the
        shared one.  Weights in MXFP4, activations in bf16.
linear  A projection with MXFP4 weights and activations quantised to MXFP4 on the way in
        (``libmoe.moe_linear_mxfp4act``): quantisation, product, optional residual, in bf16 or fp32.

MXFP4: E2M1 codes, two per byte (low nibble = even k), one E8M0 scale 2^(s - 127) per 32 consecutive k.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: The magnitudes of the eight E2M1 codes; bit 3 is the sign.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: Most weight bytes that a drawn layer holds, and most tokens by width (moe_layer_few's limits).
MOST_WEIGHTS = 3.5e9


# ------------------------------------------------------------------ cases

def _layer(name, T, H, I, E, K, shared, gate, renorm):
    return {"name": name, "op": "layer", "T": T, "H": H, "I": I, "E": E, "K": K, "shared": shared, "gate": gate,
            "renorm": renorm}


def _linear(name, T, N, K, x="bf16", out="bf16", residual=False, pad=0):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "x": x, "out": out, "residual": residual, "pad": pad}


def listed():
    return [
        # the smallest layer of this repository's tests, one token: launch latency and nothing else
        _layer("layer_tiny_1", 1, 256, 128, 8, 2, True, False, True),
        # the full-size layer of this repository (512 experts, ten chosen, a shared one), one sequence decoding
        _layer("layer_1", 1, 4096, 1024, 512, 10, True, False, True),
        # the same layer verifying one sequence's four drafted tokens and the one after them, shared expert gated
        _layer("layer_5", 5, 4096, 1024, 512, 10, True, True, True),
        # the same layer with sixteen sequences decoding: nearly all chosen experts are different ones
        _layer("layer_16", 16, 4096, 1024, 512, 10, True, False, True),
        # a layer of other widths: no power of two anywhere, no shared expert, weights not renormalised
        _layer("layer_odd_3", 3, 2080, 608, 60, 6, False, False, False),
        # few wide experts, seven tokens: experts that several tokens share
        _layer("layer_wide_7", 7, 6144, 2048, 16, 4, False, False, True),
        # a square projection of one token: latency
        _linear("linear_1", 1, 4096, 4096),
        # an odd output width and a slice of a wider activation (row stride above K), a few tokens
        _linear("linear_odd_7", 7, 1000, 1056, residual=True, pad=24),
        # an output head over a large, odd vocabulary: fp32 logits of sixteen sequences
        _linear("linear_head_16", 16, 100003, 4096, out="f32"),
        # an up projection for a batch of sixty-four decoding sequences
        _linear("linear_64", 64, 8192, 4096),
        # a prompt chunk through an output projection with its residual
        _linear("linear_1536", 1536, 4096, 4096, residual=True),
        # a long prompt: compute
        _linear("linear_8192", 8192, 8192, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"layer": work(listed()[3]), "linear": work(listed()[11])}
    while True:
        if rng.random() < 0.5:
            T = rng.randint(1, 16)
            widest = 4096 if T > 8 else 8192
            E = _log(rng, 2, 512)
            shared = rng.random() < 0.6
            case = _layer("", T, 32 * _log(rng, 1, widest // 32), 32 * _log(rng, 1, widest // 32), E,
                          rng.randint(1, min(E, 12)), shared, shared and rng.random() < 0.5, rng.random() < 0.7)
            if (E + 1) * 3 * case["H"] * case["I"] * 17 / 32 > MOST_WEIGHTS:
                continue
        else:
            case = _linear("", _log(rng, 1, 8192), _log(rng, 16, 131072), 32 * _log(rng, 1, 512),
                           rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]),
                           rng.random() < 0.3, rng.choice([0, 0, 8, 24, 5]))
        w, m = work(case), most[case["op"]]
        if w["bytes"] <= 1.6 * m["bytes"] and w["flops"] <= m["flops"]:
            del case["name"]
            return case


def _touched(E, K, T):
    """Experts that T tokens choosing K of E touch on average."""
    return E * (1.0 - (1.0 - K / E) ** T)


def work(case):
    T = case["T"]
    if case["op"] == "layer":
        H, I, E, K, s = case["H"], case["I"], case["E"], case["K"], int(case["shared"])
        expert = 3 * H * I / 2 + 3 * H * I / 32
        by = (_touched(E, K, T) + s) * expert + E * H * 2 + (H * 2 if case["gate"] else 0) + 2 * T * H * 2 + T * (K + s) * 8
        return {"bytes": int(by), "flops": int(2 * T * (K + s) * 3 * H * I + 2 * T * E * H)}
    N, K = case["N"], case["K"]
    xb, ob = (2 if case["x"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
    by = N * K / 2 + N * K / 32 + T * K * xb + T * N * ob * (2 if case["residual"] else 1)
    return {"bytes": int(by), "flops": 2 * T * N * K}


# ----------------------------------------------------------------- inputs

def _weights(g, shape):
    """Random codes [.., K / 2] and scales 2^-8 to 2^-4 [.., K / 32] of a weight of this shape."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(119, 124, (*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device=DEV, generator=g)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *n: torch.randn(n, dtype=torch.float32, device=DEV, generator=g)  # noqa: E731
    s = dict(case)
    if case["op"] == "layer":
        T, H, I, E = case["T"], case["H"], case["I"], case["E"]
        Et = E + int(case["shared"])
        s["x"] = normal(T, H).bfloat16()
        s["router"] = (normal(E, H) * (1.5 / math.sqrt(H))).bfloat16()
        s["gate_w"] = (normal(H) / math.sqrt(H)).bfloat16() if case["gate"] else None
        s["w13"], s["s13"] = _weights(g, (Et, 2 * I, H))
        s["w2"], s["s2"] = _weights(g, (Et, H, I))
        return s
    T, N, K = case["T"], case["N"], case["K"]
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    # one channel in a hundred is an outlier, as activations after a norm have them; the rows may be a slice
    wide = normal(T, K + case["pad"]) * torch.where(torch.rand(K + case["pad"], device=DEV, generator=g) < 0.01, 20.0, 1.0)
    s["x"] = wide.to(types[case["x"]])[:, :K]
    s["w"], s["s"] = _weights(g, (N, K))
    s["res"] = normal(T, N).to(types[case["out"]]) if case["residual"] else None
    return s


# ------------------------------------------------------------------ passes

def _values(codes, scales):
    """The fp32 values of an MXFP4 tensor: [.., K / 2] codes and [.., K / 32] scales -> [.., K]."""
    mag = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    nib = torch.cat([mag, -mag])
    pairs = torch.stack([nib.repeat(16), nib.repeat_interleave(16)], 1)  # byte -> (low nibble's, high nibble's)
    v = pairs[codes.int()].view(*scales.shape, 32)
    return (v * torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)[..., None]).flatten(-2)


def _quantised(x):
    """fp32 rows -> the values of their MXFP4 encoding: per 32, 2^(floor(log2 amax) - 2), nearest E2M1, ties to even."""
    b = x.view(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, -127)
    a = torch.ldexp(b.abs(), -e)
    q = (0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
         + (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float())
    return torch.ldexp(torch.copysign(q, b), e).view(x.shape)


def _plain_layer(s):
    x = s["x"].float()
    T, K = s["T"], s["K"]
    logits = x @ s["router"].float().t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    p = torch.exp(logits - top[:, :1])
    w = torch.exp(top - top[:, :1]) / p.sum(1, keepdim=True)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if s["shared"]:
        one = torch.ones((T, 1), device=DEV)
        if s["gate"]:
            one = 1.0 / (1.0 + torch.exp(-(x @ s["gate_w"].float())[:, None]))
        ids = torch.cat([ids, torch.full_like(ids[:, :1], s["E"])], 1)
        w = torch.cat([w, one], 1)
    flat = ids.reshape(-1)
    gu = torch.einsum("tjnh,th->tjn", _values(s["w13"][flat], s["s13"][flat]).view(T, -1, 2 * s["I"], s["H"]), x)
    g, u = gu[..., :s["I"]], gu[..., s["I"]:]
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.einsum("tjhi,tji->tjh", _values(s["w2"][flat], s["s2"][flat]).view(T, -1, s["H"], s["I"]), h)
    return (w[..., None] * y).sum(1).bfloat16(), ids.int(), w


def _plain_linear(s):
    y = _quantised(s["x"].float()) @ _values(s["w"], s["s"]).t()
    if s["res"] is not None:
        y = s["res"].float() + y
    return y.to(torch.bfloat16 if s["out"] == "bf16" else torch.float32)


def run(state):
    s = state
    if not own:
        return _plain_layer(s) if s["op"] == "layer" else _plain_linear(s)
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    if s["op"] == "layer":
        if "workspace" not in s:  # as a program keeps it from step to step
            s["workspace"] = libmoe.alloc_workspace_few(s["T"], s["H"], s["I"], s["E"], s["K"], s["shared"])
        return libmoe.moe_layer_few(s["x"], s["router"], s["w13"], s["s13"], s["w2"], s["s2"], s["K"], s["shared"],
                                    s["renorm"], w_shared_gate=s["gate_w"], workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = libmoe.alloc_workspace_linear(s["T"], s["N"], s["K"])
    return libmoe.moe_linear_mxfp4act(s["x"], s["w"], s["s"], residual=s["res"],
                                      out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32,
                                      workspace=s["workspace"])


# ----------------------------------------------------------- 64-bit values

def _decode64(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, c & 1
    mag = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * 2.0 ** (e - 1).double())
    v = torch.where(c >= 8, -mag, mag).double()
    return v * (2.0 ** (scales.double() - 127.0)).repeat_interleave(32, -1)


def _nearest64(x):
    """MXFP4 values of float64 rows: the nearest of the eight magnitudes, the even code of two equally near."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    step = torch.full_like(amax, 2.0 ** -127)
    for e in range(-127, 128):  # the largest power of two whose fourfold does not pass amax
        step = torch.where(amax >= 2.0 ** (e + 2), 2.0 ** e, step)
    a = (b / step[..., None]).abs()
    order = torch.tensor([E2M1[i] for i in (0, 2, 4, 6, 1, 3, 5, 7)], dtype=torch.float64, device=x.device)
    best, far = torch.zeros_like(a), torch.full_like(a, math.inf)
    for v in order:  # even codes first: an odd one has to be strictly nearer
        d = (a - v).abs()
        best, far = torch.where(d < far, v, best), torch.minimum(d, far)
    return (torch.sign(b) * best * step[..., None]).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "linear":
        xq, parts = _nearest64(x), []
        for n0 in range(0, case["N"], 16384):
            parts.append(xq @ _decode64(s["w"][n0:n0 + 16384], s["s"][n0:n0 + 16384]).t())
        y = torch.cat(parts, 1)
        return y if s["res"] is None else y + s["res"].double()
    T, K, I, E = case["T"], case["K"], case["I"], case["E"]
    Kt = K + int(case["shared"])
    logits = (x @ s["router"].double().t()).cpu().numpy()
    ids = np.zeros((T, Kt), np.int32)
    w = np.ones((T, Kt))
    out = torch.zeros_like(x)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-logits[t, e], e))[:K]
        p = np.exp(logits[t] - logits[t].max())
        p = p / p.sum()
        ids[t, :K] = order
        w[t, :K] = p[order] / (p[order].sum() if case["renorm"] else 1.0)
        if case["shared"]:
            ids[t, K] = E
            if case["gate"]:
                w[t, K] = 1.0 / (1.0 + math.exp(-float(x[t] @ s["gate_w"].double())))
    for e in sorted(set(ids.reshape(-1).tolist())):
        w13, w2 = _decode64(s["w13"][e], s["s13"][e]), _decode64(s["w2"][e], s["s2"][e])
        for t in range(T):
            for j in np.nonzero(ids[t] == e)[0]:
                g, u = w13[:I] @ x[t], w13[I:] @ x[t]
                out[t] += float(w[t, j]) * (w2 @ (g / (1.0 + torch.exp(-g)) * u))
    return out, torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
