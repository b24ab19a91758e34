"""Cases, plain forms and 64-bit values of three operators around the projections and experts of an MXFP4 decoder block.

route  Routing with softmax or sigmoid scores, a bias for balance and expert groups (``libmoe.moe_route_grouped``).
lora   Low-rank adapters of many requests beside a shared projection (``libmoe.moe_lora``).
norm   The sum over a token's expert outputs, the norm after the block, gate, scaled residual and the norm before the
       next block (``libmoe.moe_combine_norm``).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _route(name, T, E, K, score, bias, groups=1, chosen=1, top=1, renorm=True, scale=1.0, shared=False, logits="f32",
           pad=0):
    return {"name": name, "op": "route", "T": T, "E": E, "K": K, "score": score, "bias": bias, "groups": groups,
            "chosen": chosen, "top": top, "renorm": renorm, "scale": scale, "shared": shared, "logits": logits, "pad": pad}


def _lora(name, T, N, K, R, adapters, runs, x="bf16", out="bf16", residual=True, ranks=False, without=0.0, pad=0):
    return {"name": name, "op": "lora", "T": T, "N": N, "K": K, "R": R, "adapters": adapters, "runs": runs, "x": x,
            "out": out, "residual": residual, "ranks": ranks, "without": without, "pad": pad}


def _norm(name, T, H, slots=1, y="bf16", h="bf16", residual=True, post=False, gate="none", act="none", alpha=1.0, beta=1.0,
          offset=0.0, pad=0):
    return {"name": name, "op": "norm", "T": T, "H": H, "slots": slots, "y": y, "h": h, "residual": residual, "post": post,
            "gate": gate, "act": act, "alpha": alpha, "beta": beta, "offset": offset, "pad": pad}


def listed():
    return [
        # one sequence decoding, 256 experts in eight groups of which four are kept: latency
        _route("route_1", 1, 256, 8, "sigmoid", True, 8, 4, 2, scale=2.5),
        # a few sequences, a number of experts and of groups that is no power of two, bf16 logits in a wider row
        _route("route_odd_37", 37, 60, 5, "softmax", False, 6, 3, 1, renorm=False, scale=16.0, logits="bf16", pad=3),
        # a prompt chunk through this repository's layer (512 experts, ten chosen, a shared one), softmax with a bias
        _route("route_1536", 1536, 512, 10, "softmax", True, shared=True),
        # a batch of long prompts, grouped: bandwidth
        _route("route_32768", 32768, 256, 8, "sigmoid", True, 8, 4, 2, scale=2.5),
        # one sequence decoding with its adapter: latency
        _lora("lora_1", 1, 4096, 4096, 16, 32, 1),
        # sixty-four sequences decoding, most with an adapter of their own: the adapters' weights
        _lora("lora_64", 64, 8192, 4096, 16, 64, 64),
        # odd widths, ranks that differ, tokens without an adapter, fp32 rows that are slices of wider ones
        _lora("lora_odd_100", 100, 1000, 1056, 24, 7, 13, x="f32", out="f32", ranks=True, without=0.3, pad=5),
        # a batch of prompts of ragged lengths, an adapter each
        _lora("lora_8192", 8192, 4096, 4096, 64, 16, 11),
        # one sequence decoding: residual and the next block's norm
        _norm("norm_1", 1, 4096),
        # the sum over eleven expert outputs of 64 sequences, residual, the next block's norm
        _norm("norm_slots_64", 64, 4096, slots=11, y="f32"),
        # an odd width, norms on both sides, a gate per element through silu, an fp32 residual stream
        _norm("norm_odd_333", 333, 2084, y="bf16", h="f32", post=True, gate="full", act="silu", alpha=0.5, pad=3),
        # a long prompt: norms on both sides, a scale per channel
        _norm("norm_8192", 8192, 4096, post=True, gate="channel", offset=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: max((work(c)["bytes"], work(c)["flops"]) for c in listed() if c["op"] == op) for op in ("route", "lora", "norm")}
    while True:
        op = rng.choice(["route", "lora", "norm"])
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 6, 8, 8, 12, 16])
            E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
            chosen = rng.randint((groups + 1) // 2, groups)
            K = rng.randint(1, min(12, chosen * (E // groups)))
            case = _route("", _log(rng, 1, 32768), E, K, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.7, groups, chosen,
                          rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.4,
                          rng.choice(["f32", "f32", "bf16"]), rng.choice([0, 0, 0, 3, 8]))
        elif op == "lora":
            T = _log(rng, 1, 8192)
            adapters = _log(rng, 1, 64)
            case = _lora("", T, _log(rng, 16, 16384), 8 * _log(rng, 1, 2048), 8 * _log(rng, 1, 16), adapters,
                         _log(rng, 1, min(T, 128)), rng.choice(["bf16", "bf16", "bf16", "f32"]),
                         rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.random() < 0.8, rng.random() < 0.3,
                         rng.choice([0.0, 0.0, 0.2]), rng.choice([0, 0, 0, 8, 5]))
        else:
            slots = rng.choice([1, 1, 1, 2, 9, 11])
            case = _norm("", _log(rng, 1, 8192), _log(rng, 64, 8192), slots, "f32" if slots > 1 else rng.choice(["bf16", "bf16", "f32"]),
                         rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.8, rng.random() < 0.5,
                         rng.choice(["none", "none", "token", "channel", "full"]), rng.choice(["none", "sigmoid", "silu"]),
                         rng.choice([1.0, 0.5]), rng.choice([1.0, 0.75]), rng.choice([0.0, 1.0]), rng.choice([0, 0, 8, 3]))
        w = work(case)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            del case["name"]
            return case


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        by = T * E * SIZE[case["logits"]] + (4 * E if case["bias"] else 0) + T * (K + int(case["shared"])) * 8
        return {"bytes": int(by), "flops": int(4 * T * E)}
    if case["op"] == "lora":
        N, K, R = case["N"], case["K"], case["R"]
        used = min(case["adapters"], case["runs"])
        with_one = T * (1.0 - case["without"])
        by = (with_one * K * SIZE[case["x"]] + T * N * SIZE[case["out"]] * (2 if case["residual"] else 1) + used * R * (K + N) * 2 + 4 * T)
        return {"bytes": int(by), "flops": int(2 * with_one * R * (K + N))}
    H, n = case["H"], T * case["H"]
    by = n * case["slots"] * SIZE[case["y"]] + n * SIZE[case["h"]] * (2 if case["residual"] else 1) + n * 2 + 2 * H * (2 if case["post"] else 1)
    by += {"none": 0, "token": 2 * T, "channel": 2 * H, "full": 2 * n}[case["gate"]]
    return {"bytes": int(by), "flops": int(n * (case["slots"] + 6 + (4 if case["post"] else 0)))}


# ----------------------------------------------------------------- inputs

def _rows(normal, T, width, pad, dtype):
    """[T, width] rows that are slices of wider ones by `pad`."""
    return normal(T, width + pad).to(dtype)[:, :width]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *n: torch.randn(n, dtype=torch.float32, device=DEV, generator=g)  # noqa: E731
    s, T = dict(case), case["T"]
    if case["op"] == "route":
        E = case["E"]
        # some experts are liked by most tokens, which the bias (found while training) works against
        liking = 0.7 * normal(E)
        s["l"] = (1.3 * normal(T, E + case["pad"]) + torch.cat([liking, normal(case["pad"])])).to(TYPES[case["logits"]])[:, :E]
        s["b"] = None
        if case["bias"]:
            spread = 0.1 if case["score"] == "sigmoid" else 0.5 / E
            s["b"] = spread * (0.5 * normal(E) - liking)
        s["ids"] = torch.empty((T, case["K"] + int(case["shared"])), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(s["ids"].shape, dtype=torch.float32, device=DEV)
    elif case["op"] == "lora":
        N, K, R, n = case["N"], case["K"], case["R"], case["adapters"]
        rng = np.random.RandomState(seed % (1 << 32))
        # `runs` stretches of tokens, each of one request with its adapter (or none); a stretch has a token at least
        cuts = np.sort(rng.choice(T - 1, case["runs"] - 1, replace=False) + 1) if case["runs"] > 1 else []
        of_run = np.concatenate([rng.permutation(n) for _ in range(-(-case["runs"] // n))])[:case["runs"]]
        of_run = np.where(rng.rand(case["runs"]) < case["without"], -1, of_run)
        ids = np.repeat(of_run, np.diff(np.concatenate([[0], cuts, [T]])).astype(int)).astype(np.int32)
        s["adapter"] = torch.from_numpy(ids).to(DEV)
        s["rank"] = None
        if case["ranks"]:
            s["rank"] = torch.from_numpy(rng.randint(1, R + 1, n).astype(np.int32)).to(DEV)
        s["x"] = _rows(normal, T, K, case["pad"], TYPES[case["x"]])
        s["a"] = (normal(n, R, K) / math.sqrt(K)).bfloat16()
        s["bt"] = (normal(n, N, R) / math.sqrt(R)).bfloat16()
        s["scale"] = 0.25 + 0.5 * torch.rand(n, device=DEV, generator=g)
        s["res"] = _rows(normal, T, N, case["pad"], TYPES[case["out"]]) if case["residual"] else None
        s["out_rows"] = _rows(normal, T, N, case["pad"], TYPES[case["out"]])
        # which rows each adapter has, and how many of its ranks count (what a program knows from its batch)
        ranks = s["rank"].tolist() if case["ranks"] else [R] * n
        s["groups_of"] = [(int(a), torch.from_numpy(np.nonzero(ids == a)[0]).to(DEV), ranks[a]) for a in np.unique(ids) if a >= 0]
    else:
        H, S = case["H"], case["slots"]
        s["yv"] = _rows(normal, T * S, H, case["pad"], TYPES[case["y"]])
        # the residual stream has a few channels that are much larger than the others
        s["hv"] = None
        if case["residual"]:
            big = torch.where(torch.rand(H + case["pad"], device=DEV, generator=g) < 0.005, 30.0, 1.0)
            s["hv"] = (normal(T, H + case["pad"]) * big).to(TYPES[case["h"]])[:, :H]
        s["post_w"] = (1.0 - case["offset"] + 0.1 * normal(H)).bfloat16() if case["post"] else None
        s["pre_w"] = (1.0 - case["offset"] + 0.1 * normal(H)).bfloat16()
        s["gatev"] = {"none": lambda: None, "token": lambda: normal(T, 1).bfloat16(), "channel": lambda: normal(1, H).bfloat16(),
                      "full": lambda: normal(T, H).bfloat16()}[case["gate"]]()
        s["h_out"] = torch.empty((T, H), dtype=TYPES[case["h"]], device=DEV)
        s["n_out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ passes

def _plain_route(s):
    # in 64 bits: the order of values that lie next to one another decides
    x = s["l"].double()
    T, E, G, K = s["T"], s["E"], s["groups"], s["K"]
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    c = p if s["b"] is None else p + s["b"].double()
    if s["chosen"] < G:
        by_group = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0][:, :, :s["top"]].sum(2)
        best = torch.sort(by_group, dim=1, descending=True, stable=True)[1][:, :s["chosen"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        c = torch.where(kept.repeat_interleave(E // G, 1), c, -math.inf)
    ids = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :K]
    w = torch.gather(p, 1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * s["scale"]).float()
    if s["shared"]:
        ids = torch.cat([ids, torch.full_like(ids[:, :1], E)], 1)
        w = torch.cat([w, torch.ones_like(w[:, :1])], 1)
    return ids.int(), w


def _plain_lora(s):
    # (a copy: the sums below must not go into the residual itself)
    out = s["res"].to(torch.float32, copy=True) if s["res"] is not None else torch.zeros((s["T"], s["N"]), device=DEV)
    for a, rows, rank in s["groups_of"]:
        v = s["x"][rows].float() @ s["a"][a, :rank].float().t()
        out[rows] = out[rows] + s["scale"][a] * (v @ s["bt"][a, :, :rank].float().t())
    return out.to(TYPES[s["out"]])


def _plain_norm(s):
    T, H = s["T"], s["H"]
    u = s["yv"].float().view(T, s["slots"], H).sum(1) if s["slots"] > 1 else s["yv"].float()
    if s["post"]:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + 1e-6) * (s["post_w"].float() + s["offset"])
    if s["gatev"] is not None:
        z = s["gatev"].float()
        u = u * {"none": z, "sigmoid": 1.0 / (1.0 + torch.exp(-z)), "silu": z / (1.0 + torch.exp(-z))}[s["act"]]
    h = s["alpha"] * u
    if s["hv"] is not None:
        h = s["beta"] * s["hv"].float() + h
    n = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * (s["pre_w"].float() + s["offset"])
    return h.to(TYPES[s["h"]]), n.bfloat16()


def run(state):
    s = state
    if not own:
        return {"route": _plain_route, "lora": _plain_lora, "norm": _plain_norm}[s["op"]](s)
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    if s["op"] == "route":
        return libmoe.moe_route_grouped(s["l"], s["K"], s["b"], s["score"], s["groups"], s["chosen"], s["top"],
                                        with_shared=s["shared"], renormalize=s["renorm"], scale=s["scale"],
                                        topk_ids=s["ids"], topk_w=s["w"])
    if s["op"] == "lora":
        if "plan" not in s:  # made once for a batch and used by every projection of every layer
            s["plan"] = libmoe.moe_lora_plan(s["adapter"], s["adapters"])
        return libmoe.moe_lora(s["x"], s["a"], s["bt"], s["plan"], scale=s["scale"], ranks=s["rank"], residual=s["res"],
                               out=s["out_rows"])
    return libmoe.moe_combine_norm(s["yv"], s["hv"], slots=s["slots"], post_w=s["post_w"], gate=s["gatev"], gate_act=s["act"],
                                   alpha=s["alpha"], beta=s["beta"], pre_w=s["pre_w"], w_offset=s["offset"], eps=1e-6,
                                   h_out=s["h_out"], n_out=s["n_out"])


# ----------------------------------------------------------- 64-bit values

def _exact_route(case, s):
    x = s["l"].double().cpu().numpy()
    T, E, G, K = case["T"], case["E"], case["groups"], case["K"]
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + np.exp(-x))
    else:
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    c = p.copy() if s["b"] is None else p + s["b"].double().cpu().numpy()
    if case["chosen"] < G:
        size = E // G
        value = np.sort(c.reshape(T, G, size), axis=2)[:, :, size - case["top"]:].sum(2)
        # a group stays where fewer than `chosen` others come before it: larger, or as large with a lower number
        before = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & (np.arange(G)[None, :] < np.arange(G)[:, None]))
        c[np.repeat(before.sum(2) >= case["chosen"], size, axis=1)] = -np.inf
    ids = np.empty((T, K + int(case["shared"])), dtype=np.int32)
    w = np.ones((T, K + int(case["shared"])))
    for k in range(K):  # the first of the largest that are left
        ids[:, k] = c.argmax(1)
        w[:, k] = p[np.arange(T), ids[:, k]]
        c[np.arange(T), ids[:, k]] = -np.inf
    if case["renorm"]:
        w[:, :K] /= w[:, :K].sum(1, keepdims=True)
    w[:, :K] *= case["scale"]
    if case["shared"]:
        ids[:, K] = E
    return torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "lora":
        N, R = case["N"], case["R"]
        out = torch.zeros((T, N), dtype=torch.float64, device=DEV)
        if case["residual"]:
            out += s["res"]
        for a in range(case["adapters"]):
            mine = s["adapter"] == a
            if not bool(mine.any()):
                continue
            rank = R if s["rank"] is None else int(s["rank"][a])
            inner = torch.einsum("tk,rk->tr", s["x"][mine].double(), s["a"][a, :rank].double())
            out[mine] += float(s["scale"][a]) * torch.einsum("tr,nr->tn", inner, s["bt"][a, :, :rank].double())
        return out
    H, S = case["H"], case["slots"]
    y, n, hs = s["yv"].double(), [], []
    for t0 in range(0, T, 1024):
        t1 = min(T, t0 + 1024)
        u = torch.zeros((t1 - t0, H), dtype=torch.float64, device=DEV)
        for j in range(S):
            u += y[t0 * S + j:t1 * S:S]
        if case["post"]:
            u = u / torch.sqrt(u.pow(2).sum(1) / H + 1e-6)[:, None] * (s["post_w"].double() + case["offset"])
        if s["gatev"] is not None:
            z = s["gatev"].double()
            z = z if z.shape[0] == 1 else z[t0:t1]
            if case["act"] != "none":
                sig = torch.where(z >= 0, 1.0 / (1.0 + torch.exp(-z)), 1.0 - 1.0 / (1.0 + torch.exp(z)))
                z = sig if case["act"] == "sigmoid" else z * sig
            u = u * z
        h = u * case["alpha"]
        if case["residual"]:
            h = h + case["beta"] * s["hv"][t0:t1].double()
        hs.append(h)
        n.append(h / torch.sqrt(h.pow(2).sum(1) / H + 1e-6)[:, None] * (s["pre_w"].double() + case["offset"]))
    return torch.cat(hs), torch.cat(n)
