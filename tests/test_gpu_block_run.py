"""The calls between the products in a run, as a decoder block makes them: sums and norms, projection with
adapters, grouped routing, experts.  Each step is compared with its own definition on the inputs that the run
gave it; the example's decoder is captured and replayed."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import test_gpu_combine_norm as norm  # noqa: E402
import test_gpu_lora as lora  # noqa: E402
import test_gpu_route_grouped as route  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    libmoe.load()
    yield libmoe
    assert libmoe.moe_device_error() == 0


def mx(m, *shape):
    w = torch.randn((int(np.prod(shape[:-1])), shape[-1]), device="cuda") / shape[-1] ** 0.5
    codes, scales = m.moe_quantize_mxfp4(w.bfloat16())
    return codes.view(*shape[:-1], -1), scales.view(*shape[:-1], -1)


@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_a_block(m, T):
    torch.manual_seed(T)
    H, I, E, K, G = 512, 128, 32, 4, 8
    h, y = torch.randn((T, H), device="cuda").bfloat16(), torch.randn((T, H), device="cuda").bfloat16()
    w = (1.0 + 0.1 * torch.randn(H, device="cuda")).bfloat16()
    ids = lora.ids_of(T, 3, 0.3)
    plan = m.moe_lora_plan(ids, 3)
    # stream and norm, a projection with its adapters
    h1, n1 = norm.check(m, y, h=h, pre_w=w, post_w=w)
    codes, scales = mx(m, H, H)
    a, b, scale = lora.adapters(3, H, H, 16)
    z = m.moe_linear_mxfp4act(n1, codes, scales)
    want = lora.check(m, n1, a, b, ids, scale=scale, residual=z.clone())[0]
    m.moe_lora(n1, a, b, plan, scale=scale, residual=z, out=z)
    assert torch.equal(z, want)
    h2, n2 = norm.check(m, z, h=h1, pre_w=w, alpha=0.5)
    # the experts, chosen by groups: their outputs a slot, and the sum of the slots with the next norm
    router = torch.randn((E, H), device="cuda") / H ** 0.5
    bias = 0.05 * torch.randn(E, device="cuda")
    logits = n2.float() @ router.T
    eid, ew = m.moe_route_grouped(logits, K, bias, "sigmoid", G, G // 2, 2, scale=2.0)
    want_ids, want_w = route.definition(logits.cpu().numpy(), K, bias.cpu().numpy(), "sigmoid", G, G // 2, 2, scale=2.0)
    assert np.array_equal(eid[:, :K].cpu().numpy(), want_ids) and (eid[:, K] == E).all()
    assert np.allclose(ew[:, :K].cpu().numpy(), want_w, rtol=1e-5)
    (w13, s13), (w2, s2) = mx(m, E + 1, 2 * I, H), mx(m, E + 1, H, I)
    perm = m.moe_permute(eid, E + 1, 8)
    ws = m.alloc_workspace(T, H, I, E + 1, K + 1, 8)
    m.moe_ffn_gate_up(n2, w13, s13, perm, ws, m.MOE_PATH_DECODE)
    m.moe_ffn_down(w2, s2, ew, perm, ws, T, m.MOE_PATH_DECODE)
    slots = m.ffn_views(ws, T, H, I, E + 1, K + 1, 8)[1]
    h3, n3 = norm.check(m, slots, slots=K + 1, h=h2, pre_w=w)
    # the same through the layer call and the sum of its output
    out = m.moe_layer(logits, n2, w13, s13, w2, s2, K, path=m.MOE_PATH_DECODE,
                      router=dict(bias=bias, n_groups=G, topk_groups=G // 2, scale=2.0))
    assert torch.equal(out, m.moe_combine(slots, T, H, K + 1, torch.empty_like(out)))
    # h3 adds before a rounding, the layer's output is rounded first: half a bf16 step of each
    two = h2.double() + out.double()
    assert ((h3.double() - two).abs() <= 2.0 ** -8 * (h3.double().abs() + out.double().abs()) + 1e-5).all()


def test_the_example_with_adapters(m):
    import decode_step
    d = decode_step.AdapterDecoder(3, layers=2, hidden=256, inner=128, experts=8, top_k=2, vocab=500, batch=5, prompt=32, seed=1)
    prompt = torch.randint(0, 500, (5, 32), device="cuda")
    d.tokens.copy_(d.forward(prompt).argmax(-1))
    start = d.tokens.clone(), d.state.clone()
    graph = d.capture()
    said = []
    for _ in range(6):
        graph.replay()
        said.append(d.tokens.clone())
    end = d.state.clone()
    d.tokens.copy_(start[0])
    d.state.copy_(start[1])
    for want in said:
        d.step()
        assert torch.equal(d.tokens, want)
    assert torch.equal(d.state, end)
    # a sequence without an adapter does not depend on them, one with its own does
    d.tokens.copy_(start[0])
    d.state.copy_(start[1])
    before = d.forward(d.tokens[:, None]).clone()
    for pair in d.pairs:
        for a, _ in pair:
            a.mul_(-1.0)
    d.state.copy_(start[1])
    after = d.forward(d.tokens[:, None])
    none = d.adapter < 0
    assert none.any() and torch.equal(after[none], before[none])
    assert not (after[~none] == before[~none]).all(1).any()


def test_in_place_calls_one_after_another(m):
    """A stream that is updated in place by call after call, each launched while the one before still runs: rows and
    columns of neighbouring blocks share cache lines (widths that are no multiple of 128 bytes)."""
    torch.manual_seed(0)
    for T, N, tile in ((70, 200, 16), (400, 264, 128), (33, 77, 16)):
        a, b, scale = lora.adapters(3, N, 64, 16)
        x, ids = torch.randn((T, 64), device="cuda").bfloat16(), lora.ids_of(T, 3, 0.2)
        w = torch.ones(N, device="cuda").bfloat16()
        plan = m.moe_lora_plan(ids, 3, tile)
        start = torch.randn((T, N), device="cuda").bfloat16()

        def chain(h, sync):
            for _ in range(12):
                m.moe_lora(x, a, b, plan, scale=scale, residual=h, out=h)
                sync()
                m.moe_combine_norm(h, h, pre_w=w, alpha=0.25, beta=0.5, h_out=h, n_out=False)
                sync()
            return h
        want = chain(start.clone(), torch.cuda.synchronize)
        for _ in range(5):
            assert torch.equal(chain(start.clone(), lambda: None), want)
