"""Decode steps of a small MXFP4 decoder with libmoe: projections through
moe_linear_mxfp4act, the mixture-of-experts layer through moe_layer_few (up to 16
sequences), one CUDA graph per step.

    python examples/decode_step.py [--layers 4] [--batch 4] [--steps 64] [--small] [--adapters 3]

A block is  h += W_out mix(W_in norm(h));  h += moe(norm(h))  and the model ends in
norm and an fp32 output head.  `mix` (here a gated running mean, one state per
sequence) stands where a model has its attention, which libmoe does not do; the
prompt runs through the same calls, many tokens at a time, with moe_layer for
the experts.  Weights are random: the text is not.

With --adapters each sequence has a low-rank adapter of its own beside every
projection (moe_lora), experts are chosen by sigmoid scores with a bias and in
groups (moe_route_grouped), and residual and norms between the blocks are one call
(moe_combine_norm).
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Linear:
    """An MXFP4 projection with its workspace for batches of up to `tokens`."""

    def __init__(self, n, k, tokens, gen):
        import torch
        from mxfp4_mixture_experts_softmax_gb300 import libmoe
        w = torch.randn((n, k), device="cuda", generator=gen) / k ** 0.5
        self.codes, self.scales = libmoe.moe_quantize_mxfp4(w.bfloat16())
        sizes = [libmoe.moe_linear_mxfp4act_workspace_size(t, n, k) for t in (1, 16, 17, 64, 65, tokens) if t <= tokens]
        self.workspace = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def __call__(self, x, residual=None, out=None, out_dtype=None):
        from mxfp4_mixture_experts_softmax_gb300 import libmoe
        return libmoe.moe_linear_mxfp4act(x, self.codes, self.scales, residual=residual, out=out, out_dtype=out_dtype,
                                          workspace=self.workspace)


class Experts:
    """Router and expert weights of one layer, a shared expert gated per token; calls of up to `tokens`."""

    def __init__(self, hidden, inner, experts, top_k, tokens, gen):
        import torch
        from mxfp4_mixture_experts_softmax_gb300 import libmoe

        def weight(rows, k):
            w = torch.randn(((experts + 1) * rows, k), device="cuda", generator=gen) / k ** 0.5
            codes, scales = libmoe.moe_quantize_mxfp4(w.bfloat16())
            return codes.view(experts + 1, rows, k // 2), scales.view(experts + 1, rows, k // 32)
        self.k = top_k
        self.router = (torch.randn((experts, hidden), device="cuda", generator=gen) * 2 / hidden ** 0.5).bfloat16()
        self.gate = (torch.randn(hidden, device="cuda", generator=gen) / hidden ** 0.5).bfloat16()
        self.w13, self.s13 = weight(2 * inner, hidden)
        self.w2, self.s2 = weight(hidden, inner)
        # a short prompt takes the few-token layer as the decode steps do
        self.workspace = libmoe.alloc_workspace_few(min(tokens, libmoe.MOE_LAYER_FEW_MAX_T), hidden, inner, experts, top_k)

    def __call__(self, x):
        import torch
        from mxfp4_mixture_experts_softmax_gb300 import libmoe
        if x.shape[0] <= libmoe.MOE_LAYER_FEW_MAX_T:
            return libmoe.moe_layer_few(x, self.router, self.w13, self.s13, self.w2, self.s2, self.k,
                                        w_shared_gate=self.gate, workspace=self.workspace)[0]
        shared_w = torch.sigmoid(x.float() @ self.gate.float())
        _, w, perm = libmoe.moe_route_permute(x.float() @ self.router.float().T, self.k, 64, shared_w=shared_w)
        return libmoe.moe_ffn(x, self.w13, self.s13, self.w2, self.s2, w, perm)


class Decoder:
    def __init__(self, layers=4, hidden=2048, inner=1024, experts=64, top_k=8, vocab=32000, batch=4, prompt=256, seed=0):
        import torch
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        most = max(batch, batch * prompt)
        self.embed = torch.randn((vocab, hidden), device="cuda", generator=gen).bfloat16()
        self.blocks = [(Linear(2 * hidden, hidden, most, gen), Linear(hidden, hidden, most, gen),
                        Experts(hidden, inner, experts, top_k, most, gen)) for _ in range(layers)]
        self.head = Linear(vocab, hidden, batch, gen)
        self.state = torch.zeros((layers, batch, hidden), device="cuda")  # mix's running means
        self.tokens = torch.zeros(batch, dtype=torch.long, device="cuda")
        self.logits = torch.empty((batch, vocab), device="cuda")
        self.batch, self.hidden = batch, hidden

    @staticmethod
    def norm(h):
        return (h.float() * (h.float().pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()).bfloat16()

    def _mix(self, i, z):
        """z [batch * n, 2 hidden], n tokens of each sequence in order: v gated by a running mean."""
        import torch
        n = z.shape[0] // self.batch
        v, g = z.view(self.batch, n, 2, self.hidden).float().unbind(2)
        mixed = []
        for t in range(n):
            self.state[i] = 0.9 * self.state[i] + 0.1 * v[:, t]
            mixed.append(self.state[i] * g[:, t].sigmoid())
        return torch.stack(mixed, 1).flatten(0, 1).bfloat16()

    def forward(self, tokens):
        """tokens [batch, n] -> fp32 logits [batch, vocab] of the last one; advances the state."""
        h = self.embed[tokens.reshape(-1)]
        for i, (w_in, w_out, experts) in enumerate(self.blocks):
            h = w_out(self._mix(i, w_in(self.norm(h))), residual=h)
            h = h + experts(self.norm(h))
        last = h.view(self.batch, -1, self.hidden)[:, -1]  # a strided slice: the head reads it as it lies
        return self.head(self.norm(last), out=self.logits)

    def step(self):
        """One greedy step of every sequence, in place (so that it can be captured)."""
        self.tokens.copy_(self.forward(self.tokens[:, None]).argmax(-1))

    def capture(self):
        """A CUDA graph of one step (which it also runs, once before the capture)."""
        import torch
        saved = self.tokens.clone(), self.state.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step()
        torch.cuda.current_stream().wait_stream(s)
        self.tokens.copy_(saved[0])
        self.state.copy_(saved[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


class AdapterDecoder(Decoder):
    """The same model with an adapter for each sequence, grouped sigmoid routing, and sums and norms in one
    call.  n is the normed stream that a block reads, h the stream itself."""

    def __init__(self, adapters=3, rank=16, groups=4, seed=0, **size):
        import torch
        super().__init__(seed=seed, **size)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + 1)

        def pair(linear):
            n, k = linear.codes.shape[0], 2 * linear.codes.shape[1]
            a = torch.randn((adapters, rank, k), device="cuda", generator=gen) / k ** 0.5
            b = torch.randn((adapters, n, rank), device="cuda", generator=gen) / rank ** 0.5
            return a.bfloat16(), b.bfloat16()
        self.pairs = [(pair(w_in), pair(w_out)) for w_in, w_out, _ in self.blocks]
        self.scale = torch.full((adapters,), 0.5, device="cuda")
        self.adapter = (torch.arange(self.batch, device="cuda") % (adapters + 1) - 1).int()  # -1: none
        self.adapters, self.groups = adapters, groups
        self.bias = [0.05 * torch.randn(e.router.shape[0], device="cuda", generator=gen) for _, _, e in self.blocks]
        self.norm_w = torch.ones(self.hidden, device="cuda").bfloat16()

    def _experts(self, i, n):
        import torch
        from mxfp4_mixture_experts_softmax_gb300 import libmoe
        e = self.blocks[i][2]
        logits = n.float() @ e.router.float().T
        shared_w = torch.sigmoid(n.float() @ e.gate.float())
        return libmoe.moe_layer(logits, n, e.w13, e.s13, e.w2, e.s2, e.k, tile_m=8 if n.shape[0] <= 64 else 64,
                                router=dict(bias=self.bias[i], n_groups=self.groups, topk_groups=self.groups // 2, scale=2.0,
                                            shared_w=shared_w))

    def forward(self, tokens):
        from mxfp4_mixture_experts_softmax_gb300 import libmoe
        h = self.embed[tokens.reshape(-1)]
        plan = libmoe.moe_lora_plan(self.adapter.repeat_interleave(tokens.shape[1]), self.adapters)  # one a step
        _, n = libmoe.moe_combine_norm(h, pre_w=self.norm_w, h_out=False)
        for i, (w_in, w_out, _) in enumerate(self.blocks):
            (a_in, b_in), (a_out, b_out) = self.pairs[i]
            z = w_in(n)
            libmoe.moe_lora(n, a_in, b_in, plan, scale=self.scale, residual=z, out=z)
            mixed = self._mix(i, z)
            y = w_out(mixed)
            libmoe.moe_lora(mixed, a_out, b_out, plan, scale=self.scale, residual=y, out=y)
            h, n = libmoe.moe_combine_norm(y, h, pre_w=self.norm_w)
            h, n = libmoe.moe_combine_norm(self._experts(i, n), h, pre_w=self.norm_w)
        return self.head(n.view(self.batch, -1, self.hidden)[:, -1], out=self.logits)


def main():
    import torch
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=64)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--small", action="store_true", help="a tiny model")
    p.add_argument("--adapters", type=int, default=0, help="low-rank adapters, of which each sequence has one or none")
    a = p.parse_args()
    size = dict(hidden=256, inner=128, experts=8, top_k=2, vocab=1000) if a.small else {}
    if a.adapters:
        m = AdapterDecoder(a.adapters, layers=a.layers, batch=a.batch, prompt=a.prompt, **size)
    else:
        m = Decoder(layers=a.layers, batch=a.batch, prompt=a.prompt, **size)
    prompt = torch.randint(0, m.embed.shape[0], (a.batch, a.prompt), device="cuda")
    m.tokens.copy_(m.forward(prompt).argmax(-1))
    graph = m.capture()
    graph.replay()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / a.steps * 1e3
    assert libmoe.moe_device_error() == 0
    print(f"{a.layers} layers, {a.batch} sequences: {ms:.3f} ms a step, {a.batch / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
