"""Decode steps of a small MXFP4 decoder with libmoe: projections through
moe_linear_mxfp4act, the mixture-of-experts layer through moe_layer_few (up to 16
sequences), one CUDA graph per step.

    python examples/decode_step.py [--layers 4] [--batch 4] [--steps 64] [--small]

A block is  h += W_out mix(W_in norm(h));  h += moe(norm(h))  and the model ends in
norm and an fp32 output head.  `mix` (here a gated running mean, one state per
sequence) stands where a model has its attention, which libmoe does not do; the
prompt runs through the same calls, many tokens at a time, with moe_layer for
the experts.  Weights are random: the text is not.
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


def main():
    import torch
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=64)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--small", action="store_true", help="a tiny model")
    a = p.parse_args()
    size = dict(hidden=256, inner=128, experts=8, top_k=2, vocab=1000) if a.small else {}
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
