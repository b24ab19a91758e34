"""The decode example with prompts of every length class: short ones whose tokens fit the few-token
layer, and longer ones."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("batch,prompt,n", [(1, 8, 8), (2, 8, 8), (3, 5, 4), (1, 40, 9), (2, 9, 9), (17, 2, 1)])
def test_a_prompt_at_once_and_token_by_token(batch, prompt, n):
    """The same logits up to what test_a_step_against_plain_torch allows for (the layer in another
    form, h rounded in other places), and the same state."""
    from decode_step import Decoder
    m = Decoder(layers=2, hidden=256, inner=128, experts=8, top_k=2, vocab=500, batch=batch, prompt=prompt, seed=3)
    tokens = torch.randint(0, 500, (batch, n), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    whole = m.forward(tokens).clone()
    state = m.state.clone()
    m.state.zero_()
    for t in range(n):
        last = m.forward(tokens[:, t:t + 1]).clone()
    assert ((whole - last).norm() / last.norm()).item() <= 0.06
    assert ((state - m.state).norm() / m.state.norm()).item() <= 0.06
