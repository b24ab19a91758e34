"""The calls between the products from several Python threads at once, each on a stream of its own."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import test_gpu_lora as lora  # noqa: E402

BF16 = torch.bfloat16


def test_threads_side_by_side():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe as m
    m.load()
    torch.manual_seed(0)
    results, failed = {}, []

    def work(i, T, H, tile):
        # first calls are among these: each thread has kernels of its own to load
        a, b, scale = lora.adapters(3, H, H, 16 << i)
        y, h, w = torch.randn((T, H), device="cuda").to(BF16), torch.randn((T, H), device="cuda").to(BF16), torch.ones(H, device="cuda").to(BF16)
        ids, logits = lora.ids_of(T, 3, 0.2, i), torch.randn((T, 64), device="cuda")
        plan = m.moe_lora_plan(ids, 3, tile)
        torch.cuda.synchronize()

        def step(stream=None):
            h1, n1 = m.moe_combine_norm(y, h=h, pre_w=w, stream=stream)
            z = m.moe_lora(n1, a, b, plan, scale=scale, residual=h1, stream=stream)
            return (z, *m.moe_route_grouped(logits, 6, None, "sigmoid", 8, 4, 2, stream=stream))

        def run():
            try:
                torch.cuda.set_device(0)
                results[i] = [step(stream) for _ in range(40)]
            except BaseException as e:  # noqa: BLE001 (a thread's failure is the test's)
                failed.append(e)
        stream = torch.cuda.Stream()
        return threading.Thread(target=run), step

    shapes = [(70, 512, 16), (700, 264, 128), (5000, 1032, 128)]
    made = [work(i, *s) for i, s in enumerate(shapes)]
    for t, _ in made:
        t.start()
    for t, _ in made:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for i, (_, step) in enumerate(made):
        want = step()
        assert all(torch.equal(x, y) for got in results[i] for x, y in zip(got, want))
    assert m.moe_device_error() == 0
