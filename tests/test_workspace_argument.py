"""What the bindings of the few-token layer and the projection ask of a caller's workspace.  CPU
only: refused before the library is called."""
import pytest

torch = pytest.importorskip("torch")

from test_stream_argument import SIDE, few, gpu, linear, recorded  # noqa: E402,F401


@pytest.mark.parametrize("name,args", [("moe_layer_few", few), ("moe_linear_mxfp4act", linear)])
def test_refusals(recorded, name, args):  # noqa: F811
    libmoe, _ = recorded
    call = getattr(libmoe, name)
    on_host = torch.ones(1 << 20, dtype=torch.uint8)
    with pytest.raises(AssertionError, match="workspace"):
        call(**args(), workspace=on_host, stream=SIDE)
    with pytest.raises(AssertionError, match="workspace"):
        call(**args(), workspace=gpu(on_host)[::2], stream=SIDE)
    call(**args(), workspace=gpu(on_host), stream=SIDE)


def test_initialisation_refusals(recorded):  # noqa: F811
    libmoe, _ = recorded
    with pytest.raises(AssertionError, match="workspace"):
        libmoe.moe_layer_few_workspace_init(torch.ones(256, dtype=torch.uint8), stream=SIDE)


def test_sizes_count_bytes(recorded, monkeypatch):  # noqa: F811
    """A workspace of another element type counts by its bytes."""
    libmoe, _ = recorded
    sizes = []
    monkeypatch.setattr(type(libmoe._lib), "moe_linear_mxfp4act", lambda self, *a: sizes.append(a[-2]) or 0, raising=False)
    libmoe.moe_linear_mxfp4act(**linear(), workspace=gpu(torch.ones(1024, dtype=torch.int32)), stream=SIDE)
    assert sizes == [4096]


def test_the_message_names_no_other_call():
    from mxfp4_mixture_experts_softmax_gb300 import libmoe
    text = libmoe.status_string(libmoe.MOE_ERR_WORKSPACE_TOO_SMALL)
    assert "moe_ffn_workspace_size" not in text and "workspace" in text
