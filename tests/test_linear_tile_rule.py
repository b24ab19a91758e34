"""The text of the rules by which moe_linear_mxfp4act picks its kernel, as tests/test_gpu_linear_large.py
restates them: whoever changes one of them sees here that the cases there may reach other code.
CPU only: the source is read."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_mixture_experts_softmax_gb300",
                      "csrc", "linear_mxfp4.cu")


def test_the_rules_are_the_ones_restated():
    with open(SOURCE) as f:
        text = re.sub(r"\s+", " ", f.read())
    for rule in (
        "bool use_pairs(int T, int N) { return T > 64 && N >= 128; }",
        "const long long mts = (p.T + 255) / 256, most = num_sms() / 2;",
        "w256 = (mts * ((p.N + 255) / 256) + most - 1) / most, w128 = (mts * ((p.N + 127) / 128) + most - 1) / most;",
        "return 4 * w128 <= 5 * w256 ? launch_pair<128>",
        "const long long tiles = (long long)row_tiles(p.N) * ((p.T + NT - 1) / NT);",
        "while (splits < 8 && 2 * splits <= nk && tiles * 2 * splits <= 2LL * num_sms()) splits *= 2;",
        "if (p.T <= 16) return launch_stream<16, false>", "if (p.T <= 32) return launch_stream<32, false>",
        "if (p.T <= 64) return launch_stream<64, false>", "return launch_stream<128, false>",
    ):
        assert rule in text, rule
