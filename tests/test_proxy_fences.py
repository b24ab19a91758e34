"""Shared memory that ordinary stores have written goes to TMA copies only behind a fence between the two proxies: a
barrier orders ordinary accesses among themselves, not with copies to the same addresses.  CPU only: the source is
read as text."""
import re

from test_aligned_barriers import source

FENCE = "fence.proxy.async.shared::cta"


def test_adapters_rings_over_the_sums():
    """lora_prompt.cu: the epilogue's rings of residual and output lie where v's parts and their sums were."""
    text = source("lora_prompt.cu")
    # the summing warps: after their last ordinary access to that memory, before they say so
    last, ready = text.index("sums_row[c + k]"), text.index("mbar_arrive(&v_ready)")
    assert last < ready and FENCE in text[last:ready]
    # every warp that copies into it: after it has heard so, before its first copy
    run = text[text.index("if (run) {"):]
    heard = re.search(r"mbar_wait_warp\(&v_ready, 0\)", run).end()
    first = re.search(r"\bfetch\(j\)", run).start()
    assert heard < first and FENCE in run[heard:first]
