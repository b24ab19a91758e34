"""The settling of near-ties in route_grouped.cu ends by its own bound.  CPU only: the source is read as text."""
import re

from test_aligned_barriers import source


def test_the_exchange_of_neighbours_is_bounded():
    text = source("route_grouped.cu")
    text = text[text.index("int settle("):]
    loop = re.search(r"for \((int phase[^;]*);([^;]*);", text)
    bound = re.search(r"phase < (\w+)", loop.group(2))
    assert bound, loop.group(0)
    value = re.search(rf"constexpr int {bound.group(1)} = (\d+)", source("route_grouped.cu"))
    # 32 values are in order after 32 phases; two more see that nothing moves
    assert int(value.group(1) if value else bound.group(1)) >= 34
    # and the values are summed a second time at most
    assert not re.search(r"for \(;;\)|while \(true\)", text[:text.index("settle_ranks")])
