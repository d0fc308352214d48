"""Warps whose lanes wait for different barriers order their memory before they go on.  No GPU needed."""
import os
import re

from ternary_weight_dp4a_gb300 import build

CSRC = os.path.dirname(os.path.abspath(build.__file__)) + "/csrc/"


def _waits(path):
    """(name, body) of every function of the file in which a warp votes on a wait's answer."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    found = []
    for m in re.finditer(r"__forceinline__ bool (\w+)\([^)]*\) \{\n(.*?)\n\}", text, re.S):
        if "__all_sync" in m[2]:
            found.append((m[1], m[2]))
    return found


def test_a_wait_of_the_4_bit_tile_kernel_orders_memory_between_the_lanes():
    """Its fold waits for an accumulator on even lanes and for the sums of x on odd ones, and all lanes read
    both: the vote alone orders nothing, __syncwarp behind it does."""
    waits = _waits(CSRC + "tq_q4_tile.cu")
    assert [name for name, _ in waits] == ["warp_wait"]
    for name, body in waits:
        assert "__syncwarp();" in body[body.index("__all_sync"):], name


def test_a_wait_of_the_expert_tile_kernel_orders_memory_between_the_lanes():
    """Its issuing warp waits for weights, activations and an accumulator on a lane each, and one lane then reads all."""
    waits = _waits(CSRC + "tq_moe_tile.cu")
    assert [name for name, _ in waits] == ["warp_wait_alive"]
    for name, body in waits:
        assert "__syncwarp();" in body[body.index("__all_sync"):], name
