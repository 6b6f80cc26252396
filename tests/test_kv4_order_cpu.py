"""Orders in the sources of the attention block's kernels that no run without a deadlock would show."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _kernel(file, name):
    """The text of a __global__ function without its comments."""
    src = open(os.path.join(ROOT, "moe_layer_tail_gb300", "csrc", file)).read()
    src = re.sub(r"//[^\n]*", "", src)
    at = src.index(name + "(const __grid_constant__")
    depth, i = 0, src.index("{", at)
    for j in range(i, len(src)):
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        if depth == 0:
            return src[i:j]


def test_tensor_memory_is_taken_behind_the_previous_kernels():
    # a CTA that holds tensor memory while it waits for an earlier kernel locks up with one that has
    # yet to allocate its own on the same SM
    body = _kernel("k_kv4_tc.cu", "k_kv4_attn")
    alloc = [m.start() for m in re.finditer(r"tcgen05\.alloc", body)]
    waits = [m.start() for m in re.finditer(r"pdl_wait\(\)", body)]
    assert len(alloc) == 1 and waits
    # the last wait in front of the allocation stands in the same block: nothing between them closes it
    before = [w for w in waits if w < alloc[0]]
    assert before and max(waits) < alloc[0]
    between = body[before[-1]:alloc[0]]
    assert between.count("}") == 0
