"""Waits of the tree kernels that run out (no GPU).

After such a wait a role of attention's tcgen05 kernel goes on without waiting, reports, and ends.  The causal kernel's roles
walk the same items in step and may meet at barriers of a group of warps; a tree's read a list, which a warp leaves as
soon as one of its waits has run out, so that no other may wait for it without a limit."""

import os
import re

from nvfp4_w4a16_moe_skinny_gb300 import build as B

CSRC = os.path.join(B.PKG, "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, start):
    """From `start` to the end of the braces that it opens."""
    at = text.index("{", start)
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[start:end]


def test_no_barrier_without_a_limit_between_a_trees_roles():
    text = code("attention_chunk.cuh")
    arrive = block(text, text.index("bool last_to_arrive("))
    kernel = block(text, text.index("attn_chunk_kernel(const AttnJob p"))
    named = r"bar\.(?:sync|arrive|red)|barrier\.(?:cta|sync|arrive|red|cluster)"
    # named barriers: only in the causal kernel's join
    assert len(re.findall(named, arrive)) == 2
    assert not re.search(named, text.replace(arrive, "")), "a named barrier beside last_to_arrive's"
    assert len(re.findall(r"last_to_arrive<", text)) == 1
    assert "last_to_arrive<" in block(kernel, kernel.index("if (!kTree && !pc.whole)"))
    # all threads of the block meet before the roles part and after they have ended
    roles = block(kernel, kernel.index("if (warp < T::kSoft0)"))
    softmax = block(kernel, kernel.index(roles) + len(roles))
    assert "__syncthreads" not in roles + softmax and "hand_q" in softmax
