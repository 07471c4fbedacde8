"""Masks of steps without parents (kv_assign): those of chains, whatever the step held before, so that tree_attention over
a step that is used again attends by that step's tokens."""

import random

import numpy as np
import pytest
import torch

from nvfp4_w4a16_moe_skinny_gb300 import binding
from oracle import step as OS
from tests.gpu_helpers import dev
from tests.test_gpu_step import State, i32, tree
from tests.test_gpu_tree import Trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("words,new,rows", [
    (1, [1], 1), (1, [64, 0, 3, -1, 63], 140), (1, [70, 2], 80), (2, [65, 128, 64, 1], 260), (4, [300, 5], 310), (64, [4096, 9], 4110),
    (1, [1] * 700, 705), (3, [130] * 8, 1500)])
def test_chains_without_parents(lib, words, new, rows):
    """One CTA and eight; requests longer than the words hold too; rows past the last one."""
    s = State([17] * len(new), -(-(17 + max(new)) // 16) + 1, 16, spare=sum(max(0, n) // 16 + 2 for n in new))
    step = binding.Step(len(new), rows, words)
    for again in range(2):
        kv_len, held, table, free, count = s.kv_len, s.held, s.table, s.free, s.count
        want = OS.assign(table, held, free, count, kv_len, new, rows, 16, None, words)
        pages, _ = s.check(lib, new, rows, words=words, step=step)      # (fills the step with other numbers first)
        assert step.masks.tolist() == want[4]
        s.kv_len, s.held, s.table, s.free, s.count = kv_len, held, table, free, count


def test_a_tree_step_then_a_chain(lib):
    """The same step object: drafted trees, then single tokens and a short prompt attend by themselves, eagerly and captured."""
    rng = random.Random(5)
    counts, chain = [9, 20, 5], [1, 12, 20]
    s = State([30, 0, 55], 9, 16, spare=20)
    pages, step = s.up(), binding.Step(3, 40, 1)
    new, kv_len = i32(counts), i32(s.kv_len)
    lib.kv_assign(pages, kv_len, new, step, i32([p for n in counts for p in tree(rng, n)] + [-1] * 6))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        lib.kv_assign(pages, kv_len, new, step)
    for turn in range(3):
        step.masks.fill_(-1 if turn else 5)
        new.copy_(i32(chain))
        if turn == 2:
            lib.kv_assign(pages, kv_len, new, step)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert lib.device_error() == 0 and step.cu_tokens.tolist() == [0, 1, 13, 33]
        c = Trees([(n, n + a) for n, a in zip(chain, [30, 0, 55])], 4, 2, 64, 16, False, seed=turn, kind="chain")
        assert torch.equal(step.masks[:33], c.masks()) and not step.masks[33:].any()
        out, lse = lib.tree_attention(c.q, c.cache(), c.batch(), step.masks[:33], with_lse=True)
        torch.cuda.synchronize()
        c.check(out, lse)


def test_a_step_without_words_or_masks(lib):
    """No masks to write: with words and without."""
    s = State([3, 40], 8, 16, spare=9)
    step = binding.Step(2, 9, 1)
    step.c.masks = None
    s.check(lib, [4, 3], 9, step=step)
    assert torch.all(step.masks == 99)                                   # (given as NULL: left as they were)
    step = binding.Step(2, 9, 0)
    s.check(lib, [1, 2], 9, step=step)
    assert np.asarray(step.masks.shape).tolist() == [9, 0]
