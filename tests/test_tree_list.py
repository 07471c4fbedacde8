"""The list through which a tree kernel's roles get their items (csrc/tree_list.cuh), walked on the host (no GPU): roles in
random order, waits that run out, roles that leave."""

import os
import re
import shutil
import subprocess

import pytest

from nvfp4_w4a16_moe_skinny_gb300 import build as B
from tests.test_tree_waits import code

CSRC = os.path.join(B.PKG, "csrc")


def test_items_hold_still_whoever_leaves(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "tree_list")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "tree_list.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-pthread", "-I" + CSRC, "-o", exe, src], check=True)
    got = subprocess.run([exe, "300"], capture_output=True, text=True, timeout=240)
    assert (got.returncode, got.stdout) == (0, "ok\n")


def test_the_kernel_has_its_items_through_the_list_alone():
    text = code("attention_chunk.cuh")
    uses = re.findall(r"items->\w+[^;,]*", text)
    assert uses == ["items->full + i", "items->empty + i"], uses  # (their initialisation)
    assert len(re.findall(r"\bput_item\(\*items", text)) == 1
