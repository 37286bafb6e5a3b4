"""Key/value cache: what can be said of its edges without a GPU."""
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_tq4_b200", "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_registers_change_hands_by_whole_warpgroups():
    """setmaxnreg is one instruction for the four warps of a warpgroup: each share
    is taken at one place, before the roles within a warpgroup part."""
    kernel = _code("tq_tcattention.cu").split("tc_attend_kernel(", 1)[1]
    shares = [m.start() for m in re.finditer(r"a_regs_(?:more|fewer)<", kernel)]
    assert len(shares) == 2
    within = kernel.index("warp != kMmaWarp")  # warps 12 and 13..15 go separate ways
    assert max(shares) < within


@pytest.mark.parametrize("name,begin", [
    ("tq_device.cuh", "rotate_unit_lane("), ("tq_prefill.cu", "prerotate_plain_kernel("),
    ("tq_gemv.cu", "unit_product("), ("tq_gemv.cu", "load_xwords(")])
def test_activations_are_read_by_ordinary_loads(name, begin):
    """What the kernel before may still be writing (a rotary or attention output, a
    pre-rotated activation) is not asked for by the read-only path."""
    body = _code(name).split(begin, 1)[1].split("\n}\n", 1)[0]
    assert not re.search(r"\b(load4<|__ldg\(|ldg_keep\(|ldg64\(|p_ldg128\()", body)
    read_only = set(re.findall(r"(\w+)\([^)]*\)\s*\{[^{}]*\basm volatile\(\"ld\.global\.nc", _code(name)))
    assert not any(re.search(r"\b%s\(" % f, body) for f in read_only)
