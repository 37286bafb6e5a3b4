"""Key/value cache: what can be said of its edges without a GPU."""
import os
import re

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE, CUDA, UNSUP, TIMEOUT = range(9)

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


@pytest.fixture(scope="module")
def tq():
    from dequant_gemv_tq4_b200 import build as b

    b.build()
    import dequant_gemv_tq4_b200 as tq

    tq.load_library()
    return tq


class _TwoDevices:
    """Device 1 current, a workspace that is larger on device 0: stands for
    torch.cuda and the size queries where there is no GPU."""

    def __init__(self, monkeypatch, tq):
        self.current, self.asked = 1, []
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        for name in ("zeros", "empty"):
            monkeypatch.setattr(torch, name, self.allocate)
        monkeypatch.setattr(torch.Tensor, "to", lambda t, to, *a: t if isinstance(to, torch.dtype) else self.allocate(t.shape, device=to))
        for name in ("tq_kv_attention_workspace_bytes", "tq_gemm_workspace_bytes", "tq_gemm_prefill_workspace_bytes"):
            monkeypatch.setattr(tq, name, lambda *a: 256 if self.current else 512)

    def device(self, index):
        state = self

        class Guard:
            def __enter__(self):
                self.before, state.current = state.current, index

            def __exit__(self, *a):
                state.current = self.before
        return Guard()

    def allocate(self, shape, dtype=None, device=None):
        self.asked.append((shape, device))
        return self


@pytest.mark.parametrize("device,want", [(0, 0), (None, 1), (1, 1)])
def test_device_zero_is_a_device(monkeypatch, tq, device, want):
    """With device 1 current, device=0 is device 0, and a workspace's size is that device's."""
    two = _TwoDevices(monkeypatch, tq)
    tq.kv_cache(2, 1, 64, device=device)
    tq.rope_frequencies(64, device=device)
    tq.workspace(4, 64, 64, device=device)
    tq.prefill_workspace(64, 64, device=device)
    assert [d for _, d in two.asked] == [want] * 5
    tq.kv_attention_workspace(2, 1, 4, 2, 64, device=device)
    assert two.asked[-1] == (256 if want else 512, want)


def test_a_type_asked_for_is_not_dropped(tq):
    """dtype beside an output of another type is refused (before a device is looked at)."""
    codes = torch.zeros(4, 2, 2, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(4, 2, 2, 16, 4, dtype=torch.int16)
    table, one = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, out = torch.zeros(1, 1, 2, 64), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    kv = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="^out: expected torch.float32"):
        tq.kv_attention(codes, scales, table, one, q, dtype=torch.float32, out=out)
    for name in "kv":
        with pytest.raises(ValueError, match="^%s: expected torch.bfloat16" % name):
            tq.kv_read(codes, scales, table, one, one, dtype=torch.bfloat16, **{name: kv})
    # the output's own type, or none: as far as a call without a GPU goes
    for dtype in (None, torch.bfloat16):
        with pytest.raises(ValueError, match="CUDA"):
            tq.kv_attention(codes, scales, table, one, q, dtype=dtype, out=out)
    for dtype in (None, torch.float16):
        with pytest.raises(ValueError, match="CUDA"):
            tq.kv_read(codes, scales, table, one, one, dtype=dtype, k=kv)


@pytest.mark.parametrize("name,kernel", [("tq_gemv.cu", "gemv_group_kernel("), ("tq_tcgemv.cu", "tc_gemv_kernel("),
                                         ("tq_prefill.cu", "prefill_kernel(")])
def test_a_product_reports_behind_the_launch_that_clears_its_status(name, kernel):
    """A product starts while the launch before it, which clears the status word, still runs:
    nothing is reported ahead of the wait for it."""
    body = _code(name).split(kernel, 1)[1]
    assert "atomicOr(P.header" in body
    assert body.index("grid_dependency_wait()") < body.index("atomicOr(P.header")
