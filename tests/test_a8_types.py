"""The result's type of the 8-bit calls: out_dtype makes a new result, a given
y keeps its own type, and the two may not disagree."""

import pytest
import torch

import bit_weight_only_q4g64_amd as q4
from tests.gpu_helpers import DEV


def calls(dev):
    x, gamma = torch.ones((4, 256), dtype=torch.bfloat16, device=dev), torch.ones(256, device=dev)
    a = q4.Act8(torch.ones((4, 256), device=dev).to(torch.float8_e4m3fn), torch.ones((2, 4), device=dev))
    p = torch.zeros(q4.fp8b_packed_bytes(256, 256), dtype=torch.uint8, device=dev)
    return (lambda **kw: q4.rms_norm(x, gamma, 1e-5, **kw)), (lambda **kw: q4.qmm_a8_fp8b(p, None, 256, 256, a, **kw))


def test_a_type_that_is_not_ys_is_refused():
    types = (torch.bfloat16, torch.float32)
    for call in calls("cpu"):
        for t, u in (types, types[::-1]):
            with pytest.raises(ValueError, match="out_dtype"):
                call(y=torch.zeros((4, 256), dtype=t), out_dtype=u)
        with pytest.raises(ValueError, match="out_dtype"):
            call(out_dtype=torch.float16)
        with pytest.raises(ValueError, match="device"):  # the types agree: the next check speaks
            call(y=torch.zeros((4, 256)), out_dtype=torch.float32)


@pytest.mark.gpu
def test_the_results_type():
    for call, default in zip(calls(DEV), (torch.bfloat16, torch.float32)):
        assert call().dtype == default
        for t in (torch.bfloat16, torch.float32):
            y = torch.full((4, 256), 7.0, dtype=t, device=DEV)
            ref = call(out_dtype=t)
            assert ref.dtype == t
            assert call(y=y).data_ptr() == y.data_ptr() and torch.equal(y, ref)
            y.fill_(7.0)
            assert torch.equal(call(y=y, out_dtype=t), ref)
            keep = y.clone()
            with pytest.raises(ValueError):
                call(y=y, out_dtype=torch.float32 if t == torch.bfloat16 else torch.bfloat16)
            assert torch.equal(y, keep)
