"""Calls of the block's operators that the binding refuses before it looks at a device."""

import pytest
import torch

from differential_attention_03_gb300 import binding as da

BF, F32 = torch.bfloat16, torch.float32


def test_a_stream_of_another_type_than_the_one_asked_for():
    """stream_dtype says the type of s; a residual or an out of another type contradicts it."""
    x = torch.zeros(4, 8, dtype=BF)
    for kw in (dict(residual=x, stream_dtype=F32), dict(residual=x.float(), stream_dtype=BF), dict(out=x, stream_dtype=F32),
               dict(out=x.float(), stream_dtype=BF)):
        with pytest.raises(ValueError, match="stream_dtype"):
            da.residual_norm(x, **kw)
    for kw in (dict(residual=x, stream_dtype=BF), dict(out=x.float(), stream_dtype=F32), dict(stream_dtype=F32)):
        with pytest.raises(ValueError, match="CUDA"):  # (goes on to the tensors)
            da.residual_norm(x, **kw)


def test_a_gate_of_no_rows():
    """[0, D] is no gate at all to the C call (its address is NULL); with rows to gate it is a mistake."""
    x = torch.zeros(4, 8, dtype=BF)
    with pytest.raises(ValueError, match="no rows"):
        da._gate_rows(torch.zeros(0, 8), x, 0)
    for ok in (torch.zeros(8), torch.zeros(2, 8), torch.zeros(4, 8)):
        with pytest.raises(ValueError, match="CUDA"):
            da._gate_rows(ok, x, 0)
    with pytest.raises(ValueError, match="CUDA"):
        da._gate_rows(torch.zeros(0, 8), torch.zeros(0, 8, dtype=BF), 0)  # (nothing to gate)
