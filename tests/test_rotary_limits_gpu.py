"""Rotary positions on the GPU at the limits of a call."""
import pytest
import torch

from parametrized_local_linear_gb300 import plx_rotary_fwd

from helpers import device

pytestmark = pytest.mark.gpu


def test_an_output_without_its_input_is_refused():
    device()
    x = torch.zeros(9, 2, 128, dtype=torch.bfloat16, device="cuda")
    freq = torch.zeros(64, dtype=torch.float64, device="cuda")
    pos = torch.zeros(9, dtype=torch.int32, device="cuda")
    for name in "qkr":
        y = {n: None if n == name else x for n in "qkr"}
        with pytest.raises(ValueError, match=f"{name}_out without {name}"):
            plx_rotary_fwd(y["q"], y["k"], freq, y["r"], positions=pos, **{name + "_out": x.clone()})


def test_outputs_of_another_shape_are_refused():
    device()
    freq = torch.zeros(64, dtype=torch.float64, device="cuda")
    x = torch.zeros(2, 4, 9, 128, dtype=torch.bfloat16, device="cuda")
    rows, pos = x[0].transpose(0, 1), torch.zeros(9, dtype=torch.int32, device="cuda")
    for shape in ((), (128,), (9, 128), (4, 9, 128), (2, 4, 9, 64), (2, 4, 8, 128), (2, 4, 9, 128, 1)):
        out = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError, match="q_out has shape"):
            plx_rotary_fwd(x, None, freq, q_out=out)
        with pytest.raises(ValueError, match="q_out has shape"):
            plx_rotary_fwd(rows, None, freq, positions=pos, q_out=out)
