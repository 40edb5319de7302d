"""Refusals of the rotary calls (CPU only: nothing here launches a kernel)."""
import pytest
import torch

from parametrized_local_linear_gb300 import plx_rotary_bwd, plx_rotary_fwd

BF = torch.bfloat16


@pytest.mark.parametrize("name", ["q", "k", "r"])
@pytest.mark.parametrize("packed", [True, False])
def test_an_output_without_its_input_is_refused(name, packed):
    """It would be returned as None, and never written."""
    x = torch.zeros((9, 2, 128) if packed else (1, 2, 9, 128), dtype=BF)
    freq = torch.zeros(64, dtype=torch.float64)
    kw = dict(positions=torch.zeros(9, dtype=torch.int32)) if packed else {}
    for given in (("q", "k"), ("k", "r"), ("q", "r"), ("q",), ("k",), ("r",), ()):
        if name in given:
            continue
        with pytest.raises(ValueError, match=f"{name}_out without {name}"):
            plx_rotary_fwd(*(x.clone() if n in given else None for n in "qk"), freq, x.clone() if "r" in given else None,
                           **{name + "_out": x.clone()}, **kw)
        with pytest.raises(ValueError, match=f"{name}_out without {name}"):
            plx_rotary_bwd(*(x.clone() if n in given else None for n in "qk"), freq, x.clone() if "r" in given else None,
                           **{"d" + name + "_out": x.clone()}, **kw)
