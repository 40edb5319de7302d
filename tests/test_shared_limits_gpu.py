"""Decode for sequences that share prefixes where its groups are unusual: more groups
than sequences."""
import pytest
import torch

from parametrized_local_linear_gb300 import binding, plx_check_device_error, plx_decode_fwd_shared

import paged_ref as ref
from helpers import device
from test_shared_gpu import problem

pytestmark = pytest.mark.gpu

MORE_GROUPS = [  # sizes, prefix, lens, Hq, Hkv, page
    ([0] * 30 + [20], [9] * 30 + [70], [71 + 3 * i for i in range(20)], 4, 2, 16),         # tile kernel, group 30 of 20 sequences
    ([0] * 50 + [40], [0] * 50 + [4000], [4001 + i for i in range(40)], 8, 1, 64),         # split between its CTAs
    ([0] * 9 + [3] + [0] * 700 + [2], [5] * 9 + [40] + [5] * 700 + [64], [41, 40, 300, 64, 90], 4, 2, 16),  # rows kernel
    ([0] * 40 + [20, 0, 2], [1] * 40 + [65, 7, 129], [66 + i for i in range(20)] + [130, 140], 16, 1, 32),  # both
    ([0] * 99 + [1], [3] * 99 + [1], [1], 2, 1, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(MORE_GROUPS)))
def test_more_groups_than_sequences(case, fp8, monkeypatch):
    """Empty groups count: a group's number may pass the number of sequences. The debug
    build's index checks hold too, and it gives the same bits."""
    device()
    q, r, kw, (o, _, bound) = problem(*MORE_GROUPS[case], fp8)
    out = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "more groups")
    monkeypatch.setattr(binding, "_lib", binding.load_debug_lib())
    again = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    assert torch.equal(out, again)
