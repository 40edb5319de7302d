"""The paged calls at the edges of what they take: values of every size that
the e4m3 cache holds."""
import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import plx_check_device_error, plx_decode_fwd_paged, plx_prefill_fwd_paged

import paged_ref as ref
from helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ends(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=I32)


@pytest.mark.parametrize("Hq,Hkv,page", [(2, 1, 16), (4, 2, 64), (8, 1, 32), (12, 1, 16)])
@pytest.mark.parametrize("low,high", [(-40, 9), (0, 71), (60, 119), (119, -40), (10, 10)])
def test_e4m3_values_of_every_size(Hq, Hkv, page, low, high):
    """Rows of values up to 2^121 (bf16's largest are 2^128) next to ordinary
    and small ones, ascending, so that the keys a token does not see yet are the
    larger, and descending: the kernels for few and for many rows."""
    dev = device()
    n = 150
    pool = ref.Pool([n], Hkv, page, True, 3)
    k = ref.normal_rows(n, Hkv, 1).double().numpy()
    v = ref.normal_rows(n, Hkv, 2).double().numpy() * 2.0 ** np.linspace(low, high, n).round()[:, None, None]
    pool.put(0, 0, k, v)
    kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))
    for m in (1, 3, 140):
        q, r = ref.normal_rows(m, Hq, 1, 2.0), ref.normal_rows(m, Hq, 2, 0.05)
        o, _, bound = ref.reference(pool, q, r, [m])
        out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), cu_q=ends([m]).to(dev), **kw)
        plx_check_device_error()
        ref.assert_within(out, o, bound, f"prefill {m}")
        if m == 1:
            out = plx_decode_fwd_paged(q.to(dev), r.to(dev), **kw)
            plx_check_device_error()
            ref.assert_within(out, o, bound, "decode")
