"""Calls with ``stream=`` that allocate their own results: the memory must come
in the order of that stream, not of the current one."""
import pytest
import torch

from parametrized_local_linear_gb300 import (plx_check_device_error, plx_decode_fwd_paged, plx_kv_read,
                                             plx_prefill_fwd_paged)

import paged_ref as ref
from helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32
LENS = [400, 130, 70]


def _paged(dev):
    pool = ref.filled_pool(LENS, 2, 32, True, 3)
    q, r = ref.normal_rows(3, 4, 1).to(dev), ref.normal_rows(3, 4, 2, 0.05).to(dev)
    return q, r, dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))


def _decode_paged(dev):
    q, r, kw = _paged(dev)
    return lambda **s: [plx_decode_fwd_paged(q, r, **kw, **s)]


def _prefill_paged(dev):
    q, r, kw = _paged(dev)
    cu = torch.arange(4, dtype=I32, device=dev)
    return lambda **s: [plx_prefill_fwd_paged(q, r, cu_q=cu, **kw, **s)[0]]


def _read(dev):
    _, _, kw = _paged(dev)
    kw.pop("seqlens")
    cu = torch.tensor([0, 400, 530, 600], dtype=I32, device=dev)
    return lambda **s: list(plx_kv_read(cu_k=cu, T=600, **kw, **s))


CALLS = dict(decode_paged=_decode_paged, prefill_paged=_prefill_paged, read=_read)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_results_do_not_take_memory_that_queued_work_still_uses(name):
    dev = device()
    call = CALLS[name](dev)
    want = call()
    plx_check_device_error()
    s = torch.cuda.Stream()
    # Blocks of the results' sizes that work queued on the current stream has yet to write.
    junk = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for t in junk:
        t.fill_(float("nan"))
    busy = {t.data_ptr() for t in junk}
    del junk, t
    got = call(stream=s)
    assert not busy & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    plx_check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_dropped_result_is_not_reused_before_it_is_written(name):
    dev = device()
    call = CALLS[name](dev)
    want = call()
    plx_check_device_error()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = call(stream=s)
    places = {t.data_ptr() for t in got}
    del got
    fresh = [torch.zeros_like(t) for t in want for _ in range(3)]
    assert not places & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    plx_check_device_error()
    assert all(torch.count_nonzero(t) == 0 for t in fresh)
