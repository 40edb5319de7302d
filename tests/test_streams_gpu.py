"""Calls with ``stream=`` that allocate their own results: the memory must come
in the order of that stream, not of the current one."""
import pytest
import torch

from parametrized_local_linear_gb300 import (inputs, plx_check_device_error, plx_decode_fwd,
                                             plx_decode_fwd_cor, plx_decode_fwd_paged, plx_kv_read,
                                             plx_prefill_bwd, plx_prefill_fwd, plx_prefill_fwd_chunk,
                                             plx_prefill_fwd_cor, plx_prefill_fwd_f32, plx_prefill_fwd_paged,
                                             plx_prefill_fwd_train, plx_qkvr_proj)

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


def _prompt(dev, dtype=torch.bfloat16):
    return [t.to(dev) for t in inputs.prefill_inputs(2, 4, 2, 200, 128, dtype, 0.05, 17)]


def _prefill(dev):
    x = _prompt(dev)
    return lambda **s: [plx_prefill_fwd(*x, **s)[0]]


def _prefill_f32(dev):
    x = _prompt(dev, torch.float32)
    return lambda **s: [plx_prefill_fwd_f32(*x, **s)[0]]


def _chunk(dev):
    q, k, v, r = _prompt(dev)
    q, r = q[:, :, 50:].contiguous(), r[:, :, 50:].contiguous()
    return lambda **s: [plx_prefill_fwd_chunk(q, k, v, r, **s)[0]]


def _prefill_cor(dev):
    x = _prompt(dev)
    return lambda **s: [t for t in plx_prefill_fwd_cor(*x, **s) if t is not None]


def _train(dev):
    x = _prompt(dev)
    return lambda **s: list(plx_prefill_fwd_train(*x, **s))


def _backward(dev):
    x = _prompt(dev)
    out, lse, o1, sbar = plx_prefill_fwd_train(*x)
    dout = torch.randn(out.shape, device=dev).to(torch.bfloat16)
    return lambda **s: list(plx_prefill_bwd(*x, out, o1, lse, sbar, dout, **s))


def _projection(dev):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2 * 100, 512, generator=g).to(torch.bfloat16).to(dev)
    w = (torch.randn(12 * 128, 512, generator=g) / 23).to(torch.bfloat16).to(dev)
    return lambda **s: list(plx_qkvr_proj(x, w, 2, 100, 4, 2, **s))


def _packed(dev):
    q, r, k, v = (ref.normal_rows(n, h, i, c).to(dev) for n, h, i, c in
                  ((3, 4, 1, 1.0), (3, 4, 2, 0.05), (600, 2, 3, 1.0), (600, 2, 4, 1.0)))
    return q, r, k, v, torch.tensor(LENS, dtype=I32, device=dev)


def _decode(dev):
    x = _packed(dev)
    return lambda **s: [plx_decode_fwd(*x, **s)]


def _decode_cor(dev):
    x = _packed(dev)
    return lambda **s: list(plx_decode_fwd_cor(*x, **s))


CALLS = dict(decode_paged=_decode_paged, prefill_paged=_prefill_paged, read=_read, prefill=_prefill,
             prefill_f32=_prefill_f32, chunk=_chunk, prefill_cor=_prefill_cor, train=_train,
             backward=_backward, projection=_projection, decode=_decode, decode_cor=_decode_cor)


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
