"""Results and workspaces that the serving calls allocate come in the order of the call's
stream."""
import pytest
import torch

from parametrized_local_linear_gb300 import (binding, plx_check_device_error, plx_decode_fwd_shared, plx_kv_compact,
                                             plx_kv_update, plx_rotary_bwd, plx_rotary_freqs, plx_rotary_fwd)

from helpers import device
from test_moves_gpu import Cache, ints
from test_shared_gpu import problem

pytestmark = pytest.mark.gpu


def shared():
    q, r, kw, _ = problem([3], [40], [41, 40, 300], 4, 2, 16, False)
    return lambda stream: [plx_decode_fwd_shared(q, r, stream=stream, **kw)], 2  # out, workspace


def update():
    c = Cache(3, 4, 10, 16, 1, False)
    want = ints([20, 30, 5])
    return lambda stream: plx_kv_update(lens=want, stream=stream, **c.dev), 1  # workspace; in place


def compact():
    c = Cache(3, 4, 10, 16, 1, False)
    c.update([20, 30, 5])
    return lambda stream: plx_kv_compact(stream=stream, **c.dev), 3  # map, count, workspace


def rotary(fn):
    x = torch.randn(9, 4, 128, device="cuda").to(torch.bfloat16)
    freq, pos = plx_rotary_freqs(128, device="cuda")[0], ints(range(9))
    return lambda stream: fn(x, x[:, :2], freq, x, positions=pos, stream=stream), 3


@pytest.mark.parametrize("make", [shared, update, compact, lambda: rotary(plx_rotary_fwd), lambda: rotary(plx_rotary_bwd)],
                         ids=["shared", "update", "compact", "rotary_fwd", "rotary_bwd"])
@pytest.mark.parametrize("given", [True, False])
def test_every_allocation_is_in_the_order_of_the_calls_stream(make, given, monkeypatch):
    """`_empty` is asked for each, with the stream of the call; nothing that the call returns
    comes from elsewhere but what it was given."""
    device()
    call, count = make()
    side = torch.cuda.Stream() if given else None
    torch.cuda.synchronize()
    seen, plain = [], binding._empty

    def empty(shape, dtype, dev, stream):
        t = plain(shape, dtype, dev, stream)
        seen.append((stream, t.data_ptr()))
        return t

    monkeypatch.setattr(binding, "_empty", empty)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    outs = call(side)
    made = torch.cuda.memory_stats()["allocation.all.allocated"] - before
    torch.cuda.synchronize()
    assert len(seen) == count and all(s is side for s, _ in seen)
    assert made == count  # and the call allocates nothing besides
    del outs
    plx_check_device_error()
