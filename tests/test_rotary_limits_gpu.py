"""Rotary positions on the GPU at the limits of a call."""
import math
from decimal import Decimal, localcontext

import pytest
import torch

from parametrized_local_linear_gb300 import plx_check_device_error, plx_rotary_bwd, plx_rotary_freqs, plx_rotary_fwd

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


@pytest.mark.parametrize("fn,names", [(plx_rotary_fwd, "qkr"), (plx_rotary_bwd, ("dq", "dk", "dr"))])
@pytest.mark.parametrize("cu,lens,T", [([0, 5, 5, 6, 20], [5, 9, 100, 9], 23), (None, [0, 70, 0, 2], 4)])
def test_rows_of_padding(fn, names, cu, lens, T):
    """Of outputs that the call allocates, every row of a token is written; zeroed ones that
    are given stay zero in the other rows, so that sums over all rows are right."""
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(T, h, 128, generator=g).cuda() for h in (4, 2, 4)]
    ends = list(range(len(lens) + 1)) if cu is None else cu
    there = torch.zeros(T, dtype=torch.bool, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        for t in range(max(ends[b], ends[b + 1] - n), ends[b + 1]):
            there[t], pos[t] = True, n - ends[b + 1] + t
    assert 0 < there.sum() < T
    for a in x:
        a[~there] = float("nan")
    kw = dict(seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              cu_q=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    want = fn(x[0], x[1], freq, x[2], positions=pos)
    fresh = fn(x[0], x[1], freq, x[2], **kw)
    given = [torch.zeros_like(a) for a in x]
    same = fn(x[0], x[1], freq, x[2], **{n + "_out": o for n, o in zip(names, given)}, **kw)
    plx_check_device_error()
    for w, f, s, o in zip(want, fresh, same, given):
        assert s is o
        assert torch.equal(f[there], w[there]) and torch.equal(o[there], w[there]) and not o[~there].any()
        assert torch.equal(o.sum(0), torch.where(there[:, None, None], w, 0).sum(0))


def test_angles_are_as_exact_as_stated():
    """Rows (1, 0) give the cosine and the sine. Each is off by at most the angle's error,
    2 pi (2^-28 + 2^-32 + |position| (|inv_freq| 2^-54 + 2^-64)), and sincospi's 2 ulp, at most
    2^-23; the exact angle in 60 decimal digits, modulo a turn."""
    device()
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620900")
    freq, _ = plx_rotary_freqs(64, device="cuda")
    freq[20:] = torch.tensor([7.5, -3.25, 1.0, 0.999, 0.5, math.pi / 4, 1e-3, 1e-9, 0.0, 2.0, -1.0, 0.3], dtype=torch.float64)
    near = torch.randint(-(1 << 20), 1 << 20, (600,), generator=torch.Generator().manual_seed(2)).tolist()
    pos = near + [0, 1, -1, 1 << 20, 1 << 26, 1 << 28, 2**31 - 1, -2**31, 2**31 - 12345]
    x = torch.zeros(len(pos), 1, 64, device="cuda")
    x[..., :32] = 1.0
    y = plx_rotary_fwd(x, None, freq, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))[0]
    plx_check_device_error()
    y, f = y[:, 0].double().cpu(), freq.tolist()
    with localcontext() as ctx:
        ctx.prec = 60
        for t, p in enumerate(pos):
            for i in range(32):
                turns = Decimal(p) * Decimal(f[i]) / (2 * pi)
                a = 2 * math.pi * float(turns - turns.to_integral_value())
                bound = 2 * math.pi * (2.0 ** -28 + 2.0 ** -32 + abs(p) * (abs(f[i]) * 2.0 ** -54 + 2.0 ** -64)) + 2.0 ** -23
                assert abs(y[t, i].item() - math.cos(a)) <= bound and abs(y[t, 32 + i].item() - math.sin(a)) <= bound, (p, i)
