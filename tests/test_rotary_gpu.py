"""Rotary positions on the GPU against complex products in fp64: layouts, types,
positions of all kinds, in place; the backward pass against the transposed matrix
and differences; and the training step with it."""
import math

import numpy as np
import pytest
import torch

from oracle import grad as ograd
from parametrized_local_linear_gb300 import (PlxError, plx_check_device_error, plx_prefill_bwd, plx_prefill_fwd_train,
                                             plx_qkvr_proj, plx_rotary_bwd, plx_rotary_freqs, plx_rotary_fwd)

from helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32

# y = x0 c - x1 s in fp32: each of c and s = scale * cos is off by at most 3 * 2^-24 of
# the scale (sincospi 2 ulp at most 2^-24 each, the product with the scale half, the angle's 2^-33
# turns 2^-30), the two products and the sum by another 1.5 * 2^-24 of |x0 c| + |x1 s|; against
# |x0| + |x1| times the scale: 6 * 2^-24 bounds both. The output's rounding: half a step.
F32_REL = 6 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def reference(x, pos, freq, scale, interleaved, sign=1):
    """(y, bound): x [..., d] fp64 with pos broadcastable to its leading dimensions."""
    R = 2 * len(freq)
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    z = scale * np.exp(sign * 1j * (pos[..., None] * freq))
    w = (x[..., a] + 1j * x[..., b]) * z
    y, bound = x.copy(), np.zeros(x.shape)
    y[..., a], y[..., b] = w.real, w.imag
    size = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b])) * F32_REL
    bound[..., a] = bound[..., b] = size
    return y, bound


def check(got, x, pos, freq, scale, interleaved, sign=1):
    want, bound = reference(x.double().cpu().numpy(), pos, freq.cpu().numpy(), scale, interleaved, sign)
    # Angles of pos * freq in fp64 are themselves off by half a step of it, on both sides.
    bound = bound + np.abs(want) * HALF[got.dtype]
    far = np.max(np.abs(pos)) * np.max(np.abs(freq.cpu().numpy())) * 2.0 ** -51
    bound = bound + far * np.abs(scale) * np.abs(x.double().cpu().numpy()).max() * 2
    got = got.double().cpu().numpy()
    over = np.abs(got - want) - bound
    assert got.size == 0 or over.max() <= 0, f"{np.abs(got - want).max():.3e} off, {over.max():.2e} over its bound"


def rows(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R", [(128, 128), (128, 64), (128, 96), (128, 2), (128, 6), (128, 20), (128, 126), (128, 8),
                                 (64, 64), (64, 32), (64, 12), (64, 62)])
def test_layouts_and_dimensions(d, R, interleaved, dtype):
    """Both directions; heads of one and of an odd number; with and without r."""
    device()
    for B, Hq, Hkv, L in ((1, 3, 1, 1), (2, 4, 2, 37), (3, 7, 7, 130)):
        q, k, r = rows((B, Hq, L, d), dtype, 1), rows((B, Hkv, L, d), dtype, 2), rows((B, Hq, L, d), dtype, 3)
        freq, _ = plx_rotary_freqs(R, device="cuda")
        pos = np.arange(L, dtype=np.float64)
        for probe in (r, None):
            for fn, sign in ((plx_rotary_fwd, 1), (plx_rotary_bwd, -1)):
                outs = fn(q, k, freq, probe, interleaved=interleaved, scale=1.25)
                plx_check_device_error()
                assert (outs[2] is None) == (probe is None)
                for x, y in zip((q, k, probe), outs):
                    if x is not None:
                        check(y, x, pos[None, None], freq, 1.25, interleaved, sign)
                        assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_given_positions_near_and_far(dtype):
    device()
    T = 300
    freq, scale = plx_rotary_freqs(64, scaling="parts", factor=16, original_len=4096, device="cuda")
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(0, 2**31 - 1, (T,), generator=g, dtype=torch.int64)
    pos[:100] = torch.randint(0, 1 << 20, (100,), generator=g)
    pos[:6] = torch.tensor([0, 1, 2**31 - 1, -1, -1000, -2**31])
    q, k = rows((T, 5, 128), dtype, 1), rows((T, 1, 128), dtype, 2)
    p = pos.to(I32).cuda()
    for n in (T, 7, 1):  # many rows and few
        outs = plx_rotary_fwd(q[:n], k[:n], freq, positions=p[:n], scale=scale)
        plx_check_device_error()
        at = pos[:n].double().numpy()[:, None]
        check(outs[0], q[:n], at, freq, scale, False)
        check(outs[1], k[:n], at, freq, scale, False)
    # Per sequence of the contiguous layout.
    x = rows((3, 2, 50, 64), dtype, 5)
    f, _ = plx_rotary_freqs(64, device="cuda")
    y, _, _ = plx_rotary_fwd(x, None, f, positions=p[:150].view(3, 50))
    check(y, x, pos[:150].double().numpy().reshape(3, 1, 50), f, 1.0, False)


def test_angles_of_far_positions_are_not_fp32s():
    """Position 10^6 times 1 radian, mod a turn: fp32 would be off by 0.03."""
    device()
    q = torch.ones(1, 1, 64, device="cuda")
    freq = torch.full((32,), 1.0, dtype=torch.float64, device="cuda")
    y, _, _ = plx_rotary_fwd(q, None, freq, positions=torch.tensor([1000003], dtype=I32, device="cuda"))
    c, s = math.cos(1000003.0), math.sin(1000003.0)
    assert abs(y[0, 0, 0].item() - (c - s)) < 4e-7 and abs(y[0, 0, 32].item() - (c + s)) < 4e-7


def test_unusual_frequencies():
    """Above a turn a position, negative, zero; the quarters of a turn exactly."""
    device()
    freq = torch.tensor([7.5, -3.25, 0.0, 1e-9] + [math.pi / 4] * 28, dtype=torch.float64, device="cuda")
    pos = torch.arange(64, dtype=I32, device="cuda")
    q = rows((64, 2, 64), torch.float32, 1)
    y, _, _ = plx_rotary_fwd(q, None, freq, positions=pos, interleaved=True)
    check(y, q, np.arange(64.0)[:, None], freq, 1.0, True)
    assert torch.equal(y[0], q[0])


@pytest.mark.parametrize("cu,lens,T", [([0, 5, 5, 6, 20], [5, 9, 100, 40], 23), (None, [1, 70, 3], 3),
                                       ([0, 4, 9], [2, 1 << 20], 9), ([0, 300], [5000], 300)])
def test_positions_of_new_tokens(cu, lens, T):
    """As plx_kv_append places them; padding rows and rows behind the last stay."""
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    q, k, r = (rows((T, h, 128), torch.bfloat16, h) for h in (4, 2, 4))
    ends = list(range(len(lens) + 1)) if cu is None else cu
    pos = np.full(T, -1.0)
    for b, n in enumerate(lens):
        c = ends[b + 1] - ends[b]
        pos[ends[b]:ends[b + 1]] = n - c + np.arange(c)
    outs = [torch.full_like(x, 7.0) for x in (q, k, r)]
    plx_rotary_fwd(q, k, freq, r, seqlens=torch.tensor(lens, dtype=I32, device="cuda"),
                   cu_q=None if cu is None else torch.tensor(cu, dtype=I32, device="cuda"),
                   q_out=outs[0], k_out=outs[1], r_out=outs[2])
    plx_check_device_error()
    there = pos >= 0
    for x, y in zip((q, k, r), outs):
        check(y[torch.from_numpy(there)], x[torch.from_numpy(there)], pos[there][:, None], freq, 1.0, False)
        assert (y[torch.from_numpy(~there)] == 7).all()


@pytest.mark.parametrize("cu", [[0, 3, 60], [-2, 3, 6], [0, 70, 6]])
def test_bad_offsets_are_reported(cu):
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    q = rows((6, 2, 128), torch.bfloat16, 1)
    plx_rotary_fwd(q, None, freq, seqlens=torch.tensor([10, 10], dtype=I32, device="cuda"),
                   cu_q=torch.tensor(cu, dtype=I32, device="cuda"))
    with pytest.raises(PlxError):
        plx_check_device_error()


@pytest.mark.parametrize("R", [128, 40])
def test_in_place_and_strides(R):
    device()
    freq, _ = plx_rotary_freqs(R, device="cuda")
    T, Hq, Hkv = 70, 4, 2
    wide = rows((T, 2 * Hq + Hkv, 128), torch.bfloat16, 1)  # one row of heads a token
    q, k, r = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    pos = torch.arange(T, dtype=I32, device="cuda") * 3
    want = plx_rotary_fwd(q, k, freq, r, positions=pos)
    heads_first = torch.empty(Hq, T, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got, _, _ = plx_rotary_fwd(q, None, freq, positions=pos, q_out=heads_first)
    assert got is heads_first and torch.equal(got, want[0])
    # Rows with room around them, which stays as it was.
    room = torch.full((T + 1, Hq + 1, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    plx_rotary_fwd(q, None, freq, positions=pos, q_out=room[1:, 1:, 8:])
    assert torch.equal(room[1:, 1:, 8:], want[0])
    assert (room[0] == 7).all() and (room[:, 0] == 7).all() and (room[:, :, :8] == 7).all()
    same = plx_rotary_fwd(q, k, freq, r, positions=pos, q_out=q, k_out=k, r_out=r)
    plx_check_device_error()
    for a, b, c in zip(same, want, (q, k, r)):
        assert a is c and torch.equal(a, b)


def test_the_same_tensor_twice():
    """As q, k and r at once, into results of their own."""
    device()
    freq, _ = plx_rotary_freqs(64, device="cuda")
    x = rows((40, 3, 128), torch.bfloat16, 1)
    pos = torch.arange(40, dtype=I32, device="cuda")
    outs = plx_rotary_fwd(x, x, freq, x, positions=pos)
    plx_check_device_error()
    check(outs[0], x, np.arange(40.0)[:, None], freq, 1.0, False)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_values_that_are_not_finite_stay_in_their_pairs():
    device()
    freq, _ = plx_rotary_freqs(64, device="cuda")
    x = rows((4, 2, 128), torch.bfloat16, 1)
    clean, _, _ = plx_rotary_fwd(x, None, freq, positions=torch.arange(4, dtype=I32, device="cuda"))
    x[1, 0, 5], x[2, 1, 100] = float("nan"), float("inf")
    y, _, _ = plx_rotary_fwd(x, None, freq, positions=torch.arange(4, dtype=I32, device="cuda"))
    sick = torch.zeros_like(x, dtype=torch.bool)
    sick[1, 0, 5] = sick[1, 0, 37] = sick[2, 1, 100] = True
    assert torch.isnan(y[1, 0, 5]) and torch.isnan(y[1, 0, 37]) and y[2, 1, 100] == float("inf")
    assert torch.equal(y[~sick], clean[~sick])


def test_more_rows_than_a_block_and_no_rows():
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    q, k, r = rows((2, 16, 2500, 128), torch.bfloat16, 1), rows((2, 8, 2500, 128), torch.bfloat16, 2), None
    outs = plx_rotary_fwd(q, k, freq, r)
    for x, y in zip((q, k), outs):
        check(y, x, np.arange(2500.0)[None, None], freq, 1.0, False)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    y, _, _ = plx_rotary_fwd(e, None, freq, positions=torch.empty(0, dtype=I32, device="cuda"))
    assert y.shape == (0, 4, 128)


def test_backward_is_the_transpose():
    """<dy, F x> = <B dy, x> in fp32, and F by differences of one value each."""
    device()
    freq, _ = plx_rotary_freqs(48, device="cuda")
    pos = torch.tensor([3, 100000, 77], dtype=I32, device="cuda")
    x, dy = rows((3, 2, 64), torch.float32, 1), rows((3, 2, 64), torch.float32, 2)
    y, _, _ = plx_rotary_fwd(x, None, freq, positions=pos, scale=1.5)
    dx, _, _ = plx_rotary_bwd(dy, None, freq, positions=pos, scale=1.5)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    # Both sums have 384 terms, each off by F32_REL + 2^-24 of values of size 1.5 * 2.
    assert abs(a - b) <= 384 * 2 * (F32_REL + 2.0 ** -24) * 3 * (x.abs().max() * dy.abs().max()).item()
    for t, h, i in ((0, 0, 0), (1, 1, 30), (2, 0, 47), (2, 1, 50)):
        e = torch.zeros_like(x)
        e[t, h, i] = 1.0
        col, _, _ = plx_rotary_fwd(e, None, freq, positions=pos, scale=1.5)  # linear: the difference is F e
        assert abs((col.double() * dy.double()).sum().item() - dx[t, h, i].item()) <= 4 * 1.5 * 2 * F32_REL * dy.abs().max().item()


def test_two_streams_and_a_graph():
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    q, k = rows((64, 16, 128), torch.bfloat16, 1), rows((64, 8, 128), torch.bfloat16, 2)
    lens = torch.arange(64, dtype=I32, device="cuda") * 90 + 1
    want = plx_rotary_fwd(q, k, freq, seqlens=lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = plx_rotary_fwd(q, k, freq, seqlens=lens, stream=side)
    again = plx_rotary_fwd(q, k, freq, seqlens=lens)
    torch.cuda.synchronize()
    for a, b, c in zip(want[:2], got[:2], again[:2]):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(graph):
        plx_rotary_fwd(q, k, freq, seqlens=lens, q_out=qo, k_out=ko)
    lens += 5
    graph.replay()
    torch.cuda.synchronize()
    check(qo, q, (lens.double().cpu().numpy() - 1)[:, None], freq, 1.0, False)


def test_a_training_step_with_positions():
    """Projection, rotation of q, k and r, forward, backward, rotation back, against
    fp64 autograd of the whole: the layer's gradients with respect to what the
    projection gave."""
    device()
    B, L, Dm, Hq, Hkv = 2, 130, 256, 4, 2
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B * L, Dm, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((2 * Hq + 2 * Hkv) * 128, Dm, generator=g) / Dm ** 0.5)
    w[(Hq + 2 * Hkv) * 128:] *= 0.05
    freq, scale = plx_rotary_freqs(128, scaling="parts", factor=4, original_len=64, device="cuda")
    q, k, v, r = plx_qkvr_proj(x, w.to(torch.bfloat16).cuda(), B, L, Hq, Hkv)
    qr, kr, rr = plx_rotary_fwd(q, k, freq, r, scale=scale)
    out, lse, o1, sbar = plx_prefill_fwd_train(qr, kr, v, rr)
    do = torch.randn(q.shape, generator=g).to(torch.bfloat16).cuda()
    dq, dk, dv, dr = plx_prefill_bwd(qr, kr, v, rr, out, o1, lse, sbar, do)
    dq, dk, dr = plx_rotary_bwd(dq, dk, freq, dr, scale=scale)
    plx_check_device_error()

    f = freq.cpu()
    angle = torch.arange(L, dtype=torch.float64)[:, None] * f
    c, s = scale * torch.cos(angle), scale * torch.sin(angle)

    def turn(t, sign):
        a, b = t[..., :64], t[..., 64:]
        return torch.cat([a * c - sign * b * s, b * c + sign * a * s], -1)

    # Rotation in fp64 of the projection's outputs, rounded as the kernel's are, the
    # layer's gradient by autograd, then the rotation's transpose in fp64.
    want = ograd.prefill_grad(turn(q.double().cpu(), 1).to(torch.bfloat16), turn(k.double().cpu(), 1).to(torch.bfloat16),
                              v.cpu(), turn(r.double().cpu(), 1).to(torch.bfloat16), do.cpu())
    # The backward's bound is 1e-2 of a tensor's largest gradient; a pair's rotation mixes
    # two such errors (sqrt 2 * scale), and rounds once more (2^-8).
    for name, got, ref in zip(("dq", "dk", "dv", "dr"), (dq, dk, dv, dr),
                              (turn(want[0], -1), turn(want[1], -1), want[2], turn(want[3], -1))):
        top = ref.abs().max().item()
        bound = 1e-2 * top if name == "dv" else 1e-2 * max(want[0 if name == "dq" else 1 if name == "dk" else 3].abs().max().item(), top) * 2 ** 0.5 * scale + 2.0 ** -8 * top
        assert (got.double().cpu() - ref).abs().max().item() <= bound, name
