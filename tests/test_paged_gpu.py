"""The paged KV cache on the GPU against fp64: writing it (bf16 and e4m3),
reading it back, decode and chunked prefill over its pages, and all of them
together. Every slot that no sequence holds is poisoned with NaN."""
import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, plx_check_device_error, plx_decode_fwd,
                                             plx_decode_fwd_paged, plx_decode_paged_workspace_bytes,
                                             plx_kv_append, plx_kv_read, plx_prefill_fwd,
                                             plx_prefill_fwd_paged, plx_prefill_paged_workspace_bytes,
                                             plx_qkvr_proj)

import paged_ref as ref
from helpers import LSE_ABS, assert_bf16_close, device

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ends(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=I32)


def same_bits(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.uint8
    return torch.equal(a.cpu().view(kind), b.cpu().view(kind))


# ------------------------------------------------------------ append
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,Hkv,lens,counts,behind,heads_first", [
    (16, 2, [1, 40, 16, 17, 0], [1, 5, 16, 1, 0], 0, False),   # page ends inside and at a chunk's end
    (32, 8, [100, 3, 64], [70, 5, 0], 3, True),                # padding rows, rows behind, projection layout
    (64, 1, [300], [129], 0, True),
    (256, 3, [257, 256, 1], [2, 256, 1], 1, False),
    (128, 8, [9000], [4000], 0, True),
])
def test_append_stores_every_row_and_nothing_else(fp8, page, Hkv, lens, counts, behind, heads_first):
    dev = device()
    pool = ref.Pool(lens, Hkv, page, fp8, 7)
    T = sum(counts) + behind
    k, v = ref.normal_rows(T, Hkv, 1), ref.normal_rows(T, Hkv, 2, 30.0)
    kw = pool.to(dev)
    if heads_first:
        kd, vd = (x.transpose(0, 1).contiguous().to(dev).transpose(0, 1) for x in (k, v))
    else:
        kd, vd = k.to(dev), v.to(dev)
    plx_kv_append(kd, vd, seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev), **kw)
    plx_check_device_error()
    at = 0
    for b, n in enumerate(counts):
        skip = max(0, n - lens[b])  # padding
        pool.put(b, lens[b] - n + skip, k[at + skip:at + n].double().numpy(),
                 v[at + skip:at + n].double().numpy())
        at += n
    assert same_bits(kw["kpages"], pool.k) and same_bits(kw["vpages"], pool.v)
    if fp8:
        assert same_bits(kw["kscale"], pool.ks) and same_bits(kw["vscale"], pool.vs)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_one_token_each(fp8):
    """cu_q=None: a decode step's write; an empty sequence of a padded batch writes nothing."""
    dev = device()
    lens = [5, 0, 33, 16, 1]
    pool = ref.Pool(lens, 4, 16, fp8, 3)
    kw = pool.to(dev)
    k, v = ref.normal_rows(5, 4, 1), ref.normal_rows(5, 4, 2)
    plx_kv_append(k.to(dev), v.to(dev), seqlens=pool.seqlens.to(dev), **kw)
    plx_check_device_error()
    for b, n in enumerate(lens):
        if n > 0:
            pool.put(b, n - 1, k[b:b + 1].double().numpy(), v[b:b + 1].double().numpy())
    assert same_bits(kw["kpages"], pool.k) and same_bits(kw["vpages"], pool.v)
    if fp8:
        assert same_bits(kw["kscale"], pool.ks)


def test_append_e4m3_extreme_rows():
    """Zeros, the smallest and largest bf16 values, maxima at 448 and one step
    above, ties between codes, mixed magnitudes: codes and scales bit for bit."""
    dev = device()
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(40, 1, 128, generator=g) * torch.logspace(-38, 37, 40)[:, None, None]
    rows = rows.to(torch.bfloat16)
    rows[0] = 0.0
    rows[1] = 2.0 ** -133
    rows[2] = torch.finfo(torch.bfloat16).max
    rows[3, 0, 5] = -448.0
    rows[3, 0, 6:] = 0
    rows[4] = 0.0
    rows[4, 0, 9] = 450.0
    rows[5] = (torch.arange(128) * 1.0).to(torch.bfloat16)       # many ties at this scale
    rows[6] = -(torch.arange(128) + 128.0).to(torch.bfloat16)
    rows[7, 0, ::2] = 2.0 ** -20
    pool = ref.Pool([40], 1, 16, True, 3)
    kw = pool.to(dev)
    plx_kv_append(rows.to(dev), rows.to(dev), seqlens=pool.seqlens.to(dev), cu_q=ends([40]).to(dev), **kw)
    plx_check_device_error()
    pool.put(0, 0, rows.double().numpy(), rows.double().numpy())
    assert same_bits(kw["kscale"], pool.ks) and same_bits(kw["kpages"], pool.k)
    assert same_bits(kw["vpages"], pool.v)


def test_append_reports_rows_that_cannot_be_quantised():
    dev = device()
    for bad in (float("nan"), float("inf")):
        pool = ref.Pool([4], 1, 16, True, 3)
        k = ref.normal_rows(4, 1, 1)
        k[2, 0, 100] = bad
        plx_kv_append(k.to(dev), k.to(dev), seqlens=pool.seqlens.to(dev), cu_q=ends([4]).to(dev),
                      **pool.to(dev))
        with pytest.raises(PlxError) as e:
            plx_check_device_error()
        assert e.value.status == binding.PLX_ERR_INVALID_ARG
    plx_check_device_error()  # cleared


# ------------------------------------------------------------ read back
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,Hkv,lens,counts,behind", [
    (16, 2, [1, 40, 16, 17, 0], [1, 40, 16, 17, 0], 0),
    (32, 8, [100, 3, 64], [33, 0, 64], 5),               # less than the cache holds; rows behind
    (64, 3, [300], [300], 0),
    (256, 8, [2500, 700], [2500, 700], 2),
])
def test_read_back_is_exact(fp8, page, Hkv, lens, counts, behind):
    dev = device()
    pool = ref.filled_pool(lens, Hkv, page, fp8, 11)
    T = sum(counts) + behind
    k = torch.full((T, Hkv, 128), 7.0, dtype=torch.bfloat16, device=dev)
    v = k.clone()
    out = plx_kv_read(**pool.to(dev), cu_k=ends(counts).to(dev), T=T, k=k, v=v)
    plx_check_device_error()
    assert out[0] is k and out[1] is v
    want = [pool.get(b, n) for b, n in enumerate(counts)]
    for i, got in enumerate((k, v)):
        w = np.concatenate([x[i] for x in want] + [np.full((behind, Hkv, 128), 7.0)])
        assert np.array_equal(got.double().cpu().numpy(), w)


def test_append_then_read_round_trip_of_bf16():
    dev = device()
    lens = [130, 1, 64]
    pool = ref.Pool(lens, 2, 64, False, 2)
    kw = pool.to(dev)
    k, v = ref.normal_rows(195, 2, 4).to(dev), ref.normal_rows(195, 2, 5).to(dev)
    plx_kv_append(k, v, seqlens=pool.seqlens.to(dev), cu_q=ends(lens).to(dev), **kw)
    k2, v2 = plx_kv_read(**kw, cu_k=ends(lens).to(dev), T=195)
    plx_check_device_error()
    assert torch.equal(k, k2) and torch.equal(v, v2)


# ------------------------------------------------------------ decode
DECODE = [
    ([1], 2, 2, 16), ([5, 0, 33, 16, 1, 200], 4, 2, 16), ([17, 64, 63, 65], 16, 8, 32),
    ([300, 301], 8, 1, 64), ([100, 1000], 6, 2, 128), ([77, 260], 12, 4, 256), ([40, 90], 10, 2, 16),
    ([129, 31], 7, 1, 32), ([50, 700], 16, 1, 64), ([20, 130], 24, 2, 16), ([3000, 17, 5000], 16, 8, 64),
    ([0, 0], 4, 2, 16), ([4097], 16, 8, 16), ([9000], 2, 1, 256), ([70, 3], 128, 1, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,page", DECODE)
def test_decode_matches_fp64(fp8, lens, Hq, Hkv, page):
    dev = device()
    pool = ref.filled_pool(lens, Hkv, page, fp8, 21)
    q, r = ref.normal_rows(len(lens), Hq, 31), ref.normal_rows(len(lens), Hq, 32, 0.05)
    out = torch.full_like(q, float("nan")).to(dev)
    plx_decode_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev), out=out, **pool.to(dev))
    plx_check_device_error()
    o, _, bound = ref.reference(pool, q, r, [1] * len(lens))
    ref.assert_within(out, o, bound, f"paged decode {lens}")
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.count_nonzero(out[b]) == 0


def test_decode_equals_the_packed_decode():
    """Same keys, packed contiguously: the two decodes agree up to fp32
    rounding before the output's rounding (one bf16 step)."""
    dev = device()
    lens = [700, 33, 2100]
    pool = ref.filled_pool(lens, 8, 32, False, 5)
    kw = pool.to(dev)
    q, r = ref.normal_rows(3, 16, 1).to(dev), ref.normal_rows(3, 16, 2, 0.05).to(dev)
    k, v = plx_kv_read(**kw, cu_k=ends(lens).to(dev), T=sum(lens))
    sl = pool.seqlens.to(dev)
    a, b = plx_decode_fwd_paged(q, r, seqlens=sl, **kw), plx_decode_fwd(q, r, k, v, sl)
    plx_check_device_error()
    assert_bf16_close(a.double().cpu().numpy(), b.double().cpu().numpy())


def test_decode_large_probes_and_skewed_scores():
    """Probes of the queries' size, one dominating key, rows of one sign."""
    dev = device()
    lens = [200, 513]
    for fp8 in (False, True):
        pool = ref.filled_pool(lens, 2, 16, fp8, 9)
        q, r = ref.normal_rows(2, 4, 1, 4.0), ref.normal_rows(2, 4, 2, 1.0)
        out = plx_decode_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev), **pool.to(dev))
        plx_check_device_error()
        o, _, bound = ref.reference(pool, q, r, [1, 1])
        ref.assert_within(out, o, bound, "large probes")


@pytest.mark.parametrize("fp8", [False, True])
def test_scales_of_all_sizes(fp8):
    """Keys and values from 2^-60 to 2^30 (rows of very different scale)."""
    dev = device()
    n = 150
    pool = ref.Pool([n], 1, 32, fp8, 3)
    k = ref.normal_rows(n, 1, 1).double().numpy() * 2.0 ** np.linspace(-60, 0, n).round()[:, None, None]
    v = ref.normal_rows(n, 1, 2).double().numpy() * 2.0 ** np.linspace(30, -60, n).round()[:, None, None]
    pool.put(0, 0, k, v)
    q, r = ref.normal_rows(1, 2, 1, 3.0), ref.normal_rows(1, 2, 2, 0.05)
    o, _, bound = ref.reference(pool, q, r, [1])
    kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))
    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), **kw)
    ref.assert_within(out, o, bound, "decode")
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), cu_q=ends([1]).to(dev), **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "prefill")


def test_subnormal_codes_are_not_flushed():
    """Rows whose scale is set by one element, all others e4m3 subnormals:
    the bound is relative to each dimension's own values."""
    dev = device()
    n = 90
    g = torch.Generator().manual_seed(3)
    k = torch.randint(-7, 8, (n, 1, 128), generator=g).double().numpy() * 2.0 ** -9
    v = torch.randint(-7, 8, (n, 1, 128), generator=g).double().numpy() * 2.0 ** -9
    k[:, :, 0] = v[:, :, 0] = 448.0
    pool = ref.Pool([n], 1, 16, True, 3)
    pool.put(0, 0, k, v)
    q, r = ref.normal_rows(1, 4, 1, 300.0), ref.normal_rows(1, 4, 2, 10.0)
    q[:, :, 0] = r[:, :, 0] = 0
    o, _, bound = ref.reference(pool, q, r, [1])
    kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))
    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), **kw)
    ref.assert_within(out, o, bound, "decode")
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), cu_q=ends([1]).to(dev), **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "prefill")


# ------------------------------------------------------------ prefill
PREFILL = [
    # lens, counts, Hq, Hkv, page, rows behind
    ([1], [1], 2, 2, 16, 0),
    ([40, 16, 17], [40, 16, 17], 4, 2, 16, 0),                     # whole prompts
    ([100, 70, 9, 0, 64], [3, 64, 0, 0, 1], 4, 2, 16, 2),          # chunks, none, an empty sequence
    ([65, 128, 129], [65, 128, 129], 16, 8, 32, 0),
    ([5, 3], [9, 3], 4, 2, 16, 0),                                 # more tokens than keys: padding
    ([0, 4], [6, 2], 6, 2, 32, 1),                                 # a sequence of padding alone
    ([300, 700], [131, 200], 8, 1, 64, 0),
    ([200, 90], [50, 90], 6, 2, 128, 0), ([130, 61], [77, 60], 5, 1, 256, 0),
    ([90, 300], [33, 5], 7, 1, 32, 0), ([70, 40], [70, 3], 16, 1, 16, 0), ([66], [40], 24, 1, 16, 0),
    ([40, 33], [7, 33], 128, 1, 16, 0), ([50], [9], 65, 1, 16, 0),
    ([2000, 50, 1030], [4, 1, 300], 16, 8, 64, 0),
    ([1500], [700], 16, 8, 128, 0), ([4000], [1], 16, 8, 16, 0), ([6000], [130], 2, 1, 256, 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,counts,Hq,Hkv,page,behind", PREFILL)
def test_prefill_matches_fp64(fp8, lens, counts, Hq, Hkv, page, behind):
    dev = device()
    pool = ref.filled_pool(lens, Hkv, page, fp8, 41)
    T = sum(counts) + behind
    q, r = ref.normal_rows(T, Hq, 51), ref.normal_rows(T, Hq, 52, 0.05)
    out = torch.full((T, Hq, 128), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((T, Hq), 3.0, device=dev)
    plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev),
                          out=out, lse=lse, **pool.to(dev))
    plx_check_device_error()
    o, l, bound = ref.reference(pool, q, r, counts, behind)
    used = T - behind
    ref.assert_within(out[:used], o[:used], bound[:used], f"paged prefill {lens} {counts}")
    got = lse[:used].double().cpu().numpy()
    empty = np.isinf(l[:used])
    assert np.array_equal(np.isneginf(got), empty)
    assert np.max(np.abs(got[~empty] - l[:used][~empty]), initial=0) <= LSE_ABS
    assert torch.count_nonzero(out[:used][torch.from_numpy(empty).to(dev)]) == 0
    # Rows behind the last sequence are left as they were.
    assert torch.all(out[used:] == 5.0) and torch.all(lse[used:] == 3.0)


@pytest.mark.parametrize("layout", ["heads first", "padded rows", "inside a wider tensor"])
def test_prefill_strides(layout):
    dev = device()
    lens, counts, Hq, Hkv = [90, 200], [37, 141], 4, 2
    pool = ref.filled_pool(lens, Hkv, 32, True, 4)
    T = sum(counts)
    q, r = ref.normal_rows(T, Hq, 5), ref.normal_rows(T, Hq, 6, 0.05)
    kw = dict(seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev), **pool.to(dev))
    want, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), **kw)

    def place(x):
        if layout == "heads first":
            return x.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
        shape = (T, Hq, 136) if layout == "padded rows" else (T, Hq + 3, 128)
        wide = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
        view = wide[:, :, :128] if layout == "padded rows" else wide[:, 2:2 + Hq]
        view.copy_(x)
        return view

    out = place(torch.zeros_like(q))
    plx_prefill_fwd_paged(place(q), place(r), out=out, **kw)
    plx_check_device_error()
    assert torch.equal(out, want)
    base = out._base if out._base is not None else out
    if layout == "padded rows":
        assert torch.isnan(base[:, :, 128:]).all()  # nothing written beside the rows
    elif layout != "heads first":
        assert torch.isnan(base[:, :2]).all() and torch.isnan(base[:, 2 + Hq:]).all()


def test_prefill_equals_the_contiguous_prefill():
    dev = device()
    B, L, Hq, Hkv = 2, 333, 4, 2
    pool = ref.filled_pool([L] * B, Hkv, 64, False, 6)
    kw = pool.to(dev)
    q, r = ref.normal_rows(B * L, Hq, 1).to(dev), ref.normal_rows(B * L, Hq, 2, 0.05).to(dev)
    cu = ends([L] * B).to(dev)
    k, v = plx_kv_read(**kw, cu_k=cu, T=B * L)
    lse = torch.empty(B * L, Hq, device=dev)
    out, _ = plx_prefill_fwd_paged(q, r, seqlens=pool.seqlens.to(dev), cu_q=cu, lse=lse, **kw)
    f = lambda x: x.view(B, L, -1, 128).transpose(1, 2).contiguous()  # noqa: E731
    want, wl = plx_prefill_fwd(f(q), f(k), f(v), f(r), lse=torch.empty(B, Hq, L, device=dev))
    plx_check_device_error()
    assert_bf16_close(f(out).double().cpu().numpy(), want.double().cpu().numpy())
    assert (lse.view(B, L, Hq).transpose(1, 2) - wl).abs().max() <= LSE_ABS


def test_prefill_of_one_token_equals_decode():
    dev = device()
    lens = [900, 1, 64, 131]
    for fp8 in (False, True):
        pool = ref.filled_pool(lens, 2, 16, fp8, 8)
        q, r = ref.normal_rows(4, 4, 1).to(dev), ref.normal_rows(4, 4, 2, 0.05).to(dev)
        kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))
        a = plx_decode_fwd_paged(q, r, **kw)
        b, _ = plx_prefill_fwd_paged(q, r, cu_q=ends([1] * 4).to(dev), **kw)
        plx_check_device_error()
        assert_bf16_close(a.double().cpu().numpy(), b.double().cpu().numpy())


# ------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_serving_run_projection_append_prefill_decode(fp8):
    """A prompt in two chunks and two decode steps of a ragged batch, as a
    server runs them, against fp64 over the cache that the run itself wrote."""
    dev = device()
    Dm, Hq, Hkv, page = 256, 4, 2, 16
    prompts = [70, 1, 33]
    B = len(prompts)
    g = torch.Generator().manual_seed(3)
    w = torch.randn((2 * Hq + 2 * Hkv) * 128, Dm, generator=g) / Dm ** 0.5
    w[(Hq + 2 * Hkv) * 128:] *= 0.05
    w = w.to(torch.bfloat16).to(dev)
    pool = ref.Pool([n + 2 for n in prompts], Hkv, page, fp8, 12)
    kw = pool.to(dev)

    def rows(T, seed):
        x = torch.randn(T, Dm, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(dev)
        q, k, v, r = plx_qkvr_proj(x, w, 1, T, Hq, Hkv)
        return [t[0].transpose(0, 1) for t in (q, k, v, r)]

    have = [0] * B
    for step, counts in enumerate([[40, 1, 8], [30, 0, 25], [1] * B, [1] * B]):
        q, k, v, r = rows(sum(counts), step)
        have = [a + b for a, b in zip(have, counts)]
        sl = torch.tensor(have, dtype=I32, device=dev)
        cu = ends(counts).to(dev)
        plx_kv_append(k, v, seqlens=sl, cu_q=cu, **kw)
        if step < 2:
            out, _ = plx_prefill_fwd_paged(q, r, seqlens=sl, cu_q=cu, **kw)
        else:
            out = plx_decode_fwd_paged(q.contiguous(), r.contiguous(), seqlens=sl, **kw)
        plx_check_device_error()
        if fp8:
            pool.k, pool.v = kw["kpages"].cpu(), kw["vpages"].cpu()
            pool.ks, pool.vs = kw["kscale"].cpu(), kw["vscale"].cpu()
        else:
            pool.k, pool.v = kw["kpages"].cpu(), kw["vpages"].cpu()
        pool.lens = have
        o, _, bound = ref.reference(pool, q.cpu(), r.cpu(), counts)
        ref.assert_within(out, o, bound, f"step {step}")


def test_shared_prefix_pages():
    """Two sequences whose first pages are the same ones."""
    dev = device()
    pool = ref.filled_pool([100, 75], 2, 16, True, 3)
    pool.table[1, :4] = pool.table[0, :4]
    q, r = ref.normal_rows(2, 4, 1), ref.normal_rows(2, 4, 2, 0.05)
    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev), **pool.to(dev))
    plx_check_device_error()
    o, _, bound = ref.reference(pool, q, r, [1, 1])
    ref.assert_within(out, o, bound)


def _problem(dev, fp8, lens=(500, 0, 77), counts=(90, 0, 5), seed=3):
    pool = ref.filled_pool(list(lens), 2, 32, fp8, seed)
    T = sum(counts)
    q, r = ref.normal_rows(T, 4, seed).to(dev), ref.normal_rows(T, 4, seed + 1, 0.05).to(dev)
    return (q, r), dict(seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev), **pool.to(dev))


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_repeat_bit_for_bit_and_take_a_workspace(fp8):
    dev = device()
    (q, r), kw = _problem(dev, fp8)
    ws = torch.full((plx_prefill_paged_workspace_bytes(q.shape[0], 3, 4, 2, 128),), 255, dtype=torch.uint8,
                    device=dev)
    a, _ = plx_prefill_fwd_paged(q, r, **kw)
    b, _ = plx_prefill_fwd_paged(q, r, workspace=ws, **kw)
    c, _ = plx_prefill_fwd_paged(q, r, workspace=ws, **kw)
    cu = kw.pop("cu_q")
    ws = torch.full((plx_decode_paged_workspace_bytes(3, 4, 2, 128),), 255, dtype=torch.uint8, device=dev)
    qd, rd = q[:3].contiguous(), r[:3].contiguous()
    d = plx_decode_fwd_paged(qd, rd, **kw)
    e = plx_decode_fwd_paged(qd, rd, workspace=ws, **kw)
    plx_check_device_error()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(d, e) and cu is not None


def test_two_streams_at_once():
    """Calls on two streams, each with work of its own in flight."""
    dev = device()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    problems = [_problem(dev, True, (900, 300), (200, 300), 5), _problem(dev, False, (700, 64), (33, 64), 6)]
    want = [plx_prefill_fwd_paged(*rows, **kw)[0] for rows, kw in problems]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, (rows, kw)) in enumerate(zip(streams, problems)):
            with torch.cuda.stream(s):
                got[i].append(plx_prefill_fwd_paged(*rows, **kw)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
    # and by the stream argument, from another current stream
    out = torch.empty_like(want[0])
    rows, kw = problems[0]
    plx_prefill_fwd_paged(*rows, out=out, stream=streams[1], **kw)
    streams[1].synchronize()
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step_in_two_graphs(fp8):
    """Append and decode captured twice (lengths on the device advance between
    replays); replays interleave and reproduce the eager results."""
    dev = device()
    lens = [17, 300, 0, 64]
    pool = ref.filled_pool(lens, 2, 16, fp8, 3, max_len=400)
    # room for one more token each (the empty sequence stays empty)
    room = ref.Pool([n + 1 if n else 0 for n in lens], 2, 16, fp8, 3, max_len=400)
    for b, n in enumerate(lens):
        if n:
            room.put(b, 0, *pool.get(b, n))
    kw = room.to(dev)
    sl = room.seqlens.to(dev)
    data = [[ref.normal_rows(4, h, s, c).to(dev) for h, s, c in ((4, 1 + i, 1), (2, 5 + i, 1), (2, 9 + i, 1),
                                                                (4, 13 + i, 0.05))] for i in range(2)]

    def step(i, out):
        q, k, v, r = data[i]
        plx_kv_append(k, v, seqlens=sl, **kw)
        plx_decode_fwd_paged(q, r, seqlens=sl, out=out, **kw)

    want = []
    for i in range(2):
        out = torch.empty_like(data[0][0])
        step(i, out)
        want.append(out)
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(i, outs[i])
        graphs.append(graph)
    for _ in range(3):
        for i in range(2):
            outs[i].fill_(float("nan"))
            graphs[i].replay()
    torch.cuda.synchronize()
    plx_check_device_error()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_prefill_replays_in_a_graph_with_other_lengths():
    """The lengths live on the device: a captured call serves other lengths."""
    dev = device()
    (q, r), kw = _problem(dev, True, (500, 200, 77), (60, 30, 5))
    out = torch.empty_like(q)
    plx_prefill_fwd_paged(q, r, out=out, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plx_prefill_fwd_paged(q, r, out=out, **kw)
    for counts, lens in (((60, 30, 5), (500, 200, 77)), ((1, 90, 4), (499, 100, 7)), ((95, 0, 0), (100, 0, 1))):
        kw["cu_q"].copy_(ends(counts))
        kw["seqlens"].copy_(torch.tensor(lens, dtype=I32))
        graph.replay()
        got = out.clone()
        want, _ = plx_prefill_fwd_paged(q, r, **kw)
        assert torch.equal(got, want)
    plx_check_device_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_many_short_sequences(fp8):
    """More sequences than the plans' warp has lanes, empty ones among them."""
    dev = device()
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 70, 150).tolist()
    lens[3:40] = [0] * 37
    counts = [int(rng.integers(0, n + 1)) if rng.random() < 0.5 else min(n, 1) for n in lens]
    pool = ref.filled_pool(lens, 2, 16, fp8, 14)
    kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))
    for many in (counts, [min(n, 1) for n in lens], [min(n, 1 + b % 3) for b, n in enumerate(lens)]):
        T = sum(many)
        q, r = ref.normal_rows(T, 4, 1), ref.normal_rows(T, 4, 2, 0.05)
        o, _, bound = ref.reference(pool, q, r, many)
        out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), cu_q=ends(many).to(dev), **kw)
        plx_check_device_error()
        ref.assert_within(out, o, bound, "prefill")
    q, r = ref.normal_rows(150, 4, 3), ref.normal_rows(150, 4, 4, 0.05)
    o, _, bound = ref.reference(pool, q, r, [1] * 150)
    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "decode")


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (6, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_batches_of_alike_sequences(fp8, Hq, Hkv):
    """Batches of one shape with many row tiles (dealt to the CTAs in rounds
    of whole items), against the same rows of a batch that is not."""
    dev = device()
    B, n, L = 24 * (3 - Hkv), 1300, 1400
    pool = ref.filled_pool([L] * 2 + [40], Hkv, 64, fp8, 15)
    table = pool.table[[b % 2 for b in range(B)] + [2]].contiguous().to(dev)  # shared pages
    sl = torch.tensor([L] * B + [40], dtype=I32, device=dev)
    T = B * n + 7
    q, r = ref.normal_rows(T, Hq, 1).to(dev), ref.normal_rows(T, Hq, 2, 0.05).to(dev)
    kw = pool.to(dev)
    kw.pop("block_table")
    lse, lse2 = torch.empty(T, Hq, device=dev), torch.empty(B * n, Hq, device=dev)
    mixed, _ = plx_prefill_fwd_paged(q, r, block_table=table, seqlens=sl, cu_q=ends([n] * B + [7]).to(dev),
                                     lse=lse, **kw)
    alike, _ = plx_prefill_fwd_paged(q[:B * n], r[:B * n], block_table=table[:B], seqlens=sl[:B],
                                     cu_q=ends([n] * B).to(dev), lse=lse2, **kw)
    plx_check_device_error()
    assert_bf16_close(alike.double().cpu().numpy(), mixed[:B * n].double().cpu().numpy())
    assert (lse[:B * n] - lse2).abs().max() <= LSE_ABS
    rows = [0, 1, 63, 64, 128, n - 1]
    for b in (0, 11, B - 1):
        K, V = pool.get(b % 2, L)
        for h in range(Hq):
            i = torch.tensor([b * n + x for x in rows], device=dev)
            g = h // (Hq // Hkv)
            o, _, bound = ref.attend(q[i, h].double().cpu().numpy(), r[i, h].double().cpu().numpy(), K[:, g],
                                     V[:, g], np.array(rows) + L - n + 1)
            ref.assert_within(alike[i, h], o, bound, "alike")


def test_no_new_tokens():
    dev = device()
    pool = ref.filled_pool([40, 7], 2, 16, True, 3)
    kw = pool.to(dev)
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=dev)
    zero = torch.zeros(3, dtype=I32, device=dev)
    out, _ = plx_prefill_fwd_paged(none, none, seqlens=pool.seqlens.to(dev), cu_q=zero, **kw)
    assert out.shape == (0, 4, 128)
    plx_kv_append(none[:, :2], none[:, :2], seqlens=pool.seqlens.to(dev), cu_q=zero, **kw)
    assert plx_kv_read(**kw, cu_k=zero, T=0)[0].shape == (0, 2, 128)
    # rows that belong to no sequence
    for rows in (9, 200):
        q = ref.normal_rows(rows, 4, 1).to(dev)
        out = torch.full_like(q, 2.0)
        plx_prefill_fwd_paged(q, q, seqlens=pool.seqlens.to(dev), cu_q=zero, out=out, **kw)
        k = q[:, :2].contiguous()
        plx_kv_append(k, k, seqlens=pool.seqlens.to(dev), cu_q=zero, **kw)
        plx_check_device_error()
        assert torch.all(out == 2.0) and same_bits(kw["kpages"], pool.k)


def test_c_calls_allocate_their_own_workspace():
    """workspace = NULL at the C boundary: the same results."""
    import ctypes
    dev = device()
    L = binding.lib()
    p = lambda t: ctypes.c_void_p(t.data_ptr()) if t is not None else None  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for fp8 in (False, True):
        (q, r), kw = _problem(dev, fp8, (300, 80), (100, 80))
        pages = [kw[k] for k in ("kpages", "vpages", "kscale", "vscale", "block_table", "seqlens", "cu_q")]
        n, Hkv, page, d = kw["kpages"].shape
        sizes = (2, 4, Hkv, d, n, page, kw["block_table"].shape[1])
        out = torch.empty_like(q)
        s = L.plx_prefill_fwd_paged(p(q), p(r), 512, 128, *map(p, pages), p(out), 512, 128, None, q.shape[0],
                                    *sizes, None, 0, st)
        assert s == binding.PLX_OK, L.plx_last_error_message()
        want, _ = plx_prefill_fwd_paged(q, r, **kw)
        dec = torch.empty_like(q[:2])
        s = L.plx_decode_fwd_paged(p(q), p(r), *map(p, pages[:6]), p(dec), *sizes, None, 0, st)
        assert s == binding.PLX_OK, L.plx_last_error_message()
        kw.pop("cu_q")
        want_dec = plx_decode_fwd_paged(q[:2].contiguous(), r[:2].contiguous(), **kw)
        plx_check_device_error()
        assert torch.equal(out, want) and torch.equal(dec, want_dec)


# ------------------------------------------------------------ beyond 32 bits
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_32_bit_offsets(fp8):
    """A pool whose later pages start more than 2^32 bytes in: written, read
    and attended to there."""
    dev = device()
    Hkv, page, Hq, n = 8, 256, 16, 300
    per_page = Hkv * page * 128 * (1 if fp8 else 2)
    num = (1 << 32) // per_page + 40
    pages = [torch.empty(num, Hkv, page, 128, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device=dev)
             for _ in range(2)]
    scales = [torch.empty(num, Hkv, page, dtype=torch.uint8, device=dev) if fp8 else None for _ in range(2)]
    kw = dict(kpages=pages[0], vpages=pages[1], kscale=scales[0], vscale=scales[1],
              block_table=torch.tensor([[num - 1, num - 7]], dtype=I32, device=dev))
    k, v = ref.normal_rows(n, Hkv, 1), ref.normal_rows(n, Hkv, 2)
    sl, cu = torch.tensor([n], dtype=I32, device=dev), ends([n]).to(dev)
    plx_kv_append(k.to(dev), v.to(dev), seqlens=sl, cu_q=cu, **kw)
    small = ref.Pool([n], Hkv, page, fp8, 1)
    small.put(0, 0, k.double().numpy(), v.double().numpy())
    wk, wv = small.get(0, n)
    gk, gv = plx_kv_read(**kw, cu_k=cu, T=n)
    assert np.array_equal(gk.double().cpu().numpy(), wk) and np.array_equal(gv.double().cpu().numpy(), wv)
    q, r = ref.normal_rows(2, Hq, 3), ref.normal_rows(2, Hq, 4, 0.05)
    o, _, bound = ref.reference(small, q, r, [2])
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=sl, cu_q=ends([2]).to(dev), **kw)
    ref.assert_within(out, o, bound, "prefill")
    out = plx_decode_fwd_paged(q[1:].to(dev), r[1:].to(dev), seqlens=sl, **kw)
    plx_check_device_error()
    ref.assert_within(out, o[1:], bound[1:], "decode")


# ------------------------------------------------------------ bad metadata
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["page above", "page below", "length"])
def test_bad_pages_and_lengths_are_reported(fp8, bad):
    """The kernels' own bounds checks turn these into an error; the other
    sequence's results are right, and nothing outside its places is written."""
    dev = device()
    lens = [100, 60]
    pool = ref.filled_pool(lens, 2, 16, fp8, 3)
    kw = pool.to(dev)
    sl = pool.seqlens.to(dev)
    if bad == "length":
        sl[0] = kw["block_table"].shape[1] * 16 + 1
    else:
        kw["block_table"][0, 2] = pool.num_pages if bad == "page above" else -1
    q, r = ref.normal_rows(2, 4, 1), ref.normal_rows(2, 4, 2, 0.05)
    o, _, bound = ref.reference(pool, q, r, [1, 1])

    def reported():
        with pytest.raises(PlxError) as e:
            plx_check_device_error()
        assert e.value.status == binding.PLX_ERR_INVALID_ARG
        plx_check_device_error()

    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), seqlens=sl, **kw)
    reported()
    ref.assert_within(out[1:], o[1:], bound[1:], "decode")
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=sl, cu_q=ends([1, 1]).to(dev), **kw)
    reported()
    ref.assert_within(out[1:], o[1:], bound[1:], "prefill")
    if bad != "length":
        cu = ends([100, 60]).to(dev)
        k, v = plx_kv_read(**kw, cu_k=cu, T=160)
        reported()
        assert np.array_equal(k[100:].double().cpu().numpy(), pool.get(1, 60)[0])
        new = ref.normal_rows(160, 2, 9)
        plx_kv_append(new.to(dev), new.to(dev), seqlens=sl, cu_q=cu, **kw)
        reported()
        for b, at in ((0, 0), (1, 100)):
            x = new[at:at + lens[b]].double().numpy()
            keep = pool.get(0, 48)
            pool.put(b, 0, x, x)
            if b == 0:  # the bad page's 16 tokens went nowhere; that page of the pool is unchanged
                page = pool.table[0, 2].item()
                for pages, scale, got, gs in ((pool.k, pool.ks, kw["kpages"], kw["kscale"]),
                                              (pool.v, pool.vs, kw["vpages"], kw["vscale"])):
                    pages.view(torch.uint8)[page] = got.cpu().view(torch.uint8)[page]
                    if fp8:
                        scale[page] = gs.cpu()[page]
                del keep
        assert same_bits(kw["kpages"], pool.k) and same_bits(kw["vpages"], pool.v)
    else:
        cu = torch.tensor([0, kw["block_table"].shape[1] * 16 + 5, kw["block_table"].shape[1] * 16 + 8], dtype=I32)
        plx_kv_read(**kw, cu_k=cu.to(dev), T=int(cu[-1]))
        reported()


@pytest.mark.parametrize("cu", [[0, 3, 60], [0, 70, 6], [-2, 3, 6], [0, 6, 3]])
@pytest.mark.parametrize("rows", [6, 40])
def test_bad_row_offsets_are_reported(cu, rows):
    """cu_q that passes T, decreases or starts below 0 (6 rows: the kernel for
    few rows, 40: the tile kernel): reported, and the rows beside the output
    are not written."""
    dev = device()
    pool = ref.filled_pool([100, 60], 2, 16, True, 3)
    kw = pool.to(dev)
    sl = pool.seqlens.to(dev)
    guard = torch.full((rows + 100, 4, 128), 3.0, dtype=torch.bfloat16, device=dev)
    q = ref.normal_rows(rows, 4, 1).to(dev)
    bad = torch.tensor(cu, dtype=I32, device=dev)
    plx_prefill_fwd_paged(q, q, seqlens=sl, cu_q=bad, out=guard[50:50 + rows], **kw)
    with pytest.raises(PlxError) as e:
        plx_check_device_error()
    assert e.value.status == binding.PLX_ERR_INVALID_ARG
    assert torch.all(guard[:50] == 3.0) and torch.all(guard[50 + rows:] == 3.0)
    k = q[:, :2].contiguous()
    plx_kv_append(k, k, seqlens=sl, cu_q=bad, **kw)  # rows go to a place of a sequence or nowhere
    try:
        plx_check_device_error()
    except PlxError as err:
        assert err.status == binding.PLX_ERR_INVALID_ARG


def test_negative_lengths_count_as_zero():
    dev = device()
    pool = ref.filled_pool([40, 30], 2, 16, False, 3)
    kw = pool.to(dev)
    sl = torch.tensor([-5, 30], dtype=I32, device=dev)
    pool.lens[0] = 0
    q, r = ref.normal_rows(2, 4, 1), ref.normal_rows(2, 4, 2, 0.05)
    o, _, bound = ref.reference(pool, q, r, [1, 1])
    out = plx_decode_fwd_paged(q.to(dev), r.to(dev), seqlens=sl, **kw)
    ref.assert_within(out, o, bound, "decode")
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=sl, cu_q=ends([1, 1]).to(dev), **kw)
    ref.assert_within(out, o, bound, "prefill")
    k = q[:, :2].contiguous()
    plx_kv_append(k.to(dev), k.to(dev), seqlens=sl, **kw)
    plx_check_device_error()
    pool.put(1, 29, k[1:].double().numpy(), k[1:].double().numpy())
    assert same_bits(kw["kpages"], pool.k) and same_bits(kw["vpages"], pool.v)


@pytest.mark.parametrize("cu", [[-2**31, 3], [2, -2**31], [-1, 3], [0, 50]])
@pytest.mark.parametrize("rows", [4, 40])
def test_offsets_whose_difference_overflows_are_reported(cu, rows):
    """Offsets are compared before they are subtracted."""
    dev = device()
    pool = ref.filled_pool([100], 2, 16, False, 3)
    kw = pool.to(dev)
    q = ref.normal_rows(rows, 4, 1).to(dev)
    k = q[:, :2].contiguous()
    bad = torch.tensor(cu, dtype=I32, device=dev)
    guard = torch.full((rows + 100, 4, 128), 3.0, dtype=torch.bfloat16, device=dev)

    def reported(met):
        if not met:
            return plx_check_device_error()
        with pytest.raises(PlxError) as e:
            plx_check_device_error()
        assert e.value.status == binding.PLX_ERR_INVALID_ARG

    plx_prefill_fwd_paged(q, q, seqlens=pool.seqlens.to(dev), cu_q=bad, out=guard[50:50 + rows], **kw)
    reported(True)
    assert torch.all(guard[:50] == 3.0) and torch.all(guard[50 + rows:] == 3.0)
    met = cu != [2, -2**31]  # no row lies between such offsets
    plx_kv_append(k, k, seqlens=pool.seqlens.to(dev), cu_q=bad, **kw)
    reported(met)
    assert same_bits(kw["kpages"], pool.k) and same_bits(kw["vpages"], pool.v)
    gk = torch.full((rows, 2, 128), 3.0, dtype=torch.bfloat16, device=dev)
    gv = gk.clone()
    plx_kv_read(**kw, cu_k=bad, T=rows, k=gk, v=gv)
    reported(met)
    assert torch.all(gk == 3.0) and torch.all(gv == 3.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_debug_build_gives_the_same_bits(fp8, monkeypatch):
    dev = device()
    dbg = binding.load_debug_lib()

    def run():
        (q, r), kw = _problem(dev, fp8)
        k, v = q[:, :2].contiguous(), r[:, 2:].contiguous()
        plx_kv_append(k, v, **kw)
        out, lse = plx_prefill_fwd_paged(q, r, lse=torch.empty(q.shape[:2], device=dev), **kw)
        few, _ = plx_prefill_fwd_paged(q[:3], r[:3], **dict(kw, cu_q=ends([2, 0, 1]).to(dev)))
        kw.pop("cu_q")
        sl = kw.pop("seqlens")
        step = plx_decode_fwd_paged(q[:3].contiguous(), r[:3].contiguous(), seqlens=sl, **kw)
        back = plx_kv_read(cu_k=ends(sl.tolist()).to(dev), T=int(sl.sum()), **kw)
        plx_check_device_error()
        return [out, lse.view(torch.int16), few, step, *back]

    release = run()
    monkeypatch.setattr(binding, "lib", lambda: dbg)
    assert all(same_bits(a, b) for a, b in zip(release, run()))


def test_calls_from_two_host_threads():
    """Each thread with its own stream and cache, calls overlapping."""
    import threading
    dev = device()
    problems = [_problem(dev, True, (900, 300), (200, 300), 5), _problem(dev, False, (700, 64), (33, 64), 6)]
    want = [plx_prefill_fwd_paged(*rows, **kw)[0] for rows, kw in problems]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                rows, kw = problems[i]
                for _ in range(20):
                    got[i].append(plx_prefill_fwd_paged(*rows, **kw)[0])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - raised again by the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    plx_check_device_error()
    assert not errors
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts,Hq,Hkv,page,behind", [
    ([1, 200, 2, 0, 3, 17, 1], 4, 2, 16, 0),          # decodes with chunks among them: both kernels
    ([2, 1, 90, 5, 4, 1], 2, 2, 64, 3),               # one query head a kv head: up to four tokens
    ([1, 150, 1, 2, 1], 16, 2, 32, 1),                # eight: one token
    ([1, 1, 40], 12, 2, 128, 0),                      # six
    ([1] * 17 + [60, 0, 2], 4, 2, 16, 0),             # few rows on average, one long chunk
    ([8, 9, 8, 7] + [3] * 20, 4, 2, 16, 2),           # two groups of eight rows, and just above
    ([1] * 15 + [30] + [0] * 24, 18, 2, 64, 0),       # nine query heads a kv head
    ([0] * 30 + [100], 4, 2, 16, 0),                  # a long chunk alone among idle sequences
    ([1, 700, 1], 4, 2, 32, 0),                       # mostly chunk: the tile kernel alone
])
def test_mixed_chunk_lengths(fp8, counts, Hq, Hkv, page, behind):
    """Short and long chunks of one call, some with padding rows in front."""
    dev = device()
    lens = [(37 * b) % 300 + (c if b % 4 else max(c - 2, 0)) for b, c in enumerate(counts)]
    pool = ref.filled_pool(lens, Hkv, page, fp8, 11)
    T = sum(counts) + behind
    q, r = ref.normal_rows(T, Hq, 1), ref.normal_rows(T, Hq, 2, 0.05)
    o, lse_want, bound = ref.reference(pool, q, r, counts, behind)
    out = torch.full((T, Hq, 128), 3.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((T, Hq), 3.0, device=dev)
    ws = torch.full((plx_prefill_paged_workspace_bytes(T, len(counts), Hq, Hkv, 128),), 255,
                    dtype=torch.uint8, device=dev)
    plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev),
                          out=out, lse=lse, workspace=ws, **pool.to(dev))
    plx_check_device_error()
    n = sum(counts)
    assert torch.all(out[n:] == 3.0) and torch.all(lse[n:] == 3.0)
    ref.assert_within(out[:n], o[:n], bound[:n])
    got, want = lse[:n].double().cpu().numpy(), lse_want[:n]
    empty = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - want[~empty]) <= LSE_ABS)


def test_bad_row_offsets_among_mixed_chunks():
    """cu_q whose entries pass T or fall back, in a call that both kernels work on."""
    dev = device()
    pool = ref.filled_pool([100, 60, 40, 30], 2, 16, False, 3)
    kw = pool.to(dev)
    rows = 100
    guard = torch.full((rows + 200, 4, 128), 3.0, dtype=torch.bfloat16, device=dev)
    q = ref.normal_rows(rows, 4, 1).to(dev)
    top = 2**31 - 1
    for cu in ([0, top, 1, 2, 3], [0, 1, top, 2, rows], [0, -2**31, 1, 2, 3], [top - 1, top, 2, 3, rows],
               [0, 1, rows + 2, 3, 4], [-5, 1, 2, 3, rows]):
        bad = torch.tensor(cu, dtype=I32, device=dev)
        plx_prefill_fwd_paged(q, q, seqlens=pool.seqlens.to(dev), cu_q=bad, out=guard[100:100 + rows], **kw)
        with pytest.raises(PlxError) as e:
            plx_check_device_error()
        assert e.value.status == binding.PLX_ERR_INVALID_ARG
        assert torch.all(guard[:100] == 3.0) and torch.all(guard[100 + rows:] == 3.0)


@pytest.mark.parametrize("counts", [[3, 60, 1, 40, 2], [1] * 5, [2, 70, 1, 1, 30, 1, 2, 1, 9]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_that_is_not_finite_leaves_the_others_alone(counts, bad):
    """One sequence's keys, values and queries hold NaN or infinities; every
    other sequence's results are the same bits as without them."""
    dev = device()
    lens = [80 + 37 * b for b in range(len(counts))]
    pool = ref.filled_pool(lens, 2, 16, False, 3)
    T, sick = sum(counts), 1
    q, r = ref.normal_rows(T, 4, 1).to(dev), ref.normal_rows(T, 4, 2, 0.05).to(dev)
    kw, sl, cu = pool.to(dev), pool.seqlens.to(dev), ends(counts).to(dev)
    first = [row.contiguous() for row in (q[cu[1:].long() - 1], r[cu[1:].long() - 1])]

    def run():
        return [plx_prefill_fwd_paged(q, r, seqlens=sl, cu_q=cu, **kw)[0],
                plx_decode_fwd_paged(*first, seqlens=sl, **kw)]

    clean = run()
    for pages in (kw["kpages"], kw["vpages"]):
        for page in pool.table[sick, :(lens[sick] + 15) // 16].tolist():
            pages[page, :, ::3, ::5] = bad
    q[ends(counts)[sick]:ends(counts)[sick + 1], :, ::7] = bad
    dirty = run()
    plx_check_device_error()
    rows = torch.ones(T, dtype=torch.bool)
    rows[ends(counts)[sick]:ends(counts)[sick + 1]] = False
    assert same_bits(clean[0][rows.to(dev)], dirty[0][rows.to(dev)])
    others = [b for b in range(len(counts)) if b != sick]
    assert same_bits(clean[1][others], dirty[1][others])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts,Hq,Hkv", [([1] * 6, 16, 2), ([1] * 6, 4, 2), ([3, 1, 1, 1, 1, 2], 4, 2),
                                           ([2, 1, 1, 30, 40, 2], 16, 1), ([70, 50], 4, 2), ([300] * 3, 2, 2)])
def test_a_token_that_sees_one_key_gives_its_value(counts, Hq, Hkv, fp8):
    """o = v whatever the probe says: w = 1, and O2 and O1 s cancel (each first
    token of a sequence, |t| up to a few tens)."""
    dev = device()
    pool = ref.filled_pool(counts, Hkv, 16, fp8, 9)
    T, starts = sum(counts), ends(counts)[:-1].long()
    q, r = ref.normal_rows(T, Hq, 1), ref.normal_rows(T, Hq, 2, 1.0)
    out, _ = plx_prefill_fwd_paged(q.to(dev), r.to(dev), seqlens=pool.seqlens.to(dev),
                                   cu_q=ends(counts).to(dev), **pool.to(dev))
    got = out.cpu()[starts].double().numpy()
    plx_check_device_error()
    # p, 1 / l, s and the two products of the result are off by a few 2^-23
    # relative to (1 + |t|) |v|; with |t| < 64 that is below 2^-9 |v|, half a step
    # of the smallest distance of a bf16 value from its neighbours.
    for b in range(len(counts)):
        v = np.repeat(pool.get(b, 1)[1][0], Hq // Hkv, axis=0)
        assert np.array_equal(got[b], v), b
