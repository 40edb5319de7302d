"""The paged calls at the edges of what they take: values of every size that
the e4m3 cache holds, queries that are not numbers, refusals, bad metadata; the
debug build's checks."""
import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, plx_check_device_error, plx_decode_fwd_paged,
                                             plx_kv_append, plx_kv_read, plx_prefill_fwd_paged)

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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts,lens,Hq,Hkv", [([1, 1, 1], [40, 500, 33], 4, 2), ([1, 1], [500, 33], 8, 1),
                                                ([3, 2], [70, 300], 4, 2), ([130, 5], [6000, 64], 4, 2),
                                                ([1] * 9 + [300], [90] * 9 + [2000], 4, 2), ([1], [60000], 2, 1)])
@pytest.mark.parametrize("where", ["q", "r"])
def test_a_query_that_is_not_a_number_gives_nan(counts, lens, Hq, Hkv, fp8, where):
    """In its own row and nowhere else, not the zeros and -inf of a row that sees
    no key: in one kernel or two, and where the sums of several CTAs are joined."""
    dev = device()
    pool = ref.filled_pool(lens, Hkv, 32, fp8, 3)
    T = sum(counts)
    q, r = ref.normal_rows(T, Hq, 1).to(dev), ref.normal_rows(T, Hq, 2, 0.05).to(dev)
    kw = dict(seqlens=pool.seqlens.to(dev), **pool.to(dev))

    def run():
        lse = torch.empty(T, Hq, device=dev)
        out, _ = plx_prefill_fwd_paged(q, r, cu_q=ends(counts).to(dev), lse=lse, **kw)
        got = [out, lse]
        if counts == [1] * len(counts):
            got.append(plx_decode_fwd_paged(q, r, **kw))
        plx_check_device_error()
        return got

    clean = run()
    sick = torch.zeros(T, Hq, dtype=torch.bool, device=dev)
    for t, h in ((0, 1), (T - 1, 0)):
        sick[t, h] = True
        (q if where == "q" else r)[t, h, 17] = float("nan")
    dirty = run()
    for c, d in zip(clean, dirty):
        if d.dim() == 3 or where == "q":
            assert torch.isnan(d[sick]).all()
        assert torch.equal(c[~sick], d[~sick])


# ------------------------------------------------------------ refusals
def test_an_empty_workspace_is_refused():
    """Its pointer is null, which at the C boundary asks for an allocation."""
    dev = device()
    pool = ref.filled_pool([40, 7], 2, 16, True, 3)
    kw = dict(seqlens=pool.seqlens.to(dev), workspace=torch.empty(0, dtype=torch.uint8, device=dev), **pool.to(dev))
    q = ref.normal_rows(2, 4, 1).to(dev)
    with pytest.raises(ValueError, match="workspace"):
        plx_decode_fwd_paged(q, q, **kw)
    with pytest.raises(ValueError, match="workspace"):
        plx_prefill_fwd_paged(q, q, cu_q=ends([1, 1]).to(dev), **kw)


# ------------------------------------------------------------ eight rows a warp
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append_and_read_back_with_eight_rows_a_warp(fp8, heads_first):
    """Enough rows for eight a warp: chunks that start, end and change sequence
    inside a warp's eight, padding in front, rows behind, a short last group."""
    dev = device()
    lens, counts, behind = [1500, 0, 3, 901, 7, 300], [1301, 0, 9, 601, 1, 2], 5
    pool = ref.Pool(lens, 8, 32, fp8, 7)
    T = sum(counts) + behind
    assert T % 8 and T * 8 > 8 * 8 * 152
    k, v = ref.normal_rows(T, 8, 1), ref.normal_rows(T, 8, 2, 30.0)
    kw = pool.to(dev)
    kd, vd = (x.transpose(0, 1).contiguous().to(dev).transpose(0, 1) if heads_first else x.to(dev) for x in (k, v))
    plx_kv_append(kd, vd, seqlens=pool.seqlens.to(dev), cu_q=ends(counts).to(dev), **kw)
    plx_check_device_error()
    at = 0
    for b, n in enumerate(counts):
        skip = max(0, n - lens[b])  # padding
        if n > skip:
            pool.put(b, lens[b] - n + skip, k[at + skip:at + n].double().numpy(),
                     v[at + skip:at + n].double().numpy())
        at += n
    same = lambda a, b: torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert same(kw["kpages"], pool.k) and same(kw["vpages"], pool.v)
    assert not fp8 or same(kw["kscale"], pool.ks) and same(kw["vscale"], pool.vs)
    for b, n in enumerate(lens):
        if n:
            pool.put(b, 0, ref.normal_rows(n, 8, b + 10).double().numpy(), ref.normal_rows(n, 8, b + 20).double().numpy())
    kw, take = pool.to(dev), [1499, 0, 3, 900, 0, 299]
    T = sum(take) + behind
    outs = [torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    plx_kv_read(**kw, cu_k=ends(take).to(dev), T=T, k=outs[0], v=outs[1])
    plx_check_device_error()
    want = [pool.get(b, n) for b, n in enumerate(take)]
    for i, got in enumerate(outs):
        w = np.concatenate([x[i] for x in want] + [np.full((behind, 8, 128), 7.0)])
        assert np.array_equal(got.double().cpu().numpy(), w)


# ------------------------------------------------------------ bad metadata
def same_pages(kw, pool):
    pairs = [(kw["kpages"], pool.k), (kw["vpages"], pool.v)]
    if pool.fp8:
        pairs += [(kw["kscale"], pool.ks), (kw["vscale"], pool.vs)]
    kind = [torch.uint8 if a.element_size() == 1 else torch.int16 for a, _ in pairs]
    return all(torch.equal(a.cpu().view(t), b.view(t)) for (a, b), t in zip(pairs, kind))


def reported(yes=True):
    if not yes:
        return plx_check_device_error()
    with pytest.raises(PlxError) as e:
        plx_check_device_error()
    assert e.value.status == binding.PLX_ERR_INVALID_ARG
    plx_check_device_error()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_append_leaves_the_page_alone_whose_entry_is_bad(fp8, entry):
    """The page that the table should have named keeps its bytes, and so does
    every other one that no new token goes to."""
    dev = device()
    lens = [100, 60]
    pool = ref.filled_pool(lens, 2, 16, fp8, 3)
    kw = pool.to(dev)
    kw["block_table"][0, 2] = entry
    new = ref.normal_rows(160, 2, 9)
    plx_kv_append(new.to(dev), new.to(dev), seqlens=pool.seqlens.to(dev), cu_q=ends(lens).to(dev), **kw)
    reported()
    page = pool.table[0, 2].item()
    tensors = [t for t in (pool.k, pool.v, pool.ks, pool.vs) if t is not None]
    before = [t.view(torch.uint8)[page].clone() for t in tensors]
    for b, at in ((0, 0), (1, 100)):
        x = new[at:at + lens[b]].double().numpy()
        pool.put(b, 0, x, x)
    for t, old in zip(tensors, before):
        assert not torch.equal(t.view(torch.uint8)[page], old)  # the tokens would have shown
        t.view(torch.uint8)[page] = old
    assert same_pages(kw, pool)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [6, 40])
@pytest.mark.parametrize("cu,met,stored", [
    ([0, 3, 60], True, [(0, 97, 0, 3)]),    # the second sequence passes T
    ([0, 70, 6], True, []),                 # the first does
    ([-2, 3, 6], True, [(1, 57, 3, 6)]),    # the first starts below 0
    ([0, 6, 3], False, [(0, 94, 0, 6)]),    # the second falls back: no row lies between its offsets
])
def test_append_with_bad_offsets_writes_only_the_good_sequences(fp8, rows, cu, met, stored):
    dev = device()
    pool = ref.filled_pool([100, 60], 2, 16, fp8, 3)
    kw = pool.to(dev)
    k, v = ref.normal_rows(rows, 2, 1), ref.normal_rows(rows, 2, 2)
    plx_kv_append(k.to(dev), v.to(dev), seqlens=pool.seqlens.to(dev),
                  cu_q=torch.tensor(cu, dtype=I32, device=dev), **kw)
    reported(met)
    for b, pos, i0, i1 in stored:
        pool.put(b, pos, k[i0:i1].double().numpy(), v[i0:i1].double().numpy())
    assert same_pages(kw, pool)


@pytest.mark.parametrize("counts", [[3, 60, 1, 40, 2], [1] * 5, [2, 70, 1, 1, 30, 1, 2, 1, 9]])
@pytest.mark.parametrize("code,E", [(0x7F, 120), (0xFF, 255), (0x7E, 254)])
def test_an_e4m3_sequence_that_is_not_finite_leaves_the_others_alone(counts, code, E):
    """One sequence's pages hold NaN codes or scales that overflow, its queries
    NaN; every other sequence's results are the same bits as without them."""
    dev = device()
    lens = [80 + 37 * b for b in range(len(counts))]
    pool = ref.filled_pool(lens, 2, 16, True, 3)
    T, sick = sum(counts), 1
    q, r = ref.normal_rows(T, 4, 1).to(dev), ref.normal_rows(T, 4, 2, 0.05).to(dev)
    kw, sl, cu = pool.to(dev), pool.seqlens.to(dev), ends(counts).to(dev)
    first = [row.contiguous() for row in (q[cu[1:].long() - 1], r[cu[1:].long() - 1])]

    def run():
        return [plx_prefill_fwd_paged(q, r, seqlens=sl, cu_q=cu, **kw)[0],
                plx_decode_fwd_paged(*first, seqlens=sl, **kw)]

    clean = run()
    for pages, scales in ((kw["kpages"], kw["kscale"]), (kw["vpages"], kw["vscale"])):
        for page in pool.table[sick, :(lens[sick] + 15) // 16].tolist():
            pages.view(torch.uint8)[page, :, ::3, ::5] = code
            scales[page, :, ::3] = E
    rows = slice(sum(counts[:sick]), sum(counts[:sick + 1]))
    q[rows, :, ::7] = float("nan")
    dirty = run()
    plx_check_device_error()
    others = torch.ones(T, dtype=torch.bool)
    others[rows] = False
    bits = lambda x: x.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(clean[0][others.to(dev)]), bits(dirty[0][others.to(dev)]))
    keep = [b for b in range(len(counts)) if b != sick]
    assert torch.equal(bits(clean[1][keep]), bits(dirty[1][keep]))


# ------------------------------------------------------------ debug build
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,counts,Hq,Hkv,page,behind", [
    ([1], [1], 2, 2, 16, 0), ([100, 70, 9, 0, 64], [3, 64, 0, 0, 1], 4, 2, 16, 2), ([5, 3], [9, 3], 4, 2, 16, 0),
    ([40, 33], [7, 33], 128, 1, 16, 0), ([50], [9], 65, 1, 32, 0), ([2000, 50, 1030], [4, 1, 300], 16, 8, 64, 0),
    ([6000], [130], 2, 1, 256, 0), ([300, 20, 40] + [90] * 9, [100, 2, 3] + [1] * 9, 4, 2, 16, 1),
    ([260] * 4, [256] * 4, 64, 32, 128, 0), ([500] * 17, [1] * 16 + [300], 4, 2, 16, 0)])
def test_debug_build_passes_its_checks(fp8, lens, counts, Hq, Hkv, page, behind, monkeypatch):
    """Valid calls of every form (few rows, tiles, both, rounds of whole items,
    split items): no check fails, and the bits are the release library's."""
    dev = device()
    pool = ref.filled_pool(lens, Hkv, page, fp8, 5)
    T, B = sum(counts) + behind, len(lens)
    q, r = ref.normal_rows(T, Hq, 1).to(dev), ref.normal_rows(T, Hq, 2, 0.05).to(dev)
    qd, rd = ref.normal_rows(B, Hq, 3).to(dev), ref.normal_rows(B, Hq, 4, 0.05).to(dev)
    k, v = ref.normal_rows(T, Hkv, 5).to(dev), ref.normal_rows(T, Hkv, 6).to(dev)
    sl, cu = pool.seqlens.to(dev), ends(counts).to(dev)
    cu_k = ends([max(n, 0) for n in lens]).to(dev)

    def run():
        kw = pool.to(dev)
        plx_kv_append(k, v, seqlens=sl, cu_q=cu, **kw)
        out, lse = torch.zeros_like(q), torch.zeros(T, Hq, device=dev)
        plx_prefill_fwd_paged(q, r, seqlens=sl, cu_q=cu, out=out, lse=lse, **kw)
        step = plx_decode_fwd_paged(qd, rd, seqlens=sl, **kw)
        back = plx_kv_read(cu_k=cu_k, T=int(cu_k[-1]), **kw)
        plx_check_device_error()
        return [out, lse.view(torch.int16), step, *back, kw["kpages"], kw["vpages"]]

    release = run()
    dbg = binding.load_debug_lib()
    monkeypatch.setattr(binding, "lib", lambda: dbg)
    for a, b in zip(release, run()):
        kind = torch.int16 if a.element_size() == 2 else torch.uint8
        assert torch.equal(a.view(kind), b.view(kind))
