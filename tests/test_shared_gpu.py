"""Decode for sequences that share prefixes, against fp64, and the calls around it
as a server makes them: rotate, append, prefill, fork, append, decode, free, compact."""
import random

import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, plx_check_device_error, plx_decode_fwd_paged,
                                             plx_decode_fwd_shared, plx_decode_shared_workspace_bytes,
                                             plx_kv_append, plx_kv_compact, plx_kv_update, plx_prefill_fwd_paged,
                                             plx_qkvr_proj, plx_rotary_freqs, plx_rotary_fwd)

import paged_ref as ref
from helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ends(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=I32, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def cache(sizes, prefix, lens, Hq, Hkv, page, fp8, seed=3, hide=True):
    """A pool in which every group's sequences begin with the same keys, each with its
    own pages: but for the first of a group, the whole ones in front of a sequence's own
    keys are then taken out of its table, and the slots in front of them get NaN (hide)."""
    pool = ref.filled_pool(lens, Hkv, page, fp8, seed)
    b = 0
    for n, p in zip(sizes, prefix):
        for i in range(b + 1, b + n):
            m = min(p, lens[i], lens[b])
            if m > 0:
                k, v = pool.get(b, m)
                pool.put(i, 0, k, v)
        b += n
    B = len(lens)
    q, r = ref.normal_rows(B, Hq, seed + 1), ref.normal_rows(B, Hq, seed + 2, 0.05)
    kw = pool.to("cuda")
    b = 0
    for n, p in zip(sizes, prefix):
        if hide:
            for i in range(b + 1, b + n):
                kw["block_table"][i, :max(0, p) // page] = -7
                if p % page and lens[i] > p:  # the shared slots of its first own page
                    at = pool.table[i, p // page].item()
                    for name in ("kpages", "vpages"):
                        kw[name].view(torch.uint8 if fp8 else torch.int16)[at, :, :p % page] = 0x7F if fp8 else 0x7FC0
                    if fp8:
                        kw["kscale"][at, :, :p % page] = kw["vscale"][at, :, :p % page] = 255
        b += n
    kw.update(seqlens=pool.seqlens.cuda(), cu_g=ends(sizes), prefix_lens=ints(prefix))
    return pool, q.cuda(), r.cuda(), kw


def problem(*args, **kw):
    """Queries, probes and arguments of a call, and what it gives in fp64."""
    pool, q, r, args = cache(*args, **kw)
    return q, r, args, ref.reference(pool, q.cpu(), r.cpu(), [1] * len(pool.lens))


CASES = [
    # sizes, prefix, lens, Hq, Hkv, page
    ([1], [1], [1], 2, 1, 16),
    ([3], [40], [41, 40, 300], 4, 2, 16),                       # one that ends with the prefix
    ([2, 3], [64, 100], [65, 200, 100, 101, 164], 4, 2, 32),    # whole pages; a partial one
    ([4, 1, 2], [0, 70, 33], [5, 0, 80, 1, 71, 33, 500], 8, 1, 16),  # no prefix, an empty sequence
    ([5], [200], [230, 10, 0, 199, 201], 4, 4, 64),             # shorter than the prefix, and empty
    ([2, 0, 2], [31, 7, 129], [32, 50, 130, 400], 6, 2, 128),   # an empty group, three heads a kv head
    ([70], [513], [514 + 7 * i for i in range(70)], 4, 2, 16),  # several row tiles
    ([9, 20], [1000, 65], [1000 + i for i in range(9)] + [65 + 3 * i for i in range(20)], 16, 1, 256),
    ([3], [5000], [5001, 5100, 5000], 4, 2, 64),                # split between CTAs
    ([2], [47], [48, 63], 2, 2, 16),                            # starts inside a page and a tile
    ([2] * 12, [90] * 12, [100] * 24, 4, 2, 32),                # alike groups
    ([3, 2], [64, 64], [64, 64, 64, 64, 64], 4, 2, 64),         # no keys behind any prefix
    ([2], [300], [301, 320], 128, 1, 32),                       # a whole tile of query heads
    ([2], [300], [301, 320], 96, 1, 32),                        # heads that do not fill one
    ([1] * 8 + [20] + [2] * 3, [100] * 8 + [333] + [50] * 3, [101] * 8 + [340] * 20 + [60] * 6, 4, 2, 16),  # both kernels
    ([9] * 5, [90, 90, 90, 64, 1], [100] * 45, 4, 2, 32),       # row tiles that few sequences fill
    ([12, 9], [130, 70], [131, 20, 0, 129, 130] + [150] * 7 + [70] * 9, 4, 2, 16),  # shorter than the prefix there
    ([40], [4000], [4001 + i for i in range(40)], 8, 1, 64),    # split, and several row tiles
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sizes,prefix,lens,Hq,Hkv,page", CASES)
def test_shared_decode_matches_fp64(sizes, prefix, lens, Hq, Hkv, page, fp8):
    device()
    q, r, kw, (o, _, bound) = problem(sizes, prefix, lens, Hq, Hkv, page, fp8)
    out = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "shared")
    ws = torch.empty(plx_decode_shared_workspace_bytes(len(lens), Hq, Hkv, 128), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # what an earlier call left
    again = plx_decode_fwd_shared(q, r, out=torch.empty_like(q), workspace=ws, **kw)
    plx_check_device_error()
    assert torch.equal(out, again)


def some_rows(out, q, r, pool, bs):
    """Rows `bs` of a decode against fp64."""
    G = q.shape[1] // pool.Hkv
    for b in bs:
        n = pool.lens[b]
        K, V = pool.get(b, n)
        for h in range(q.shape[1]):
            o, _, bound = ref.attend(q[b:b + 1, h].double().cpu().numpy(), r[b:b + 1, h].double().cpu().numpy(),
                                     K[:, h // G], V[:, h // G], [n])
            assert np.all(np.abs(out[b, h].double().cpu().numpy() - o[0]) <= bound[0]), (b, h)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_alike_groups(fp8):
    """So many row tiles that the CTAs take whole ones in rounds; shared pages."""
    device()
    n, groups, page = 33, 58, 16
    B = n * groups
    pool = ref.Pool([70] * B, 16, page, fp8, 3)
    g = torch.Generator().manual_seed(4)
    for name in ("k", "v"):
        x = getattr(pool, name)
        if fp8:  # codes of up to 15 (0x57), scales 2^-3 and 2^-4
            codes = torch.randint(0, 0x58, x.shape, generator=g, dtype=torch.uint8)
            setattr(pool, name, (codes + 128 * torch.randint(0, 2, x.shape, generator=g, dtype=torch.uint8)
                                 ).view(torch.float8_e4m3fn))
            setattr(pool, name + "s", torch.randint(123, 125, x.shape[:3], generator=g, dtype=torch.uint8))
        else:
            x.copy_(torch.randn(x.shape, generator=g))
    for b in range(B):
        pool.table[b, :4] = pool.table[b - b % n, :4]
    q, r = ref.normal_rows(B, 16, 5).cuda(), ref.normal_rows(B, 16, 6, 0.05).cuda()
    out = plx_decode_fwd_shared(q, r, seqlens=pool.seqlens.cuda(), cu_g=ends([n] * groups),
                                prefix_lens=ints([64] * groups), **pool.to("cuda"))
    plx_check_device_error()
    some_rows(out, q, r, pool, random.Random(1).sample(range(B), 40))


@pytest.mark.parametrize("fp8", [False, True])
def test_more_sequences_than_are_looked_up_ahead(fp8):
    """600 sequences in groups of two, and some in none."""
    device()
    sizes, prefix = [2] * 290, [20 + b % 40 for b in range(290)]
    lens = [p + 1 + b % 7 for b, p in enumerate(prefix) for _ in range(2)] + [5] * 20
    pool, q, r, kw = cache(sizes, prefix, lens, 2, 1, 16, fp8)
    out = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    some_rows(out, q, r, pool, range(len(lens)))


@pytest.mark.parametrize("fp8", [False, True])
def test_random_groups(fp8):
    """Sizes of all kinds, some sequences in no group."""
    device()
    for seed in range(8):
        rng = random.Random(seed)
        page, (Hq, Hkv) = rng.choice([16, 32, 64, 128, 256]), rng.choice([(4, 2), (8, 1), (6, 2), (3, 3), (20, 2)])
        sizes = [rng.choice([0, 1, 2, 3, 8] if seed % 2 else [0, 9, 20, 33]) for _ in range(rng.randint(1, 6))]
        prefix, lens = [], []
        for n in sizes:
            p = rng.choice([0, 1, rng.randint(1, 700)])
            prefix.append(p)
            mine = [p + rng.choice([0, 1, rng.randint(0, 300)]) for _ in range(n)]
            mine[1:] = [m if rng.random() < 0.8 else rng.randint(0, p) for m in mine[1:]]
            lens += mine
        lens += [rng.randint(0, 200) for _ in range(rng.randint(0 if lens else 1, 3))]
        q, r, kw, (o, _, bound) = problem(sizes, prefix, lens, Hq, Hkv, page, fp8, seed)
        out = plx_decode_fwd_shared(q, r, **kw)
        plx_check_device_error()
        ref.assert_within(out, o, bound, f"groups {seed}")


def test_equals_the_paged_decode():
    """On a cache whose rows really share pages, at the sizes of a server: both calls
    are within the bound of the same values, so within twice of each other."""
    device()
    B, Hq, Hkv, page, p, n = 24, 16, 8, 64, 3000, 200
    whole = p // page
    pages = whole + B * (-(-(p + n) // page) - whole)
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = (torch.randn(pages, Hkv, page, 128, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.empty(B, -(-(p + n) // page), dtype=I32, device="cuda")
    table[:, :whole] = torch.arange(whole, dtype=I32, device="cuda")
    table[:, whole:] = torch.arange(whole, pages, dtype=I32, device="cuda").view(B, -1)
    own = table[:, whole].long()
    kp[own, :, :p % page], vp[own, :, :p % page] = kp[own[0], :, :p % page], vp[own[0], :, :p % page]
    lens = ints([p + 1 + 8 * b for b in range(B)])
    q = torch.randn(B, Hq, 128, device="cuda", generator=g).to(torch.bfloat16)
    r = (torch.randn(B, Hq, 128, device="cuda", generator=g) * 0.05).to(torch.bfloat16)
    a = plx_decode_fwd_paged(q, r, kp, vp, table, lens)
    b = plx_decode_fwd_shared(q, r, kp, vp, table, lens, ends([B]), ints([p]))
    plx_check_device_error()
    # Bound of each: 2^-8 (2 sum w |v| + ... + |o|), w uniform-like: |v| averages 0.8, t 0.05 * 11 |v|.
    assert (a.float() - b.float()).abs().max().item() <= 2 * 1.02 * 2.0 ** -8 * (1 + 0.8 * (1 + 0.6 + 0.6) + 0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", ["q", "r"])
def test_a_query_that_is_not_a_number_gives_nan(fp8, where):
    device()
    for sizes, prefix, lens in (([4], [3000], [3001, 3100, 0, 50]), ([2, 3], [64, 0], [65, 64, 7, 8, 9])):
        q, r, kw, _ = problem(sizes, prefix, lens, 4, 2, 32, fp8)
        clean = plx_decode_fwd_shared(q, r, **kw)
        (q if where == "q" else r)[1, 2, 17] = float("nan")
        dirty = plx_decode_fwd_shared(q, r, **kw)
        plx_check_device_error()
        sick = torch.zeros(len(lens), 4, dtype=torch.bool, device="cuda")
        sick[1, 2] = True
        assert torch.isnan(dirty[sick]).all() and torch.equal(clean[~sick], dirty[~sick])


@pytest.mark.parametrize("fp8", [False, True])
def test_one_key_gives_its_value(fp8):
    device()
    q, r, kw, _ = problem([3, 1], [1, 0], [1, 1, 1, 1], 4, 2, 16, fp8)
    r *= 400  # probes whose covariance term would show
    out = plx_decode_fwd_shared(q, r, **kw)
    one = plx_decode_fwd_paged(q[3:], r[3:], kw["kpages"], kw["vpages"], kw["block_table"][3:].contiguous(),
                               kw["seqlens"][3:], kw["kscale"], kw["vscale"])
    plx_check_device_error()
    assert torch.equal(out[3:], one)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("bad", ["prefix", "ends below", "ends above", "ends decrease", "page", "length"])
def test_bad_groups_are_reported(bad):
    device()
    sizes, prefix, lens = [2, 2], [40, 64], [41, 90, 70, 100]
    q, r, kw, (o, _, bound) = problem(sizes, prefix, lens, 4, 2, 16, False, hide=False)
    if bad == "prefix":
        kw["prefix_lens"][0] = 42
    elif bad == "ends below":
        kw["cu_g"][0] = -5
    elif bad == "ends above":
        kw["cu_g"][2] = 60
    elif bad == "ends decrease":
        kw["cu_g"][1] = 5
    elif bad == "page":
        kw["block_table"][0, 1] = 10**6
    else:
        kw["seqlens"][0] = 10**6
    out = plx_decode_fwd_shared(q, r, **kw)
    with pytest.raises(PlxError) as e:
        plx_check_device_error()
    assert e.value.status == binding.PLX_ERR_INVALID_ARG
    if bad == "prefix":  # taken for none: every sequence has all of its keys
        ref.assert_within(out, o, bound, "without its prefix")
    out = plx_decode_fwd_shared(*problem(sizes, prefix, lens, 4, 2, 16, False)[:2],
                                **problem(sizes, prefix, lens, 4, 2, 16, False)[2])
    plx_check_device_error()
    ref.assert_within(out, o, bound, "afterwards")


def test_two_graphs_share_a_workspace_and_repeat():
    device()
    q, r, kw, (o, _, bound) = problem([5, 3], [700, 90], [701, 800, 0, 900, 750, 91, 95, 300], 4, 2, 32, True)
    ws = torch.empty(plx_decode_shared_workspace_bytes(8, 4, 2, 128), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    plx_decode_fwd_shared(q, r, workspace=ws, **kw)
    torch.cuda.synchronize()
    graphs = []
    for x in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plx_decode_fwd_shared(q, r, out=x, workspace=ws, **kw)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    plx_check_device_error()
    ref.assert_within(outs[0], o, bound, "replayed")
    assert torch.equal(outs[0], outs[1])


def test_two_streams_at_once():
    device()
    a = problem([4], [1500], [1501, 1600, 1550, 2000], 4, 2, 16, False, 3)
    b = problem([2, 2], [64, 500], [65, 100, 501, 700], 4, 2, 64, True, 4)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = [plx_decode_fwd_shared(x[0], x[1], stream=s, **x[2]) for x, s in zip((a, b), side)]
        torch.cuda.synchronize()
        for x, out in zip((a, b), outs):
            ref.assert_within(out, x[3][0], x[3][2], "two streams")
    plx_check_device_error()


def test_pages_past_32_bit_offsets():
    """A prefix and own keys behind 4 GB of the pool, in both kernels."""
    device()
    for sizes, Hq in (([3], 8), ([6, 3], 32)):  # few rows; 24 and 12 rows a kv head
        n, Hkv, page, B = 9000, 8, 256, sum(sizes)
        kp = torch.zeros(n, Hkv, page, 128, dtype=torch.bfloat16, device="cuda")
        vp = torch.zeros_like(kp)
        kp[n - 40:], vp[n - 40:] = torch.randn(2, 40, Hkv, page, 128, device="cuda").to(torch.bfloat16)
        first = [sum(sizes[:g]) for g in range(len(sizes))]
        table = torch.zeros(B, 2, dtype=I32, device="cuda")
        for g, b in enumerate(first):
            table[b:b + sizes[g], 0] = n - 1 - g
        table[:, 1] = torch.arange(n - 20, n - 20 + B, device="cuda")
        lens = ints([260 + b for b in range(B)])
        q, r = (ref.normal_rows(B, Hq, 3, x).cuda() for x in (1.0, 0.05))
        out = plx_decode_fwd_shared(q, r, kp, vp, table, lens, ends(sizes), ints([256] * len(sizes)))
        plx_check_device_error()
        for b in range(B):
            K, V = (torch.cat([x[table[b, 0].item()], x[table[b, 1].item()]], 1)[:, :260 + b].double().cpu().numpy()
                    for x in (kp, vp))
            for h in range(Hq):
                o, _, bound = ref.attend(q[b:b + 1, h].double().cpu().numpy(), r[b:b + 1, h].double().cpu().numpy(),
                                         K[h // (Hq // Hkv)], V[h // (Hq // Hkv)], [260 + b])
                assert np.all(np.abs(out[b, h].double().cpu().numpy() - o[0]) <= bound[0]), (b, h)
        del kp, vp


def test_calls_from_two_host_threads():
    """Each with a stream, a cache and queries of its own: rotate, update, decode."""
    import threading
    device()
    freq, _ = plx_rotary_freqs(128, device="cuda")
    jobs = []
    for seed in (3, 4):
        q, r, kw, (o, _, bound) = problem([3, 40], [300, 70], [301, 320, 5] + [90] * 40, 4, 2, 32, seed == 4, seed)
        x = ref.normal_rows(64, 4, seed).cuda()
        pos = torch.arange(64, dtype=I32, device="cuda") * seed
        want = plx_rotary_fwd(x, None, freq, positions=pos)[0]
        jobs.append((q, r, kw, o, bound, x, pos, want))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        q, r, kw, o, bound, x, pos, want = job
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                table = torch.zeros(4, 4, dtype=I32, device="cuda")
                lens, refs = (torch.zeros(k, dtype=I32, device="cuda") for k in (4, 12))
                pages = torch.zeros(2, 12, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
                for i in range(20):
                    out = plx_decode_fwd_shared(q, r, **kw)
                    y = plx_rotary_fwd(x, None, freq, positions=pos)[0]
                    grown = min(40, 2 * i + 2)
                    plx_kv_update(pages[0], pages[1], table, lens, refs, ints([grown, grown, 0, 0]),
                                  src=ints([0, 0, -1, -1]))
                torch.cuda.current_stream().synchronize()
                ref.assert_within(out, o, bound, "thread")
                assert torch.equal(y, want) and lens.tolist() == [40, 40, 0, 0]
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    plx_check_device_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_debug_build_gives_the_same_bits(fp8, monkeypatch):
    device()
    cases = [problem(*c, fp8) for c in CASES[1:]]
    want = [plx_decode_fwd_shared(q, r, **kw) for q, r, kw, _ in cases]
    plx_check_device_error()
    monkeypatch.setattr(binding, "_lib", binding.load_debug_lib())
    got = [plx_decode_fwd_shared(q, r, **kw) for q, r, kw, _ in cases]
    plx_check_device_error()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_sampling_several_continuations(fp8):
    """Two prompts are projected, rotated, appended and prefilled; each is forked into
    three rows, which grow by tokens of their own; one ends, the pool is compacted,
    and a row is forked again. Every decode is checked against fp64 on what the cache
    holds, and the prompt's last token against the prefill."""
    device()
    Hq, Hkv, page, Dm, B = 4, 2, 16, 256, 6
    g = torch.Generator().manual_seed(12)
    w = (torch.randn((2 * Hq + 2 * Hkv) * 128, Dm, generator=g) / Dm ** 0.5)
    w[(Hq + 2 * Hkv) * 128:] *= 0.05
    w = w.to(torch.bfloat16).cuda()
    freq, scale = plx_rotary_freqs(64, scaling="linear", factor=2.0, device="cuda")
    pages = 40
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pool = dict(kpages=torch.zeros(pages, Hkv, page, 128, device="cuda").to(dt),
                vpages=torch.zeros(pages, Hkv, page, 128, device="cuda").to(dt),
                kscale=torch.ones(pages, Hkv, page, dtype=torch.uint8, device="cuda") if fp8 else None,
                vscale=torch.ones(pages, Hkv, page, dtype=torch.uint8, device="cuda") if fp8 else None)
    tables = dict(block_table=torch.zeros(B, 8, dtype=I32, device="cuda"),
                  seqlens=torch.zeros(B, dtype=I32, device="cuda"))
    refs = torch.zeros(pages, dtype=I32, device="cuda")

    def tokens(n):
        x = torch.randn(n, Dm, generator=g).to(torch.bfloat16).cuda()
        return [t[0].transpose(0, 1) for t in plx_qkvr_proj(x, w, 1, n, Hq, Hkv)]  # [n, H, 128]

    def rotated(q, k, r, cu):
        return [t.contiguous() for t in
                plx_rotary_fwd(q, k, freq, r, seqlens=tables["seqlens"], cu_q=cu, scale=scale)]

    def exact(q, r, rows):
        """fp64 on the cache's contents, for the last token of each of `rows`."""
        host = ref.Pool([int(n) for n in tables["seqlens"].tolist()], Hkv, page, fp8, 0)
        host.k, host.v = pool["kpages"].cpu(), pool["vpages"].cpu()
        if fp8:
            host.ks, host.vs = pool["kscale"].cpu(), pool["vscale"].cpu()
        host.table = tables["block_table"].cpu()
        return ref.reference(host, q.cpu(), r.cpu(), [1] * B)

    # Prompts in rows 0 and 3.
    plx_kv_update(page_refs=refs, lens=ints([45, 0, 0, 64, 0, 0]), **pool, **tables)
    cu = ints([0, 45, 45, 45, 109, 109, 109])
    q, k, v, r = tokens(109)
    q, k, r = rotated(q, k, r, cu)
    plx_kv_append(k, v.contiguous(), cu_q=cu, **pool, **tables)
    prompt, _ = plx_prefill_fwd_paged(q, r, cu_q=cu, **pool, **tables)
    # Forks; each row then takes a token of its own.
    src, lens, cu_g, prefix = ints([0, 0, 0, 3, 3, 3]), [45, 45, 45, 64, 64, 64], ints([0, 3, 6]), ints([45, 64])
    plx_kv_update(page_refs=refs, lens=ints(lens), src=src, **pool, **tables)
    last = torch.tensor([44] * 3 + [108] * 3, device="cuda")
    out = plx_decode_fwd_shared(q[last].contiguous(), r[last].contiguous(), cu_g=cu_g, prefix_lens=prefix, **pool, **tables)
    plx_check_device_error()
    o, _, bound = exact(q[last], r[last], range(B))
    ref.assert_within(out, o, bound, "forked")
    ref.assert_within(prompt[last], o, bound, "prefill")
    for step in range(20):
        lens = [n + 1 for n in lens]
        if step == 9:
            lens[1] = 0  # a row ends
        if step > 9:
            lens[1] = 0
        plx_kv_update(page_refs=refs, lens=ints(lens), **pool, **tables)
        if step == 12:
            plx_kv_compact(page_refs=refs, **pool, **tables)
        if step == 15:  # row 1 is taken up again, from row 2 and its last tokens
            lens[1] = lens[2]
            plx_kv_update(page_refs=refs, lens=ints(lens), src=ints([0, 2, 2, 3, 4, 5]), **pool, **tables)
        assert tables["seqlens"].tolist() == lens
        live = torch.tensor([n > 0 for n in lens], device="cuda")
        q, k, v, r = tokens(B)
        cu = ends([int(n > 0) for n in lens])
        some = lambda t: t[live].contiguous()  # noqa: E731
        qs, ks, rs = rotated(some(q), some(k), some(r), cu)
        plx_kv_append(ks, some(v), cu_q=cu, **pool, **tables)
        q, r = q.contiguous(), r.contiguous()
        q[live], r[live] = qs, rs
        out = plx_decode_fwd_shared(q, r, cu_g=cu_g, prefix_lens=prefix, **pool, **tables)
        plx_check_device_error()
        o, _, bound = exact(q, r, range(B))
        ref.assert_within(out, o, bound, f"step {step}")
        assert not out[~live].any()
    plx_kv_update(page_refs=refs, lens=ints([0] * B), **pool, **tables)
    assert not refs.any()
