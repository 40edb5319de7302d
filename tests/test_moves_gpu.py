"""The page bookkeeping of a paged KV cache on the GPU: rows that take over others'
pages, are cut, grown and emptied, and the compaction of the pool, against a host
reference; contents by reading sequences back."""
import random

import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, plx_check_device_error, plx_kv_compact,
                                             plx_kv_compact_workspace_bytes, plx_kv_read, plx_kv_update,
                                             plx_kv_update_workspace_bytes)

import moves_ref
from helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Cache:
    """A pool whose every slot holds bits of its own, and tables on both sides."""

    def __init__(self, B, width, num_pages, page, Hkv, fp8, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.width, self.n, self.page, self.fp8, self.Hkv = B, width, num_pages, page, fp8, Hkv
        shape = (num_pages, Hkv, page, 128)
        def codes(*s):  # every e4m3 code but NaN (0x7f, 0xff)
            return (torch.randint(0, 127, s, generator=g, dtype=torch.uint8)
                    + 128 * torch.randint(0, 2, s, generator=g, dtype=torch.uint8))
        if fp8:
            self.pools = [codes(*shape), codes(*shape), codes(*shape[:3]) % 127 + 1, codes(*shape[:3]) % 127 + 1]
        else:
            self.pools = [torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2)]
        self.table = [[-7] * width for _ in range(B)]
        self.lens, self.refs = [0] * B, [0] * num_pages
        d = [x.cuda() for x in self.pools]
        self.dev = dict(kpages=d[0].view(torch.float8_e4m3fn) if fp8 else d[0],
                        vpages=d[1].view(torch.float8_e4m3fn) if fp8 else d[1],
                        kscale=d[2] if fp8 else None, vscale=d[3] if fp8 else None,
                        block_table=ints(self.table), seqlens=ints(self.lens), page_refs=ints(self.refs))

    def host_update(self, want, src):
        rows, self.lens, self.refs, copies = moves_ref.update(self.table, self.lens, self.refs, want, src, self.page)
        for a, b, n in copies:
            for x in self.pools:
                x[b, :, :n] = x[a, :, :n]
        for b, row in enumerate(rows):
            self.table[b][:len(row)] = row
        return rows

    def update(self, want, src=None, **kw):
        rows = self.host_update(want, src)
        got = plx_kv_update(lens=ints(want), src=None if src is None else ints(src), **self.dev, **kw)
        self.dev.update(zip(("block_table", "seqlens", "page_refs"), got))
        return rows

    def compact(self, **kw):
        rows, refs, to, used = moves_ref.compact(self.table, self.lens, self.refs, self.page)
        pools = [x.clone() for x in self.pools]
        for a, b in enumerate(to):
            if b >= 0:
                for x, y in zip(pools, self.pools):
                    x[b] = y[a]
        self.pools, self.refs = pools, refs
        for b, row in enumerate(rows):
            self.table[b][:len(row)] = row
        table, counts, page_map, n = plx_kv_compact(**self.dev, **kw)
        self.dev.update(block_table=table, page_refs=counts)
        assert page_map.tolist() == to and n.tolist() == [used]

    def check(self):
        plx_check_device_error()
        assert self.dev["seqlens"].tolist() == self.lens
        assert self.dev["page_refs"].tolist() == self.refs
        assert self.dev["block_table"].tolist() == self.table
        names = ("kpages", "vpages", "kscale", "vscale")
        for x, name in zip(self.pools, names):
            y = self.dev[name].cpu()
            kind = torch.int16 if x.element_size() == 2 else torch.uint8
            assert torch.equal(x.view(kind), y.view(kind)), name
        # Counts are the rows' use; a partial last page is its row's alone.
        use = [0] * self.n
        for b, n in enumerate(self.lens):
            for p in self.table[b][:-(-n // self.page)]:
                use[p] += 1
        assert use == self.refs
        for b, n in enumerate(self.lens):
            if n % self.page:
                assert use[self.table[b][n // self.page]] == 1

    def tokens(self, b, n):
        at = [(self.table[b][i // self.page], i % self.page) for i in range(n)]
        return [torch.stack([x[p, :, s] for p, s in at]) if at else x[:0, :, 0] for x in self.pools]


def random_step(rng, c, spread):
    B, cap = c.B, c.width * c.page
    src = None if rng.random() < 0.3 else [
        b if rng.random() < 0.5 else rng.randrange(-1, B) for b in range(B)]
    want = []
    for b in range(B):
        s = b if src is None else src[b]
        have = 0 if s < 0 else c.lens[s]
        kind = rng.random()
        n = (have + rng.randint(0, 3) if kind < 0.4 else rng.randint(0, max(have, 1)) if kind < 0.6 else
             have // c.page * c.page if kind < 0.7 else have if kind < 0.8 else rng.randint(0, spread))
        want.append(min(n, cap))
    return want, src


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,width,num_pages,page,Hkv", [(5, 9, 24, 16, 2), (1, 3, 5, 32, 1), (40, 12, 300, 16, 3),
                                                        (7, 4, 20, 256, 1), (12, 6, 30, 64, 2)])
@pytest.mark.parametrize("in_place", [True, False])
def test_random_steps(B, width, num_pages, page, Hkv, fp8, in_place):
    """Forks, reorders, cuts, growth, rows that run out of pages, and compactions,
    one after the other on the same cache."""
    device()
    rng = random.Random(B * 1000 + page + fp8)
    c = Cache(B, width, num_pages, page, Hkv, fp8, seed=B)
    for step in range(30):
        want, src = random_step(rng, c, width * page)
        before = [c.tokens(b, n) for b, n in enumerate(c.lens)]
        lens = list(c.lens)
        outs = {}
        if not in_place:  # entries behind a row's pages are left as they were: so is the buffer
            outs = dict(block_table_out=ints(c.table), seqlens_out=torch.full_like(c.dev["seqlens"], 99),
                        page_refs_out=torch.full_like(c.dev["page_refs"], 99))
        c.update(want, src, **outs)
        c.check()
        for b in range(B):  # the kept tokens are the old row's
            s = b if src is None else src[b]
            kept = 0 if s < 0 else min(lens[s], c.lens[b])
            for x, y in zip(c.tokens(b, kept), before[s]):
                assert torch.equal(x, y[:kept])
        if step % 5 == 4:
            outs = {} if in_place else dict(block_table_out=ints(c.table),
                                            page_refs_out=torch.full_like(c.dev["page_refs"], 99))
            c.compact(**outs)
            c.check()


def test_inputs_are_left_alone_out_of_place():
    device()
    c = Cache(4, 6, 20, 16, 2, False)
    c.update([40, 16, 0, 5])
    old = {k: c.dev[k].clone() for k in ("block_table", "seqlens", "page_refs")}
    kw = dict(c.dev)
    outs = dict(block_table_out=torch.full((4, 6), -3, dtype=I32, device="cuda"),
                seqlens_out=torch.empty_like(old["seqlens"]), page_refs_out=torch.empty_like(old["page_refs"]))
    t, s, r = plx_kv_update(lens=ints([41, 41, 20, 0]), src=ints([0, 0, 1, 2]), **kw, **outs)
    plx_check_device_error()
    for k, v in old.items():
        assert torch.equal(kw[k], v)
    rows, lens, refs, _ = moves_ref.update(c.table, c.lens, c.refs, [41, 41, 20, 0], [0, 0, 1, 2], 16)
    assert s.tolist() == lens and r.tolist() == refs
    assert t.tolist() == [row + [-3] * (6 - len(row)) for row in rows]


def test_a_fork_reads_back_like_its_parent():
    device()
    c = Cache(6, 8, 60, 16, 2, True)
    c.update([100, 0, 0, 0, 0, 0])
    c.update([100, 101, 100, 37, 96, 0], [0, 0, 0, 0, 0, -1])
    c.check()
    cu = ints(np.cumsum([0] + c.lens).tolist())
    names = ("kpages", "vpages", "kscale", "vscale", "block_table")
    k, v = plx_kv_read(cu_k=cu, T=sum(c.lens), **{n: c.dev[n] for n in names})
    plx_check_device_error()
    for n, at in zip((100, 37, 96), (201, 301, 338)):
        assert torch.equal(k[at:at + n], k[:n]) and torch.equal(v[at:at + n], v[:n])
    assert torch.equal(k[100:200], k[:100])


def test_rows_that_find_no_pages():
    """From the first one that does not fit on, none gets any: they end with what they
    keep, and lose a partial page that they would have had to copy."""
    device()
    c = Cache(5, 8, 8, 16, 1, False)
    c.update([40, 20, 0, 0, 0])  # 3 + 2 pages: 3 free
    c.check()
    c.update([40, 20 + 32, 40, 40, 16], [0, 1, 0, 1, -1])
    c.check()
    # Row 2 copies a page and row 1 grows by two: three. Row 3 finds none, and row 4 neither.
    assert c.lens == [40, 52, 40, 16, 0]


def test_freed_pages_serve_the_same_call():
    device()
    c = Cache(3, 4, 4, 16, 2, True)
    c.update([64, 0, 0])
    c.update([0, 64, 0], [-1, -1, -1])
    c.check()
    c.update([64, 10, 0], [1, 1, -1])  # a permutation, with a cut page that is whole elsewhere: no page for a copy
    c.check()
    assert c.lens == [64, 0, 0]


@pytest.mark.parametrize("n,free", [(1, 0), (1, 1), (4096, 0), (4097, 4097), (30000, 9000), (70001, 35000)])
def test_pools_of_all_sizes(n, free):
    """Counts and ranks over many blocks; pages of one kv head of 16 slots."""
    device()
    rng = random.Random(n)
    B = 50
    used = rng.sample(range(n), n - free)
    width = max(1, -(-len(used) // B) + 3)
    c = Cache(B, width, n, 16, 1, True)
    for i, p in enumerate(used):
        c.table[i % B][i // B] = p
        c.lens[i % B] += 16
        c.refs[p] = 1
    c.dev.update(block_table=ints(c.table), seqlens=ints(c.lens), page_refs=ints(c.refs))
    c.compact()
    c.check()
    c.update([min(k + 33, width * 16) if i % 3 else 5 for i, k in enumerate(c.lens)])
    c.check()


@pytest.mark.parametrize("B", [3, 64, 700])
def test_steps_that_need_nothing_or_too_much(B):
    """Back to back on one stream: rows that keep partial pages and need no other,
    and rows of which most find none."""
    device()
    c = Cache(B, 4, 2 * B, 16, 1, True, seed=B)
    c.update([1 + b % 30 for b in range(B)])
    for i in range(60):
        same = list(c.lens)
        if i % 3 == 2:
            same = [min(64, n + 20) for n in same]
        c.update(same, [b for b in range(B)] if i % 2 else None)
        if i % 3 == 2:
            c.update([max(1, n - 25 - b % 7) if n else 0 for b, n in enumerate(c.lens)])
    c.check()


def test_many_rows():
    """More rows than the planning block has threads."""
    device()
    B = 2500
    c = Cache(B, 3, 5000, 16, 1, False)
    c.update([1 + b % 40 for b in range(B)])
    c.check()
    rng = random.Random(3)
    src = [rng.randrange(-1, B) for _ in range(B)]
    c.update([0 if s < 0 else min(48, c.lens[s] + 1) for s in src], src)
    c.check()


def test_pages_held_by_something_else():
    """A count above the rows' use keeps a page: whole, and as a partial last page."""
    device()
    c = Cache(2, 4, 12, 16, 1, False)
    c.update([40, 0])
    pages = c.table[0][:3]
    for p in (pages[0], pages[2]):
        c.refs[p] += 1
    c.dev["page_refs"] = ints(c.refs)
    c.update([41, 0])  # the last page is held: copied
    assert c.dev["page_refs"].tolist() == c.refs and c.dev["block_table"].tolist() == c.table
    assert c.table[0][2] != pages[2] and c.refs[pages[2]] == 1
    c.update([0, 0])
    assert c.dev["page_refs"].tolist() == c.refs and sum(c.refs) == 2
    plx_check_device_error()


def test_one_workspace_two_graphs_and_another_stream():
    """A step captured in place and replayed, its workspace shared with another graph
    on the same stream; then the same on a side stream."""
    device()
    c = Cache(8, 6, 60, 16, 2, True, seed=5)
    c.update([17 + 5 * b for b in range(8)])
    want, src = c.dev["seqlens"].clone(), ints(list(range(8)))
    ws = torch.empty(max(plx_kv_update_workspace_bytes(8, 60, 6), plx_kv_compact_workspace_bytes(60)),
                     dtype=torch.uint8, device="cuda")
    page_map, used = torch.empty(60, dtype=I32, device="cuda"), torch.empty(1, dtype=I32, device="cuda")
    plx_kv_compact(**c.dev, workspace=ws, page_map=page_map, used=used)  # attributes before the capture
    c.compact(workspace=ws)
    step, pack = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(step, stream=side):
        plx_kv_update(lens=want, src=src, workspace=ws, **c.dev)
    with torch.cuda.graph(pack, stream=side):
        plx_kv_compact(workspace=ws, page_map=page_map, used=used, **c.dev)
    rng = random.Random(8)
    with torch.cuda.stream(side):
        for _ in range(12):
            lens, rows = random_step(rng, c, 96)
            rows = list(range(8)) if rows is None else rows
            want.copy_(ints(lens))
            src.copy_(ints(rows))
            step.replay()
            c.host_update(lens, rows)
            pack.replay()
            moved, c.refs, to, n = moves_ref.compact(c.table, c.lens, c.refs, 16)
            old = [x.clone() for x in c.pools]
            for a, b in enumerate(to):
                if b >= 0:
                    for x, y in zip(c.pools, old):
                        x[b] = y[a]
            for b, row in enumerate(moved):
                c.table[b][:len(row)] = row
            side.synchronize()
            assert page_map.tolist() == to and used.tolist() == [n]
            c.check()


def test_calls_on_a_given_stream():
    device()
    side = torch.cuda.Stream()
    c = Cache(4, 6, 40, 16, 2, False)
    c.update([30, 0, 0, 0])
    torch.cuda.synchronize()
    want, src = ints([31, 31, 12, 0]), ints([0, 0, 0, -1])
    torch.cuda.synchronize()
    c.host_update([31, 31, 12, 0], [0, 0, 0, -1])
    plx_kv_update(lens=want, src=src, stream=side, **c.dev)
    out = plx_kv_compact(stream=side, **c.dev)
    side.synchronize()
    rows, c.refs, to, n = moves_ref.compact(c.table, c.lens, c.refs, 16)
    assert out[2].tolist() == to and out[3].tolist() == [n]
    assert c.dev["page_refs"].tolist() == c.refs


# ------------------------------------------------------------ bad tables
def reported(status=binding.PLX_ERR_INVALID_ARG):
    with pytest.raises(PlxError) as e:
        plx_check_device_error()
    assert e.value.status == status


@pytest.mark.parametrize("src,want", [([4, 1, 2, 3], [5, 16, 20, 0]), ([-2, 1, 2, 3], [5, 16, 20, 0]),
                                      ([2**31 - 1, 1, 2, 3], [5, 16, 20, 0]), ([0, 1, 2, 3], [97, 16, 20, 0]),
                                      ([0, 1, 2, 3], [2**31 - 1, 16, 20, 0])])
def test_rows_out_of_range_stay_as_they_were(src, want):
    device()
    c = Cache(4, 6, 30, 16, 1, False)
    c.update([33, 40, 50, 7])
    got = plx_kv_update(lens=ints(want), src=ints(src), **c.dev)
    reported()
    c.dev.update(zip(("block_table", "seqlens", "page_refs"), got))
    c.host_update([33] + want[1:], [0] + src[1:])
    c.check()


def test_negative_lengths_count_as_zero():
    device()
    c = Cache(3, 4, 10, 16, 1, True)
    c.update([20, 30, 40])
    c.update([-5, 30, -2**31], [0, 1, 1])
    c.check()
    assert c.lens == [0, 30, 0]


@pytest.mark.parametrize("bad", [-1, 30, 2**31 - 1, -2**31])
@pytest.mark.parametrize("where", [0, 2])  # a whole page, a partial last one
def test_pages_that_do_not_exist_are_reported(bad, where):
    device()
    c = Cache(4, 6, 30, 16, 1, False)
    c.update([40, 40, 0, 16])
    c.dev["block_table"][0, where] = bad
    plx_kv_update(lens=ints([41, 50, 40, 0]), src=ints([0, 1, 0, 3]), **c.dev)
    reported()
    assert c.dev["seqlens"].tolist()[1] == 50  # the others go on
    plx_kv_compact(**c.dev)
    if where == 0:
        reported()
        assert c.dev["block_table"][0, 0].item() == bad


def test_lengths_that_the_table_cannot_hold_are_reported():
    device()
    c = Cache(2, 3, 10, 16, 1, False)
    c.update([20, 30])
    c.dev["seqlens"][0] = 1000
    plx_kv_update(lens=ints([21, 31]), **c.dev)
    reported()
    assert c.dev["seqlens"].tolist()[1] == 31
    c.dev["seqlens"][0] = 1000
    plx_kv_compact(**c.dev)
    reported()


def test_a_used_page_with_a_count_of_zero_is_reported():
    device()
    c = Cache(2, 3, 10, 16, 1, False)
    c.update([20, 30])
    c.dev["page_refs"][c.table[1][0]] = 0
    plx_kv_compact(**c.dev)
    reported()


def test_pools_past_32_bit_offsets():
    """Pages behind 4 GB of a pool, to and from."""
    device()
    n, Hkv, page = 9000, 8, 256  # 512 KB of K a page: 4.7 GB
    kp = torch.zeros(n, Hkv, page, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table, refs = torch.full((2, 2), -7, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    refs[:n - 3] = 1  # all but the last three are held elsewhere
    table[0, 0], refs[n - 1] = n - 1, 1
    x = torch.randn(Hkv, page, 128, device="cuda").to(torch.bfloat16)
    kp[n - 1], vp[n - 1] = x, -x
    lens = ints([100, 0])
    t, s, r = plx_kv_update(kp, vp, table, lens, refs, ints([100, 100]), src=ints([0, 0]))
    plx_check_device_error()
    assert t[:, 0].tolist() == [n - 1, n - 3] and s.tolist() == [100, 100]
    assert torch.equal(kp[n - 3, :, :100], x[:, :100]) and torch.equal(vp[n - 3, :, :100], -x[:, :100])
    assert not kp[n - 3, :, 100:].any() and not kp[n - 2].any()
    refs[:] = 0
    refs[t[:, 0].long()] = 1
    t, r, to, used = plx_kv_compact(kp, vp, t, s, refs)
    plx_check_device_error()
    assert t[:, 0].tolist() == [1, 0] and used.tolist() == [2]
    assert torch.equal(kp[1], x) and torch.equal(vp[0, :, :100], -x[:, :100])


def test_debug_build_gives_the_same(monkeypatch):
    device()
    c = Cache(6, 6, 40, 16, 2, True)
    c.update([30, 50, 0, 0, 16, 1])
    monkeypatch.setattr(binding, "_lib", binding.load_debug_lib())
    c.update([31, 50, 40, 12, 0, 20], [0, 1, 1, 0, -1, 5])
    c.check()
    c.compact()
    c.check()
