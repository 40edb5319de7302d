"""Decode for sequences that share prefixes where its groups are unusual: more groups
than sequences, and groups whose first sequences have ended."""
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, plx_check_device_error, plx_decode_fwd_shared,
                                             plx_kv_append, plx_kv_update)

import paged_ref as ref
from helpers import device
from test_shared_gpu import I32, ends, problem

pytestmark = pytest.mark.gpu

MORE_GROUPS = [  # sizes, prefix, lens, Hq, Hkv, page
    ([0] * 30 + [20], [9] * 30 + [70], [71 + 3 * i for i in range(20)], 4, 2, 16),         # tile kernel, group 30 of 20 sequences
    ([0] * 50 + [40], [0] * 50 + [4000], [4001 + i for i in range(40)], 8, 1, 64),         # split between its CTAs
    ([0] * 9 + [3] + [0] * 700 + [2], [5] * 9 + [40] + [5] * 700 + [64], [41, 40, 300, 64, 90], 4, 2, 16),  # rows kernel
    ([0] * 40 + [20, 0, 2], [1] * 40 + [65, 7, 129], [66 + i for i in range(20)] + [130, 140], 16, 1, 32),  # both
    ([0] * 99 + [1], [3] * 99 + [1], [1], 2, 1, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(MORE_GROUPS)))
def test_more_groups_than_sequences(case, fp8, monkeypatch):
    """Empty groups count: a group's number may pass the number of sequences. The debug
    build's index checks hold too, and it gives the same bits."""
    device()
    q, r, kw, (o, _, bound) = problem(*MORE_GROUPS[case], fp8)
    out = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    ref.assert_within(out, o, bound, "more groups")
    monkeypatch.setattr(binding, "_lib", binding.load_debug_lib())
    again = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    assert torch.equal(out, again)


ENDED = [  # sizes, sequences in front of each group's that have ended, prefix, lens (of the others), Hq, Hkv, page
    ([3], [1], [40], [41, 40, 300], 4, 2, 16),                                     # rows kernel
    ([3, 2, 1], [2, 0, 1], [64, 100, 30], [65, 200, 0, 101, 164, 31], 4, 2, 32),   # one in the middle, too
    ([20, 33], [5, 0], [333, 70], [334 + 3 * i for i in range(20)] + [71 + i for i in range(33)], 4, 2, 16),  # tile kernel
    ([3, 20], [7, 1], [100, 333], [101, 20, 150] + [340] * 20, 4, 2, 16),          # both, fewer keys than the prefix
    ([40], [24], [4000], [4001 + i for i in range(40)], 8, 1, 64),                 # split between CTAs
    ([0, 2, 0], [4, 1, 3], [500, 129, 7], [130, 400], 6, 2, 128),                  # all of a group
    ([1], [299], [100], [110], 4, 2, 16),                                          # one of 300 is left
    ([33, 2], [260, 135], [90, 31], [91 + i for i in range(33)] + [32, 31], 4, 2, 32),
    ([1, 3], [600, 41], [17, 64], [18, 65, 0, 70], 2, 1, 16),                      # more than are looked up ahead
    ([2] * 290, [1] * 290, [20 + b % 40 for b in range(290)],
     [20 + b % 40 + 1 + i for b in range(290) for i in range(2)], 2, 1, 16),       # 870 sequences
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(ENDED)))
def test_a_group_whose_first_sequences_have_ended(case, fp8, monkeypatch):
    """The shared keys are only in the pages of the first sequence that has keys (the
    others' entries for them do not exist); ended ones have no entries at all."""
    device()
    sizes, gone, prefix, lens, Hq, Hkv, page = ENDED[case]
    q0, r0, kw, (o, _, bound) = problem(sizes, prefix, lens, Hq, Hkv, page, fp8)
    at, b = [], 0  # where the sequences with lens are in the batch
    for n, dead in zip(sizes, gone):
        at += range(b + dead, b + dead + n)
        b += dead + n
    live = torch.tensor(at, device="cuda")

    def among(x, fill):
        y = torch.full((b, *x.shape[1:]), fill, dtype=x.dtype, device="cuda")
        y[live] = x
        return y

    q, r = among(q0, float("nan")), among(r0, float("nan"))
    kw.update(block_table=among(kw["block_table"], -7), seqlens=among(kw["seqlens"], 0),
              cu_g=ends([n + dead for n, dead in zip(sizes, gone)]))
    out = plx_decode_fwd_shared(q, r, **kw)
    plx_check_device_error()
    ref.assert_within(out[live], o, bound, "behind ended ones")
    over = torch.ones(b, dtype=torch.bool, device="cuda")
    over[live] = False
    assert not out[over].any()
    kw["seqlens"][over] = -3  # below zero is none, too
    assert torch.equal(out, plx_decode_fwd_shared(q, r, **kw))
    plx_check_device_error()
    monkeypatch.setattr(binding, "_lib", binding.load_debug_lib())
    assert torch.equal(out, plx_decode_fwd_shared(q, r, **kw))
    plx_check_device_error()


def test_a_first_sequence_with_a_length_out_of_range_is_reported():
    """It counts as one without keys: the others have theirs."""
    device()
    q, r, kw, (o, _, bound) = problem([3], [40], [41, 50, 300], 4, 2, 16, False)
    kw["block_table"][1] = kw["block_table"][0]  # the first one's pages hold the shared keys
    kw["seqlens"][0], kw["seqlens"][1] = 10**6, 41
    out = plx_decode_fwd_shared(q, r, **kw)
    with pytest.raises(PlxError) as e:
        plx_check_device_error()
    assert e.value.status == binding.PLX_ERR_INVALID_ARG
    ref.assert_within(out[2:], o[2:], bound[2:], "behind a bad length")


def test_the_prompts_continuations_end_one_after_the_other():
    """Eight forks of a prompt; the first one ends, then the next, until none is left."""
    device()
    B, Hq, Hkv, page, p = 8, 4, 2, 16, 70
    g = torch.Generator().manual_seed(5)
    ints = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    cache = dict(kpages=torch.zeros(40, Hkv, page, 128, dtype=torch.bfloat16, device="cuda"),
                 vpages=torch.zeros(40, Hkv, page, 128, dtype=torch.bfloat16, device="cuda"),
                 block_table=torch.zeros(B, 8, dtype=I32, device="cuda"), seqlens=torch.zeros(B, dtype=I32, device="cuda"))
    refs = torch.zeros(40, dtype=I32, device="cuda")

    def rows(n, heads, scale=1.0):
        return (torch.randn(n, heads, 128, generator=g) * scale).to(torch.bfloat16).cuda()

    plx_kv_update(page_refs=refs, lens=ints([p] + [0] * 7), **cache)
    plx_kv_append(rows(p, Hkv), rows(p, Hkv), cu_q=ints([0] + [p] * 8), **cache)
    plx_kv_update(page_refs=refs, lens=ints([p] * 8), src=ints([0] * 8), **cache)
    for gone in range(9):
        lens = [0 if b < gone else p + gone + 1 for b in range(B)]
        plx_kv_update(page_refs=refs, lens=ints(lens), **cache)
        n = B - gone
        if n > 0:
            plx_kv_append(rows(n, Hkv), rows(n, Hkv), cu_q=ends([int(k > 0) for k in lens]), **cache)
        q, r = rows(B, Hq), rows(B, Hq, 0.05)
        out = plx_decode_fwd_shared(q, r, cu_g=ints([0, 8]), prefix_lens=ints([p]), **cache)
        plx_check_device_error()
        host = ref.Pool(lens, Hkv, page, False, 0)
        host.k, host.v, host.table = (cache[x].cpu() for x in ("kpages", "vpages", "block_table"))
        o, _, bound = ref.reference(host, q.cpu(), r.cpu(), [1] * B)
        ref.assert_within(out, o, bound, f"{gone} have ended")
    assert not refs.any()
