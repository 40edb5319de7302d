"""Refusals of the rotary, page bookkeeping and shared-prefix calls, the frequencies,
and pins of the host references (CPU only: nothing here launches a kernel)."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

from parametrized_local_linear_gb300 import (PlxError, binding, build, plx_decode_fwd_shared, plx_kv_compact,
                                             plx_kv_update, plx_rotary_bwd, plx_rotary_freqs, plx_rotary_fwd)

import moves_ref
import paged_ref as ref

P = ctypes.c_void_p(4096)
Q = ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4104)
INV, UNS = binding.PLX_ERR_INVALID_ARG, binding.PLX_ERR_UNSUPPORTED
I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


# ------------------------------------------------------------ C refusals
def _shared(lib, **kw):
    a = dict(q=P, r=P, kp=P, vp=P, ks=None, vs=None, table=P, sl=P, cu=P, pre=P, out=P, ng=1, B=2, Hq=4, Hkv=2,
             d=128, n=8, page=16, width=4, ws=None, wsb=0)
    a.update(kw)
    return lib.plx_decode_fwd_shared(*a.values(), None)


def _update(lib, **kw):
    a = dict(kp=P, vp=P, ks=None, vs=None, table=P, sl=P, refs=P, src=None, lens=P, to=Q, so=Q, ro=Q, B=2, Hkv=2,
             d=128, n=8, page=16, width=4, ws=None, wsb=0)
    a.update(kw)
    return lib.plx_kv_update(*a.values(), None)


def _compact(lib, **kw):
    a = dict(kp=P, vp=P, ks=None, vs=None, table=P, sl=P, refs=P, to=Q, ro=Q, map=P, used=P, B=2, Hkv=2, d=128, n=8,
             page=16, width=4, ws=None, wsb=0)
    a.update(kw)
    return lib.plx_kv_compact(*a.values(), None)


CALLS = {"shared": _shared, "update": _update, "compact": _compact}


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("kw,status,word", [
    (dict(kp=None), INV, b"null"), (dict(vp=None), INV, b"null"), (dict(table=None), INV, b"null"),
    (dict(sl=None), INV, b"null"), (dict(ks=P), INV, b"both"), (dict(B=0), INV, b">= 1"), (dict(n=0), INV, b">= 1"),
    (dict(width=0), INV, b">= 1"), (dict(d=64), UNS, b"head dim"), (dict(page=48), UNS, b"page_size"),
    (dict(kp=ODD), INV, b"aligned"), (dict(n=1 << 26), UNS, b"2^31"), (dict(width=(1 << 26) + 1), UNS, b"2^30"),
    (dict(ws=P, wsb=8), INV, b"workspace"), (dict(ws=ODD, wsb=1 << 40), INV, b"workspace"),
])
def test_cache_arguments_are_checked(lib, call, kw, status, word):
    assert CALLS[call](lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=None), INV, b"null"), (dict(out=None), INV, b"null"), (dict(cu=None), INV, b"cu_g"),
    (dict(pre=None), INV, b"prefix_lens"), (dict(ng=0), INV, b"ngroups"), (dict(ng=(1 << 24) + 1), UNS, b"2^24"), (dict(Hq=3), INV, b"multiple"),
    (dict(Hq=512), UNS, b"at most 128"), (dict(r=ODD), INV, b"aligned"), (dict(B=1 << 23), UNS, b"2^24"),
])
def test_shared_arguments_are_checked(lib, kw, status, word):
    assert _shared(lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(refs=None), INV, b"null"), (dict(lens=None), INV, b"null"), (dict(so=None), INV, b"null"),
    (dict(to=P), INV, b"all of the outputs"), (dict(ro=P, so=P), INV, b"all of the outputs"),
    (dict(B=(1 << 20) + 1), UNS, b"2^20"),
])
def test_update_arguments_are_checked(lib, kw, status, word):
    assert _update(lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(refs=None), INV, b"null"), (dict(map=None), INV, b"null"), (dict(used=None), INV, b"null"),
    (dict(to=P), INV, b"both of the outputs"),
])
def test_compact_arguments_are_checked(lib, kw, status, word):
    assert _compact(lib, **kw) == status
    assert word in lib.plx_last_error_message()


def _turn(lib, fn="plx_rotary_fwd", st=None, **kw):
    # sequence, token, head of q, k, r, q_out, k_out, r_out
    strides = [2 * 4 * 128, 128, 2 * 128] * 6 if st is None else st
    V = [ctypes.c_void_p(4096 * i) for i in range(1, 7)]
    a = dict(q=V[0], k=V[1], r=V[2], qo=V[3], ko=V[4], ro=V[5], strides=(ctypes.c_longlong * 18)(*strides), pos=None, sl=None, cu=None,
             freq=P, scale=1.0, nseq=0, B=3, L=2, Hq=4, Hkv=4, d=128, R=128, near=0, dtype=0)
    a.update(kw)
    return getattr(lib, fn)(*a.values(), None)


@pytest.mark.parametrize("fn", ["plx_rotary_fwd", "plx_rotary_bwd"])
@pytest.mark.parametrize("kw,status,word", [
    (dict(strides=None), INV, b"null"), (dict(freq=None), INV, b"null"), (dict(L=-1), INV, b">= 1"),
    (dict(Hq=0), INV, b">= 1"), (dict(d=96), UNS, b"head dim"), (dict(R=0), INV, b"rotary_dim"),
    (dict(R=130), INV, b"rotary_dim"), (dict(R=7), INV, b"rotary_dim"), (dict(dtype=2), INV, b"dtype"),
    (dict(pos=P, sl=P), INV, b"exclude"), (dict(cu=P), INV, b"cu_q"), (dict(sl=P, nseq=2), INV, b"packed"),
    (dict(sl=P, nseq=0, B=1), INV, b"nseq"), (dict(sl=P, nseq=3, B=1), INV, b"one row"),
    (dict(q=None, k=None, r=None, qo=None, ko=None, ro=None), INV, b"all null"),
    (dict(qo=None), INV, b"both"), (dict(k=None), INV, b"both"), (dict(r=ODD), INV, b"aligned"),
    (dict(B=1 << 20, L=1 << 12), UNS, b"2^31"), (dict(qo=P, st=[1024, 128, 256] * 3 + [2048, 128, 256] * 3), INV, b"same strides"),
    (dict(ko=P), INV, b"output is q"), (dict(qo=Q, k=Q, ko=Q), INV, b"output is k"), (dict(ro=ctypes.c_void_p(5 * 4096)), INV, b"output is"),
    (dict(st=[1024, 128, 0] * 6), INV, b"multiples"), (dict(st=[1024, 132, 256] * 6), INV, b"multiples"),
    (dict(st=[1024, 128, 256] * 3 + [1024, 128, 128] * 3), INV, b"overlap"),
    (dict(st=[1024, 128, 256] * 3 + [512, 128, 256] * 3), INV, b"overlap"),
])
def test_rotary_arguments_are_checked(lib, fn, kw, status, word):
    assert _turn(lib, fn, **kw) == status
    assert word in lib.plx_last_error_message()


def test_no_rows_is_a_call_that_does_nothing(lib):
    assert _turn(lib, L=0) == binding.PLX_OK
    assert _turn(lib, B=0) == binding.PLX_OK


def test_workspace_sizes(lib):
    assert lib.plx_decode_shared_workspace_bytes(4, 16, 8, 128) > lib.plx_decode_paged_workspace_bytes(4, 16, 8, 128)
    assert lib.plx_decode_shared_workspace_bytes(4, 12, 8, 128) == 0
    assert lib.plx_decode_shared_workspace_bytes(0, 16, 8, 128) == 0
    assert lib.plx_kv_update_workspace_bytes(4, 100, 10) > 0 and lib.plx_kv_update_workspace_bytes(4, 0, 10) == 0
    assert lib.plx_kv_compact_workspace_bytes(100) > 0 and lib.plx_kv_compact_workspace_bytes(0) == 0


# ------------------------------------------------------------ frequencies
def test_frequencies():
    f, s = plx_rotary_freqs(64, base=500000.0)
    want = 500000.0 ** (-np.arange(32) / 32)
    assert s == 1.0 and f.dtype == torch.float64 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    assert np.allclose(plx_rotary_freqs(64, base=500000.0, scaling="linear", factor=4.0)[0].numpy(), want / 4, rtol=1e-14)
    f, s = plx_rotary_freqs(64, scaling="base", factor=4.0)
    plain = plx_rotary_freqs(64)[0]
    assert s == 1.0 and f[0] == 1.0 and math.isclose(f[31], plain[31] / 4, rel_tol=1e-13)
    f, s = plx_rotary_freqs(64, scaling="parts", factor=8.0, original_len=4096)
    turns = 4096 * plain.numpy() / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(8.0) + 1)
    for i in range(32):
        keep = min(1.0, max(0.0, (turns[i] - 1) / 31))
        assert math.isclose(f[i], plain[i] * keep + plain[i] / 8 * (1 - keep), rel_tol=1e-13)
    assert f[0] == plain[0] and math.isclose(f[31], plain[31] / 8, rel_tol=1e-14)
    one, s = plx_rotary_freqs(64, scaling="parts", factor=1.0, original_len=4096)
    assert s == 1.0 and torch.allclose(one, plain, rtol=1e-15, atol=0)


@pytest.mark.parametrize("kw,word", [
    (dict(rotary_dim=7), "rotary_dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(base=0.0), "base"),
    (dict(base=float("nan")), "base"), (dict(scaling="linear", factor=0.5), "factor"),
    (dict(scaling="base", rotary_dim=2, factor=2.0), "above 2"), (dict(scaling="parts", factor=2.0), "original_len"),
    (dict(scaling="parts", factor=2.0, original_len=10, beta_slow=32.0), "beta_fast"),
])
def test_frequency_refusals(kw, word):
    with pytest.raises(PlxError, match=word):
        plx_rotary_freqs(**dict(dict(rotary_dim=64), **kw))
    with pytest.raises(ValueError, match="scaling"):
        plx_rotary_freqs(64, scaling="another")


# ------------------------------------------------------------ binding refusals
def _cache(fp8=False):
    pool = ref.Pool([20, 3], 2, 16, fp8, 1)
    kw = pool.to("cpu")
    kw["seqlens"] = pool.seqlens
    return kw, pool.num_pages


def _py(call, fp8=False, **over):
    kw, n = _cache(fp8)
    if call == "shared":
        kw.update(q=torch.zeros(2, 4, 128, dtype=BF), r=torch.zeros(2, 4, 128, dtype=BF),
                  cu_g=torch.zeros(2, dtype=I32), prefix_lens=torch.zeros(1, dtype=I32))
    else:
        kw["page_refs"] = torch.zeros(n, dtype=I32)
    if call == "update":
        kw["lens"] = torch.zeros(2, dtype=I32)
    kw.update(over)
    return dict(shared=plx_decode_fwd_shared, update=plx_kv_update, compact=plx_kv_compact)[call](**kw)


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("fp8", [False, True])
def test_host_tensors_are_rejected(call, fp8):
    with pytest.raises(ValueError, match="CUDA"):
        _py(call, fp8)


@pytest.mark.parametrize("call,name", [("shared", "seqlens"), ("shared", "cu_g"), ("shared", "prefix_lens"),
                                       ("update", "seqlens"), ("update", "page_refs"), ("update", "lens"),
                                       ("compact", "seqlens"), ("compact", "page_refs")])
def test_missing_tensors_are_rejected(call, name):
    with pytest.raises(TypeError, match=name):
        _py(call, **{name: None})


def test_shapes_are_rejected():
    with pytest.raises(ValueError, match="q must be"):
        _py("shared", q=torch.zeros(3, 4, 128, dtype=BF))
    with pytest.raises(ValueError, match="r must be"):
        _py("shared", r=torch.zeros(2, 3, 128, dtype=BF))
    with pytest.raises(ValueError, match="cu_g"):
        _py("shared", cu_g=torch.zeros(3, dtype=I32))
    with pytest.raises(ValueError, match="prefix_lens"):
        _py("shared", prefix_lens=torch.zeros(1, 1, dtype=I32))
    for call in ("update", "compact"):
        with pytest.raises(ValueError, match="seqlens"):
            _py(call, seqlens=torch.zeros(3, dtype=I32))


def _rot(**kw):
    a = dict(q=torch.zeros(2, 4, 9, 128, dtype=BF), k=torch.zeros(2, 2, 9, 128, dtype=BF),
             inv_freq=torch.zeros(64, dtype=torch.float64))
    a.update(kw)
    return plx_rotary_fwd(**a)


@pytest.mark.parametrize("kw,error,word", [
    (dict(), ValueError, "CUDA"), (dict(q=None, k=None), ValueError, "all None"),
    (dict(q=torch.zeros(2, 4, 9, 128, dtype=torch.float16)), TypeError, "bfloat16"),
    (dict(q=torch.zeros(9, 128, dtype=BF)), ValueError, r"\[T, H, d\]"),
    (dict(k=torch.zeros(2, 2, 8, 128, dtype=BF)), ValueError, "k has shape"),
    (dict(r=torch.zeros(2, 3, 9, 128, dtype=BF)), ValueError, "r has shape"),
    (dict(q_out=torch.zeros(2, 4, 9, 64, dtype=BF)), ValueError, "q_out has shape"),
    (dict(k=torch.zeros(2, 0, 9, 128, dtype=BF)), ValueError, "no heads"),
])
def test_rotary_tensors_are_checked(kw, error, word):
    with pytest.raises(error, match=word):
        _rot(**kw)


def test_rotary_bwd_checks_its_tensors_too():
    with pytest.raises(ValueError, match="all None"):
        plx_rotary_bwd(None, None, torch.zeros(4, dtype=torch.float64))


def test_results_are_allocated_in_the_order_of_the_calls_stream():
    import inspect
    for fn in (binding.plx_decode_fwd_shared, binding.plx_kv_compact, binding._rotary):
        assert "torch.empty" not in inspect.getsource(fn) and "_empty(" in inspect.getsource(fn)


# ------------------------------------------------------------ the host reference
def test_reference_update_by_hand():
    # Two rows of 20 tokens in pages of 16; row 2 forks row 0 and grows, row 3 takes a cut of row 1.
    rows, lens, refs, copies = moves_ref.update([[5, 1], [2, 0], [], []], [20, 20, 0, 0], [1, 1, 1, 0, 0, 1, 0, 0],
                                                [20, 33, 34, 16], [0, 1, 0, 1], 16)
    # Row 0 keeps page 1, row 2 copies it into the lowest free page after row 1's growth took 3.
    assert rows == [[5, 1], [2, 0, 3], [5, 4, 6], [2]] and lens == [20, 33, 34, 16]
    assert refs == [1, 1, 2, 1, 1, 2, 1, 0] and copies == [(1, 4, 4)]


def test_reference_compact_by_hand():
    rows, refs, to, used = moves_ref.compact([[6, 1], [1, 4], [9]], [20, 32, 0], [0, 2, 0, 0, 1, 0, 1, 0], 16)
    assert used == 3 and to == [-1, 1, -1, -1, 0, -1, 2, -1]
    assert rows == [[2, 1], [1, 0], []] and refs == [1, 2, 1, 0, 0, 0, 0, 0]


def test_reference_update_keeps_counts():
    rng = random.Random(2)
    table, lens, refs = [[] for _ in range(6)], [0] * 6, [0] * 25
    for _ in range(200):
        src = [rng.randrange(-1, 6) for _ in range(6)]
        want = [rng.randint(0, 70) for _ in range(6)]
        table, lens, refs, copies = moves_ref.update(table, lens, refs, want, src, 16)
        use = [0] * 25
        for row, n in zip(table, lens):
            assert len(row) == moves_ref.pages_of(n, 16)
            for p in row:
                use[p] += 1
        assert use == refs
        assert all(use[row[n // 16]] == 1 for row, n in zip(table, lens) if n % 16)
        table, refs, _, used = moves_ref.compact(table, lens, refs, 16)
        assert all(n > 0 for n in refs[:used]) and not any(refs[used:])


@pytest.mark.parametrize("name,at_least", [("paged_moves.cu", 2), ("paged_decode.cu", 5), ("paged_prefill.cu", 6)])
def test_the_debug_build_checks_the_kernels(name, at_least):
    import os
    with open(os.path.join(build.CSRC, name)) as f:
        assert f.read().count("PLX_IN_BOUNDS(") >= at_least
