"""The paged KV cache's refusals, and the pins of its fp64 reference (CPU only:
nothing here launches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from parametrized_local_linear_gb300 import (binding, build, plx_decode_fwd_paged, plx_kv_append,
                                             plx_kv_read, plx_prefill_fwd_paged)

import paged_ref as ref

P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


# ------------------------------------------------------------ the reference
def test_reference_quantiser_agrees_with_torch_conversion():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(64, 128, generator=g) * torch.logspace(-3, 3, 64)[:, None]).to(torch.bfloat16)
    x[3] = 0
    x[5, 0] = 448.0
    codes, E = ref.quantise(x.double().numpy())
    scaled = torch.from_numpy(np.ldexp(x.double().numpy(), (127 - E.astype(int))[:, None]))
    want = scaled.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    back = ref.dequantise(codes, E)
    amax = np.abs(x.double().numpy()).max(1, keepdims=True)
    # Half a step of e4m3 (2^-4 relative), or half the subnormal step 2^-9 of
    # a row scaled so that its maximum is above 224.
    assert np.all(np.abs(back - x.double().numpy()) <=
                  np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, amax / 224 * 2.0 ** -10))
    assert E[3] == 1


@pytest.mark.parametrize("amax,E", [(448.0, 127), (449.0, 128), (224.0, 126), (225.0, 127), (1.75, 119),
                                    (1.7578125, 120), (0.0, 1), (2.0 ** -133, 1)])
def test_reference_scale_is_the_smallest(amax, E):
    x = np.zeros((1, 128))
    x[0, 7] = -amax
    assert ref.quantise(x)[1][0] == E


def test_reference_attention_equals_the_oracle():
    """The dense fp64 definition against the oracle that forms Sigma."""
    n, L, Hq, Hkv = 5, 40, 4, 2
    pool = ref.filled_pool([L], Hkv, 16, True, 3)
    q, r = ref.normal_rows(n, Hq, 8), ref.normal_rows(n, Hq, 9, 0.05)
    o, lse, _ = ref.reference(pool, q, r, [n])
    K, V = pool.get(0, L)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x.transpose(1, 0, 2)))[None]  # noqa: E731
    want, wl = oracle.prefill(q.double().transpose(0, 1)[None], t(K), t(V),
                              r.double().transpose(0, 1)[None])
    assert np.allclose(o, want[0].transpose(1, 0, 2), rtol=0, atol=1e-12)
    assert np.allclose(lse, wl[0].T, rtol=0, atol=1e-12)


# ------------------------------------------------------------ C refusals
def _append(lib, **kw):
    a = dict(k=P, v=P, ts=256, hs=128, kp=P, vp=P, ks=None, vs=None, table=P, sl=P, cu=P, T=4, B=2, Hkv=2,
             d=128, n=8, page=16, width=4)
    a.update(kw)
    return lib.plx_kv_append(*a.values(), None)


def _read(lib, **kw):
    a = dict(kp=P, vp=P, ks=None, vs=None, table=P, cu=P, k=P, v=P, T=4, B=2, Hkv=2, d=128, n=8, page=16,
             width=4)
    a.update(kw)
    return lib.plx_kv_read(*a.values(), None)


def _decode(lib, **kw):
    a = dict(q=P, r=P, kp=P, vp=P, ks=None, vs=None, table=P, sl=P, out=P, B=2, Hq=4, Hkv=2, d=128, n=8,
             page=16, width=4, ws=None, wsb=0)
    a.update(kw)
    return lib.plx_decode_fwd_paged(*a.values(), None)


def _prefill(lib, **kw):
    a = dict(q=P, r=P, ts=512, hs=128, kp=P, vp=P, ks=None, vs=None, table=P, sl=P, cu=P, out=P, ots=512,
             ohs=128, lse=None, T=4, B=2, Hq=4, Hkv=2, d=128, n=8, page=16, width=4, ws=None, wsb=0)
    a.update(kw)
    return lib.plx_prefill_fwd_paged(*a.values(), None)


CALLS = {"append": _append, "read": _read, "decode": _decode, "prefill": _prefill}
INV, UNS = binding.PLX_ERR_INVALID_ARG, binding.PLX_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("kw,status,word", [
    (dict(kp=None), INV, b"null"), (dict(vp=None), INV, b"null"), (dict(table=None), INV, b"null"),
    (dict(ks=P), INV, b"both"), (dict(vs=P), INV, b"both"), (dict(B=0), INV, b">= 1"),
    (dict(Hkv=0), INV, b">= 1"), (dict(n=0), INV, b">= 1"), (dict(width=0), INV, b">= 1"),
    (dict(d=64), UNS, b"head dim"), (dict(page=8), UNS, b"page_size"), (dict(page=48), UNS, b"page_size"),
    (dict(page=512), UNS, b"page_size"), (dict(page=0), UNS, b"page_size"),
    (dict(kp=ctypes.c_void_p(4104)), INV, b"aligned"), (dict(n=1 << 30, Hkv=4, Hq=4), UNS, b"2^31"),
    (dict(width=1 << 27), UNS, b"2^31"),
])
def test_cache_arguments_are_checked(lib, call, kw, status, word):
    if call in ("append", "read"):
        kw = {k: v for k, v in kw.items() if k != "Hq"}
    assert CALLS[call](lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(sl=None), INV, b"seqlens"), (dict(T=-1), INV, b"T"), (dict(cu=None, T=3), INV, b"cu_q"),
    (dict(k=None), INV, b"null"), (dict(v=ctypes.c_void_p(4098)), INV, b"aligned"),
    (dict(ts=0), INV, b"strides"), (dict(hs=64), INV, b"strides"), (dict(ts=260), INV, b"strides"),
    (dict(hs=1 << 39), INV, b"strides"), (dict(T=1 << 30, Hkv=2), UNS, b"too large"),
])
def test_append_arguments_are_checked(lib, kw, status, word):
    assert _append(lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(cu=None), INV, b"cu_k"), (dict(T=-1), INV, b"T"), (dict(k=None), INV, b"null"),
    (dict(v=ctypes.c_void_p(4098)), INV, b"aligned"), (dict(T=1 << 30), UNS, b"too large"),
])
def test_read_arguments_are_checked(lib, kw, status, word):
    assert _read(lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=None), INV, b"null"), (dict(out=None), INV, b"null"), (dict(sl=None), INV, b"null"),
    (dict(Hq=3), INV, b"multiple"), (dict(Hq=512, Hkv=2), UNS, b"at most 128"),
    (dict(r=ctypes.c_void_p(4104)), INV, b"aligned"), (dict(B=1 << 23), UNS, b"2^24"),
    (dict(ws=P, wsb=8), INV, b"workspace"), (dict(ws=ctypes.c_void_p(4104), wsb=1 << 40), INV, b"workspace"),
])
def test_decode_arguments_are_checked(lib, kw, status, word):
    assert _decode(lib, **kw) == status
    assert word in lib.plx_last_error_message()


@pytest.mark.parametrize("kw,status,word", [
    (dict(q=None), INV, b"null"), (dict(cu=None), INV, b"null"), (dict(sl=None), INV, b"null"),
    (dict(T=-1), INV, b"T"), (dict(Hq=3), INV, b"multiple"), (dict(Hq=512), UNS, b"at most 128"),
    (dict(ts=0), INV, b"strides"), (dict(ohs=0), INV, b"strides"), (dict(ots=136, ohs=136), INV, b"overlap"),
    (dict(out=ctypes.c_void_p(4104)), INV, b"aligned"), (dict(T=1 << 30), UNS, b"too large"),
    (dict(ws=P, wsb=8), INV, b"workspace"), (dict(ws=ctypes.c_void_p(4104), wsb=1 << 40), INV, b"workspace"),
])
def test_prefill_arguments_are_checked(lib, kw, status, word):
    assert _prefill(lib, **kw) == status
    assert word in lib.plx_last_error_message()


def test_no_rows_is_a_call_that_does_nothing(lib):
    assert _append(lib, T=0, k=None, v=None) == binding.PLX_OK
    assert _read(lib, T=0, k=None, v=None) == binding.PLX_OK
    assert _prefill(lib, T=0, q=None, r=None, out=None) == binding.PLX_OK


def test_workspace_sizes(lib):
    assert lib.plx_decode_paged_workspace_bytes(4, 16, 8, 128) > 0
    assert lib.plx_decode_paged_workspace_bytes(4, 12, 8, 128) == 0
    assert lib.plx_decode_paged_workspace_bytes(0, 16, 8, 128) == 0
    assert lib.plx_prefill_paged_workspace_bytes(100, 4, 16, 8, 128) > 0
    assert lib.plx_prefill_paged_workspace_bytes(-1, 4, 16, 8, 128) == 0
    assert lib.plx_prefill_paged_workspace_bytes(100, 4, 16, 7, 128) == 0


# ------------------------------------------------------------ binding refusals
def _args(fp8=False):
    pool = ref.Pool([20, 3], 2, 16, fp8, 1)
    kw = pool.to("cpu")
    kw["seqlens"] = pool.seqlens
    return kw


def _py(call, kw, **over):
    bf = torch.bfloat16
    kw = dict(kw)
    if call == "append":
        a = dict(k=torch.zeros(5, 2, 128, dtype=bf), v=torch.zeros(5, 2, 128, dtype=bf),
                 cu_q=torch.zeros(3, dtype=torch.int32), **kw)
        fn = plx_kv_append
    elif call == "read":
        kw.pop("seqlens")
        a = dict(cu_k=torch.zeros(3, dtype=torch.int32), T=5, **kw)
        fn = plx_kv_read
    elif call == "decode":
        a = dict(q=torch.zeros(2, 4, 128, dtype=bf), r=torch.zeros(2, 4, 128, dtype=bf), **kw)
        fn = plx_decode_fwd_paged
    else:
        a = dict(q=torch.zeros(5, 4, 128, dtype=bf), r=torch.zeros(5, 4, 128, dtype=bf),
                 cu_q=torch.zeros(3, dtype=torch.int32), **kw)
        fn = plx_prefill_fwd_paged
    a.update(over)
    return fn(**a)


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("fp8", [False, True])
def test_host_tensors_are_rejected(call, fp8):
    with pytest.raises(ValueError, match="CUDA"):
        _py(call, _args(fp8))


@pytest.mark.parametrize("call", sorted(CALLS))
def test_wrong_shapes_and_types_are_rejected(call):
    a = _args(True)
    with pytest.raises(ValueError, match="vpages"):
        _py(call, a, vpages=a["vpages"][:1])
    with pytest.raises(ValueError, match="vscale"):
        _py(call, a, vscale=None)
    with pytest.raises(ValueError, match="kscale"):
        _py(call, a, kscale=a["kscale"][:, :1])
    with pytest.raises(TypeError, match="kpages"):
        _py(call, a, kscale=None, vscale=None)  # codes without their scales
    if call != "decode":  # there the rows' own check comes first
        with pytest.raises(ValueError, match="block_table"):
            _py(call, a, block_table=a["block_table"][0])
    with pytest.raises(ValueError, match="kpages"):
        _py(call, a, kpages=a["kpages"][0])
    if call != "read":
        with pytest.raises(ValueError, match="seqlens"):
            _py(call, a, seqlens=a["seqlens"][:1])
    with pytest.raises(TypeError, match="kpages"):
        _py(call, _args(False), kpages=torch.zeros(4, 2, 16, 128), vpages=torch.zeros(4, 2, 16, 128))


def test_row_shapes_are_rejected():
    a, bf = _args(), torch.bfloat16
    with pytest.raises(ValueError, match="v has shape"):
        _py("append", a, v=torch.zeros(4, 2, 128, dtype=bf))
    with pytest.raises(ValueError, match="q must be"):
        _py("decode", a, q=torch.zeros(3, 4, 128, dtype=bf))
    with pytest.raises(ValueError, match="r must be"):
        _py("decode", a, out=torch.zeros(2, 4, 128, dtype=bf), r=torch.zeros(2, 3, 128, dtype=bf))
    with pytest.raises(ValueError, match="r has shape"):
        _py("prefill", a, r=torch.zeros(5, 3, 128, dtype=bf))
    with pytest.raises(ValueError, match="T must be"):
        _py("read", a, T=-1)


@pytest.mark.parametrize("call", sorted(CALLS))
def test_a_table_past_2_to_30_positions_is_rejected(lib, call):
    """Positions plus a tile stay inside 32 bits."""
    assert CALLS[call](lib, width=(1 << 26) + 1) == UNS  # 2^30 + 16 positions
    assert b"2^30" in lib.plx_last_error_message()


@pytest.mark.parametrize("call", sorted(CALLS))
def test_2_to_31_rows_of_pages_are_rejected(lib, call):
    """Rows of a page tensor are counted in 32 bits."""
    assert CALLS[call](lib, n=1 << 26) == UNS  # 2^26 pages x 2 heads x 16 slots
    assert b"2^31" in lib.plx_last_error_message()


@pytest.mark.parametrize("call,name", [("append", "seqlens"), ("decode", "seqlens"), ("prefill", "seqlens"),
                                       ("prefill", "cu_q"), ("read", "cu_k")])
def test_missing_lengths_and_offsets_are_rejected(call, name):
    with pytest.raises(TypeError, match=name):
        _py(call, _args(), **{name: None})


# ------------------------------------------------------------ memory of results
def test_results_are_allocated_in_the_order_of_the_calls_stream(monkeypatch):
    import inspect
    order = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            order.append(self.stream)

        def __exit__(self, *exc):
            order.append(None)

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: order.append("empty") or empty(*a, **kw))
    t = binding._empty((3, 2), torch.bfloat16, torch.device("cpu"), "another")
    assert order == ["another", "empty", None] and t.shape == (3, 2) and t.dtype is torch.bfloat16
    binding._empty((3, 2), torch.bfloat16, torch.device("cpu"), None)
    assert order[3:] == ["empty"]
    for fn in (binding.plx_decode_fwd_paged, binding.plx_prefill_fwd_paged, binding.plx_kv_read,
               binding._workspace):
        assert "torch.empty" not in inspect.getsource(fn)


# ------------------------------------------------------------ debug build
@pytest.mark.parametrize("name,at_least", [("paged_cache.cu", 2), ("paged_decode.cu", 4), ("paged_prefill.cu", 6)])
def test_the_debug_build_checks_the_paged_kernels(name, at_least):
    """The header promises a check before each TMA copy and each indexed store:
    page boxes, rows of pages and results, records, parts and their tables."""
    import os
    from parametrized_local_linear_gb300 import build
    with open(os.path.join(build.CSRC, name)) as f:
        assert f.read().count("PLX_IN_BOUNDS(") >= at_least
