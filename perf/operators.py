"""The paged-cache operators, as cases to measure: writing a KV cache (bf16 or
e4m3 with a scale per token and head), reading it back, decode and chunked
prefill over its pages.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the
framework's calls. ``exact`` evaluates the definitions in fp64.
"""
import math
import random

import torch

own = False

D = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A decode step's write: one new token for each of 64 sequences (latency).
        dict(name="append_one_token_each_e4m3", op="append", fp8=True, Hq=16, Hkv=8, page=16, B=64,
             q_lo=1, q_hi=1, k_lo=100, k_hi=8192, mix=1, heads_first=False),
        # The write of a batch of prompts, straight from the projection's layout.
        dict(name="append_prompts_e4m3", op="append", fp8=True, Hq=16, Hkv=8, page=64, B=16,
             q_lo=1, q_hi=4096, k_lo=4096, k_hi=8192, mix=2, heads_first=True),
        # The same without quantisation, a few long chunks.
        dict(name="append_chunks_bf16", op="append", fp8=False, Hq=16, Hkv=8, page=32, B=3,
             q_lo=1000, q_hi=9000, k_lo=9000, k_hi=20000, mix=3, heads_first=True),
        # Moving sequences out of the pool: a few short ones, and a large batch.
        dict(name="read_short_bf16", op="read", fp8=False, Hq=16, Hkv=8, page=16, B=5,
             q_lo=1, q_hi=1, k_lo=1, k_hi=700, mix=4, heads_first=False),
        dict(name="read_long_e4m3", op="read", fp8=True, Hq=16, Hkv=8, page=64, B=8,
             q_lo=1, q_hi=1, k_lo=4096, k_hi=32768, mix=5, heads_first=False),
        # One user's next token.
        dict(name="decode_one_bf16", op="decode", fp8=False, Hq=16, Hkv=8, page=16, B=1,
             q_lo=1, q_hi=1, k_lo=1777, k_hi=1777, mix=6, heads_first=False),
        # The batched decode workload (64 sequences of 8192 keys) on 8-bit pages.
        dict(name="decode_batch_e4m3", op="decode", fp8=True, Hq=16, Hkv=8, page=64, B=64,
             q_lo=1, q_hi=1, k_lo=8192, k_hi=8192, mix=7, heads_first=False),
        # The ragged long-context decode workload on bf16 pages.
        dict(name="decode_ragged_bf16", op="decode", fp8=False, Hq=16, Hkv=8, page=32, B=8,
             q_lo=1, q_hi=1, k_lo=16384, k_hi=131072, mix=8, heads_first=False),
        # Checking a few drafted tokens of each sequence.
        dict(name="prefill_drafts_e4m3", op="prefill", fp8=True, Hq=16, Hkv=8, page=16, B=16,
             q_lo=1, q_hi=5, k_lo=500, k_hi=6000, mix=9, heads_first=False),
        # A chunk of a long prompt.
        dict(name="prefill_long_chunk_bf16", op="prefill", fp8=False, Hq=16, Hkv=8, page=64, B=1,
             q_lo=2048, q_hi=2048, k_lo=32768, k_hi=32768, mix=10, heads_first=True),
        # Continuous batching: chunks of all lengths over contexts of all lengths.
        dict(name="prefill_mixed_e4m3", op="prefill", fp8=True, Hq=16, Hkv=8, page=32, B=12,
             q_lo=1, q_hi=700, k_lo=1000, k_hi=16000, mix=11, heads_first=False),
        # Whole prompts (the 0.6B-like prefill shape).
        dict(name="prefill_prompts_bf16", op="prefill", fp8=False, Hq=16, Hkv=8, page=128, B=4,
             q_lo=4096, q_hi=4096, k_lo=4096, k_hi=4096, mix=12, heads_first=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "read", "decode", "prefill"])
        Hq, Hkv = rng.choice([(16, 8), (16, 8), (8, 8), (4, 2), (8, 1), (12, 4), (16, 2), (16, 1)])
        B = _log_int(rng, 1, 64)
        k_hi = _log_int(rng, 1, 131072)
        k_lo = _log_int(rng, max(1, k_hi // 16), k_hi)
        q_hi = _log_int(rng, 1, 8192) if op in ("append", "prefill") else 1
        q_hi = min(q_hi, k_hi)
        case = dict(op=op, fp8=rng.random() < 0.5, Hq=Hq, Hkv=Hkv, page=rng.choice([16, 32, 64, 128, 256]),
                    B=B, q_lo=_log_int(rng, 1, q_hi), q_hi=q_hi, k_lo=k_lo, k_hi=k_hi,
                    mix=rng.randrange(1 << 20), heads_first=rng.random() < 0.5)
        qn, kn = lengths(case)
        cells = B * max(kn) * Hkv
        if sum(kn) * Hkv > 4_200_000 or cells > 8_400_000:
            continue
        if op == "prefill" and B * Hq * max(qn) * max(kn) > 1_070_000_000:
            continue
        if op in ("append", "read") and max(sum(qn), sum(kn) if op == "read" else 0) * Hkv > 1_000_000:
            continue
        return case


def lengths(case):
    """New tokens and keys (new ones included) of every sequence."""
    rng = random.Random(case["mix"])
    qn, kn = [], []
    for _ in range(case["B"]):
        k = rng.randint(case["k_lo"], case["k_hi"])
        kn.append(k)
        qn.append(min(k, rng.randint(case["q_lo"], case["q_hi"])))
    return qn, kn


# ---------------------------------------------------------------- inputs
def _quantise(x):
    """e4m3 codes and biased scale exponents of the rows (last axis) of x: the
    smallest exponent E >= 1 with max|x| <= 448 * 2^(E - 127)."""
    x = x.float()
    amax = x.abs().amax(-1)
    frac, ex = torch.frexp(amax)  # amax = frac * 2^ex, frac in [0.5, 1)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8) + 127
    e = torch.where(amax > 0, e, torch.ones_like(e)).clamp(1, 253)
    codes = (x * _power_of_two(254 - e).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, e.to(torch.uint8)


def _power_of_two(e):
    """2^(e - 127) in fp32, 1 <= e <= 254, from its bits."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    qn, kn = lengths(case)
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["page"]
    npages = [(k + P - 1) // P for k in kn]
    width, total = max(npages), sum(npages) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(npages):
        table[b, :n] = order[at:at + n]
        at += n
    ends = [0]
    for n in (qn if case["op"] != "read" else kn):
        ends.append(ends[-1] + n)
    T = ends[-1]
    s = dict(case=case, table=table, T=T, max_q=max(qn), max_k=max(kn),
             seqlens=torch.tensor(kn, dtype=torch.int32, device=dev),
             cu=torch.tensor(ends, dtype=torch.int32, device=dev))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    def rows(heads, scale):
        if case["heads_first"]:  # as the projection writes them
            return (normal(heads, T, D) * scale).transpose(0, 1)
        return normal(T, heads, D) * scale

    for name in ("k", "v"):
        pool = normal(total, Hkv, P, D)  # what earlier sequences left is in the pages too
        if case["fp8"]:
            s[name + "pages"], s[name + "scale"] = _quantise(pool)
        else:
            s[name + "pages"], s[name + "scale"] = pool, None
    if case["op"] == "append":
        s["k"], s["v"] = rows(Hkv, 1.0), rows(Hkv, 1.0)
    elif case["op"] == "decode":
        s["q"], s["r"] = normal(B, Hq, D), normal(B, Hq, D) * 0.05
    elif case["op"] == "prefill":
        s["q"], s["r"] = rows(Hq, 1.0), rows(Hq, 0.05)
    return s


# ---------------------------------------------------------------- plain forms
def _row_places(s, row_count):
    """Sequence and position of each of the packed rows."""
    rows = torch.arange(row_count, device=s["table"].device)
    seq = torch.searchsorted(s["cu"].long(), rows, right=True) - 1
    return seq, rows - s["cu"].long()[seq]


def _plain_append(s):
    P = s["case"]["page"]
    seq, i = _row_places(s, s["T"])
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = s["seqlens"].long()[seq] - n[seq] + i
    page, slot = s["table"].long()[seq, pos // P], pos % P
    for name in ("k", "v"):
        if s["case"]["fp8"]:
            codes, e = _quantise(s[name])
            s[name + "pages"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[name + "scale"][page, :, slot] = e
        else:
            s[name + "pages"][page, :, slot] = s[name]
    return [s["kpages"], s["vpages"]] + ([s["kscale"], s["vscale"]] if s["case"]["fp8"] else [])


def _fetch(s, name, page, slot):
    """fp32 cache rows at (page, slot): [..., Hkv, D]."""
    if s["case"]["fp8"]:
        codes = s[name + "pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
        return codes * _power_of_two(s[name + "scale"][page, :, slot]).unsqueeze(-1)
    return s[name + "pages"][page, :, slot].float()


def _plain_read(s):
    P = s["case"]["page"]
    seq, pos = _row_places(s, s["T"])
    page, slot = s["table"].long()[seq, pos // P], pos % P
    return [_fetch(s, "k", page, slot).to(torch.bfloat16), _fetch(s, "v", page, slot).to(torch.bfloat16)]


def _plain_attention(s, q, r, pos):
    """q, r fp32 [B, n, Hq, D]; query (b, i) sees the keys 0 .. pos[b, i]."""
    P, Hkv = s["case"]["page"], s["case"]["Hkv"]
    B, n, Hq, _ = q.shape
    G = Hq // Hkv
    key = torch.arange(s["max_k"], device=q.device)
    inside = key < s["seqlens"].long()[:, None]
    page = s["table"].long()[:, key // P]
    slot = (key % P).expand(B, -1)
    K = _fetch(s, "k", page, slot).permute(0, 2, 3, 1)  # [B, Hkv, D, keys]
    V = _fetch(s, "v", page, slot).permute(0, 2, 1, 3)  # [B, Hkv, keys, D]
    V = V.masked_fill(~inside[:, None, :, None], 0.0)

    def grouped(x):
        return x.reshape(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)

    hidden = (key > pos[:, :, None]).repeat_interleave(G, dim=1)[:, None]  # [B, 1, n G, keys]
    S = (grouped(q) @ K) / math.sqrt(D)
    S = S.masked_fill(hidden, -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    W = torch.exp(S - m)
    l = W.sum(-1, keepdim=True)
    W = W / torch.where(l > 0, l, torch.ones_like(l))
    O1 = W @ V
    W = W * (grouped(r) @ K).masked_fill(hidden, 0.0)
    O = O1 - W @ V + O1 * W.sum(-1, keepdim=True)

    def ungrouped(x):
        return x.reshape(B, Hkv, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, -1)

    return ungrouped(O), ungrouped(m + torch.log(l))[..., 0]


def _plain_decode(s):
    pos = s["seqlens"].long()[:, None] - 1
    out, _ = _plain_attention(s, s["q"].float()[:, None], s["r"].float()[:, None], pos)
    return [out[:, 0].to(torch.bfloat16)]


def _plain_prefill(s):
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["max_q"], device=n.device)
    row = (s["cu"].long()[:-1, None] + i).clamp(max=s["T"] - 1)
    pos = s["seqlens"].long()[:, None] - n[:, None] + i
    out, lse = _plain_attention(s, s["q"][row].float(), s["r"][row].float(), pos)
    seq, i = _row_places(s, s["T"])
    return [out[seq, i].to(torch.bfloat16), lse[seq, i]]


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        plain = {"append": _plain_append, "read": _plain_read, "decode": _plain_decode,
                 "prefill": _plain_prefill}
        return plain[op](s)
    import parametrized_local_linear_gb300 as plx
    scales = dict(kscale=s["kscale"], vscale=s["vscale"])
    if op == "append":
        plx.plx_kv_append(s["k"], s["v"], s["kpages"], s["vpages"], s["table"], s["seqlens"],
                          cu_q=s["cu"], **scales)
        return [s["kpages"], s["vpages"]] + ([s["kscale"], s["vscale"]] if s["case"]["fp8"] else [])
    if op == "read":
        return list(plx.plx_kv_read(s["kpages"], s["vpages"], s["table"], s["cu"], s["T"], **scales))
    if op == "decode":
        return [plx.plx_decode_fwd_paged(s["q"], s["r"], s["kpages"], s["vpages"], s["table"],
                                         s["seqlens"], **scales)]
    lse = torch.empty(s["T"], s["case"]["Hq"], dtype=torch.float32, device=s["q"].device)
    return list(plx.plx_prefill_fwd_paged(s["q"], s["r"], s["kpages"], s["vpages"], s["table"],
                                          s["seqlens"], s["cu"], lse=lse, **scales))


def work(case):
    qn, kn = lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    row = 2 * ((D + 1) if case["fp8"] else 2 * D)  # one token's K and V of one kv head in the cache
    table = 4 * sum((k + case["page"] - 1) // case["page"] for k in kn)
    meta = table + 8 * case["B"]
    T, keys = sum(qn), sum(kn)
    if case["op"] == "append":
        return dict(bytes=T * Hkv * (4 * D + row) + meta, flops=0)
    if case["op"] == "read":
        return dict(bytes=keys * Hkv * (4 * D + row) + meta, flops=0)
    pairs = sum(sum(range(k - q + 1, k + 1)) for q, k in zip(qn, kn))
    side = T * Hq * D * 2 * 3 + (4 * T * Hq if case["op"] == "prefill" else 0)
    return dict(bytes=keys * Hkv * row + side + meta, flops=8 * D * Hq * pairs)


# ---------------------------------------------------------------- fp64
def exact(case, seed):
    s = prepare(case, seed)
    qn, kn = lengths(case)
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["page"]
    G = Hq // Hkv
    if case["op"] == "append":
        return _exact_append(s, qn, kn)
    table = s["table"].tolist()

    def sequence(name, b, h, n):
        """fp64 [n, D]: the first n tokens of kv head h of sequence b."""
        ids = torch.tensor(table[b][:(n + P - 1) // P], device=s["table"].device, dtype=torch.long)
        pages = s[name + "pages"]
        if case["fp8"]:
            x = pages.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(s[name + "scale"][ids, h].double() - 127.0)[..., None]
        else:
            x = pages[ids, h].double()
        return x.reshape(-1, D)[:n]

    if case["op"] == "read":
        outs = []
        for name in ("k", "v"):
            out = torch.empty(s["T"], Hkv, D, dtype=torch.float64, device=s["table"].device)
            at = 0
            for b, n in enumerate(kn):
                for h in range(Hkv):
                    out[at:at + n, h] = sequence(name, b, h, n)
                at += n
            outs.append(out)
        return outs

    def attend(q, r, K, V, pos):
        """The definition: softmax weights, then the centred cross-covariance
        applied to the probe. Rows q, r [m, D]; row i sees keys 0 .. pos[i]."""
        z = q.double() @ K.T / math.sqrt(D)
        z.masked_fill_(torch.arange(K.shape[0], device=z.device) > pos[:, None], -math.inf)
        lse = torch.logsumexp(z, 1)
        w = torch.exp(z - lse[:, None])
        mean_v, mean_k = w @ V, w @ K
        r = r.double()
        w = w * (r @ K.T - (r * mean_k).sum(1, keepdim=True))  # w_j (k_j - mu) . rho
        return mean_v - (w @ V - w.sum(1, keepdim=True) * mean_v), lse

    dev = s["q"].device
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=dev)
    step = max(1, 24_000_000 // max(kn))
    at = 0
    for b, (n, k) in enumerate(zip(qn, kn)):
        for h in range(Hkv):
            K, V = sequence("k", b, h, k), sequence("v", b, h, k)
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                pos = torch.arange(k - n + i0, k - n + i1, device=dev)
                for hq in range(h * G, (h + 1) * G):
                    rows = slice(at + i0, at + i1)
                    out[rows, hq], lse[rows, hq] = attend(s["q"][rows, hq], s["r"][rows, hq], K, V, pos)
        at += n
    return [out] if case["op"] == "decode" else [out, lse]


def _exact_append(s, qn, kn):
    """The pages after the write; the codes and exponents by searching the
    definition: e4m3 neighbours in fp64, ties to the even code."""
    P, fp8 = s["case"]["page"], s["case"]["fp8"]
    dev = s["table"].device
    code_values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().to(dev)
    middles = (code_values[1:] + code_values[:-1]) / 2
    outs, scales = [], []
    for name in ("k", "v"):
        pages = s[name + "pages"].double()
        exps = s[name + "scale"].clone() if fp8 else None
        at = 0
        for b, (n, k) in enumerate(zip(qn, kn)):
            pos = torch.arange(k - n, k, device=dev)
            page, slot = s["table"][b].long()[pos // P], pos % P
            x = s[name][at:at + n].double()
            if fp8:
                amax = x.abs().amax(-1)
                e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -140) / E4M3_MAX) - 1e-12) + 127
                e = e.clamp(1, 253)
                y = x * torch.exp2(127 - e)[..., None]
                a = y.abs()
                lo = torch.searchsorted(middles, a.contiguous())  # middles[lo - 1] < a <= middles[lo]
                tie = (lo < 126) & (a == middles[lo.clamp(max=125)]) & (lo % 2 == 1)
                x = torch.copysign(code_values[lo + tie], y)
                exps[page, :, slot] = e.to(torch.uint8)
            pages[page, :, slot] = x
            at += n
        outs.append(pages)
        scales.append(exps)
    return outs + (scales if fp8 else [])
