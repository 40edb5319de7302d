"""Positions, forked sequences and shared prefixes, as cases to measure: rotary
positions (forward and backward), the bookkeeping of a paged KV cache between two
steps of a server (fork, reorder, grow, trim, free), its compaction, and decode
for sequences that share a prefix.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the
framework's calls. ``exact`` evaluates the definitions in fp64.
"""
import math
import random

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A decode step: one new token for each of 64 sequences (latency).
        dict(name="rotary_decode_step", op="rotary", dtype="bf16", back=False, where="lengths", B=64, L=1,
             Hq=16, Hkv=8, d=128, rd=128, interleaved=False, probe=True, scaling="none", far=8192, mix=1),
        # The 0.6B-like training forward, in the projection's layout.
        dict(name="rotary_training_fwd", op="rotary", dtype="bf16", back=False, where="order", B=4, L=4096,
             Hq=16, Hkv=8, d=128, rd=128, interleaved=False, probe=True, scaling="none", far=4096, mix=2),
        # Gradients of packed documents; half of the head rotates, in neighbouring pairs.
        dict(name="rotary_partial_bwd", op="rotary", dtype="bf16", back=True, where="given", B=1, L=5531,
             Hq=16, Hkv=8, d=128, rd=64, interleaved=True, probe=False, scaling="none", far=5531, mix=3),
        # The fp32 path at far positions of a scaled context.
        dict(name="rotary_long_fp32", op="rotary", dtype="fp32", back=False, where="given", B=2, L=2049,
             Hq=4, Hkv=2, d=64, rd=64, interleaved=False, probe=True, scaling="parts", far=1000000, mix=4),
        # A decode step's pages: every sequence grows by a token, a few end.
        dict(name="update_step_e4m3", op="update", fork=False, fp8=True, Hq=16, Hkv=8, page=16, groups=64,
             each=1, p_lo=64, p_hi=4096, s_lo=1, s_hi=2000, spare=300, mix=5),
        # A step of eight beams for each of eight prompts: rows take over others' pages.
        dict(name="update_beams_bf16", op="update", fork=True, fp8=False, Hq=16, Hkv=8, page=64, groups=8,
             each=8, p_lo=2048, p_hi=8192, s_lo=1, s_hi=500, spare=200, mix=6),
        # A small pool with holes (latency), and one that large batches have left.
        dict(name="compact_small_e4m3", op="compact", fp8=True, Hq=16, Hkv=8, page=16, groups=8, each=2,
             p_lo=16, p_hi=500, s_lo=1, s_hi=200, spare=150, mix=7),
        dict(name="compact_large_bf16", op="compact", fp8=False, Hq=16, Hkv=8, page=64, groups=32, each=2,
             p_lo=512, p_hi=4096, s_lo=512, s_hi=4096, spare=3500, mix=8),
        # Four continuations of a short prompt (latency).
        dict(name="shared_four_bf16", op="shared", fp8=False, Hq=16, Hkv=8, page=16, groups=1, each=4,
             p_lo=1777, p_hi=1777, s_lo=1, s_hi=100, spare=3, mix=9),
        # Many continuations of one long prompt.
        dict(name="shared_samples_bf16", op="shared", fp8=False, Hq=16, Hkv=8, page=64, groups=1, each=64,
             p_lo=32768, p_hi=32768, s_lo=1, s_hi=1024, spare=3, mix=10),
        # A batch of users behind a few common instructions, on 8-bit pages.
        dict(name="shared_instructions_e4m3", op="shared", fp8=True, Hq=16, Hkv=8, page=64, groups=5, each=20,
             p_lo=2000, p_hi=8000, s_lo=50, s_hi=4000, spare=3, mix=11),
        # A large group with few kv heads over the longest prefix.
        dict(name="shared_wide_bf16", op="shared", fp8=False, Hq=16, Hkv=2, page=128, groups=1, each=100,
             p_lo=100000, p_hi=100000, s_lo=1, s_hi=500, spare=3, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    while True:
        op = rng.choice(["rotary", "update", "compact", "shared", "shared"])
        Hq, Hkv = rng.choice([(16, 8), (16, 8), (8, 8), (4, 2), (8, 1), (12, 4), (16, 2), (16, 1)])
        mix = rng.randrange(1 << 20)
        if op == "rotary":
            where = rng.choice(["order", "given", "lengths"])
            L = _log_int(rng, 1, 16384)
            B = _log_int(rng, 1, 64)
            dtype = rng.choice(["bf16", "bf16", "fp32"])
            d = rng.choice([128, 128, 64])
            if B * L * (2 * Hq + Hkv) * d * (2 if dtype == "bf16" else 4) > 4 * 4096 * 40 * 256:
                continue
            return dict(op=op, dtype=dtype, back=rng.random() < 0.4, where=where, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d,
                        rd=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                        interleaved=rng.random() < 0.5, probe=rng.random() < 0.6,
                        scaling=rng.choice(["none", "none", "linear", "parts"]),
                        far=max(L, _log_int(rng, 64, 1 << 20)), mix=mix)
        case = dict(op=op, fp8=rng.random() < 0.5, Hq=Hq, Hkv=Hkv, page=rng.choice([16, 32, 64, 128, 256]),
                    groups=_log_int(rng, 1, 64), each=_log_int(rng, 1, 100))
        case["p_hi"] = _log_int(rng, 1, 100000)
        case["p_lo"] = _log_int(rng, max(1, case["p_hi"] // 8), case["p_hi"])
        case["s_hi"] = _log_int(rng, 1, 4096)
        case["s_lo"] = _log_int(rng, 1, case["s_hi"])
        case["spare"] = 3 if op == "shared" else _log_int(rng, 3, 2000)
        case["mix"] = mix
        if op == "update":
            case["fork"] = rng.random() < 0.6
        sizes, prefix, suffix = lengths(case)
        own_keys = sum(suffix) + len(suffix) * case["page"]
        held = (sum(prefix) + own_keys) * Hkv + case["spare"] * case["page"] * Hkv
        pairs = sum(n * p for n, p in zip(sizes, prefix)) + sum(suffix)
        widest = max(p for p in prefix) + max(suffix)
        if case["groups"] * case["each"] > 256 or held > 3_000_000:
            continue
        if op == "shared" and (Hq * pairs > 160_000_000 or len(suffix) * max(suffix) * Hkv > 1_000_000
                               or case["groups"] * max(prefix) * (Hkv + Hq * max(sizes) / 16) > 20_000_000):
            continue
        if op != "shared" and len(suffix) * widest / case["page"] > 200_000:
            continue
        return case


def lengths(case):
    """Sequences of every group, its prefix's tokens, and each sequence's own behind it."""
    rng = random.Random(case["mix"])
    sizes = [rng.randint((case["each"] + 1) // 2, case["each"]) if case["groups"] > 1 else case["each"]
             for _ in range(case["groups"])]
    prefix = [rng.randint(case["p_lo"], case["p_hi"]) for _ in sizes]
    suffix = [rng.randint(case["s_lo"], case["s_hi"]) for _ in range(sum(sizes))]
    return sizes, prefix, suffix


def next_step(case, sizes, lens):
    """The rows that a step's sequences come from (None: their own) and their new lengths."""
    rng = random.Random(case["mix"] + 1)
    B = len(lens)
    if case["fork"]:
        src, at = [], 0
        for n in sizes:
            src += [at + rng.randrange(n) for _ in range(n)]
            at += n
        return src, [lens[s] + 1 for s in src]
    ended = [b for b in range(B) if rng.random() < 0.05]
    return None, [0 if b in ended else lens[b] + 1 for b in range(B)]


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


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(case):
    """Radians a position of each pair (fp64), and the factor of cos and sin."""
    base, factor, original = 10000.0, 8.0, 4096.0
    half = case["rd"] // 2
    f = base ** (-torch.arange(half, dtype=torch.float64) / half)
    scale = 1.0
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "parts":  # by the turns that a pair makes over the original length
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    return f.cuda(), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_rotary(case, g) if case["op"] == "rotary" else _prepare_cache(case, g)


def _prepare_rotary(case, g):
    B, L = case["B"], case["L"]
    rng = random.Random(case["mix"])
    f, scale = _frequencies(case)
    s = dict(case=case, inv_freq=f, scale=scale, positions=None, seqlens=None, cu=None)

    def rows(heads, std):
        shape = (B, heads, L, case["d"]) if case["where"] == "order" else (B * L, heads, case["d"])
        return (torch.randn(shape, generator=g, device="cuda") * std).to(DTYPES[case["dtype"]])

    s["q"], s["k"] = rows(case["Hq"], 1.0), rows(case["Hkv"], 1.0)
    s["r"] = rows(case["Hq"], 0.05) if case["probe"] else None
    if case["where"] == "given":  # documents one after the other, from any position
        starts = [rng.randint(0, max(0, case["far"] - L)) for _ in range(B)]
        s["positions"] = torch.cat([torch.arange(a, a + L, dtype=torch.int32) for a in starts]).cuda()
    elif case["where"] == "lengths":
        s["seqlens"] = _ints([rng.randint(L, case["far"]) for _ in range(B)])
        s["cu"] = _ints([b * L for b in range(B + 1)])
    return s


def _prepare_cache(case, g):
    """A pool in which every group's sequences share the full pages of its prefix;
    the first tokens of their own pages repeat the rest of it."""
    P, Hkv = case["page"], case["Hkv"]
    sizes, prefix, suffix = lengths(case)
    lens, B = [], sum(sizes)
    for n, p in zip(sizes, prefix):
        lens += [p + t for t in suffix[len(lens):len(lens) + n]]
    src, new_lens = next_step(case, sizes, lens) if case["op"] == "update" else (None, lens)
    width = max(-(-n // P) for n in lens + new_lens)
    shared = [p // P for p in prefix]
    used = sum(shared) + sum(-(-n // P) for n in lens) - sum(n * h for n, h in zip(sizes, shared))
    total = used + case["spare"]
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    refs = torch.zeros(total, dtype=torch.int32, device="cuda")
    pages, scales = {}, {}
    for name in ("k", "v"):
        x = torch.randn(total, Hkv, P, D, generator=g, device="cuda").to(torch.bfloat16)
        pages[name], scales[name] = _quantise(x) if case["fp8"] else (x, None)
    at = b = 0
    for n, p, h in zip(sizes, prefix, shared):
        table[b:b + n, :h] = order[at:at + h]
        refs[order[at:at + h].long()] = n
        at += h
        for i in range(b, b + n):
            m = -(-lens[i] // P) - h
            table[i, h:h + m] = order[at:at + m]
            at += m
        if p % P:  # the rest of the prefix, in each sequence's own page
            first, rest = table[b, h].long(), table[b + 1:b + n, h].long()
            for x in [pages["k"], pages["v"]] + ([scales["k"], scales["v"]] if case["fp8"] else []):
                x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
                x[rest, :, :p % P] = x[first, :, :p % P]
        b += n
    mine = torch.arange(width, device="cuda") >= torch.tensor(shared, device="cuda").repeat_interleave(
        torch.tensor(sizes, device="cuda"))[:, None]
    mine &= torch.arange(width, device="cuda") < (_ints(lens)[:, None] + P - 1) // P
    refs[table[mine].long()] = 1
    s = dict(case=case, table=table, refs=refs, seqlens=_ints(lens), max_own=max(suffix), max_prefix=max(prefix),
             kpages=pages["k"], vpages=pages["v"], kscale=scales["k"], vscale=scales["v"])
    if case["op"] == "shared":
        ends = [0]
        for n in sizes:
            ends.append(ends[-1] + n)
        s["cu"], s["prefix"], s["most"] = _ints(ends), _ints(prefix), max(sizes)
        s["q"] = torch.randn(B, case["Hq"], D, generator=g, device="cuda").to(torch.bfloat16)
        s["r"] = (torch.randn(B, case["Hq"], D, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    else:  # the second set of tables of a program that switches between two
        s["table_out"], s["refs_out"] = torch.zeros_like(table), torch.zeros_like(refs)
        s["seqlens_out"] = torch.zeros_like(s["seqlens"])
        s["lens"], s["src"] = _ints(new_lens), None if src is None else _ints(src)
        s["map"], s["used"] = torch.zeros_like(refs), _ints([0])
    return s


# ---------------------------------------------------------------- plain forms
def _plain_rotary(s):
    case = s["case"]
    rd, pairs_apart = case["rd"], not case["interleaved"]
    if case["where"] == "order":
        pos = torch.arange(case["L"], device="cuda")
    elif case["where"] == "given":
        pos = s["positions"]
    else:
        n = s["cu"][1:] - s["cu"][:-1]
        pos = (s["seqlens"] - n)[:, None] + torch.arange(case["L"], device="cuda")
        pos = pos.reshape(-1)
    angle = pos.double()[:, None] * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    if case["where"] != "order":
        cos, sin = cos[:, None], sin[:, None]  # one for all heads of a row
    if case["back"]:
        sin = -sin

    def turn(x):
        if x is None:
            return None
        y = x.float()
        a, b = (y[..., :rd // 2], y[..., rd // 2:rd]) if pairs_apart else (y[..., 0:rd:2], y[..., 1:rd:2])
        u, v = a * cos - b * sin, b * cos + a * sin
        both = torch.cat([u, v], -1) if pairs_apart else torch.stack([u, v], -1).flatten(-2)
        return torch.cat([both, y[..., rd:]], -1).to(x.dtype)

    return [y for y in (turn(s["q"]), turn(s["k"]), turn(s["r"])) if y is not None]


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _pools(s):
    return [s["kpages"], s["vpages"]] + ([s["kscale"], s["vscale"]] if s["case"]["fp8"] else [])


def _count(pages, where, total):
    """How many of the table entries `where` name each page."""
    at = torch.where(where, pages, total).flatten()
    return torch.zeros(total + 1, dtype=torch.int64, device="cuda").scatter_add_(0, at, torch.ones_like(at))[:total]


def _plain_update(s):
    P, total = s["case"]["page"], s["refs"].numel()
    B, width = s["table"].shape
    old, lens, row = s["seqlens"].long(), s["lens"].long(), torch.arange(B, device="cuda")
    src = row if s["src"] is None else s["src"].long()
    col = torch.arange(width, device="cuda")
    table = s["table"].long()
    pages = table[src]
    kept = torch.minimum(lens, old[src])
    full, part = kept // P, kept % P
    refs = (s["refs"].long() - _count(table, col < ((old + P - 1) // P)[:, None], total)
            + _count(pages, col < full[:, None], total))
    # A partial last page stays with the first row that has it, if no other row has all of it.
    last = torch.where(part > 0, pages.gather(1, full.clamp(max=width - 1)[:, None])[:, 0], total)
    first = torch.full((total + 1,), B, device="cuda").scatter_reduce_(0, last, row, "amin")
    alone = torch.cat([refs == 0, torch.zeros(1, dtype=torch.bool, device="cuda")])
    stays = alone[last] & (first[last] == row)
    copies = (part > 0) & ~stays
    refs = refs + _count(last[:, None], stays[:, None], total)
    # The rows take the lowest free pages in their order, while all that a row needs is there.
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    keep = full + stays.long()
    need = (lens + P - 1) // P - keep
    ends = need.cumsum(0)
    fits = (need == 0) | (ends <= (refs == 0).sum())
    new = torch.where(fits, lens, torch.where(copies, full * P, kept))
    fresh = free[((ends - need)[:, None] + col - keep[:, None]).clamp(0, total - 1)]
    inside = col < ((new + P - 1) // P)[:, None]
    mixed = torch.where(col < keep[:, None], pages, fresh)
    s["table_out"].copy_(torch.where(inside, mixed, s["table_out"].long()))
    s["seqlens_out"].copy_(new)
    s["refs_out"].copy_(refs + _count(fresh, inside & (col >= keep[:, None]), total))
    moved = (copies & fits).nonzero()[:, 0]
    to, back = mixed[moved, full[moved]], last[moved]
    slot = torch.arange(P, device="cuda") < part[moved, None]
    k, v = _bits(s["kpages"]), _bits(s["vpages"])
    cut = slot[:, None, :, None]
    k[to] = torch.where(cut, k[back], k[to])
    v[to] = torch.where(cut, v[back], v[to])
    if s["case"]["fp8"]:
        cut = slot[:, None, :]
        s["kscale"][to] = torch.where(cut, s["kscale"][back], s["kscale"][to])
        s["vscale"][to] = torch.where(cut, s["vscale"][back], s["vscale"][to])
    return [s["table_out"], s["seqlens_out"], s["refs_out"]] + _pools(s)


def _plain_compact(s):
    P, total = s["case"]["page"], s["refs"].numel()
    page = torch.arange(total, device="cuda")
    used = s["refs"] > 0
    count = used.sum()
    back, to = (used & (page >= count)).nonzero()[:, 0], (~used & (page < count)).nonzero()[:, 0]
    moved = torch.where(used, page, -1)
    moved[back] = to
    inside = torch.arange(s["table"].shape[1], device="cuda") < ((s["seqlens"] + P - 1) // P)[:, None]
    s["table_out"].copy_(torch.where(inside, moved[s["table"].long()], s["table_out"].long()))
    refs = s["refs"].clone()
    refs[to], refs[back] = refs[back], 0
    s["refs_out"].copy_(refs)
    k, v = _bits(s["kpages"]), _bits(s["vpages"])
    k[to], v[to] = k[back], v[back]
    if s["case"]["fp8"]:
        s["kscale"][to], s["vscale"][to] = s["kscale"][back], s["vscale"][back]
    s["map"].copy_(moved)
    s["used"].copy_(count)
    return [s["table_out"], s["refs_out"], s["map"], s["used"]] + _pools(s)


def _fetch(s, name, page, slot):
    """fp32 cache rows at (page, slot): [..., Hkv, D]."""
    if s["case"]["fp8"]:
        codes = s[name + "pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
        return codes * _power_of_two(s[name + "scale"][page, :, slot]).unsqueeze(-1)
    return s[name + "pages"][page, :, slot].float()


def _plain_shared(s):
    """Scores against the prefix, once for a group, and against each sequence's own keys; one softmax over both."""
    case = s["case"]
    P, Hkv, G, n = case["page"], case["Hkv"], case["Hq"] // case["Hkv"], s["most"]
    B, table = s["table"].shape[0], s["table"].long()
    cu, prefix, lens = s["cu"].long(), s["prefix"].long(), s["seqlens"].long()
    groups = prefix.numel()
    group = torch.searchsorted(cu, torch.arange(B, device="cuda"), right=True) - 1
    place = group * n + torch.arange(B, device="cuda") - cu[group]  # in the groups padded to n sequences
    key = torch.arange(s["max_prefix"], device="cuda")
    page, slot = table[cu[:-1]][:, key // P], (key % P).expand(groups, -1)
    Kp, Vp = (_fetch(s, x, page, slot).transpose(1, 2) for x in "kv")  # [groups, Hkv, keys, D]
    pos = prefix[group][:, None] + torch.arange(s["max_own"], device="cuda")
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1))
    Ko, Vo = (_fetch(s, x, page, pos % P).transpose(1, 2) for x in "kv")  # [B, Hkv, keys, D]

    def padded(x):  # [B, Hkv, G, X] -> [groups, Hkv, n G, X]
        y = torch.zeros(groups * n, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[place] = x
        return y.reshape(groups, n, Hkv, G, -1).transpose(1, 2).reshape(groups, Hkv, n * G, -1)

    def single(y):
        return y.reshape(groups, Hkv, n, G, -1).transpose(1, 2).reshape(groups * n, Hkv, G, -1)[place]

    q, r = s["q"].float().reshape(B, Hkv, G, D), s["r"].float().reshape(B, Hkv, G, D)
    qp, rp = padded(q), padded(r)
    hidden_p = (key >= prefix[group][:, None])[:, None, None]
    hidden_o = (pos >= lens[:, None])[:, None, None]
    Sp = (single(qp @ Kp.transpose(2, 3)) / math.sqrt(D)).masked_fill(hidden_p, -math.inf)
    So = (q @ Ko.transpose(2, 3) / math.sqrt(D)).masked_fill(hidden_o, -math.inf)
    m = torch.maximum(Sp.amax(-1, keepdim=True), So.amax(-1, keepdim=True))
    Wp, Wo = torch.exp(Sp - m), torch.exp(So - m)
    l = Wp.sum(-1, keepdim=True) + Wo.sum(-1, keepdim=True)
    Wp, Wo = Wp / l, Wo / l
    O1 = single(padded(Wp) @ Vp) + Wo @ Vo
    Wp, Wo = Wp * single(rp @ Kp.transpose(2, 3)), Wo * (r @ Ko.transpose(2, 3))
    O2 = single(padded(Wp) @ Vp) + Wo @ Vo
    sigma = Wp.sum(-1, keepdim=True) + Wo.sum(-1, keepdim=True)
    return [(O1 - O2 + O1 * sigma).reshape(B, case["Hq"], D).to(torch.bfloat16)]


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        plain = {"rotary": _plain_rotary, "update": _plain_update, "compact": _plain_compact,
                 "shared": _plain_shared}
        return plain[op](s)
    import parametrized_local_linear_gb300 as plx
    if op == "rotary":
        turn = plx.plx_rotary_bwd if s["case"]["back"] else plx.plx_rotary_fwd
        outs = turn(s["q"], s["k"], s["inv_freq"], s["r"], positions=s["positions"], seqlens=s["seqlens"],
                    cu_q=s["cu"], interleaved=s["case"]["interleaved"], scale=s["scale"])
        return [y for y in outs if y is not None]
    scales = dict(kscale=s["kscale"], vscale=s["vscale"])
    if op == "update":
        outs = plx.plx_kv_update(s["kpages"], s["vpages"], s["table"], s["seqlens"], s["refs"], s["lens"],
                                 src=s["src"], block_table_out=s["table_out"], seqlens_out=s["seqlens_out"],
                                 page_refs_out=s["refs_out"], **scales)
        return list(outs) + _pools(s)
    if op == "compact":
        outs = plx.plx_kv_compact(s["kpages"], s["vpages"], s["table"], s["seqlens"], s["refs"],
                                  block_table_out=s["table_out"], page_refs_out=s["refs_out"],
                                  page_map=s["map"], used=s["used"], **scales)
        return list(outs) + _pools(s)
    return [plx.plx_decode_fwd_shared(s["q"], s["r"], s["kpages"], s["vpages"], s["table"], s["seqlens"],
                                      s["cu"], s["prefix"], **scales)]


def work(case):
    if case["op"] == "rotary":
        rows = case["B"] * case["L"]
        heads = case["Hq"] * (2 if case["probe"] else 1) + case["Hkv"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=2 * rows * heads * case["d"] * size + 4 * case["rd"], flops=3 * rows * heads * case["rd"])
    P, Hq, Hkv = case["page"], case["Hq"], case["Hkv"]
    sizes, prefix, suffix = lengths(case)
    row = Hkv * 2 * ((D + 1) if case["fp8"] else 2 * D)  # one token's K and V
    lens = []
    for n, p in zip(sizes, prefix):
        lens += [p + t for t in suffix[len(lens):len(lens) + n]]
    shared = [p // P for p in prefix]
    entries = sum(-(-n // P) for n in lens)
    used = sum(shared) + entries - sum(n * h for n, h in zip(sizes, shared))
    total = used + case["spare"]
    if case["op"] == "update":
        src, new = next_step(case, sizes, lens)
        tails = 0  # tokens of the copied last pages: all but one of a page's rows copy it
        for s in set(src or []):
            tails += (src.count(s) - 1) * (lens[s] % P)
        after = sum(-(-n // P) for n in new)
        return dict(bytes=2 * tails * row + 4 * (entries + after + 2 * total + 4 * len(lens)), flops=0)
    if case["op"] == "compact":  # the expected share of the used pages that lie behind the first `used`
        moved = used * (total - used) // total
        return dict(bytes=2 * moved * P * row + 4 * (2 * entries + 3 * total + len(lens)), flops=0)
    keys = sum(prefix) + sum(suffix)
    pairs = sum(n * p for n, p in zip(sizes, prefix)) + sum(suffix)
    side = len(lens) * (Hq * D * 2 * 3 + 4) + 8 * len(sizes) + 4 * entries
    return dict(bytes=keys * row + side, flops=8 * D * Hq * pairs)


# ---------------------------------------------------------------- fp64
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    if case["op"] == "shared":
        return _exact_shared(s)
    return _exact_update(s) if case["op"] == "update" else _exact_compact(s)


def _exact_rotary(s):
    """Every pair as a complex number, times scale e^(i angle)."""
    case = s["case"]
    if case["where"] == "order":
        pos = list(range(case["L"])) * case["B"]
    elif case["where"] == "given":
        pos = s["positions"].tolist()
    else:
        pos = [n - case["L"] + i for n in s["seqlens"].tolist() for i in range(case["L"])]
    angle = torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None] * s["inv_freq"]
    z = torch.polar(torch.full_like(angle, s["scale"]), -angle if case["back"] else angle)
    outs = []
    for x in (s["q"], s["k"], s["r"]):
        if x is None:
            continue
        y = x.double()
        if y.dim() == 4:
            y = y.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])
        i = torch.arange(case["rd"] // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rd"] // 2)
        w = torch.complex(y[..., a], y[..., b]) * z[:, None]
        y = y.clone()
        y[..., a], y[..., b] = w.real, w.imag
        if x.dim() == 4:
            y = y.reshape(x.shape[0], x.shape[2], x.shape[1], x.shape[3]).transpose(1, 2).contiguous()
        outs.append(y)
    return outs


def _exact_update(s):
    """Row by row, on the host."""
    P = s["case"]["page"]
    table, old, lens = s["table"].tolist(), s["seqlens"].tolist(), s["lens"].tolist()
    src = list(range(len(old))) if s["src"] is None else s["src"].tolist()
    refs = s["refs"].tolist()
    for b, n in enumerate(old):
        for p in table[b][:-(-n // P)]:
            refs[p] -= 1
    rows, tails = [], []
    for b, a in enumerate(src):
        kept = min(lens[b], old[a])
        rows.append(table[a][:kept // P])
        tails.append((table[a][kept // P], kept % P) if kept % P else None)
        for p in rows[b]:
            refs[p] += 1
    whole = {p for row in rows for p in row}
    copies, given = [], set()
    for b, tail in enumerate(tails):
        copies.append(tail is not None and (tail[0] in whole or tail[0] in given))
        if tail is not None and not copies[b]:
            given.add(tail[0])
            rows[b].append(tail[0])
            refs[tail[0]] += 1
    free = [p for p, n in enumerate(refs) if n == 0]
    full = [len(r) for r in rows]
    at, new, out = 0, list(lens), s["table_out"].clone()
    pools = [x.clone() for x in _pools(s)]
    for b in range(len(src)):
        need = -(-lens[b] // P) - full[b]
        if need and at + need > len(free):
            at = len(free) + 1  # no page for a later row either
            new[b] = full[b] * P if copies[b] or tails[b] is None else full[b] * P - P + tails[b][1]
            continue
        take = free[at:at + need]
        at += need
        for p in take:
            refs[p] = 1
        if copies[b]:
            for x, y in zip(pools, _pools(s)):
                _bits(x)[take[0], :, :tails[b][1]] = _bits(y)[tails[b][0], :, :tails[b][1]]
        rows[b] = rows[b] + take
    for b, row in enumerate(rows):
        out[b, :len(row)] = _ints(row)
    return [out, _ints(new), _ints(refs)] + pools


def _exact_compact(s):
    P = s["case"]["page"]
    table, lens, refs = s["table"].tolist(), s["seqlens"].tolist(), s["refs"].tolist()
    used = [p for p, n in enumerate(refs) if n > 0]
    holes = [p for p in range(len(used)) if refs[p] == 0]
    moves = dict(zip([p for p in used if p >= len(used)], holes))
    new = [0] * len(refs)
    for p in used:
        new[moves.get(p, p)] = refs[p]
    out = s["table_out"].clone()
    for b, n in enumerate(lens):
        m = -(-n // P)
        out[b, :m] = _ints([moves.get(p, p) for p in table[b][:m]])
    pools = [x.clone() for x in _pools(s)]
    for x, y in zip(pools, _pools(s)):
        for a, b in moves.items():
            _bits(x)[b] = _bits(y)[a]
    return [out, _ints(new), _ints([moves.get(p, p) if n > 0 else -1 for p, n in enumerate(refs)]),
            _ints([len(used)])] + pools


def _exact_shared(s):
    """The definition for each sequence over all of its own pages: softmax
    weights, then the centred cross-covariance applied to the probe."""
    case = s["case"]
    P, Hkv, G = case["page"], case["Hkv"], case["Hq"] // case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seqlens"].tolist()):
        ids = s["table"][b, :(n + P - 1) // P].long()

        def keys(name):
            pages = s[name + "pages"]
            if case["fp8"]:
                x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                x = x * torch.exp2(s[name + "scale"][ids].double() - 127.0)[..., None]
            else:
                x = pages[ids].double()
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n]

        K, V = keys("k"), keys("v")
        q, r = (s[x][b].double().reshape(Hkv, G, D) for x in "qr")
        w = torch.softmax(q @ K.transpose(1, 2) / math.sqrt(D), -1)
        mean_k, mean_v = w @ K, w @ V
        w = w * (r @ K.transpose(1, 2) - (r * mean_k).sum(-1, keepdim=True))  # w_j (k_j - mu) . rho
        out[b] = (mean_v - (w @ V - w.sum(-1, keepdim=True) * mean_v)).reshape(-1, D)
    return [out]
