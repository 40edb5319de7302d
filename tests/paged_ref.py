"""fp64 CPU reference of the paged KV cache operators, and pools to run them on.

A ``Pool`` holds pages whose every unused slot is poisoned (bf16 NaN; e4m3 NaN
codes under exponent 255), so that a result that used one is not finite."""
import math

import numpy as np
import torch

D = 128
# One rounding to bf16, round to nearest: half a step, relative (8 significant
# bits); raised by 2% for the fp32 accumulations (relative 2e-5 at most here).
BF16_HALF = 2.0 ** -8 * 1.02


def e4m3_values():
    """The 127 finite non-negative e4m3 values in code order, from the format:
    1-4-3 bits, bias 7, subnormals below 2^-6, code 127 is NaN."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


def quantise(x):
    """(codes uint8, exponents uint8) of rows x (fp64 [..., d]): the smallest
    E >= 1 with max|x| <= 448 * 2^(E - 127), then the nearest code, ties to
    the even one. By search in fp64, no bit arithmetic on the inputs."""
    x = np.asarray(x, dtype=np.float64)
    vals = e4m3_values()
    amax = np.abs(x).max(-1)
    E = np.ones(amax.shape, dtype=np.int64)
    while True:
        low = amax > 448.0 * np.ldexp(1.0, E - 127)
        if not low.any():
            break
        E = E + low
    y = np.ldexp(x, (127 - E)[..., None])
    a = np.abs(y)
    hi = np.minimum(np.searchsorted(vals, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - vals[lo], vals[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == vals[hi], hi, code)
    return (code + 128 * np.signbit(y)).astype(np.uint8), E.astype(np.uint8)


def dequantise(codes, E):
    vals = np.concatenate([e4m3_values(), [np.nan]])
    vals = np.concatenate([vals, -vals])
    return np.ldexp(vals[codes], (E.astype(np.int64) - 127)[..., None])


class Pool:
    """Poisoned pages, a random page for every (sequence, page), CPU tensors."""

    def __init__(self, lens, Hkv, page, fp8, seed, max_len=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.page, self.fp8 = list(lens), Hkv, page, fp8
        need = [(max(n, 0) + page - 1) // page for n in lens]
        width = max(1, max(need), -(-(max_len or 0) // page))
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)  # never read
        at = 0
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = order[at]
                at += 1
        shape = (self.num_pages, Hkv, page, D)
        if fp8:
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
            self.v = self.k.clone()
            self.ks = torch.full(shape[:3], 255, dtype=torch.uint8)
            self.vs = self.ks.clone()
        else:
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            self.v = self.k.clone()
            self.ks = self.vs = None
        self.seqlens = torch.tensor(lens, dtype=torch.int32)

    def put(self, b, pos, k, v):
        """Store fp64 rows k, v [n, Hkv, d] (bf16 values) at pos .. of sequence b."""
        p = np.arange(pos, pos + k.shape[0])
        page, slot = self.table[b].numpy()[p // self.page], p % self.page
        for pages, scale, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
            if self.fp8:
                c, E = quantise(x)
                pages.view(torch.uint8).numpy()[page, :, slot] = c
                scale.numpy()[page, :, slot] = E
            else:
                pages[torch.from_numpy(page).long(), :, torch.from_numpy(slot)] = torch.from_numpy(
                    np.ascontiguousarray(x)).to(torch.bfloat16)

    def get(self, b, n):
        """fp64 numpy (k, v) [n, Hkv, d]: the first n positions of sequence b."""
        p = np.arange(n)
        page, slot = self.table[b].numpy()[p // self.page], p % self.page
        out = []
        for pages, scale in ((self.k, self.ks), (self.v, self.vs)):
            if self.fp8:
                out.append(dequantise(pages.view(torch.uint8).numpy()[page, :, slot],
                                      scale.numpy()[page, :, slot]))
            else:
                out.append(pages[torch.from_numpy(page).long(), :, torch.from_numpy(slot)].double().numpy())
        return out

    def to(self, dev):
        """Device tensors, as keyword arguments of the binding's calls."""
        return dict(kpages=self.k.to(dev), vpages=self.v.to(dev), block_table=self.table.to(dev),
                    kscale=self.ks.to(dev) if self.fp8 else None,
                    vscale=self.vs.to(dev) if self.fp8 else None)


def normal_rows(n, heads, seed, scale=1.0):
    """bf16 [n, heads, d] ~ N(0, scale^2)."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, D, generator=g) * scale).to(torch.bfloat16)


def filled_pool(lens, Hkv, page, fp8, seed, **kw):
    pool = Pool(lens, Hkv, page, fp8, seed, **kw)
    for b, n in enumerate(lens):
        if n > 0:
            pool.put(b, 0, normal_rows(n, Hkv, seed + 100 + b).double().numpy(),
                     normal_rows(n, Hkv, seed + 500 + b).double().numpy())
    return pool


def attend(Q, R, K, V, nkeys):
    """The definition in fp64 (torch): rows Q, R [m, d], row i sees the first
    nkeys[i] of K, V. Returns (o, lse, bound): bound [m, d] on |o_gpu - o| of
    a kernel that rounds the weights p_j and the products p_j t_j to bf16 once
    before the value products, and the output once:
      2^-8 ((1 + |s|) sum_j w_j |v_j| + sum_j w_j |t_j| (|v_j| + |O1|) + |o|)
    since o = O1 (1 + s) - O2, the denominator uses unrounded p, and s unrounded
    p_j t_j (long chunks) or those of O2 (few rows): a p_j t_j that is off by e
    enters o as -e v_j or as e (O1 - v_j)."""
    Q, R, K, V = (torch.as_tensor(np.asarray(x, dtype=np.float64)) for x in (Q, R, K, V))
    nkeys = torch.as_tensor(nkeys)
    m = Q.shape[0]
    if K.shape[0] == 0 or m == 0:
        z = torch.zeros(m, D, dtype=torch.float64)
        return z.numpy(), np.full(m, -np.inf), z.numpy()
    z = Q @ K.T / math.sqrt(D)
    z = z.masked_fill(torch.arange(K.shape[0])[None] >= nkeys[:, None], -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.where(nkeys[:, None] > 0, torch.exp(z - lse[:, None]), torch.zeros(()).double())
    mean_v, mean_k = w @ V, w @ K
    t = R @ K.T
    c = w * (t - (R * mean_k).sum(1, keepdim=True))
    o = mean_v - (c @ V - c.sum(1, keepdim=True) * mean_v)
    s = (w * t).sum(1, keepdim=True)
    bound = BF16_HALF * ((1 + s.abs()) * (w @ V.abs()) + (w * t.abs()) @ V.abs()
                         + mean_v.abs() * (w * t.abs()).sum(1, keepdim=True) + o.abs())
    return o.numpy(), lse.numpy(), bound.numpy() + 1e-6


def reference(pool, q, r, counts, rows_behind=0):
    """(o, lse, bound) of the packed new tokens: q, r bf16 [T, Hq, d], counts[b]
    new tokens of each sequence, the last ones of its pool.lens[b] keys."""
    T, Hq, _ = q.shape
    G = Hq // pool.Hkv
    o, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    at = 0
    for b, n in enumerate(counts):
        length = max(pool.lens[b], 0)
        K, V = pool.get(b, length)
        nkeys = np.maximum(length - n + np.arange(n) + 1, 0)
        for h in range(Hq):
            x = attend(q[at:at + n, h].double().numpy(), r[at:at + n, h].double().numpy(), K[:, h // G],
                       V[:, h // G], nkeys)
            o[at:at + n, h], lse[at:at + n, h], bound[at:at + n, h] = x
        at += n
    assert at + rows_behind == T
    return o, lse, bound


def assert_within(got, ref, bound, what=""):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - ref) - bound
    if got.size:
        print(f"{what}: max err / bound = {np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3f}")
    assert got.size == 0 or np.max(over) <= 0, (
        f"{what}: {np.max(np.abs(got - ref)):.3e} off, {np.max(over):.2e} over its bound")
