"""Plain fp64 forms of the paged-cache operators and the inputs of their tests (numpy, CPU).

Written from the definitions: a cache is a pair of page arrays, position j of sequence b is slot
j % page of page table[b, j // page].  bf16 values are held in float64 exactly.
"""
import math

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8  # largest relative rounding error of bf16: half of torch.finfo(torch.bfloat16).eps


def bf16(x):
    """x rounded to bf16 the way the kernels do (fp32 first), as float64."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().bfloat16().double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A cache with random content in every slot and a table that hands out its pages in no order."""

    def __init__(self, seed, lens_cap, Hkv, d, page, bits, spare=2, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-int(n) // page) for n in lens_cap]
        self.page, self.bits, self.d, self.Hkv = page, bits, d, Hkv
        P = sum(need) + spare
        W = max([1] + need) if width is None else width
        order = torch.randperm(P, generator=g).tolist()
        table = torch.full((len(need), W), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = table
        if bits == 16:
            self.k, self.v = (torch.randn(P, Hkv, page, d, generator=g).bfloat16() for _ in range(2))
            self.ks = self.vs = None
        else:
            self.k, self.v = (torch.randint(0, 256, (P, Hkv, page, d // 2), generator=g, dtype=torch.uint8)
                              for _ in range(2))
            self.ks, self.vs = (torch.stack([0.1 + 0.4 * torch.rand(P, Hkv, page, generator=g),
                                             -3 + torch.rand(P, Hkv, page, generator=g)], -1).bfloat16()
                                for _ in range(2))

    def cuda(self):
        for n in ("k", "v", "ks", "vs", "table"):
            t = getattr(self, n)
            setattr(self, n, None if t is None else t.cuda())
        return self

    @property
    def kw(self):
        return {} if self.bits == 16 else {"k_scales": self.ks, "v_scales": self.vs}

    def dense(self, b, n):
        """Exact k, v of the first n positions of sequence b, [n, Hkv, d] float64 (nothing rounded)."""
        ids = self.table[b].cpu().tolist()
        out = []
        for x, s in ((self.k.cpu(), self.ks), (self.v.cpu(), self.vs)):
            y = np.zeros((n, self.Hkv, self.d))
            for j in range(n):
                row = x[ids[j // self.page], :, j % self.page]
                if self.bits == 16:
                    y[j] = f64(row)
                else:
                    sc = f64(s.cpu()[ids[j // self.page], :, j % self.page])
                    c = row.numpy().astype(np.int64)
                    y[j, :, 0::2] = sc[:, 1:] + sc[:, :1] * (c & 15)
                    y[j, :, 1::2] = sc[:, 1:] + sc[:, :1] * (c >> 4)
            out.append(y)
        return out


def visible(pos, n, causal, vec, b, h):
    """Which of n keys a row at position pos of head h sees; vec: four [B, Hm, Nm] arrays or Nones."""
    see = np.ones(n, bool)
    if causal:
        see &= np.arange(n) <= pos
    for lo, hi in ((vec[0], vec[1]), (vec[2], vec[3])):
        if lo is not None:
            m = min(n, lo.shape[2])
            hm = 0 if lo.shape[1] == 1 else h
            see[:m] &= ~((lo[b, hm, :m] <= pos) & (pos < hi[b, hm, :m]))
    return see


def attention(q, cache, lens, vec=(None,) * 4, start=None, causal=True, scale=None):
    """o, lse in float64, and the bounds of their errors.

    The kernel rounds each weight (with 4 bits: weight times scale) to bf16 before the second product and the
    result once more: |do| <= 2^-8 sum w |v| + 2^-8 |o|.  With 4 bits the rounded weight multiplies scale * (code - 8)
    and the rest of the value is summed in fp32: |v| there is |scale (code - 8)|.  Scores are sums
    of d products in fp32, at most 2^-23 of sum |q k| a term, which moves each weight by twice delta
    relatively.  With 4 bits scale * (16 + code) is multiplied, from -24 scale sum(q) on: running sums of at most
    55 scale sum |q|, rounded twice for every 16 products; sum(q) times minimum + 8 scale comes to it.  2^-16 covers
    exp2, the running sums over the keys and the merge."""
    B, Nq, Hq, d = q.shape
    G = Hq // cache.Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    qq = f64(q)
    vec = [None if x is None else x.cpu().numpy().astype(np.int64) for x in vec]
    o, lse = np.zeros((B, Nq, Hq, d)), np.full((B, Hq, Nq), -np.inf)
    o_tol, lse_tol = np.zeros((B, Nq, Hq, d)), np.full((B, Hq, Nq), 1e-30)
    for b in range(B):
        n = int(lens[b])
        k, v = cache.dense(b, n)
        size_k, size_v = np.abs(k), np.abs(v)
        if cache.bits == 4 and n:
            # codes and scales apart: |scale (code - 8)| and |minimum + 8 scale| are what is summed
            ids = cache.table[b].cpu().tolist()
            sk, sv = (np.stack([f64(s.cpu()[ids[j // cache.page], :, j % cache.page]) for j in range(n)])
                      for s in (cache.ks, cache.vs))
            mid_k, mid_v = (s[..., 1:] + 8 * s[..., :1] for s in (sk, sv))
            size_k = (55 * d / 8 * sk[..., :1] / (d + 4) + np.abs(mid_k)) * np.ones(d)
            size_v = np.abs(v - mid_v)
        first = n - Nq if start is None else int(start[b])
        for i in range(Nq):
            for h in range(Hq):
                see = visible(first + i, n, causal, vec, b, h)
                if not see.any():
                    continue
                kk, vv = k[see, h // G], v[see, h // G]
                s = scale * (kk @ qq[b, i, h])
                m = s.max()
                w = np.exp(s - m)
                lse[b, h, i] = m + math.log(w.sum())
                w /= w.sum()
                o[b, i, h] = w @ vv
                delta = scale * (d + 4) * 2.0 ** -23 * (size_k[see, h // G] @ np.abs(qq[b, i, h])).max()
                spread = w @ size_v[see, h // G]
                o_tol[b, i, h] = HALF_BF16 * (spread + np.abs(o[b, i, h])) * (1 + HALF_BF16) + \
                    (2 * delta + 2.0 ** -16) * (w @ np.abs(vv) + spread)
                lse_tol[b, h, i] = delta + 2.0 ** -20 * (1 + abs(lse[b, h, i]))
    return o, lse, o_tol, lse_tol


def rotate(x, c, s, interleaved):
    """Rows x [.., d] with the first 2 * len(c) values turned, float64."""
    r = c.shape[-1]
    y = x.copy()
    a, b = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if interleaved else (np.arange(r), np.arange(r, 2 * r))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x):
    """(codes, scale, minimum) of rows of bf16 values: the nearest of 16 steps, ties to even."""
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    scale = bf16((hi - lo) / 15)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(scale > 0, np.clip(np.rint((x - lo) / scale), 0, 15), 0)
    return code.astype(np.int64), scale[..., 0], lo[..., 0]
