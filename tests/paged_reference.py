"""Plain references of the norm and rotation and of the paged cache, in 64 bits
on the CPU, with the error bounds that their kernels are held to."""
from __future__ import annotations

import math

import torch

HALF = 2.0 ** -8        # rounding to bfloat16: at most half a step, relative to the value
U = 2.0 ** -24          # rounding to fp32


def cdiv(a, b):
    return -(-a // b)


def norm_rotate(x, norm, w, cos, sin, pos, interleaved, eps):
    """x [n, H, d] bf16, pos [n]: (result, size of each value's pair) in fp64."""
    x = x.double()
    if norm == "head":
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    elif norm == "token":
        x = x / torch.sqrt(x.pow(2).mean((-2, -1), keepdim=True) + eps)
    if norm != "none" and w is not None:
        x = x * w.double()
    if cos is None:
        return x, x.abs()
    c, s = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    y0, y1, r = a * c - b * s, a * s + b * c, (a.abs() + b.abs()) * (c.abs() + s.abs())
    if interleaved:
        return torch.stack((y0, y1), -1).flatten(-2), torch.stack((r, r), -1).flatten(-2)
    return torch.cat((y0, y1), -1), torch.cat((r, r), -1)


def assert_norm_rotate(got, ref, size, norm, values):
    """One rounding to bf16, and fp32 arithmetic on terms of at most `size`: the
    mean square's sum has `values` terms, added by lanes (at most 64 in a row),
    across lanes and warps (at most 21 more) and halved by the root; scale,
    weight, two products, a sum: 6 more."""
    k = (85 / 2 + 8 if norm != "none" else 0) + 6
    off = (got.double() - ref).abs() - (HALF * (1 + k * U) * ref.abs() + k * U * size)
    assert off.max().item() <= 0, f"beyond its bound by {off.max().item()}"


def plan(n_new, lens, table, free, free_count, page, max_pages, T):
    """The lists of one step, request after request.  Returns (lens, table, free,
    free_count, cu, slots, positions, complaint)."""
    lens, table, free = list(lens), [list(r) for r in table], list(free)
    top, bad = free_count, False
    for s, n in enumerate(n_new):
        if n == -1:
            for j in range(cdiv(lens[s], page)):
                free[top] = table[s][j]
                top += 1
    cu, slots, positions, open_ = [0], [], [], True
    for s, n in enumerate(n_new):
        if n < -1 or lens[s] + max(n, 0) > max_pages * page:
            n, bad = 0, True
        old = cdiv(lens[s], page)
        k = max(n, 0)
        need = cdiv(lens[s] + k, page) - old if k else 0
        if open_ and (need > top or len(slots) + k > T):
            open_, bad = False, True
        if not open_:
            k = need = 0
        for j in range(need):
            top -= 1
            table[s][old + j] = free[top]
        for i in range(k):
            at = lens[s] + i
            positions.append(at)
            slots.append(table[s][at // page] * page + at % page)
        lens[s] = 0 if n == -1 else lens[s] + k
        cu.append(len(slots))
    slots += [-1] * (T - len(slots))
    positions += [0] * (T - len(positions))
    return lens, table, free, top, cu, slots, positions, bad


def budget(n, keep):
    keep = torch.tensor(keep, dtype=torch.float32).item()
    return min(max(int(math.floor(keep * n + 0.5)), 1), n) if n else 0


def topk(P, n, keep, recent):
    """Kept pages of one row (P fp32 [>= n])."""
    kb = budget(n, keep)
    r = min(recent, kb)
    key = [float(x) if x > 0 else 0.0 for x in P[:n - r].tolist()]
    best = sorted(range(n - r), key=lambda j: (-key[j], j))[:kb - r]
    return sorted(best) + list(range(n - r, n))


def select(q, kbar, lens, page, d):
    """P of one row in fp64, and the bound of the scores' errors: q [G, d], kbar
    [n, d].  A product's d terms are exact and summed in fp32 in any order, with
    truncation: at most (d/16 + 16) steps of 2^-23 of the terms' sizes, twice
    (numerator and the row's sum)."""
    q, kbar = q.double(), kbar.double()
    n = kbar.shape[0]
    size = torch.full((n,), float(page), dtype=torch.float64)
    if n:
        size[-1] = lens - (n - 1) * page
    x = q @ kbar.T / math.sqrt(d) + size.log()
    a = (q.abs() @ kbar.abs().T / math.sqrt(d)).max().item() if n else 0.0
    return torch.softmax(x, -1).mean(0), 2 * (d / 16 + 16) * 2 * U * a


def attention(q, keys, values, d):
    """q [G, d] over keys, values [n, d] in fp64: (O, sum p |v|, bound of the
    scores' errors as in select)."""
    q, keys, values = q.double(), keys.double(), values.double()
    p = torch.softmax(q @ keys.T / math.sqrt(d), -1)
    a = (q.abs() @ keys.abs().T / math.sqrt(d)).max().item()
    return p @ values, p @ values.abs(), 2 * (d / 16 + 16) * 2 * U * a


def assert_attention(got, ref, size, eps, n):
    """One rounding to bf16; weights off by the scores' errors, by 2^-16 (two
    bf16 parts) and 2^-20 (exponentials, joins); sums of n terms in fp32, 16 at
    a time in at least four parts."""
    rel = math.expm1(eps) + 2.0 ** -16 + 2.0 ** -20 + (n / 64 + 40) * 2 * U
    off = (got.double() - ref).abs() - (HALF * ref.abs() + rel * (1 + HALF) * size)
    assert off.max().item() <= 0, f"beyond its bound by {off.max().item()}"


class Cache:
    """A cache with distinct pages in random order, in CPU memory; what no
    sequence holds is NaN."""

    def __init__(self, lens, Hkv, d, page, seed, max_pages=None, spare=3, kscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.d, self.Hkv = list(lens), page, d, Hkv
        pages = [cdiv(n, page) for n in lens]
        self.max_pages = max_pages or max(max(pages), 1)
        self.num_pages = sum(pages) + spare
        perm = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        nan = float("nan")
        self.K = torch.full((self.num_pages, Hkv, page, d), nan, dtype=torch.bfloat16)
        self.V = torch.full((self.num_pages, Hkv, page, d), nan, dtype=torch.bfloat16)
        self.ksum = torch.full((self.num_pages, Hkv, d), nan, dtype=torch.bfloat16)
        self.keys, self.values = [], []
        for s, n in enumerate(lens):
            k = (kscale * torch.randn(n, Hkv, d, generator=g)).to(torch.bfloat16)
            v = torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16)
            self.keys.append(k)
            self.values.append(v)
            for j in range(pages[s]):
                p = perm.pop()
                self.table[s, j] = p
                m = min(page, n - j * page)
                self.K[p, :, :m] = k[j * page:j * page + m].transpose(0, 1)
                self.V[p, :, :m] = v[j * page:j * page + m].transpose(0, 1)
                self.ksum[p] = self.K[p, :, :m].float().mean(1).to(torch.bfloat16)
        self.free = perm
