"""Plain 64-bit forms of the token-mixing operators, with for each output the
sum of its terms' magnitudes, from which the tests derive their tolerances.
Sequence by sequence and head by head, from the definitions alone."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def half_step(dtype) -> float:
    """Largest relative error of rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half the spacing of dtype's subnormals: the absolute part of a rounding."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def rotate(x, pos, freqs, interleaved=False, amp=1.0):
    """x [rows][heads][dim] (any type) -> (rotated, magnitudes), 64-bit."""
    x = x.to(F64)
    rot = 2 * len(freqs)
    y, mag = x.clone(), x.abs()
    ang = pos.to(F64)[:, None] * torch.as_tensor(freqs, dtype=F64)[None]
    c, s = amp * torch.cos(ang)[:, None], amp * torch.sin(ang)[:, None]
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    m = abs(amp) * (x[..., a].abs() + x[..., b].abs())
    mag[..., a] = m
    mag[..., b] = m
    return y, mag


def attend(q, k, v, first, scale, causal=True, window=0):
    """One head, one sequence: q [n][d] at places first.., k and v [len][d] -> (o, weighted
    magnitudes of v, largest sum of a score's magnitudes); a row that sees nothing gives 0."""
    n, L = q.shape[0], k.shape[0]
    q, k = q.to(F64), k.to(F64)
    p = first + torch.arange(n)[:, None]
    j = torch.arange(L)[None]
    seen = (j <= p) if causal else torch.ones(n, L, dtype=torch.bool)
    if window:
        seen = seen & (j > p - window)
    s = torch.where(seen, (q @ k.T) * scale, -math.inf)
    mags = torch.where(seen, (q.abs() @ k.abs().T) * abs(scale), 0.0).amax(1) if L else torch.zeros(n, dtype=F64)
    top = s.amax(1, keepdim=True) if L else torch.zeros(n, 1, dtype=F64)
    top = torch.where(torch.isfinite(top), top, 0.0)
    w = torch.exp(s - top)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0)
    vv = v.to(F64)
    o = torch.zeros(n, v.shape[1], dtype=F64)
    a = torch.zeros_like(o)
    for i in range(n):                         # unseen rows of v are not touched at all
        at = seen[i].nonzero()[:, 0]
        o[i] = w[i, at] @ vv[at]
        a[i] = w[i, at] @ vv[at].abs()
    return o, a, mags


def linear(q, k, v, g, state, scale=1.0):
    """One head, one sequence, token by token: -> (o, state, and the same of the magnitudes)."""
    S, A = state.to(F64).clone(), state.to(F64).abs()
    o, ao = [], []
    for t in range(q.shape[0]):
        d = math.exp(float(g[t]))
        S = d * S + torch.outer(k[t].to(F64), v[t].to(F64))
        A = d * A + torch.outer(k[t].to(F64).abs(), v[t].to(F64).abs())
        o.append(scale * (q[t].to(F64) @ S))
        ao.append(abs(scale) * (q[t].to(F64).abs() @ A))
    z = torch.zeros(0, v.shape[1], dtype=F64)
    return (torch.stack(o) if o else z), S, (torch.stack(ao) if ao else z), A


def paged(n_pages, page_size, heads, dim, dtype, gen, head_major=False, fill=None):
    """A CPU pool [pages][page_size][heads][dim] (a permuted view if head_major)."""
    shape = (n_pages, heads, page_size, dim) if head_major else (n_pages, page_size, heads, dim)
    x = torch.randn(shape, generator=gen).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype)
    return x.transpose(1, 2) if head_major else x


def table_of(lengths, page_size, gen, spare=2, cols=0):
    """(table, pages of the pool): every sequence's pages its own, in random order."""
    need = [(l + page_size - 1) // page_size for l in lengths]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen).to(torch.int32)
    t = torch.full((len(lengths), max([1, cols] + need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = order[at:at + n]
        at += n
    return t, pool


def gather(pool, table, s, length, head):
    """[length][dim] of one head of sequence s."""
    ps = pool.shape[1]
    j = torch.arange(length)
    return pool[table[s, j // ps].long(), j % ps, head]
