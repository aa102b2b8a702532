"""Plain references of the attention and cache calls in 64 bits, and the error
bounds their 16-bit results have to meet.

The bound of an attention output o = sum_j p_j v_j (p normalised), with
A = sum_j p_j |v_j| and h = eps / 2 the half step of the type:
  h |o|         the output's one rounding
  h (A + |o|)   each p rounded once before it meets V, in the sum or not
  (2 g S + 2^-18) A   fp32 scores off by g S (g = D 2^-24, S the largest
                scale sum |q_i k_i|), in numerator and denominator; exp2 and
                the fp32 sums
and, for fp16, steps of 2^-25 where p or o leave the normal range.
"""

from __future__ import annotations

import torch


def attend(q, k, v, seen, scale):
    """q [R][D], k and v [N][D] doubles, seen [R] visible keys of each row.
    Returns (o, A, S): the output, its absolute sum, the score scale.  Hidden
    keys are left out, not multiplied by zero."""
    r, d = q.shape
    o = torch.zeros(r, d, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    s = torch.zeros(r, 1, dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return o, a, s
    hidden = torch.arange(k.shape[0], device=q.device)[None] >= seen[:, None]
    x = (q @ k.T * scale).masked_fill(hidden, float("-inf"))
    top = x.amax(1, keepdim=True)
    rows = seen > 0
    p = torch.where(rows[:, None], torch.exp(x - torch.where(rows[:, None], top, 0.0)), 0.0)
    p = p / torch.where(rows[:, None], p.sum(1, keepdim=True), 1.0)
    finite = torch.isfinite(v)
    clean = torch.where(finite, v, 0.0)
    o, a = p @ clean, p @ clean.abs()
    if not bool(finite.all()):
        sees = (~hidden).double()
        for kind, value in ((v == float("inf"), float("inf")), (v == float("-inf"), float("-inf")),
                            (torch.isnan(v), float("nan"))):
            o = o + torch.where(sees @ kind.double() > 0, value, 0.0)
    kf = torch.where(torch.isfinite(k), k, 0.0)
    s = (q.abs() @ kf.abs().T * scale).masked_fill(hidden, 0.0).amax(1, keepdim=True)
    return o, a, s


def bound(o, a, s, d, keys, dtype, vmax):
    h = torch.finfo(dtype).eps / 2
    t = h * (2 * o.abs() + a) * (1 + 4 * h) + (2 * d * 2.0**-24 * s + 2.0**-18) * a
    return t + (keys * 2.0**-25 * vmax + 2.0**-25 if dtype == torch.float16 else 0.0) + 1e-30


def check(got, o, a, s, keys, vmax):
    """Asserts that got [R][D] meets the bound around o (equal where o is no
    finite number)."""
    dtype, got = got.dtype, got.double()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isnan(got), torch.isnan(o)), "NaN where none belongs, or none where one does"
    odd = ~fine & ~torch.isnan(o)
    assert torch.equal(got[odd], o[odd]), "infinities differ"
    err, tol = (got - o).abs()[fine], bound(o, a, s, o.shape[1], keys, dtype, vmax)[fine]
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3g} times its bound"


def gather(pages, row, n, head):
    """The first n tokens of one head out of the pages that a table row lists;
    pages that do not exist read as zeros."""
    page = pages.shape[2]
    out = torch.zeros(n, pages.shape[3], dtype=torch.float64, device=pages.device)
    for c in range(-(-n // page)):
        p = int(row[c])
        m = min(page, n - c * page)
        if 0 <= p < pages.shape[0]:
            out[c * page:c * page + m] = pages[p, head, :m].double()
    return out


def tables_for(lens, page, g, spare=3, width=None, fill=-1):
    """A shuffled table for sequences of these lengths and the pool's size."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = width or max(need + [1]) + 1
    rows, at = [], 0
    for m in need:
        rows.append(order[at:at + m] + [fill] * (width - m))
        at += m
    return torch.tensor(rows, dtype=torch.int32).reshape(len(lens), width), pages
