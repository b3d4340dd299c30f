"""Plain 64-bit forms of the grouped products and of MXFP4, on the CPU, and the bounds that the kernels' results are held
to.  Shared by the CPU and the GPU tests."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def padded(cols):
    return -(-cols // 128) * 128


def mx_encode(x):
    """(codes, scales) of float rows by the definition: nearest grid value, ties to the even code."""
    rows, cols = x.shape
    v = torch.zeros(rows, padded(cols), dtype=torch.float64)
    v[:, :cols] = x.double()
    v = v.reshape(rows, -1, 32)
    amax = v.abs().amax(dim=2)
    bad = ~torch.isfinite(amax)
    e = torch.frexp(torch.where(bad, 1.0, amax))[1] - 3  # floor(log2) - 2
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    y = torch.where(bad[..., None], 0.0, v / torch.exp2(e.double())[..., None])
    d = (y.abs()[..., None] - GRID).abs()
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])  # even codes win ties
    code = order[d[..., order].argmin(dim=-1)]
    code = code + torch.where(torch.signbit(y), 8, 0)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
    code = code.reshape(rows, -1, 2)
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8), scale


def mx_decode(q, s, cols):
    n = torch.stack([q & 15, q >> 4], dim=-1).reshape(q.shape[0], -1).long()
    v = GRID[n & 7] * torch.where(n >= 8, -1.0, 1.0)
    f = torch.where(s == 255, math.nan, torch.exp2(s.double() - 127))
    return (v * f.repeat_interleave(32, dim=1))[:, :cols]


def gathered(x, row_tok, n_rows):
    """x's rows in 64 bits as the products read them: zeros for tokens out of range."""
    if row_tok is None:
        return x.double()[:n_rows]
    t = row_tok.long()
    ok = (t >= 0) & (t < x.shape[0])
    return torch.where(ok[:, None], x.double()[t.clamp(0, x.shape[0] - 1)], 0.0)


def groups(offsets, n_rows, E):
    if offsets is None:
        return [(0, 0, n_rows)]
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(E)]


def product(rows, w, offsets, n_rows):
    """(sums, sums of magnitudes) of every grouped row: rows [n_rows][K], w [E][N][K] in 64 bits."""
    y = torch.zeros(n_rows, w.shape[1], dtype=torch.float64)
    m = torch.zeros_like(y)
    for e, a, b in groups(offsets, n_rows, w.shape[0]):
        y[a:b] = rows[a:b] @ w[e].T
        m[a:b] = rows[a:b].abs() @ w[e].abs().T
    return y, m


def in_groups(offsets, n_rows):
    """Which rows belong to a group."""
    r = torch.arange(n_rows)
    return torch.ones(n_rows, dtype=torch.bool) if offsets is None else (r >= int(offsets[0])) & (r < int(offsets[-1]))


def sum_bound(m, length, step):
    """How far an fp32 sum of `length` exact products may be off.  A matrix instruction adds `step` products to its
    accumulator in any order, with at most step additions, and length / step instructions follow one another: at most
    step + length / step roundings on any product's way, each at most 2^-23 of the sum of magnitudes m (2^-24 were every
    addition rounded to nearest)."""
    return (step + -(-length // step)) * 2.0 ** -23 * m


def rounded(ref, bound, dtype):
    """`bound` and the rounding of the result to dtype: half a step relative to the value, or half the smallest step."""
    f = torch.finfo(dtype)
    return bound + (ref.abs() + bound) * (f.eps / 2) + f.smallest_normal * f.eps / 2


def silu(g):
    return g / (1 + torch.exp(-g))
