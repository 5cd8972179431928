"""Plain references in 64 bits of the packed and paged operators, and the
element-wise bounds their results are held to.

Bounds.  A result computed in fp32 from products that are exact or rounded once
differs from the definition by
  * the scores: a sum of D products errs by at most (D + 4) steps of 2^-23 of
    sum |q k| (truncating accumulators included); a score's error e changes its
    weight by a factor e^(+-e), and the normalised row by at most 2 e;
  * the base-2 exponential and the scaling before it: 2^-20 of the weight;
  * the sums over n keys: n steps of 2^-23 of sum p |v| (and of sum p);
  * a P rounded to bf16 for the product: 2^-8 of sum p |v|;
  * the rounding to the element type: eps / 2 of |y|.
"""
import math

import torch

POISON = float("nan")


def attention_rows(q, k, v, allowed, scale):
    """y, sum p |v| and max_j scale * sum |q k| of rows q (n, D) over keys k, v
    (m, D); allowed (n, m).  Rows without a key are zeros."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T) * scale
    s = s.masked_fill(~allowed, -math.inf)
    top = s.amax(1, keepdim=True) if s.shape[1] else torch.full((q.shape[0], 1), -math.inf, dtype=s.dtype, device=s.device)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total.clamp(min=1e-300), torch.zeros_like(e))
    size = ((q.abs() @ k.abs().T) * scale).masked_fill(~allowed, 0.0)
    size = size.amax(1, keepdim=True) if size.shape[1] else torch.zeros_like(top)
    return p @ v, p @ v.abs(), size


def bound(y, pv, size, D, n, dtype, p_bf16):
    u = torch.finfo(dtype).eps / 2
    e = (D + 4) * 2.0 ** -23 * size + 2.0 ** -20 + n * 2.0 ** -23
    return 2 * e * pv + (2.0 ** -8 * pv if p_bf16 else 0.0) + u * y.abs() + 1e-30


def check(got, y, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - y).abs() - tol
    assert float(over.max()) <= 0, f"{what}: over its bound by {float(over.max())}, error {float((got - y).abs().max())}"


def turn_fraction(pos: int, f: float) -> float:
    """frac(pos * f / 2 pi) in [0, 1) with the exact value of the fp32 f: whole
    numbers against 400 bits of 1 / 2 pi (Machin's formula)."""
    m, e = math.frexp(f)
    m, e = int(m * (1 << 24)), e - 24  # f = m * 2^e
    num = pos * m * _INV_2PI
    shift = _BITS - e
    return ((num >> (shift - 60)) % (1 << 60)) / float(1 << 60)


_BITS = 400


def _arctan_inv(x, bits):
    total, term, k = 0, (1 << bits) // x, 0
    while term:
        total += (-term if k & 1 else term) // (2 * k + 1)
        term //= x * x
        k += 1
    return total


_INV_2PI = (1 << (2 * _BITS)) // (2 * 4 * (4 * _arctan_inv(5, _BITS) - _arctan_inv(239, _BITS)))


def rotate_rows(x, pos, inv, sections, R, interleaved):
    """x (rows, H, D) turned by pos (axes, rows) * inv (R/2): the result in 64
    bits and its bound's scale |a| + |b| per element."""
    rows = x.shape[0]
    cos = torch.empty((rows, R // 2), dtype=torch.float64)
    sin = torch.empty_like(cos)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    pos, inv = pos.tolist(), inv.tolist()
    for r in range(rows):
        for i in range(R // 2):
            t = 2 * math.pi * turn_fraction(pos[axis[i]][r], inv[i])
            cos[r, i], sin[r, i] = math.cos(t), math.sin(t)
    x = x.detach().cpu().double()
    y, size = x.clone(), x.abs()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    c, s = cos[:, None], sin[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def rotary_bound(y, size, dtype):
    """The angle (at most half a turn) rounded to fp32 and sincospi's two steps:
    2^-21 on cos and sin; two products and a sum: 2^-22; the element type's
    rounding."""
    return size * (2.0 ** -21 + 2.0 ** -22) + torch.finfo(dtype).eps / 2 * y.abs()


def pages_for(lens, page_size, gen, spare=3, width_spare=1):
    """(pool size, table): random distinct pages for these lengths; -1 elsewhere."""
    need = [(n + page_size - 1) // page_size for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen)
    table = torch.full((len(lens), max(need + [0]) + width_spare), -1, dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pool, table
