"""Plain 64-bit forms of the E4M3 cache's operators and of the norms with their
rotation, for the tests. Torch float64 on whatever device the inputs are on;
nothing calls the library."""
from __future__ import annotations

import math

import torch

from tests import draft_util as du

TOP, LEAST = 448.0, 2.0 ** -80
U = 2.0 ** -24  # half a step of fp32


# ------------------------------------------------------------------ E4M3 blocks

def e4m3(x):
    """float64 rounded to the nearest E4M3 value, ties to even, saturated: 4 significant bits, steps of 2^-9 at least."""
    step = torch.exp2((torch.frexp(x)[1].double() - 4).clamp(min=-9.0))
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def fp32(x):
    return x.float().double()


def append_block(codes, scale, kept, new):
    """One block of a head and plane: codes [block, D] (values, float64) with its first `kept` tokens in use and their
    scale, new [n, D] (float64) behind them. Returns (codes, scale)."""
    codes = codes.clone()
    most = float(new.abs().max())  # NaN where there is one
    n = new.shape[0]
    if kept and scale != 0:
        if not math.isfinite(most) or math.isnan(scale):
            scale = math.nan
        else:
            limit, times = float(fp32(torch.tensor(scale, dtype=torch.float64) * TOP)), 1.0
            while most > limit * times:
                times *= 2
            if times > 1:
                codes[:kept] = e4m3(codes[:kept] / times)
            scale *= times
    elif not math.isfinite(most):
        scale = math.nan
    else:
        scale = max(float(fp32(torch.tensor(most, dtype=torch.float64) / TOP)), LEAST) if most else 0.0
    if scale == 0 or math.isnan(scale):
        codes[kept: kept + n] = 0
    else:
        codes[kept: kept + n] = e4m3(fp32(new / scale))
    return codes, scale


def append_row(codes, scales, block, start, new):
    """A row's tokens of a head and plane: codes [C, D], scales [blocks] (float64), new [n, D] at `start`; in place."""
    n, t = new.shape[0], 0
    while t < n:
        j = (start + t) // block
        kept = start + t - j * block
        m = min(block - kept, n - t)
        lo = j * block
        hi = min(lo + block, codes.shape[0])
        codes[lo: hi], scales[j] = append_block(codes[lo: hi], float(scales[j]), kept, new[t: t + m])
        t += m


# ------------------------------------------------------------------- attention

def attention(q, k, ks, v, vs, ok, scale):
    """One row and kv head: q [G, T, D], k and v codes [n, D], ks and vs the tokens' scales [n], ok [T, n] ->
    out, sum p |v|, max sum |q k| scale, sums for the bounds (all float64). Hidden tokens take no part."""
    q, kk = q.double(), k.double() * ks.double()[:, None]
    vv = v.double() * vs.double()[:, None]
    hidden = ~torch.from_numpy(ok).to(q.device)
    dead = hidden.all(0)
    kk = torch.where(dead[:, None], 0.0, kk)
    vv = torch.where(dead[:, None], 0.0, vv)
    s = (torch.einsum("gtd,nd->gtn", q, kk) * scale).masked_fill(hidden, -math.inf)
    top = s.nan_to_num(nan=-math.inf).amax(-1, keepdim=True)
    p = (s - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp().masked_fill(hidden, 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    clean = torch.nan_to_num(vv)
    out = p @ clean
    for j in torch.nonzero(torch.isnan(vv).any(-1))[:, 0].tolist():  # only the queries that see it
        out[:, ~hidden[:, j]] = math.nan
    size = (torch.einsum("gtd,nd->gtn", q.abs(), torch.nan_to_num(kk.abs())) * scale).masked_fill(hidden, 0.0)
    sum_k = (torch.nan_to_num(kk.abs()).sum(-1) * scale)                                   # [n]
    coarse = (q.abs().amax(-1, keepdim=True) * torch.where(hidden, 0.0, sum_k)).amax(-1, keepdim=True)
    peak = (torch.nan_to_num(p) * torch.nan_to_num(torch.where(dead, 0.0, vs.double()))).amax(-1, keepdim=True)
    return out, torch.nan_to_num(p) @ clean.abs(), size.amax(-1, keepdim=True), coarse, peak


def attention_tolerance(out, pv, size, coarse, peak, D, n, out_dtype, wide):
    """Bound of one output element. First as a chain of drafted tokens (draft_util.tree_tolerance), and one more
    rounding of each K and V value (code times scale): D + 5 for D + 3, 2^-23 more. (A step of the tensor cores' sums
    takes 32 products and the sum before; each is cut at 2^-25 of the largest, the sum rounded: 33 2^-25 + 2^-23 a step, less
    than 32 of the chain's 2^-23.) Then what the parts leave out.
    bf16 queries: q is held in two E4M3 parts, off by 2^-14 where q's largest element is 2^7 or more
    (2^-21 of it, for each product); a score and the reference (a score and the logarithm of V's scale) are added in fp32
    (three roundings of |s| + |log2 scale| + 9 <= 1.45 size + 40, and 2^-21 for weights times scale); a weight in four E4M3 parts is
    off by 2^-16 of itself, and by at most 2^-26 of the largest weight times scale (parts of 2^5 and more for that,
    steps of 2^-9 / 16^3), times a code of up to 448.
    fp32 queries (wide): six parts, each of which leaves 2^-4 of what it is given: q off by 2^-24 of each element, and by
    half a step of the last part, 2^-10 / 16^5 = 2^-30, where q's largest is 2^7 or more: 2^-37 of it. Three more roundings of
    the score (products with the scale, the parts' sum), and room for |log2 scale| up to 80: eight of them. A weight off by 2^-24 of
    itself and by 2^-30 / 2^5 of the largest; its product with the scale 2^-24."""
    rel = 2 * (D + 5) * 2.0 ** -23 * size + 2 * 2.0 ** -22 + 2 * (n + 40) * 2.0 ** -23 + 2.0 ** -23
    tol = rel * pv
    if wide:
        tol = tol + pv * (2 * 2.0 ** -37 * coarse + 2 * 2.0 ** -24 * size + 2 * 8 * 2.0 ** -24 * (1.45 * size + 40) + 3 * 2.0 ** -24)
        tol = tol + n * 2.0 ** -35 * TOP * peak
    else:
        tol = tol + pv * (2 * 2.0 ** -21 * coarse + 2 * 3 * 2.0 ** -24 * (1.45 * size + 40) + 2 * 2.0 ** -21 + 2.0 ** -16)
        tol = tol + n * 2.0 ** -26 * TOP * peak
    return tol + torch.finfo(out_dtype).eps / 2 * (out.abs() + tol) + 1e-37


# ---------------------------------------------------------- norms and rotation

def norm_rope(x, weight, offset, eps, positions, freq, style, magnitude=1.0):
    """x [..., T, D]: norm times (weight + offset), then the rotation (freq None: none). float64 result, and the size
    of every element for the bound: |y| of a plain element, |y| + |its partner| of a rotated one."""
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * (weight.double() + offset)
    if freq is None:
        return y, y.abs()
    out, size = du.rotate(y, positions, freq, style, magnitude)
    return out, torch.where(size > 0, size, y.abs())


def norm_tolerance(want, size, dtype, positions, freq):
    """The sum of D <= 1024 squares is one of a lane's up to 64 terms, one after another, and of 5 steps among lanes:
    off by 70 U; times the rounded 1 / D, plus eps: 73 U. A square root halves that; its own rounding and the
    quotient's 1 U each: 39 U. x times it, w + offset, their product: 3 U: 42 U of |y|. The rotation 8 U of both elements
    (draft_util.rotation_tolerance) and the angle's share; then half a step of the output type."""
    angle = 0.0
    if freq is not None and positions.numel():
        angle = positions.double().abs().max().item() * float(max(freq))
    tol = size * (50 * U + 4 * 2.0 ** -53 * angle)
    return tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + 1e-44
