"""Plain 64-bit forms of the operators around drafted tokens, and seeded
inputs for their tests. Everything here is torch float64 on whatever device the
inputs are on; nothing calls the library."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF, INTERLEAVED = 0, 1


# ------------------------------------------------------------ rotary positions

def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Radians per position of each pair (numpy float64)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        k = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = (1 - k) * f / factor + k * f
    return f


def rotate(x, positions, freq, style, magnitude=1.0):
    """x [..., T, D] at positions [..., T] (broadcast against x's leading axes): float64 result, and the
    size |x| + |y| of every element's pair (for tolerances; 0 where elements are copied)."""
    x = x.double()
    r = 2 * len(freq)
    angle = positions.double()[..., None] * torch.from_numpy(freq).to(x.device)
    c, s = angle.cos() * magnitude, angle.sin() * magnitude
    out, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(r // 2, device=x.device)
    a, b = (i, i + r // 2) if style == HALF else (2 * i, 2 * i + 1)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * magnitude
    return out, size


def rotation_tolerance(want, size, dtype, positions, freq):
    """Rounding of the rotation. In fp32 steps u = 2^-24 of (|x| + |y|): the half-turn argument in [-1, 1] is off by
    u / 2, so the angle by pi u / 2 < 2 u; sincospif by at most 2 ulp (2 u); times the magnitude, times x or y, the
    difference: 1 u each. 7 u, taken as 8. The table carries 53 bits and so does this reference: the angle differs by
    2 * 2^-53 of it. Then half a step of the output type; copied elements (size 0) are exact."""
    angle = positions.double().abs().max().item() * float(np.max(freq)) if positions.numel() else 0.0
    tol = size * (8 * 2.0 ** -24 + 4 * 2.0 ** -53 * angle)
    step = torch.finfo(dtype).eps / 2
    return torch.where(size > 0, tol + step * (want.abs() + tol), torch.zeros_like(tol))


# ------------------------------------------------------------- tree attention

def random_trees(rng, batch, nodes, depth_bias=0.5):
    """Trees in topological order: bool [B, T, T] of ancestors and self, depths [B, T]."""
    sees = np.zeros((batch, nodes, nodes), bool)
    depth = np.zeros((batch, nodes), np.int32)
    for b in range(batch):
        for i in range(nodes):
            p = int(rng.integers(-1, i)) if rng.random() < depth_bias else max(-1, i - 2)
            if p >= 0:
                sees[b, i] = sees[b, p]
                depth[b, i] = depth[b, p] + 1
            sees[b, i, i] = True
    return sees, depth


def pack_mask(sees):
    """bool [B, T, T] -> int64 [B, T, ceil(T / 64)] (the uint64 words' bits)."""
    batch, nodes, _ = sees.shape
    words = -(-nodes // 64)
    padded = np.zeros((batch, nodes, words * 64), bool)
    padded[:, :, :nodes] = sees
    return np.packbits(padded, axis=-1, bitorder="little").view("<u8").astype(np.uint64).view(np.int64)


def visible(length, count, sees, positions, window):
    """bool [count, length] of one row: which cached tokens each node attends. sees [T, T] or None (a chain),
    positions [T] or None."""
    prefix = length - count
    ok = np.ones((count, length), bool)
    ok[:, prefix:] = np.tril(np.ones((count, count), bool)) if sees is None else sees[:count, :count]
    if window >= 0:
        at = prefix + np.arange(count) if positions is None else np.maximum(positions[:count].astype(np.int64), prefix)
        where = np.concatenate((np.arange(prefix), at))
        ok &= at[:, None] - where[None] <= window
    return ok


def tree_attention(q, k, v, ok, scale):
    """One row and kv head: q [G, T, D], k and v [n, D], ok [T, n] -> out, sum p |v|, sqrt(sum p^2 v^2), max |score
    error per unit of rounding| (all float64). Hidden tokens take no part, whatever they hold."""
    q, k, v = q.double(), k.double(), v.double()
    hidden = ~torch.from_numpy(ok).to(q.device)
    s = torch.einsum("gtd,nd->gtn", q, k) * scale
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    p = p.masked_fill(hidden, 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    dead = hidden.all(0)
    clean = torch.where(dead[:, None], torch.zeros_like(v), v)
    out = p @ clean
    bad = ~torch.isfinite(clean).all(-1)
    if bad.any():  # 0 * inf: only the nodes that see such a token get it
        finite = torch.where(torch.isfinite(clean), clean, torch.zeros_like(clean))
        out = p @ finite
        for j in torch.nonzero(bad)[:, 0].tolist():
            sees = ~hidden[:, j]
            out[:, sees] += torch.where(torch.isfinite(v[j]), torch.zeros_like(v[j]), v[j])
        clean = finite
    size = torch.einsum("gtd,nd->gtn", q.abs(), torch.nan_to_num(k.abs(), posinf=0.0)) * scale
    size = size.masked_fill(hidden, 0.0).amax(-1, keepdim=True)
    return out, p @ clean.abs(), (p.square() @ clean.square()).sqrt(), size


def tree_tolerance(out, pv, size, D, n, out_dtype, p_bf16):
    """Bound of one output element. Scores: D products summed in fp32, one product with the scale, the subtraction of
    the maximum: (D + 3) * 2^-23 of sum |q k| scale (2^-23 a step: the tensor cores may truncate), which is the relative
    error of a weight and of the sum of weights alike: twice. exp2 2^-22, the two sums over n tokens n * 2^-23 each
    (2 * 2^-23 a partial result and a merge more). A weight rounded to bf16 is off by 2^-8 of itself. All of it times
    sum p |v|. Then half a step of the output type."""
    rel = 2 * (D + 3) * 2.0 ** -23 * size + 2 * 2.0 ** -22 + 2 * (n + 40) * 2.0 ** -23
    if p_bf16:
        rel = rel + 2.0 ** -8
    tol = rel * pv
    return tol + torch.finfo(out_dtype).eps / 2 * (out.abs() + tol) + 1e-37
