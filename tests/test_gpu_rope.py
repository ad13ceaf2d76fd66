"""GPU parity of the rotary operators (ol_rope_rows, ol_rope_append) against the
formula in 64 bits: both pairings, whole and partial rotation, every scaling,
fp32 and bf16, odd sizes, strided, broadcast and in-place views, far and
negative positions; appends to contiguous and paged caches with ragged counts
and separate rotation positions, which leave every other slot as it was."""
import numpy as np
import pytest
import torch

import place_kv_cache_gb300 as ol
from tests import draft_util as du
from tests.gpu_util import DEV, canaries_intact, guarded

pytestmark = pytest.mark.gpu
SCALINGS = {"none": ol.OL_ROPE_UNSCALED, "linear": ol.OL_ROPE_LINEAR, "ntk": ol.OL_ROPE_NTK,
            "by_parts": ol.OL_ROPE_BY_PARTS}
CODE = {torch.float32: ol.OL_F32, torch.bfloat16: ol.OL_BF16}


def rotation(rot, style, scaling="none", factor=1.0, magnitude=1.0):
    freq = du.frequencies(rot, scaling=scaling, factor=factor, original=4096.0)
    return freq, ol.rope(rot, style=style, scaling=SCALINGS[scaling], factor=factor, original_len=4096.0,
                         magnitude=magnitude, device=DEV)


def check(got, want, size, positions, freq):
    tol = du.rotation_tolerance(want, size, got.dtype, positions, freq)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off - tol).max()):.3e} more than the bound"


# dtype, B, H, T, D, rot
SIZES = [
    ("bf16", 1, 1, 1, 128, 128), ("bf16", 3, 40, 1, 128, 128), ("bf16", 2, 5, 37, 128, 64), ("bf16", 2, 3, 9, 96, 48),
    ("bf16", 1, 7, 3, 80, 80), ("bf16", 2, 2, 5, 80, 40), ("bf16", 1, 2, 4, 20, 6), ("bf16", 1, 3, 2, 7, 4),
    ("f32", 2, 9, 17, 128, 128), ("f32", 1, 4, 3, 64, 32), ("f32", 2, 3, 5, 6, 2), ("f32", 1, 2, 3, 1024, 1024),
    ("f32", 1, 1, 2047, 96, 48), ("bf16", 70, 1, 2, 256, 256), ("f32", 2, 2, 2, 5, 2), ("bf16", 1, 2, 2, 1000, 998),
]


@pytest.mark.parametrize("style", [ol.OL_ROPE_HALF, ol.OL_ROPE_INTERLEAVED], ids=["half", "interleaved"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_rope_rows(size, style):
    dt, B, H, T, D, rot = size
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    gen = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn((B, T, H, D), generator=gen, device=DEV, dtype=dtype).transpose(1, 2)  # token-major
    freq, rope = rotation(rot, style)
    first = torch.randint(0, 100000, (B,), generator=gen, device=DEV, dtype=torch.int32)
    positions = (first[:, None] + torch.arange(T, device=DEV, dtype=torch.int32)).contiguous()
    buf, payload = guarded(B * H * T * D * x.element_size())
    out = payload.view(dtype).view(B, H, T, D)
    before = x.clone()
    for per_token, at in ((True, positions), (False, first)):
        out.fill_(float("nan"))
        ol.ol_rope_rows(rope, CODE[dtype], B, H, T, D, x, out, at, per_token)
        want, extent = du.rotate(x, positions[:, None], freq, style)
        check(out, want, extent, positions, freq)
        assert torch.equal(out[..., rot:], x[..., rot:])
    assert torch.equal(x, before) and canaries_intact(buf)


@pytest.mark.parametrize("scaling,factor,magnitude", [("linear", 4.0, 1.0), ("ntk", 8.0, 1.0),
                                                      ("by_parts", 8.0, 1.2079), ("none", 1.0, 0.5)])
@pytest.mark.parametrize("positions", [[0, 1, 2, 3], [131071, 1000003, 16777217, 2147483647],
                                       [-1, -7, -100000, -2147483648]], ids=["near", "far", "negative"])
def test_rope_scalings_and_positions(scaling, factor, magnitude, positions):
    freq, rope = rotation(128, ol.OL_ROPE_HALF, scaling, factor, magnitude)
    x = torch.randn((1, 3, 4, 128), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    at = torch.tensor([positions], dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    ol.ol_rope_rows(rope, ol.OL_F32, 1, 3, 4, 128, x, out, at, True)
    want, size = du.rotate(x, at[:, None], freq, ol.OL_ROPE_HALF, magnitude)
    check(out, want, size, at, freq)


@pytest.mark.parametrize("style", [ol.OL_ROPE_HALF, ol.OL_ROPE_INTERLEAVED])
def test_rope_in_place_broadcast_and_unaligned_views(style):
    freq, rope = rotation(64, style)
    gen = torch.Generator(device=DEV).manual_seed(6)
    at = torch.tensor([[3, 900], [77, 5]], dtype=torch.int32, device=DEV)
    qkv = torch.randn((2, 2, 9, 64), generator=gen, device=DEV, dtype=torch.bfloat16)
    q = qkv.transpose(1, 2)[:, :5]
    want, size = du.rotate(q, at[:, None], freq, style)
    rest = qkv[:, :, 5:].clone()
    ol.ol_rope_rows(rope, ol.OL_BF16, 2, 5, 2, 64, q, q, at, True)
    check(q, want, size, at, freq)
    assert torch.equal(qkv[:, :, 5:], rest)
    # one vector for every head and row, rotated to each position
    one = torch.randn((1, 1, 2, 64), generator=gen, device=DEV, dtype=torch.bfloat16).expand(2, 3, 2, 64)
    out = torch.empty((2, 3, 2, 64), device=DEV, dtype=torch.bfloat16)
    ol.ol_rope_rows(rope, ol.OL_BF16, 2, 3, 2, 64, one, out, at, True)
    check(out, *du.rotate(one, at[:, None], freq, style), at, freq)
    # a view that starts at an odd element
    flat = torch.randn(1 + 2 * 3 * 2 * 64, generator=gen, device=DEV, dtype=torch.bfloat16)
    odd = flat[1:].view(2, 3, 2, 64)
    ol.ol_rope_rows(rope, ol.OL_BF16, 2, 3, 2, 64, odd, out, at, True)
    check(out, *du.rotate(odd, at[:, None], freq, style), at, freq)


def test_rope_of_nothing():
    _, rope = rotation(64, ol.OL_ROPE_HALF)
    at = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.empty((0, 2, 1, 64), device=DEV)
    ol.ol_rope_rows(rope, ol.OL_F32, 0, 2, 1, 64, x, x, at, True)
    x = torch.empty((2, 2, 0, 64), device=DEV)
    ol.ol_rope_rows(rope, ol.OL_F32, 2, 2, 0, 64, x, x, at, False)
    torch.cuda.synchronize()


# ------------------------------------------------------------------- the append

def make_cache(layout, dtype, B, H, C, D, page, rng):
    """A poisoned cache with guard bytes: (guard buffer, tensor, descriptor, slot(b, t) -> index of a token's heads)."""
    if layout == "contiguous":
        shape = (2, B, H, C, D)
    else:
        M = -(-C // page)
        P = B * M + 2
        table = rng.permutation(P)[: B * M].astype(np.int32).reshape(B, M)
        shape = (2, P, H, page, D)
    size = 4 if dtype == torch.float32 else 2
    buf, payload = guarded(int(np.prod(shape)) * size)
    cache = payload.view(dtype).view(shape)
    cache.fill_(float("nan"))
    if layout == "contiguous":
        return buf, cache, ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(cache), lambda b, t: (b, slice(None), t)
    table_d = torch.from_numpy(table).to(DEV)
    return (buf, cache, ol.OL_LAYOUT_PAGED, ol.paged_kv(cache, table_d, table),
            lambda b, t: (int(table[b, t // page]), slice(None), t % page))


APPENDS = [
    # layout, dtype, B, Hq, Hkv, D, rot, page, C, T, starts, counts, separate angles
    ("contiguous", "bf16", 3, 28, 4, 128, 128, 0, 64, 1, [0, 63, 17], None, False),
    ("paged", "bf16", 3, 32, 8, 128, 128, 16, 64, 1, [0, 63, 16], None, False),
    ("paged", "bf16", 4, 28, 4, 128, 64, 16, 96, 21, [0, 75, 15, 3], [21, 21, 0, 5], True),
    ("contiguous", "f32", 2, 6, 3, 80, 40, 0, 50, 33, [17, 0], [33, 1], False),
    ("paged", "f32", 2, 4, 4, 64, 64, 5, 43, 13, [2, 30], [12, 13], True),
    ("contiguous", "bf16", 1, 2, 1, 20, 6, 0, 9, 9, [0], None, False),
    ("contiguous", "bf16", 2, 16, 2, 256, 256, 0, 300, 257, [40, 0], [257, 100], False),
    ("paged", "bf16", 2, 0, 2, 96, 96, 32, 64, 7, [30, 57], None, True),
]


@pytest.mark.parametrize("style", [ol.OL_ROPE_HALF, ol.OL_ROPE_INTERLEAVED], ids=["half", "interleaved"])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:10])))
def test_rope_append(case, style):
    layout, dt, B, Hq, H, D, rot, page, C, T, starts, counts, separate = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    rng = np.random.default_rng(21)
    gen = torch.Generator(device=DEV).manual_seed(22)
    buf, cache, code, desc, slot = make_cache(layout, dtype, B, H, C, D, page, rng)
    qkv = torch.randn((B, T, Hq + 2 * H, D), generator=gen, device=DEV, dtype=dtype).transpose(1, 2)
    q, k, v = qkv.split((Hq, H, H), dim=1)
    starts_h = np.array(starts, np.int32)
    counts_h = None if counts is None else np.array(counts, np.int32)
    n = [T] * B if counts is None else counts
    angles = torch.randint(0, 5000, (B, T), generator=gen, device=DEV, dtype=torch.int32) if separate else None
    at = angles if separate else torch.from_numpy(starts_h).to(DEV)[:, None] + torch.arange(T, device=DEV)
    freq, rope = rotation(rot, style, "by_parts", 4.0, 1.1)
    q_out = torch.full((B, Hq, T, D), 7.0, device=DEV, dtype=dtype) if Hq else None
    before = cache.clone()
    ol.ol_reset_stats()
    ol.ol_rope_append(code, desc, cache, rope, T, k, v, Hq, q if Hq else None, q_out, starts_h,
                      torch.from_numpy(starts_h).to(DEV), counts_h,
                      None if counts is None else torch.from_numpy(counts_h).to(DEV), angles)
    torch.cuda.synchronize()
    stats = ol.ol_last_call_stats()
    assert stats["calls"] == 1
    assert stats["storage_append_copied_bytes"] == 2 * sum(n) * H * D * cache.element_size()
    wk, sk = du.rotate(k, at[:, None], freq, style, 1.1)
    tol = du.rotation_tolerance(wk, sk, dtype, at, freq)
    for b in range(B):
        for t in range(n[b]):
            s = slot(b, starts[b] + t)
            assert bool(((cache[0][s].double() - wk[b, :, t]).abs() <= tol[b, :, t]).all())
            assert torch.equal(cache[1][s], v[b, :, t])
            before[0][s], before[1][s] = cache[0][s], cache[1][s]
    bits = torch.int32 if dt == "f32" else torch.int16
    assert torch.equal(cache.view(bits), before.view(bits))  # every other slot as it was
    assert canaries_intact(buf)
    if Hq:
        wq, sq = du.rotate(q, at[:, None], freq, style, 1.1)
        tol = du.rotation_tolerance(wq, sq, dtype, at, freq)
        for b in range(B):
            assert bool(((q_out[b, :, : n[b]].double() - wq[b, :, : n[b]]).abs() <= tol[b, :, : n[b]]).all())
            assert bool((q_out[b, :, n[b]:] == 7.0).all())


def test_rope_append_in_place_q_of_a_fused_projection():
    rng = np.random.default_rng(31)
    B, Hq, H, D, T, C = 2, 4, 2, 64, 3, 8
    _, cache, code, desc, _ = make_cache("contiguous", torch.bfloat16, B, H, C, D, 0, rng)
    qkv = torch.randn((B, T, Hq + 2 * H, D), device=DEV, dtype=torch.bfloat16).transpose(1, 2)
    q, k, v = qkv.split((Hq, H, H), dim=1)
    freq, rope = rotation(D, ol.OL_ROPE_HALF)
    start = np.array([1, 5], np.int32)
    at = torch.from_numpy(start).to(DEV)[:, None] + torch.arange(T, device=DEV)
    want, size = du.rotate(q, at[:, None], freq, ol.OL_ROPE_HALF)
    wk, _ = du.rotate(k, at[:, None], freq, ol.OL_ROPE_HALF)
    kept = qkv[:, Hq:].clone()
    ol.ol_rope_append(code, desc, cache, rope, T, k, v, Hq, q, q, start, torch.from_numpy(start).to(DEV))
    check(q, want, size, at, freq)
    assert torch.equal(qkv[:, Hq:], kept)
    for b in range(B):
        got = cache[0, b, :, start[b]: start[b] + T].double()
        assert float((got - wk[b]).abs().max()) < 0.05
        assert torch.equal(cache[1, b, :, start[b]: start[b] + T], v[b])


def test_rope_append_keeps_bits_of_v_and_of_the_unrotated_part():
    """Infinities and NaN in V and in the unrotated elements pass through; they do not reach other elements."""
    rng = np.random.default_rng(32)
    _, cache, code, desc, _ = make_cache("contiguous", torch.float32, 1, 1, 4, 64, 0, rng)
    k = torch.randn((1, 1, 1, 64), device=DEV)
    v = torch.randn((1, 1, 1, 64), device=DEV)
    v[..., 5], v[..., 6] = float("inf"), float("nan")
    k[..., 40] = float("nan")
    _, rope = rotation(32, ol.OL_ROPE_HALF)
    start = np.array([2], np.int32)
    ol.ol_rope_append(code, desc, cache, rope, 1, k, v, 0, None, None, start, torch.from_numpy(start).to(DEV))
    assert torch.equal(cache[1, 0, 0, 2].view(torch.int32), v[0, 0, 0].view(torch.int32))
    assert torch.equal(cache[0, 0, 0, 2, 32:].view(torch.int32), k[0, 0, 0, 32:].view(torch.int32))
    assert bool(torch.isfinite(cache[0, 0, 0, 2, :32]).all())


def test_rope_append_captured_replays_with_device_positions():
    rng = np.random.default_rng(33)
    B, H, D, C, T = 2, 2, 64, 32, 2
    _, cache, code, desc, slot = make_cache("paged", torch.bfloat16, B, H, C, D, 16, rng)
    freq, rope = rotation(D, ol.OL_ROPE_INTERLEAVED)
    k = torch.randn((B, H, T, D), device=DEV, dtype=torch.bfloat16)
    v = torch.randn((B, H, T, D), device=DEV, dtype=torch.bfloat16)
    start_h = np.array([0, 4], np.int32)
    start = torch.from_numpy(start_h).to(DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ol.ol_rope_append(code, desc, cache, rope, T, k, v, 0, None, None, start_h, start)
    for now in ([3, 9], [15, 30], [31, -1]):  # the last: token 1 of row 0 and row 1 have no place
        cache.fill_(0)
        start.copy_(torch.tensor(now, dtype=torch.int32))
        k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        written = 0
        for b in range(B):
            for t in range(T):
                p = now[b] + t
                if now[b] < 0 or p >= C:
                    continue
                want, size = du.rotate(k[b, :, t], torch.full((H,), p, device=DEV), freq, ol.OL_ROPE_INTERLEAVED)
                tol = du.rotation_tolerance(want, size, torch.bfloat16, start, freq)
                assert bool(((cache[0][slot(b, p)].double() - want).abs() <= tol + 1e-6).all())
                written += 2 * H
        assert int((cache != 0).any(-1).sum()) == written


def test_offsets_past_32_bits():
    """A cache of 2.25e9 elements: tokens appended at a row's end and kept there are those of a small cache; vectors
    that lie 1.1e9 elements apart are rotated in place."""
    H, D, C, T = 8, 128, 1100000, 6
    gen = torch.Generator(device=DEV).manual_seed(77)
    big = torch.zeros((2, 1, H, C, D), device=DEV, dtype=torch.bfloat16)
    small = torch.zeros((2, 1, H, 16, D), device=DEV, dtype=torch.bfloat16)
    k, v = (torch.randn((1, H, T, D), generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    rope = ol.rope(D, device=DEV)
    at = torch.arange(C - T, C, dtype=torch.int32, device=DEV).view(1, T)
    for cache, start in ((big, C - T), (small, 10)):
        first = np.array([start], np.int32)
        first_d = torch.from_numpy(first).to(DEV)
        ol.ol_rope_append(ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(cache), cache, rope, T, k, v, 0, None, None, first, first_d,
                          angles_dev=at)
    torch.cuda.synchronize()
    assert torch.equal(big[:, :, :, C - T:], small[:, :, :, 10:]) and bool((small[:, :, :, 10:] != 0).any())
    kept = torch.tensor([[1, 2, 5, 0, 0, 0]], dtype=torch.int32, device=DEV)
    first = np.array([C - T], np.int32)
    ol.ol_tree_keep(ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(big), big, T, first, torch.from_numpy(first).to(DEV), kept,
                    torch.tensor([3], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(big[:, :, :, C - T: C - 3], small[:, :, :, [11, 12, 15]])
    flat, stride = big.view(-1), 1120000000
    ends = [flat[i * stride: i * stride + 4 * D] for i in range(3 if 2 * stride + 4 * D <= flat.numel() else 2)]
    for e in ends:
        e.copy_(torch.randn(4 * D, generator=gen, device=DEV))
    want = [torch.empty((1, 2, 2, D), device=DEV, dtype=torch.bfloat16) for _ in ends]
    where = torch.tensor([[5, 900]] * len(ends), dtype=torch.int32, device=DEV)
    for e, w in zip(ends, want):
        ol.ol_rope_rows(rope, ol.OL_BF16, 1, 2, 2, D, e.view(1, 2, 2, D), w, where[:1], True)
    view = ol.Rows(big.data_ptr(), stride, 2 * D, D)
    ol.ol_rope_rows(rope, ol.OL_BF16, len(ends), 2, 2, D, view, view, where, True)
    torch.cuda.synchronize()
    assert len(ends) == 3 and all(torch.equal(e.view(1, 2, 2, D), w) for e, w in zip(ends, want))
