"""GPU parity of ol_norm_rope_rows against the formula in 64 bits: both pairings,
whole, partial and no rotation, weights with and without an offset, fp32 and bf16,
head sizes from one element to 1024, strided, broadcast, unaligned and in-place
views, q or k alone, far positions, vectors of zeros, large and non-finite elements."""
import numpy as np
import pytest
import torch

import place_kv_cache_gb300 as ol
from tests import draft_util as du
from tests import fp8_util as fu
from tests.gpu_util import DEV, canaries_intact, guarded

pytestmark = pytest.mark.gpu
CODE = {torch.float32: ol.OL_F32, torch.bfloat16: ol.OL_BF16}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
STYLES = pytest.mark.parametrize("style", [ol.OL_ROPE_HALF, ol.OL_ROPE_INTERLEAVED], ids=["half", "interleaved"])


def check(got, want, size, positions, freq):
    tol = fu.norm_tolerance(want, size, got.dtype, positions, freq)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off - tol).max()):.3e} more than the bound"


# dtype, B, Hq, Hk, T, D, rot (0: norms alone)
SIZES = [
    ("bf16", 1, 28, 4, 1, 128, 128), ("bf16", 3, 32, 8, 1, 128, 128), ("bf16", 2, 5, 1, 37, 128, 64),
    ("bf16", 2, 3, 3, 9, 96, 48), ("bf16", 1, 7, 2, 3, 80, 80), ("bf16", 2, 2, 1, 5, 80, 40), ("bf16", 1, 2, 1, 4, 20, 6),
    ("bf16", 1, 3, 1, 2, 7, 4), ("bf16", 2, 4, 2, 3, 64, 0), ("bf16", 2, 2, 1, 3, 1, 0), ("bf16", 70, 1, 1, 2, 256, 256),
    ("bf16", 1, 2, 2, 2, 1000, 998), ("bf16", 1, 2, 1, 3, 1024, 1024), ("f32", 2, 9, 3, 17, 128, 128),
    ("f32", 1, 4, 1, 3, 64, 32), ("f32", 2, 3, 1, 5, 6, 2), ("f32", 1, 2, 1, 3, 1024, 1024), ("f32", 1, 2, 1, 3, 1024, 0),
    ("f32", 1, 1, 1, 1023, 96, 48), ("f32", 2, 2, 2, 2, 5, 2), ("f32", 1, 2, 1, 2, 1023, 0), ("f32", 1, 2, 1, 2, 1022, 1022),
]


@STYLES
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_norm_rope_rows(size, style):
    dt, B, Hq, Hk, T, D, rot = size
    dtype = TORCH[dt]
    gen = torch.Generator(device=DEV).manual_seed(5)
    qkv = torch.randn((B, T, Hq + 2 * Hk, D), generator=gen, device=DEV, dtype=dtype) * 3  # a projection's output
    q, k, _ = qkv.transpose(1, 2).split((Hq, Hk, Hk), dim=1)
    qw, kw = torch.randn(D, generator=gen, device=DEV).to(dtype), \
        torch.randn(D, generator=gen, device=DEV).to(dtype)
    freq = du.frequencies(rot) if rot else None
    rope = ol.rope(rot, style=style, device=DEV) if rot else None
    first = torch.randint(0, 100000, (B,), generator=gen, device=DEV, dtype=torch.int32)
    positions = (first[:, None] + torch.arange(T, device=DEV, dtype=torch.int32)).contiguous()
    bufs = [guarded(B * H * T * D * qkv.element_size() + 16) for H in (Hq, Hk)]
    q_out, k_out = (p[: B * H * T * D * qkv.element_size()].view(dtype).view(B, H, T, D)
                    for (_, p), H in zip(bufs, (Hq, Hk)))
    before = qkv.clone()
    for per_token, at, weights, offset in ((True, positions, (qw, kw), 0.0), (False, first, (qw, None), 1.0)):
        q_out.fill_(float("nan"))
        k_out.fill_(float("nan"))
        ol.ol_norm_rope_rows(rope, ol.head_norm(*weights, eps=1e-5, weight_offset=offset), CODE[dtype], B, T, D, Hq, q,
                             q_out, Hk, k, k_out, at if rot else None, per_token)
        for x, w, got in ((q, weights[0], q_out), (k, weights[1], k_out)):
            want, extent = fu.norm_rope(x, w, offset, 1e-5, positions[:, None], freq, style)
            check(got, want, extent, positions, freq)
    assert torch.equal(qkv, before) and all(canaries_intact(b) for b, _ in bufs)


@STYLES
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_place_in_a_projection(dt, style):
    dtype, B, Hq, Hk, T, D = TORCH[dt], 2, 6, 2, 5, 128
    gen = torch.Generator(device=DEV).manual_seed(6)
    qkv = torch.randn((B, T, Hq + 2 * Hk, D), generator=gen, device=DEV, dtype=dtype)
    before = qkv.clone()
    views = lambda x: x.transpose(1, 2).split((Hq, Hk, Hk), dim=1)  # noqa: E731
    q, k, v = views(qkv)
    q0, k0, v0 = views(before)
    freq, rope = du.frequencies(64), ol.rope(64, style=style, device=DEV)
    at = torch.tensor([0, 77777], dtype=torch.int32, device=DEV)
    positions = (at[:, None] + torch.arange(T, device=DEV, dtype=torch.int32)).contiguous()
    ol.ol_norm_rope_rows(rope, ol.head_norm(), CODE[dtype], B, T, D, Hq, q, q, Hk, k, k, at, False)
    for x, got in ((q0, q), (k0, k)):
        want, extent = fu.norm_rope(x, None, 0.0, 1e-6, positions[:, None], freq, style)
        check(got, want, extent, positions, freq)
    assert torch.equal(v, v0)


@STYLES
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_one_kind_alone_and_unaligned_views(shift, style):
    B, H, T, D = 2, 3, 4, 64
    gen = torch.Generator(device=DEV).manual_seed(7)
    flat = torch.randn(B * H * T * (D + 3) + 16, generator=gen, device=DEV).bfloat16()
    x = flat[shift: shift + B * H * T * (D + 3)].view(B, H, T, D + 3)[..., :D]
    out = torch.full((B * H * T * D + 16,), 7.0, device=DEV, dtype=torch.bfloat16)
    y = out[shift: shift + B * H * T * D].view(B, H, T, D)
    freq, rope = du.frequencies(D), ol.rope(D, style=style, device=DEV)
    at = torch.arange(B * T, device=DEV, dtype=torch.int32).view(B, T) * 1000
    w = torch.randn(D, generator=gen, device=DEV).bfloat16()
    want, extent = fu.norm_rope(x, w, 0.0, 1e-6, at[:, None], freq, style)
    ol.ol_norm_rope_rows(rope, ol.head_norm(w), ol.OL_BF16, B, T, D, H, x, y, 0, None, None, at, True)
    check(y, want, extent, at, freq)
    y.zero_()
    ol.ol_norm_rope_rows(rope, ol.head_norm(None, w), ol.OL_BF16, B, T, D, 0, None, None, H, x, y, at, True)
    check(y, want, extent, at, freq)
    assert bool((out[:shift] == 7).all()) and bool((out[shift + B * H * T * D:] == 7).all())


def test_far_positions_and_a_broadcast_input():
    B, H, T, D = 1, 4, 3, 128
    x = torch.randn((1, 1, T, D), device=DEV)
    freq, rope = du.frequencies(D), ol.rope(D, device=DEV)
    at = torch.tensor([[2 ** 31 - 1, -5, 1000000]], dtype=torch.int32, device=DEV)
    y = torch.empty((B, H, T, D), device=DEV)
    ol.ol_norm_rope_rows(rope, ol.head_norm(), ol.OL_F32, B, T, D, H, x.expand(B, H, T, D), y, 0, None, None, at, True)
    want, extent = fu.norm_rope(x.expand(B, H, T, D), None, 0.0, 1e-6, at[:, None], freq, ol.OL_ROPE_HALF)
    check(y, want, extent, at, freq)


def test_zeros_large_and_nonfinite_vectors_stay_apart():
    B, H, T, D = 1, 8, 2, 128
    x = torch.randn((B, H, T, D), device=DEV).bfloat16()
    x[0, 1] = 0
    x[0, 2] *= 1e12
    x[0, 3] *= 1e-12
    x[0, 4, 0, 5] = float("inf")
    x[0, 5, 1, 7] = float("nan")
    rope = ol.rope(D, device=DEV)
    at = torch.zeros((B, T), dtype=torch.int32, device=DEV)
    y = torch.full_like(x, 3.0)
    ol.ol_norm_rope_rows(rope, ol.head_norm(), ol.OL_BF16, B, T, D, H, x, y, 0, None, None, at, True)
    bad = torch.zeros((B, H, T), dtype=torch.bool, device=DEV)
    bad[0, 4, 0] = bad[0, 5, 1] = True
    freq = du.frequencies(D)
    want, extent = fu.norm_rope(x.masked_fill(bad[..., None], 1.0), None, 0.0, 1e-6, at[:, None], freq, ol.OL_ROPE_HALF)
    check(y[~bad], want[~bad], extent[~bad], at, freq)
    assert bool(torch.isnan(y[bad]).any(-1).all())
    assert bool((y[0, 1] == 0).all())


@STYLES
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D, rot", [(128, 64), (96, 48), (80, 64), (64, 16), (72, 16), (120, 104), (48, 16)])
def test_an_infinity_past_the_rotated_part(D, rot, dt, style):
    """The vector's norm is infinite: every other element, its neighbours of the tail among them, comes out as 0."""
    x = torch.randn((1, 3, 1, D), device=DEV, dtype=TORCH[dt])
    for at in (rot, D - 1, (rot + D) // 2):
        z = x.clone()
        z[0, 1, 0, at] = float("-inf")
        y = torch.full_like(x, 3.0)
        ol.ol_norm_rope_rows(ol.rope(rot, style=style, device=DEV), ol.head_norm(), CODE[TORCH[dt]], 1, 1, D, 3, z, y, 0,
                             None, None, torch.tensor([9], dtype=torch.int32, device=DEV), False)
        rest = torch.arange(D, device=DEV) != at
        assert bool(torch.isnan(y[0, 1, 0, at])) and bool((y[0, 1, 0][rest] == 0).all())
        assert bool((y[0, ::2].abs() > 0).any(-1).all()) and bool(torch.isfinite(y[0, ::2]).all())


def test_streams_graphs_and_two_rotations():
    """A captured call replays with the positions it finds; calls on two streams at once keep apart."""
    B, H, T, D = 4, 8, 1, 128
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn((B, H, T, D), generator=gen, device=DEV).bfloat16()
    freq, rope = du.frequencies(D), ol.rope(D, device=DEV)
    at = torch.arange(B, device=DEV, dtype=torch.int32)
    y = torch.empty_like(x)
    call = lambda s=None: ol.ol_norm_rope_rows(rope, ol.head_norm(), ol.OL_BF16, B, T, D, H, x, y, 0, None, None,  # noqa
                                               at, False, stream=s)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    at.add_(4321)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want, extent = fu.norm_rope(x, None, 0.0, 1e-6, at[:, None, None], freq, ol.OL_ROPE_HALF)
    check(y, want, extent, at, freq)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    z = torch.empty_like(x)
    for _ in range(20):
        call()
        ol.ol_norm_rope_rows(rope, ol.head_norm(), ol.OL_BF16, B, T, D, H, x, z, 0, None, None, at, False, stream=other)
    torch.cuda.synchronize()
    check(y, want, extent, at, freq)
    assert torch.equal(y, z)


def test_no_rows_or_tokens_is_no_work():
    x = torch.zeros((1, 1, 1, 64), device=DEV)
    y = torch.full_like(x, 5.0)
    ol.ol_norm_rope_rows(None, ol.head_norm(), ol.OL_F32, 0, 1, 64, 1, x, y, 0, None, None, None, False)
    ol.ol_norm_rope_rows(None, ol.head_norm(), ol.OL_F32, 1, 0, 64, 1, x, y, 0, None, None, None, False)
    torch.cuda.synchronize()
    assert bool((y == 5).all())
