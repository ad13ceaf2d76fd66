"""GPU parity of the E4M3 cache's operators against plain 64-bit forms: the
quantising append (bit-exact codes and scales, whole buffers), reading back
(exact), attention on both kernels. Contiguous and paged caches, all block sizes,
odd head sizes and lengths, ragged counts, windows, blocks that grow, zeros,
infinities and NaN, poison in every slot past a row, views of any strides, replayed
and concurrent calls, lengths and pages that disagree on the device."""
import math

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
E4M3 = torch.float8_e4m3fn


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Cache:
    """An E4M3 cache whose every code and scale is NaN until something is put there."""

    def __init__(self, B, H, C, D, block, page=0, seed=1):
        self.B, self.H, self.D, self.block, self.page = B, H, D, block, page
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.table = None
        if page:
            M = -(-C // page)
            C = M * page
            self.table = self.rng.permutation(B * M + 2)[: B * M].astype(np.int32).reshape(B, M)
            shape, per = (2, B * M + 2, H, page, D), page // block
        else:
            shape, per = (2, B, H, C, D), -(-C // block)
        self.C = C
        self.codes_buf, codes = guarded(int(np.prod(shape)))
        self.codes = codes.view(shape).fill_(0x7F)
        n = int(np.prod(shape[:3])) * per
        self.scales_buf, scales = guarded(-(-n // 4) * 16)
        self.scales = scales[: 4 * n].view(torch.float32).view(*shape[:3], per).fill_(float("nan"))
        self.table_d = None if self.table is None else dev(self.table)
        self.desc = ol.fp8_kv(self.codes, self.scales, self.table_d, self.table, block=block)

    def row(self, plane, b):
        """(codes [H, C, D], scales [H, C / block]) of a row as float64 copies."""
        if self.table is None:
            return self.codes[plane, b].view(E4M3).double(), self.scales[plane, b].double()
        pages = self.table[b].tolist()
        return (torch.cat([self.codes[plane, p].view(E4M3).double() for p in pages], 1),
                torch.cat([self.scales[plane, p].double() for p in pages], 1))

    def put_row(self, plane, b, codes, scales):
        c8, s32 = codes.to(E4M3).view(torch.uint8), scales.float()
        if self.table is None:
            self.codes[plane, b], self.scales[plane, b] = c8, s32
            return
        per = self.page // self.block
        for i, p in enumerate(self.table[b].tolist()):
            self.codes[plane, p] = c8[:, i * self.page: (i + 1) * self.page]
            self.scales[plane, p] = s32[:, i * per: (i + 1) * per]

    def fill(self, lens, spread=0.5):
        """Rows of random codes, blocks of random scales, the slots behind them still NaN."""
        for b, n in enumerate(lens):
            if n == 0:
                continue
            for plane in (0, 1):
                codes, scales = self.row(plane, b)
                new = torch.randn((self.H, n, self.D), generator=self.gen, device=DEV, dtype=torch.float64) * 140
                codes[:, :n] = fu.e4m3(new)
                m = -(-n // self.block)
                scales[:, :m] = torch.exp(torch.randn((self.H, m), generator=self.gen, device=DEV, dtype=torch.float64)
                                          * spread).float().double() / 140
                self.put_row(plane, b, codes, scales)

    def expected(self, start, counts, k, v):
        """Bytes of codes and scales after an append (the operator's definition)."""
        keep = self.codes.clone(), self.scales.clone()
        for plane, x in ((0, k), (1, v)):
            for b in range(self.B):
                n = int(counts[b])
                if n == 0:
                    continue
                codes, scales = self.row(plane, b)
                raw = codes.clone()
                for g in range(self.H):
                    fu.append_row(codes[g], scales[g], self.block, int(start[b]), x[b, g, :n].double())
                codes = torch.where(torch.isnan(raw) & torch.isnan(codes), raw, codes)
                self.put_row(plane, b, codes, scales)
        want = self.codes.clone(), self.scales.clone()
        self.codes.copy_(keep[0])
        self.scales.copy_(keep[1])
        return want

    def append(self, start, counts, k, v, ragged=True, stream=None):
        T = k.shape[2]
        ol.ol_fp8kv_append(self.desc, self.codes, CODE[k.dtype], T, k, v, np.array(start, np.int32),
                           dev(np.array(start, np.int32)), np.array(counts, np.int32) if ragged else None,
                           dev(np.array(counts, np.int32)) if ragged else None, stream=stream)

    def same(self, want):
        torch.cuda.synchronize()
        assert torch.equal(self.codes, want[0])
        assert torch.equal(self.scales.nan_to_num(nan=-1.0), want[1].nan_to_num(nan=-1.0))
        assert torch.equal(torch.isnan(self.scales), torch.isnan(want[1]))
        assert canaries_intact(self.codes_buf) and canaries_intact(self.scales_buf)


# ------------------------------------------------------------------------ append

# dtype, B, H, C, D, block, page, T, start, counts
APPENDS = [
    ("bf16", 1, 1, 64, 128, 16, 0, 1, [0], None), ("bf16", 1, 2, 64, 128, 16, 0, 1, [63], None),
    ("bf16", 3, 2, 100, 128, 16, 16, 1, [5, 16, 31], None), ("bf16", 3, 2, 100, 64, 32, 64, 37, [0, 31, 60], [37, 0, 35]),
    ("bf16", 2, 4, 300, 128, 64, 0, 200, [7, 100], [193, 200]), ("bf16", 2, 1, 300, 256, 128, 128, 256, [0, 127], None),
    ("bf16", 2, 3, 77, 80, 16, 0, 33, [44, 1], None), ("bf16", 1, 1, 17, 16, 128, 0, 17, [0], None),
    ("f32", 2, 2, 100, 128, 16, 16, 5, [14, 95], None), ("f32", 2, 2, 260, 256, 128, 0, 129, [130, 0], [128, 129]),
    ("bf16", 2, 2, 200, 128, 16, 48, 50, [40, 95], None), ("bf16", 2, 1, 600, 64, 32, 256, 300, [255, 31], [300, 7]),
    ("f32", 1, 8, 64, 96, 32, 32, 64, [0], None), ("f32", 4, 2, 50, 48, 16, 0, 3, [47, 0, 15, 29], [3, 2, 1, 0]),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:8])))
def test_append_is_exact(case):
    dt, B, H, C, D, block, page, T, start, counts = case
    c = Cache(B, H, C, D, block, page)
    c.fill(start)
    n = [T] * B if counts is None else counts
    # a projection's output; tokens of very different sizes, so that blocks grow
    kv = torch.randn((B, T, 2 * H, D), generator=c.gen, device=DEV)
    kv = (kv * torch.exp(2 * torch.randn((B, T, 2 * H, 1), generator=c.gen, device=DEV))).to(TORCH[dt])
    k, v = kv.transpose(1, 2).chunk(2, dim=1)
    want = c.expected(start, n, k, v)
    c.append(start, n, k, v, ragged=counts is not None)
    c.same(want)
    c.append(start, n, k, v, ragged=counts is not None)  # the same again: nothing grows any more, the codes stay
    first = c.codes.clone(), c.scales.clone()
    want = c.expected(start, n, k, v)
    c.append(start, n, k, v, ragged=counts is not None)
    c.same(want)
    assert torch.equal(c.codes, first[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_append_of_unaligned_views(dt, shift):
    B, H, T, D = 2, 2, 9, 80
    c = Cache(B, H, 64, D, 16, 16)
    c.fill([3, 20])
    flat = torch.randn(2 * B * H * T * (D + 1) + 16, generator=c.gen, device=DEV).to(TORCH[dt])
    k, v = flat[shift: shift + 2 * B * H * T * (D + 1)].view(2, B, H, T, D + 1)[..., :D]
    want = c.expected([3, 20], [T, T], k, v)
    c.append([3, 20], [T, T], k, v)
    c.same(want)


def test_token_by_token_grows_without_drift():
    """Blocks that grow token by token: exact against the definition, and every value stays within half a step of its
    own (2^-4 of it) or of the block's smallest (2^-10 of the final scale)."""
    B, H, C, D, block = 2, 2, 64, 64, 32
    c = Cache(B, H, C, D, block)
    x = torch.randn((2, B, H, C, D), generator=c.gen, device=DEV)
    x = (x * torch.exp2(torch.arange(C, device=DEV) % block / 2.0)[:, None]).bfloat16()
    for t in range(C):
        k, v = x[:, :, :, t: t + 1]
        want = c.expected([t] * B, [1] * B, k, v)
        c.append([t] * B, [1] * B, k, v, ragged=False)
        c.same(want)
    for plane in (0, 1):
        for b in range(B):
            codes, scales = c.row(plane, b)
            wide = scales.repeat_interleave(block, 1)[:, :C, None]
            off = (codes * wide - x[plane, b].double()).abs()
            # a code is off by half a step of 2^-3 of its value at first; below 2^-6 of the scale each doubling of the
            # scale rounds to steps of 2^-9, halves that add up to less than one step
            assert bool((off <= 2.0 ** -4 * x[plane, b].double().abs() * (1 + 2.0 ** -20) + 2.0 ** -9 * wide).all())


def test_values_at_the_border():
    """Zeros, values below every code, the smallest scale, the largest numbers, infinities and NaN: each in its block."""
    B, H, D, block = 1, 8, 16, 16
    c = Cache(B, H, 48, D, block)
    k = torch.randn((B, H, 40, D), generator=c.gen, device=DEV)
    k[0, 0] = 0
    k[0, 1, :16] *= 1e-38
    k[0, 2] = torch.where(k[0, 2] > 0, 3.3e38, -1e-3)
    k[0, 3, 3, 3] = float("inf")
    k[0, 4, 20, 1] = float("nan")
    k[0, 5, 0, 0] = -float("inf")
    k[0, 6, :20] = 0                       # a block that is 0 at first
    k[0, 7] = 2.0 ** -130
    k[0, 7, :, 0] = 1.0
    v = k.flip(1).contiguous()
    want = c.expected([0], [20], k[:, :, :20], v[:, :, :20])
    c.append([0], [20], k[:, :, :20], v[:, :, :20])
    c.same(want)
    assert math.isnan(float(c.scales[0, 0, 3, 0])) and not math.isnan(float(c.scales[0, 0, 3, 1]))
    assert float(c.scales[0, 0, 0, 0]) == 0 and float(c.scales[0, 0, 1, 0]) == fu.LEAST
    want = c.expected([20], [20], k[:, :, 20:], v[:, :, 20:])
    c.append([20], [20], k[:, :, 20:], v[:, :, 20:])
    c.same(want)
    assert math.isnan(float(c.scales[0, 0, 4, 1])) and float(c.scales[0, 0, 6, 1]) > 0
    k[0, 3] = 1.0                          # begun anew
    want = c.expected([0], [4], k[:, :, :4], v[:, :, :4])
    c.append([0], [4], k[:, :, :4], v[:, :, :4])
    c.same(want)
    assert not math.isnan(float(c.scales[0, 0, 3, 0]))


def test_append_reads_positions_and_counts_on_the_device():
    """A captured append replays with what it finds: other positions, counts past the call's and places past the
    cache, which are left out."""
    B, H, D, T = 3, 2, 64, 4
    c = Cache(B, H, 64, D, 16, 16)
    c.fill([0, 0, 40])
    k, v = torch.randn((2, B, H, T, D), generator=c.gen, device=DEV)
    pos, cnt = dev(np.array([0, 0, 0], np.int32)), dev(np.array([4, 4, 4], np.int32))
    host = np.zeros(3, np.int32), np.full(3, 4, np.int32)
    call = lambda: ol.ol_fp8kv_append(c.desc, c.codes, ol.OL_F32, T, k, v, host[0], pos, host[1], cnt)  # noqa: E731
    keep = c.codes.clone(), c.scales.clone()
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.codes.copy_(keep[0])
    c.scales.copy_(keep[1])
    pos.copy_(dev(np.array([62, 64, 40], np.int32)))  # row 0: two places in the cache; row 1: none
    cnt.copy_(dev(np.array([4, 4, 3], np.int32)))
    want = c.expected([62, 0, 40], [2, 0, 3], k, v)
    graph.replay()
    c.same(want)
    c.codes.copy_(keep[0])
    c.scales.copy_(keep[1])
    pos.copy_(dev(np.array([-1, 0, 40], np.int32)))
    cnt.copy_(dev(np.array([4, 5, -3], np.int32)))
    graph.replay()
    c.same(keep)


# -------------------------------------------------------------------------- read

# dtype, B, H, C, D, block, page, T, start, counts
READS = [
    ("bf16", 1, 1, 64, 128, 16, 0, 1, [0], None), ("bf16", 3, 2, 100, 128, 16, 16, 50, [5, 16, 31], [50, 0, 7]),
    ("bf16", 2, 4, 300, 64, 64, 64, 200, [7, 100], [193, 200]), ("bf16", 2, 1, 300, 256, 128, 0, 300, [0, 0], None),
    ("f32", 2, 3, 77, 80, 16, 0, 33, [44, 1], None), ("f32", 2, 2, 260, 256, 128, 128, 129, [130, 0], [128, 129]),
    ("f32", 1, 1, 17, 16, 32, 0, 17, [0], None), ("bf16", 2, 2, 40, 48, 32, 32, 40, [0, 0], None),
]


@pytest.mark.parametrize("shift", [0, 1], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("case", READS, ids=lambda c: "-".join(map(str, c[:8])))
def test_read_is_exact(case, shift):
    dt, B, H, C, D, block, page, T, start, counts = case
    n = [T] * B if counts is None else counts
    c = Cache(B, H, C, D, block, page)
    c.fill([s + m for s, m in zip(start, n)])
    c.scales[0, 0, 0, 0] = 0.0
    es = TORCH[dt].itemsize
    buf, payload = guarded((2 * B * H * T * D + 16) * es)
    flat = payload.view(TORCH[dt]).fill_(-7.0)
    out = flat[shift: shift + 2 * B * H * T * D].view(B, T, 2 * H, D).transpose(1, 2)
    k, v = out.chunk(2, dim=1)
    args = (np.array(start, np.int32), dev(np.array(start, np.int32)),
            None if counts is None else np.array(n, np.int32), None if counts is None else dev(np.array(n, np.int32)))
    want = out.clone()
    for plane in (0, 1):
        for b in range(B):
            codes, scales = c.row(plane, b)
            value = (codes.float() * scales.float().repeat_interleave(block, 1)[:, : codes.shape[1], None])
            want[b, plane * H: (plane + 1) * H, : n[b]] = value[:, start[b]: start[b] + n[b]].to(TORCH[dt])
    ol.ol_fp8kv_read(c.desc, CODE[TORCH[dt]], T, k, None, *args)
    torch.cuda.synchronize()
    assert torch.equal(k, want[:, :H]) and bool((v == -7).all())
    k.fill_(-7.0)
    ol.ol_fp8kv_read(c.desc, CODE[TORCH[dt]], T, None, v, *args)
    torch.cuda.synchronize()
    assert torch.equal(v, want[:, H:]) and bool((k == -7).all())
    ol.ol_fp8kv_read(c.desc, CODE[TORCH[dt]], T, k, v, *args)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((flat[:shift] == -7).all()) and bool((flat[shift + out.numel():] == -7).all()) and canaries_intact(buf)


# --------------------------------------------------------------------- attention

class Attention:
    def __init__(self, dt, B, Hq, H, D, block, page, T, lens, counts=None, window=-1, out=None, seed=1, spare=3,
                 spread=0.5):
        self.dtype, self.Hq, self.T, self.window = TORCH[dt], Hq, T, window
        self.lens = np.array(lens, np.int32)
        self.ragged = counts is not None
        self.counts = np.full(B, T, np.int32) if counts is None else np.array(counts, np.int32)
        self.out_dtype = TORCH[out or dt]
        self.c = c = Cache(B, H, max(int(self.lens.max()), 1) + spare, D, block, page, seed)
        c.fill(self.lens, spread)
        self.q = torch.randn((B, Hq, T, D), generator=c.gen, device=DEV).to(self.dtype)
        self.lens_d, self.counts_d = dev(self.lens), dev(self.counts)
        self.ws_bytes = ol.ol_workspace_size_fp8kv(B, Hq, H, D, T)
        self.ws_buf, self.ws = guarded(self.ws_bytes)
        ol.ol_workspace_init(self.ws, self.ws_bytes)
        self.out_buf, payload = guarded(self.q.numel() * self.out_dtype.itemsize)
        self.out = payload.view(self.out_dtype).view(self.q.shape).fill_(-77.0)
        self.wide = self.dtype == torch.float32

    def call(self, scale=0.0, stream=None, out=None, ws=None):
        c = self.c
        ol.ol_fp8kv_attention(c.desc, CODE[self.dtype], self.q, self.Hq, self.T, self.lens, self.lens_d,
                              self.counts if self.ragged else None, self.counts_d if self.ragged else None, scale,
                              self.window, self.out if out is None else out, CODE[self.out_dtype],
                              self.ws if ws is None else ws, self.ws_bytes, stream=stream)

    def check(self, scale=None, lens=None, counts=None, status=ol.OL_DEVICE_OK):
        torch.cuda.synchronize()
        assert ol.ol_workspace_status(self.ws) == status
        c, D = self.c, self.c.D
        scale = 1 / math.sqrt(D) if scale is None else scale
        lens, counts = self.lens if lens is None else lens, self.counts if counts is None else counts
        G = self.Hq // c.H
        worst = 0.0
        for b in range(c.B):
            n, t = int(lens[b]), int(counts[b])
            assert bool((self.out[b, :, t:] == -77.0).all()), "an output past the row's count was written"
            if t == 0:
                continue
            ok = du.visible(n, t, None, None, self.window)
            (kc, ks), (vc, vs) = c.row(0, b), c.row(1, b)
            ks, vs = (x.repeat_interleave(c.block, 1)[:, :n] for x in (ks, vs))
            for g in range(c.H):
                q = self.q[b, g * G: (g + 1) * G, :t]
                want, *sizes = fu.attention(q, kc[g, :n], ks[g], vc[g, :n], vs[g], ok, scale)
                got = self.out[b, g * G: (g + 1) * G, :t].double()
                tol = fu.attention_tolerance(want, *sizes, D, n, self.out_dtype, self.wide)
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                off = ((got - want).abs() / tol)[~torch.isnan(want)]
                if off.numel():
                    worst = max(worst, float(off.max()))
        assert worst <= 1, f"{worst:.2f} of the bound"
        assert canaries_intact(self.out_buf) and canaries_intact(self.ws_buf)
        assert canaries_intact(c.codes_buf) and canaries_intact(c.scales_buf)


# dtype, B, Hq, H, D, block, page, T, lens, counts, window, out
SHAPES = [
    ("bf16", 1, 1, 1, 128, 16, 0, 1, [1], None, -1, None), ("bf16", 1, 28, 4, 128, 128, 0, 1, [4097], None, -1, None),
    ("bf16", 5, 8, 2, 128, 16, 16, 1, [1, 15, 16, 17, 129], None, -1, "f32"),
    ("bf16", 4, 8, 8, 128, 16, 16, 1, [128, 127, 1000, 3], None, -1, None),
    ("bf16", 3, 16, 2, 128, 32, 64, 4, [4, 300, 129], None, -1, None),
    ("bf16", 3, 32, 8, 128, 64, 0, 4, [500, 2000, 4], [4, 3, 0], -1, "f32"),
    ("bf16", 2, 28, 4, 128, 64, 64, 64, [900, 64], [64, 17], -1, None),
    ("bf16", 2, 8, 1, 128, 16, 16, 17, [40, 333], None, 20, None),
    ("bf16", 2, 8, 2, 128, 128, 128, 3, [1000, 700], None, 0, None),
    ("bf16", 3, 8, 2, 128, 16, 32, 1, [1000, 5, 200], None, 100, "f32"),
    ("bf16", 2, 4, 2, 64, 16, 0, 1, [777, 30], None, -1, None), ("bf16", 2, 14, 2, 64, 32, 32, 5, [300, 64], None, -1, "f32"),
    ("bf16", 2, 8, 1, 64, 64, 64, 33, [129, 2000], None, 150, None),
    ("bf16", 2, 4, 2, 80, 16, 16, 3, [100, 33], None, -1, None), ("bf16", 1, 4, 4, 256, 64, 0, 2, [300], None, 40, None),
    ("f32", 2, 8, 2, 128, 16, 16, 1, [513, 2], None, -1, None), ("f32", 2, 16, 2, 80, 32, 32, 5, [400, 100], [5, 2], 60, None),
    ("f32", 1, 4, 1, 64, 128, 0, 40, [200], None, -1, None), ("f32", 2, 2, 2, 256, 16, 16, 2, [90, 2], None, -1, "bf16"),
    ("f32", 3, 4, 2, 16, 16, 16, 2, [70, 2, 31], None, -1, None), ("f32", 2, 12, 4, 160, 32, 0, 9, [70, 200], None, -1, None),
    ("bf16", 40, 8, 2, 128, 16, 16, 1, list(range(1, 41)), None, -1, None),
    ("bf16", 3, 8, 2, 128, 16, 48, 2, [500, 49, 129], None, -1, None), ("bf16", 2, 8, 2, 64, 16, 80, 3, [700, 81], None, 333, None),
    ("bf16", 2, 8, 2, 128, 32, 256, 1, [1000, 257], None, -1, None), ("f32", 2, 8, 2, 128, 16, 48, 2, [200, 49], None, -1, None),
    ("bf16", 5, 8, 2, 128, 16, 16, 4, [0, 4, 700, 0, 33], [0, 4, 1, 0, 3], -1, None),
    ("f32", 3, 8, 2, 80, 16, 16, 4, [0, 4, 70], [0, 4, 1], -1, None),
    ("bf16", 3, 28, 4, 128, 32, 32, 512, [512, 600, 900], [512, 1, 77], -1, None),
    ("bf16", 2, 64, 1, 64, 64, 0, 7, [300, 1000], [7, 3], 64, "f32"), ("bf16", 33, 4, 4, 128, 16, 0, 1, [9] * 33, None, 3, None),
    # heads that the tensor cores take with zeros behind, and those of two halves
    ("bf16", 3, 8, 2, 16, 16, 16, 3, [50, 400, 3], None, -1, "f32"), ("bf16", 2, 28, 4, 48, 32, 0, 2, [131, 700], None, 90, None),
    ("bf16", 2, 16, 2, 80, 128, 0, 1, [1000, 129], None, -1, "f32"), ("bf16", 2, 8, 1, 96, 16, 48, 9, [300, 60], [9, 4], -1, None),
    ("bf16", 5, 8, 2, 112, 16, 16, 3, [0, 3, 700, 0, 33], [0, 3, 1, 0, 2], -1, "f32"),
    ("bf16", 2, 4, 2, 144, 16, 16, 2, [257, 31], None, -1, "f32"), ("bf16", 2, 8, 2, 160, 64, 64, 4, [600, 64], None, 130, None),
    ("bf16", 1, 28, 4, 256, 128, 0, 1, [4097], None, -1, "f32"), ("bf16", 4, 32, 8, 256, 16, 16, 1, [128, 127, 1000, 3], None, -1, None),
    ("bf16", 3, 28, 4, 256, 32, 32, 40, [512, 600, 90], [40, 1, 17], -1, None),
    ("bf16", 2, 16, 1, 240, 64, 128, 7, [900, 7], None, 20, "f32"),
    # fp32 queries: more columns than a unit has, long rows, heads of two halves
    ("f32", 1, 28, 4, 128, 128, 0, 1, [4097], None, -1, None), ("f32", 3, 32, 8, 128, 32, 64, 9, [500, 129, 9], [9, 0, 4], -1, None),
    ("f32", 2, 14, 2, 64, 64, 0, 33, [2000, 64], None, 150, None), ("f32", 2, 16, 2, 256, 16, 16, 5, [700, 77], [5, 3], -1, None),
    ("f32", 40, 4, 4, 112, 16, 16, 1, list(range(1, 41)), None, -1, "bf16"),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c[:8] + c[10:])))
def test_attention(case):
    a = Attention(*case)
    a.call()
    a.check()
    a.out.fill_(-77.0)
    a.call(scale=0.3)
    a.check(scale=0.3)


@pytest.mark.parametrize("Hq,H,D,T,seed", [(8, 8, 128, 1, 1), (28, 4, 128, 3, 2), (16, 2, 64, 9, 3), (12, 4, 96, 2, 4), (8, 2, 80, 3, 5),
                                           (8, 8, 256, 2, 6), (28, 4, 192, 3, 7)])
def test_drawn_rows(Hq, H, D, T, seed):
    """Batches past one warp's, of lengths and counts of every kind, in pages in any order."""
    rng = np.random.default_rng(seed)
    lens = np.minimum(np.exp(rng.uniform(0, 7.5, 50)).astype(np.int32), 1500)
    counts = np.minimum(rng.integers(0, T + 1, 50), lens).astype(np.int32)
    a = Attention("bf16" if D != 96 else "f32", 50, Hq, H, D, 16, 32, T, lens, counts, -1 if seed % 2 else 100, seed=seed)
    a.call()
    a.check()


def test_shares_of_the_pool():
    """Rows long enough that the last tiles go to whoever is done first: right, and the same bits every time."""
    lens = [11000 + 37 * b for b in range(30)]  # 90 tiles a row and head: more than 64 for each of 304 CTAs
    a = Attention("bf16", 30, 32, 8, 128, 128, 0, 1, lens, out="f32")
    a.call()
    first = a.out.clone()
    for _ in range(4):
        a.out.fill_(-77.0)
        a.call()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first)
    for b in (0, 13, 29):  # against the definition
        ok = du.visible(lens[b], 1, None, None, -1)
        (kc, ks), (vc, vs) = a.c.row(0, b), a.c.row(1, b)
        ks, vs = (x.repeat_interleave(128, 1)[:, : lens[b]] for x in (ks, vs))
        for g in range(8):
            want, *sizes = fu.attention(a.q[b, g * 4: g * 4 + 4], kc[g, : lens[b]], ks[g], vc[g, : lens[b]], vs[g], ok,
                                        128 ** -0.5)
            tol = fu.attention_tolerance(want, *sizes, 128, lens[b], torch.float32, False)
            assert bool(((first[b, g * 4: g * 4 + 4].double() - want).abs() <= tol).all())
    assert ol.ol_workspace_status(a.ws) == ol.OL_DEVICE_OK


@pytest.mark.parametrize("D,C", [(128, 1 << 25), (16, 1 << 30)])
def test_past_32_bit_offsets(D, C):
    """Codes past 2^32 bytes, and (heads of 16) more than 2^31 vectors: append, read back, attention at a cache's end."""
    H, T, block, window = 2 if D == 128 else 1, 3, 128, 200
    if torch.cuda.mem_get_info()[0] < 2 * H * C * D * 1.3:
        pytest.skip("no room")
    c = Cache.__new__(Cache)
    c.B, c.H, c.D, c.block, c.page, c.C, c.table, c.table_d = 1, H, D, block, 0, C, None, None
    c.gen = torch.Generator(device=DEV).manual_seed(3)
    c.codes = torch.empty((2, 1, H, C, D), dtype=torch.uint8, device=DEV)
    c.scales = torch.empty((2, 1, H, C // block), device=DEV)
    c.desc = ol.fp8_kv(c.codes, c.scales, block=block)
    first = C - 260
    at = first // block * block
    k, v = torch.randn((2, 1, H, 260, D), generator=c.gen, device=DEV).bfloat16()
    c.scales[..., at // block] = 1.0
    c.append([first], [260], k, v, ragged=False)
    want = []
    for plane, x in ((0, k), (1, v)):
        tail = c.codes[plane, 0, :, at:].view(E4M3).double()
        scales = c.scales[plane, 0, :, at // block:].double()
        for g in range(H):
            codes, s = tail[g].clone(), torch.ones_like(scales[g])
            fu.append_row(codes, s, block, first - at, x[0, g].double())
            assert torch.equal(codes[first - at:], tail[g, first - at:]) and torch.equal(s, scales[g])
        want.append((tail, scales))
    out = torch.empty((2, 1, H, 260, D), device=DEV)
    start = np.array([first], np.int32)
    ol.ol_fp8kv_read(c.desc, ol.OL_F32, 260, out[0], out[1], start, dev(start))
    for plane in (0, 1):
        values = (want[plane][0].float() * want[plane][1].float().repeat_interleave(block, 1)[..., None])[:, first - at:]
        assert torch.equal(out[plane, 0], values)
    lens = np.array([C], np.int32)
    for dtype in (torch.bfloat16, torch.float32):
        q = torch.randn((1, 2 * H, T, D), generator=c.gen, device=DEV).to(dtype)
        y = torch.empty_like(q)
        n = ol.ol_workspace_size_fp8kv(1, 2 * H, H, D, T)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        ol.ol_workspace_init(ws, n)
        ol.ol_fp8kv_attention(c.desc, CODE[dtype], q, 2 * H, T, lens, dev(lens), None, None, 0.0, window, y, CODE[dtype], ws, n)
        assert ol.ol_workspace_status(ws) == ol.OL_DEVICE_OK
        m = C - at
        ok = du.visible(C - at, T, None, None, window)
        for g in range(H):
            wide = [s[g].repeat_interleave(block)[:m] for _, s in want]
            exact, *sizes = fu.attention(q[0, 2 * g: 2 * g + 2], want[0][0][g], wide[0], want[1][0][g], wide[1], ok, D ** -0.5)
            tol = fu.attention_tolerance(exact, *sizes, D, m, dtype, dtype == torch.float32)
            assert bool(((y[0, 2 * g: 2 * g + 2].double() - exact).abs() <= tol).all())


def test_scales_that_no_append_writes():
    """A negative or infinite scale under an append makes its block NaN, and ends."""
    c = Cache(1, 3, 32, 64, 16)
    c.fill([8])
    c.scales[:, 0, 0, 0], c.scales[:, 0, 1, 0], c.scales[:, 0, 2, 0] = -1.0, float("inf"), 1e-44
    k, v = torch.randn((2, 1, 3, 2, 64), generator=c.gen, device=DEV)
    c.append([8], [2], k, v)
    torch.cuda.synchronize()
    assert bool(torch.isnan(c.scales[:, 0, :2, 0]).all())
    grown = c.scales[:, 0, 2, 0].double()
    most = torch.stack((k, v))[:, 0, 2].abs().amax((1, 2)).double()
    assert bool((448 * grown >= most * (1 - 2.0 ** -23)).all()) and bool((448 * grown < 2.1 * most).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scales_far_apart_zero_and_small(dt):
    """Blocks whose scales differ by many orders, of zero, and at the smallest: weights and sums keep their share."""
    a = Attention(dt, 2, 8, 2, 128, 16, 16, 3, [700, 130], spread=3.0)
    a.c.scales[1, :, :, :] = torch.where(torch.rand(a.c.scales[1].shape, generator=a.c.gen, device=DEV) < 0.2, 0.0,
                                         a.c.scales[1])
    a.c.codes[1][(a.c.scales[1] == 0).repeat_interleave(16, 2)] = 0
    a.call()
    a.check()
    tiny = Attention(dt, 1, 4, 1, 128, 16, 0, 1, [200])
    tiny.c.scales[1] = fu.LEAST
    tiny.call()
    tiny.check()
    tiny.c.scales[1] = 0.0
    tiny.c.codes[1] = 0
    tiny.out.fill_(-77.0)
    tiny.call()
    torch.cuda.synchronize()
    assert bool((tiny.out == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scales_of_v_from_the_least_to_large(dt):
    """Blocks of V from 2^-80 to 2^60, and of scale 0 whatever their codes: no token loses its part of the sum."""
    a = Attention(dt, 2, 8, 2, 128, 16, 16, 3, [700, 130], out="f32")
    some = torch.tensor([2.0 ** -80, 2.0 ** -40, 1.0, 2.0 ** 40, 2.0 ** 60, 0.0], device=DEV)
    a.c.scales[1] = some[torch.randint(0, 6, a.c.scales[1].shape, generator=a.c.gen, device=DEV)]
    a.call()
    a.check()
    a.c.scales[1] = some[torch.randint(0, 2, a.c.scales[1].shape, generator=a.c.gen, device=DEV) * 5]  # 2^-80 and 0
    a.out.fill_(-77.0)
    a.call()
    a.check()


def test_a_cache_of_no_tokens():
    a = Attention("bf16", 2, 8, 2, 128, 16, 0, 3, [5, 7], [3, 3])
    a.c.desc.capacity = 0
    a.lens[:], a.counts[:] = 0, 0
    a.call()
    torch.cuda.synchronize()
    assert bool((a.out == -77.0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_heavy_token_among_many(dt):
    """One token with most of the weight and thousands that share the rest: none of their weight is lost."""
    n = 8000
    a = Attention(dt, 1, 4, 1, 128, 16, 0, 1, [n], out="f32", spread=0.0)
    q = a.q[0, :, 0].double()
    a.q[0, 1:] = a.q[0, :1]
    a.c.codes[0, 0, 0, :n] = 0
    lead = q[0] * 20
    a.c.codes[0, 0, 0, 4000] = fu.e4m3(lead * (11.0 / float(lead @ q[0] * 128 ** -0.5) * 140)).to(E4M3).view(torch.uint8)
    a.c.codes[1, 0, 0, :n] = fu.e4m3(torch.full((n, 128), 100.0, device=DEV, dtype=torch.float64)).to(E4M3).view(torch.uint8)
    a.c.codes[1, 0, 0, 4000] = 0
    a.call()
    a.check()


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_nan_blocks_reach_only_those_that_see_them(dt, D):
    a = Attention(dt, 2, 4, 1, D, 16, 16, 40, [100, 300], window=64)
    c = a.c
    for plane, b, block in ((0, 0, 5), (1, 1, 17)):
        p = int(c.table[b, block])
        c.scales[plane, p, 0, 0] = float("nan")
    a.call()
    a.check()
    assert bool(torch.isnan(a.out).any()) and not bool(torch.isnan(a.out).all())


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_what_no_query_sees_is_not_read(dt, D):
    """Below a window and past a row: NaN codes and scales, and table entries that name no page."""
    a = Attention(dt, 2, 4, 2, D, 16, 16, 2, [500, 333], window=50, spare=40)
    c = a.c
    for b, n in enumerate(a.lens.tolist()):
        first = max(0, n - a.T - a.window) // 16
        for i in list(range(first)) + list(range(-(-n // 16), c.table.shape[1])):
            p = int(c.table[b, i])
            c.codes[:, p] = 0x7F
            c.scales[:, p] = float("nan")
    a.call()
    a.check()
    good = a.out.clone()
    table = c.table.copy()
    for b, n in enumerate(a.lens.tolist()):
        first = max(0, n - a.T - a.window) // 16
        table[b, :first] = -1
        table[b, -(-n // 16):] = 1 << 20
    c.table_d.copy_(dev(table))
    desc, c.desc = c.desc, ol.fp8_kv(c.codes, c.scales, c.table_d, table, block=16)
    a.out.fill_(-77.0)
    a.call()
    torch.cuda.synchronize()
    assert torch.equal(a.out, good) and ol.ol_workspace_status(a.ws) == ol.OL_DEVICE_OK
    c.desc = desc


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_lengths_on_the_device(dt):
    """A captured call replays with the lengths, counts and queries it finds; lengths past the capacity and counts past
    the call's are clamped and recorded."""
    a = Attention(dt, 3, 8, 2, 128, 16, 16, 4, [600, 600, 600], [4, 4, 4])
    a.call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call()
    for lens, counts in (([600, 17, 4], [1, 4, 0]), ([1, 600, 128], [1, 2, 3])):
        a.lens_d.copy_(dev(np.array(lens, np.int32)))
        a.counts_d.copy_(dev(np.array(counts, np.int32)))
        a.q.normal_(generator=a.c.gen)
        a.out.fill_(-77.0)
        graph.replay()
        a.check(lens=lens, counts=counts)
    a.lens_d.copy_(dev(np.array([10 ** 6, -4, 600], np.int32)))
    a.counts_d.copy_(dev(np.array([4, 2, 9], np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(a.ws) == ol.OL_DEVICE_GUARD
    a.c.table_d[0, 0] = -1
    a.lens_d.copy_(dev(np.array([600, 600, 600], np.int32)))
    a.counts_d.copy_(dev(np.array([4, 4, 4], np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(a.ws) == ol.OL_DEVICE_GUARD
    assert canaries_intact(a.out_buf) and canaries_intact(a.ws_buf)


def test_the_same_call_gives_the_same_bits():
    a = Attention("bf16", 6, 8, 2, 128, 16, 16, 2, [3000, 1, 129, 800, 2, 77], [2, 1, 2, 2, 1, 2], out="f32")
    a.call()
    first = a.out.clone()
    for _ in range(5):
        a.out.fill_(-77.0)
        a.call()
        assert torch.equal(a.out, first)


def test_two_streams_with_their_own_workspaces():
    a = Attention("bf16", 4, 8, 2, 128, 32, 32, 1, [3000, 40, 700, 1500])
    a.call()
    torch.cuda.synchronize()
    first = a.out.clone()
    ws = torch.empty(a.ws_bytes, dtype=torch.uint8, device=DEV)
    ol.ol_workspace_init(ws, a.ws_bytes)
    other, out = torch.cuda.Stream(), torch.empty_like(a.out)
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a.call()
        a.call(stream=other, out=out, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(a.out, first) and torch.equal(out, first)


def test_the_workspace_serves_a_tree_call_too():
    a = Attention("bf16", 2, 8, 2, 128, 16, 0, 3, [900, 400])
    dense = torch.randn((2, 2, 2, 512, 128), generator=a.c.gen, device=DEV).bfloat16()
    lens = np.array([500, 400], np.int32)
    out = torch.empty_like(a.q)
    for _ in range(3):
        ol.ol_tree_attention(ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(dense), a.q, 8, 3, lens, dev(lens), None, None, None,
                             None, 0.0, -1, out, ol.OL_BF16, a.ws, a.ws_bytes)
        a.call()
    a.check()


# ------------------------------------------------------ the operators as they are used

def test_the_pool_in_a_captured_call():
    """The shares' counter is 0 again after every replay, also of a graph with two calls."""
    a = Attention("f32", 16, 8, 8, 128, 64, 0, 1, [20000 + b for b in range(16)], seed=4)  # 156 tiles a row and head: 65 a CTA
    a.call()
    first = a.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call()
        a.call()
    for _ in range(3):
        a.out.fill_(-77.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, first)
    assert ol.ol_workspace_status(a.ws) == ol.OL_DEVICE_OK


@pytest.mark.parametrize("dt,D,window", [("bf16", 128, -1), ("f32", 64, 20), ("bf16", 256, -1)])
def test_a_captured_decode_step(dt, D, window):
    """Norms with rotation, append and attention in one graph: replayed with the positions it finds, it leaves the cache
    and gives the outputs of the calls one by one."""
    B, Hq, H, block, steps = 3, 8, 2, 16, 20
    start = [5, 40, 0]
    one, two = (Cache(B, H, 64, D, block, 16, seed=11) for _ in range(2))
    for c in (one, two):
        c.fill(start)
    assert torch.equal(one.codes, two.codes) and torch.equal(one.scales[~one.scales.isnan()], two.scales[~two.scales.isnan()])
    rope, norm, dtype = ol.rope(D, device=DEV), ol.head_norm(), TORCH[dt]
    qkv = torch.zeros((B, 1, Hq + 2 * H, D), device=DEV, dtype=dtype)
    q, k, v = qkv.transpose(1, 2).split((Hq, H, H), dim=1)
    qr, kr = torch.empty((B, Hq, 1, D), device=DEV, dtype=dtype), torch.empty((B, H, 1, D), device=DEV, dtype=dtype)
    at, lens = np.array(start, np.int32), np.array(start, np.int32) + 1
    at_d, lens_d = dev(at), dev(lens)
    n = ol.ol_workspace_size_fp8kv(B, Hq, H, D, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    ol.ol_workspace_init(ws, n)

    def step(c, out, at, lens):
        ol.ol_norm_rope_rows(rope, norm, CODE[dtype], B, 1, D, Hq, q, qr, H, k, kr, at_d, False)
        ol.ol_fp8kv_append(c.desc, c.codes, CODE[dtype], 1, kr, v, at, at_d)
        ol.ol_fp8kv_attention(c.desc, CODE[dtype], qr, Hq, 1, lens, lens_d, None, None, 0.0, window, out, CODE[dtype], ws, n)

    outs = [torch.empty((B, Hq, 1, D), device=DEV, dtype=dtype) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, outs[0], at, lens)
    for i in range(steps):
        qkv.normal_(generator=one.gen)
        at_d.copy_(dev(at + i))
        lens_d.copy_(dev(lens + i))
        graph.replay()
        step(two, outs[1], at + i, lens + i)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and not bool(outs[0].isnan().any())
    assert torch.equal(one.codes, two.codes)
    assert torch.equal(one.scales.nan_to_num(nan=-1.0), two.scales.nan_to_num(nan=-1.0))
    assert ol.ol_workspace_status(ws) == ol.OL_DEVICE_OK


@pytest.mark.parametrize("page", [0, 32])
def test_a_prompt_then_steps(page):
    """A projection's output normed and rotated, appended, attended: a ragged prompt in chunks, then single tokens; the
    cache is that of the definition, read back it gives the values, attention is that of the cache."""
    B, Hq, H, D, block, C = 3, 8, 2, 128, 32, 160
    c = Cache(B, H, C, D, block, page, seed=9)
    G = c.gen
    rope, freq = ol.rope(D, device=DEV), du.frequencies(D)
    qw, kw = (1 + 0.2 * torch.randn((2, D), generator=G, device=DEV)).bfloat16()
    norm = ol.head_norm(qw, kw, eps=1e-6)
    length = np.zeros(B, np.int32)
    for T, counts in ((64, [64, 33, 1]), (16, [16, 0, 16]), (1, [1, 1, 1]), (1, [1, 1, 1]), (1, [0, 1, 1])):
        counts = np.array(counts, np.int32)
        qkv = torch.randn((B, T, Hq + 2 * H, D), generator=G, device=DEV).bfloat16()
        q, k, v = qkv.transpose(1, 2).split((Hq, H, H), dim=1)
        at, counts_d = dev(length), dev(counts)
        positions = at[:, None, None] + torch.arange(T, device=DEV, dtype=torch.int32)
        wants = [fu.norm_rope(x, w, 0.0, 1e-6, positions, freq, 0) for x, w in ((q, qw), (k, kw))]
        ol.ol_norm_rope_rows(rope, norm, ol.OL_BF16, B, T, D, Hq, q, q, H, k, k, at, False)
        for x, (want, extent) in zip((q, k), wants):
            tol = fu.norm_tolerance(want, extent, torch.bfloat16, positions, freq)
            assert bool(((x.double() - want).abs() <= tol).all())
        want = c.expected(length, counts, k, v)
        ol.ol_fp8kv_append(c.desc, c.codes, ol.OL_BF16, T, k, v, length, at, counts, counts_d)
        c.same(want)
        length = (length + counts).astype(np.int32)
        a = Attention.__new__(Attention)
        a.c, a.dtype, a.out_dtype, a.Hq, a.T, a.window, a.ragged = c, torch.bfloat16, torch.bfloat16, Hq, T, -1, True
        a.lens, a.counts, a.lens_d, a.counts_d, a.wide = length, counts, dev(length), counts_d, False
        a.q = q.contiguous()
        a.ws_bytes = ol.ol_workspace_size_fp8kv(B, Hq, H, D, T)
        a.ws_buf, a.ws = guarded(a.ws_bytes)
        ol.ol_workspace_init(a.ws, a.ws_bytes)
        a.out_buf, payload = guarded(a.q.numel() * 2)
        a.out = payload.view(torch.bfloat16).view(a.q.shape).fill_(-77.0)
        a.call()
        a.check()
    k, v = torch.zeros((2, B, H, int(length.max()), D), device=DEV)
    ol.ol_fp8kv_read(c.desc, ol.OL_F32, int(length.max()), k, v, np.zeros(B, np.int32), dev(np.zeros(B, np.int32)),
                     length, dev(length))
    torch.cuda.synchronize()
    for b in range(B):
        codes, scales = c.row(0, b)
        n = int(length[b])
        assert torch.equal(k[b, :, :n], (codes.float() * scales.float().repeat_interleave(block, 1)[:, :C, None])[:, :n])
