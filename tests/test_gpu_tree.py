"""GPU parity of tree attention (ol_tree_attention) and of the accepted path's
move (ol_tree_keep) against a plain 64-bit form: contiguous and paged caches,
bf16 and fp32, head sizes and groups on both kernels, one to 512 nodes, rows
without prefix, without nodes, with hidden nodes, ragged counts, windows,
infinities and NaN in what is hidden, poison in every slot past a row, replayed
and concurrent calls, lengths and pages that disagree on the device."""
import math

import numpy as np
import pytest
import torch

import place_kv_cache_gb300 as ol
from tests import draft_util as du
from tests.gpu_util import DEV, canaries_intact, guarded

pytestmark = pytest.mark.gpu
CODE = {torch.float32: ol.OL_F32, torch.bfloat16: ol.OL_BF16}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


class Tree:
    """A cache of poisoned slots with the rows' tokens in place, q, trees and the call on them."""

    def __init__(self, dt, layout, B, Hq, H, D, page, nodes, lens, counts=None, window=-1, mask="tree", out=None,
                 seed=1, spare=3, positions=True):
        self.dtype, self.B, self.Hq, self.H, self.D, self.nodes, self.window = TORCH[dt], B, Hq, H, D, nodes, window
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.lens = np.array(lens, np.int32)
        self.counts = np.full(B, nodes, np.int32) if counts is None else np.array(counts, np.int32)
        self.ragged = counts is not None
        self.out_dtype = TORCH[out or dt]
        C = max(int(self.lens.max()), 1) + spare
        self.layout, self.page, self.table = layout, page, None
        if layout == "contiguous":
            shape = (2, B, H, C, D)
        else:
            M = -(-C // page)
            self.table = self.rng.permutation(B * M + 2)[: B * M].astype(np.int32).reshape(B, M)
            shape = (2, B * M + 2, H, page, D)
        self.cache = torch.full(shape, float("nan"), device=DEV, dtype=self.dtype)
        for b in range(B):
            n = int(self.lens[b])
            for plane in (0, 1):
                self.put(plane, b, torch.randn((H, n, D), generator=self.gen, device=DEV, dtype=self.dtype))
        self.q = torch.randn((B, Hq, nodes, D), generator=self.gen, device=DEV, dtype=self.dtype)
        if mask == "tree":
            self.sees, depth = du.random_trees(self.rng, B, nodes)
        elif mask == "random":  # any bits: rows that see nothing drafted, later tokens, not themselves
            self.sees, depth = self.rng.random((B, nodes, nodes)) < 0.3, self.rng.integers(0, 9, (B, nodes))
        elif mask == "empty":
            self.sees, depth = np.zeros((B, nodes, nodes), bool), np.zeros((B, nodes), np.int64)
        else:
            self.sees, depth = None, np.broadcast_to(np.arange(nodes), (B, nodes))
        self.at = ((self.lens - self.counts)[:, None] + depth).astype(np.int32) if positions else None
        self.mask = None if self.sees is None else torch.from_numpy(du.pack_mask(self.sees)).to(DEV)
        self.at_d = None if self.at is None else torch.from_numpy(self.at).to(DEV)
        self.lens_d, self.counts_d = torch.from_numpy(self.lens).to(DEV), torch.from_numpy(self.counts).to(DEV)
        if layout == "contiguous":
            self.code, self.desc = ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(self.cache, access=ol.OL_READ_ONLY)
        else:
            self.table_d = torch.from_numpy(self.table).to(DEV)
            self.code = ol.OL_LAYOUT_PAGED
            self.desc = ol.paged_kv(self.cache, self.table_d, self.table, access=ol.OL_READ_ONLY)
        self.ws_bytes = ol.ol_workspace_size_tree(B, Hq, H, D, nodes)
        self.ws_buf, self.ws = guarded(self.ws_bytes)
        ol.ol_workspace_init(self.ws, self.ws_bytes)
        self.out_buf, payload = guarded(B * Hq * nodes * D * (4 if self.out_dtype == torch.float32 else 2))
        self.out = payload.view(self.out_dtype).view(B, Hq, nodes, D)
        self.out.fill_(-77.0)

    def row(self, plane, b, n):
        if self.table is None:
            return self.cache[plane, b, :, :n]
        pages = [self.cache[plane, p] for p in self.table[b, : -(-n // self.page)].tolist()]
        return torch.cat(pages, 1)[:, :n] if pages else self.cache[plane, 0, :, :0]

    def put(self, plane, b, x, first=0):
        for t0 in range(0, x.shape[1], self.page or x.shape[1] or 1):
            part = x[:, t0: t0 + self.page] if self.page else x
            if self.page:
                assert first % self.page == 0
                self.cache[plane, int(self.table[b, (first + t0) // self.page]), :, : part.shape[1]] = part
            else:
                self.cache[plane, b, :, first: first + part.shape[1]] = part

    def token(self, plane, b, t):
        """View [Hkv, D] of one cached token."""
        return self.cache[plane, b, :, t] if self.table is None else \
            self.cache[plane, int(self.table[b, t // self.page]), :, t % self.page]

    def call(self, stream=None, scale=0.0):
        ol.ol_tree_attention(self.code, self.desc, self.q, self.Hq, self.nodes, self.lens, self.lens_d,
                             self.counts if self.ragged else None, self.counts_d if self.ragged else None, self.mask,
                             self.at_d, scale, self.window, self.out, CODE[self.out_dtype], self.ws, self.ws_bytes,
                             stream=stream)

    def check(self, scale=None, lens=None, counts=None, status=ol.OL_DEVICE_OK):
        torch.cuda.synchronize()
        assert ol.ol_workspace_status(self.ws) == status
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        lens, counts = self.lens if lens is None else lens, self.counts if counts is None else counts
        G = self.Hq // self.H
        for b in range(self.B):
            n, t = int(lens[b]), int(counts[b])
            assert bool((self.out[b, :, t:] == -77.0).all()), "an output past the row's count was written"
            if t == 0:
                continue
            ok = du.visible(n, t, None if self.sees is None else self.sees[b],
                            None if self.at is None else self.at[b], self.window)
            k, v = self.row(0, b, n), self.row(1, b, n)
            for g in range(self.H):
                q = self.q[b, g * G: (g + 1) * G, :t]
                want, pv, rms, size = du.tree_attention(q, k[g], v[g], ok, scale)
                got = self.out[b, g * G: (g + 1) * G, :t].double()
                weights = self.dtype == torch.bfloat16
                tol = du.tree_tolerance(want, pv, size, self.D, n, self.out_dtype, weights)
                fine = torch.isfinite(want)
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
                off = ((got - want).abs() - tol)[fine]
                assert not off.numel() or float(off.max()) <= 0, \
                    f"row {b} head {g}: {float(off.max()):.3e} more than the bound"
                if weights and bool(fine.all()):
                    # roundings of the weights are independent: their root mean square is at most 2^-8 / sqrt(3) of
                    # sqrt(sum p^2 v^2), the output's 2^-8 / sqrt(3) of itself; 2 covers the spread of a finite sample
                    # (and the fp32 part is added whole)
                    step = torch.finfo(self.out_dtype).eps / 2
                    rest = du.tree_tolerance(want, pv, size, self.D, n, torch.float64, False)
                    bound = 2 * ((2.0 ** -8 / 3 ** 0.5 * rms).norm() + (step / 3 ** 0.5 * want).norm()) + rest.norm()
                    assert float((got - want).norm()) <= float(bound)
        assert canaries_intact(self.out_buf) and canaries_intact(self.ws_buf)


CASES = [
    # dt, layout, B, Hq, Hkv, D, page, nodes, lens, counts, window, mask, out
    # --- bf16, the tensor-core kernel's head sizes
    ("bf16", "contiguous", 1, 1, 1, 128, 0, 1, [1]),
    ("bf16", "contiguous", 1, 28, 4, 128, 0, 8, [4097 + 8]),
    ("bf16", "contiguous", 3, 32, 8, 128, 0, 16, [16, 17, 700]),
    ("bf16", "contiguous", 2, 8, 8, 128, 0, 5, [127, 130]),
    ("bf16", "contiguous", 2, 16, 2, 64, 0, 63, [64, 513]),
    ("bf16", "contiguous", 2, 32, 8, 128, 0, 64, [300, 64]),
    ("bf16", "contiguous", 2, 14, 2, 128, 0, 65, [65, 400]),
    ("bf16", "contiguous", 1, 16, 1, 64, 0, 200, [1111]),
    ("bf16", "contiguous", 1, 4, 2, 128, 0, 512, [512 + 77]),
    ("bf16", "contiguous", 5, 12, 4, 128, 0, 7, [7, 128, 129, 255, 1000], [7, 0, 1, 3, 6]),
    ("bf16", "contiguous", 3, 8, 2, 128, 0, 9, [0, 9, 5], [0, 9, 5]),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 12, [12, 600], None, -1, "random"),
    ("bf16", "contiguous", 3, 8, 2, 128, 0, 6, [6, 128, 600], None, -1, "empty"),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 33, [33, 600], None, -1, "chain"),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 10, [500, 60], None, 0, "tree"),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 10, [500, 600], None, 3, "tree"),
    ("bf16", "contiguous", 3, 8, 2, 64, 0, 10, [500, 200, 10], [10, 2, 9], 150, "random"),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 40, [500, 60], None, 20, "chain"),
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 4, [300, 60], None, -1, "tree", "f32"),
    ("bf16", "paged", 3, 32, 8, 128, 16, 16, [16, 100, 1000]),
    ("bf16", "paged", 2, 28, 4, 128, 64, 256, [256, 900]),
    ("bf16", "paged", 3, 8, 2, 128, 48, 7, [7, 130, 500], [3, 7, 0]),
    ("bf16", "paged", 2, 8, 2, 64, 128, 20, [333, 20]),
    ("bf16", "paged", 2, 8, 2, 128, 256, 20, [600, 20]),
    ("bf16", "paged", 2, 8, 2, 128, 16, 10, [500, 300], None, 100, "tree"),
    ("bf16", "paged", 40, 8, 2, 128, 16, 3, list(range(3, 203, 5))),
    ("bf16", "contiguous", 170, 4, 4, 64, 0, 2, [2 + (7 * i) % 300 for i in range(170)]),
    # many tiles and several segments a CTA, one and two query tiles, both head sizes
    ("bf16", "contiguous", 4, 32, 8, 128, 0, 64, [6000, 1000, 4001, 6500]),
    ("bf16", "paged", 4, 32, 8, 128, 16, 64, [6000, 1000, 4001, 6500]),
    ("bf16", "paged", 4, 32, 8, 128, 16, 16, [6000, 1000, 4001, 6500], [16, 3, 16, 1]),
    ("bf16", "contiguous", 4, 32, 8, 64, 0, 40, [6000, 1000, 4001, 6500]),
    ("bf16", "contiguous", 4, 32, 8, 64, 0, 9, [6000, 1000, 4001, 6500]),
    ("bf16", "paged", 60, 28, 4, 128, 32, 64, [64 + (37 * i) % 700 for i in range(60)]),
    ("bf16", "paged", 60, 28, 4, 128, 32, 6, [6 + (37 * i) % 700 for i in range(60)]),
    # --- CUDA cores
    ("bf16", "paged", 2, 8, 2, 128, 8, 10, [100, 33]),
    ("bf16", "paged", 2, 8, 2, 128, 7, 10, [100, 33]),
    ("bf16", "contiguous", 2, 6, 2, 96, 0, 11, [100, 11]),
    ("bf16", "contiguous", 1, 6, 2, 256, 0, 11, [257]),
    ("bf16", "contiguous", 1, 3, 1, 20, 0, 4, [77]),
    ("f32", "contiguous", 1, 1, 1, 4, 0, 1, [1]),
    ("f32", "contiguous", 2, 6, 3, 5, 0, 3, [40, 3]),
    ("f32", "contiguous", 3, 28, 4, 128, 0, 8, [8, 500, 1500], [8, 3, 0]),
    ("f32", "paged", 2, 16, 2, 80, 16, 33, [400, 33], None, -1, "random"),
    ("f32", "paged", 2, 16, 2, 64, 5, 40, [400, 40], None, 50, "tree", "bf16"),
    ("f32", "contiguous", 2, 4, 1, 256, 0, 70, [200, 70], None, 10, "chain"),
    ("f32", "contiguous", 2, 4, 1, 192, 0, 6, [200, 6], None, -1, "empty"),
    # every CTA with several segments, units of one and of two and more row groups
    ("f32", "paged", 16, 16, 4, 128, 16, 24, [24 + (211 * i) % 2500 for i in range(16)]),
    ("f32", "contiguous", 30, 8, 4, 64, 0, 7, [7 + (97 * i) % 1500 for i in range(30)], [i % 8 for i in range(30)]),
    ("bf16", "paged", 12, 16, 4, 96, 32, 20, [20 + (211 * i) % 2500 for i in range(12)], None, 300, "random"),
    # the widest trees on both kernels, any mask, a window among the drafted tokens
    ("bf16", "contiguous", 2, 8, 2, 128, 0, 512, [512, 1500], [512, 300], 64, "random"),
    ("bf16", "paged", 2, 2, 2, 64, 16, 511, [511, 900], None, 100, "chain"),
    ("f32", "contiguous", 1, 2, 1, 64, 0, 512, [700], None, -1, "random"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:8]) + ("" if len(c) < 11 else
                                                                                       f"-w{c[10]}-{c[11]}"))
def test_tree_attention(case):
    t = Tree(*case)
    t.call()
    t.check()


@pytest.mark.parametrize("seed", range(60))
def test_random_trees(seed):
    """Shapes drawn over both kernels: heads, pages, groups, lengths, counts, windows, masks, output types."""
    rng = np.random.default_rng(1000 + seed)
    dt = "f32" if rng.random() < 0.25 else "bf16"
    D = int(rng.choice([64, 128, 128, 64, 96, 40] if dt == "bf16" else [64, 128, 33]))
    layout, page = ("contiguous", 0) if rng.random() < 0.5 else ("paged", int(rng.choice([16, 16, 32, 48, 64, 128, 10])))
    H, G = int(rng.integers(1, 6)), int(rng.integers(1, 9))
    nodes = int(rng.choice([1, 2, 5, 8, 17, 33, 64, 90]))
    B = int(rng.integers(1, 41 if nodes < 20 else 7))
    counts = None
    if rng.random() < 0.5:
        counts = rng.integers(0, nodes + 1, B)
    prefix = rng.integers(0, int(rng.choice([3, 140, 1500])), B)
    lens = prefix + (nodes if counts is None else counts)
    window = int(rng.choice([-1, -1, 0, 7, 130, 1000]))
    t = Tree(dt, layout, B, H * G, H, D, page, nodes, lens, counts, window, str(rng.choice(["tree", "random", "chain"])),
             str(rng.choice(["f32", "bf16"])), seed=seed)
    t.call()
    t.check()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", [
    # layout, B, Hq, H, D, page, nodes, lens: rows of few tokens, where a weight's rounding is not averaged away
    ("contiguous", 3, 8, 8, 128, 0, 1, [2, 3, 9]),
    ("contiguous", 4, 28, 4, 128, 0, 8, [8, 11, 30, 90]),
    ("contiguous", 3, 16, 2, 64, 0, 7, [7, 9, 140]),
    ("contiguous", 3, 32, 8, 128, 0, 64, [64, 70, 130]),
    ("contiguous", 2, 16, 2, 64, 0, 33, [33, 36]),
    ("paged", 4, 8, 2, 128, 16, 5, [5, 7, 20, 140]),
    ("paged", 3, 32, 8, 128, 16, 40, [40, 43, 150]),
    ("paged", 3, 28, 4, 128, 64, 50, [50, 60, 131]),
    ("paged", 2, 8, 2, 64, 128, 6, [6, 150]),
], ids=lambda c: "-".join(map(str, c[:7])))
def test_weights_of_the_tensor_core_kernel_keep_16_bits(case, out):
    """V is multiplied by a weight's leading 8 bits and by the bf16 of its remainder, as in the decode and chunked steps:
    of a weight in [1, 2) the remainder is below 2^-7, where bf16 numbers lie 2^-15 apart: off by at most 2^-16."""
    layout, B, Hq, H, D, page, nodes, lens = case
    t = Tree("bf16", layout, B, Hq, H, D, page, nodes, lens, out=out, seed=23)
    t.call()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK
    G, step = Hq // H, torch.finfo(t.out_dtype).eps / 2
    for b in range(B):
        n = int(t.lens[b])
        ok = du.visible(n, nodes, t.sees[b], t.at[b], -1)
        for g in range(H):
            want, pv, _, size = du.tree_attention(t.q[b, g * G: (g + 1) * G], t.row(0, b, n)[g], t.row(1, b, n)[g], ok,
                                                  D ** -0.5)
            tol = du.tree_tolerance(want, pv, size, D, n, torch.float64, False) + 2.0 ** -16 * pv
            tol = tol + step * (want.abs() + tol)
            off = (t.out[b, g * G: (g + 1) * G].double() - want).abs() - tol
            assert float(off.max()) <= 0, f"row {b} head {g}: {float(off.max()):.3e} more than the bound"


def test_tree_attention_explicit_scale_and_no_positions():
    t = Tree("bf16", "contiguous", 2, 8, 2, 128, 0, 9, [200, 100], positions=False)
    t.call(scale=0.25)
    t.check(scale=0.25)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 128)])
def test_hidden_infinities_and_nan(dt, D):
    """K and V of a drafted token that some nodes see and others do not: only those that see it are touched."""
    t = Tree(dt, "paged", 2, 8, 2, D, 16, 12, [150, 60], seed=9)
    for b in range(2):
        first = int(t.lens[b]) - 12
        t.sees[b, :, 4:9] = False
        t.sees[b, 3, 4], t.sees[b, 5, 5], t.sees[b, 7, 6], t.sees[b, 8, 7] = True, True, True, True
        t.token(1, b, first + 4)[:, 3] = float("inf")
        t.token(1, b, first + 5)[:, D - 1] = float("nan")
        t.token(1, b, first + 6)[:] = -float("inf")
        t.token(1, b, first + 7)[:, 0] = float("inf")
        t.token(0, b, first + 8)[:] = float("nan")      # seen by none
        t.token(1, b, first + 8)[:] = float("nan")
    t.mask = torch.from_numpy(du.pack_mask(t.sees)).to(DEV)
    t.call()
    t.check()
    assert not torch.isfinite(t.out[:, :, 3, 3]).any() and torch.isfinite(t.out[:, :, 0]).all()


@pytest.mark.parametrize("far", [0, 1, 300])
@pytest.mark.parametrize("dt,layout,page,H,Hq,D,nodes", [
    ("bf16", "contiguous", 0, 2, 8, 128, 12), ("bf16", "paged", 16, 2, 8, 128, 12), ("bf16", "paged", 64, 2, 8, 64, 9),
    ("bf16", "contiguous", 0, 2, 8, 128, 64), ("bf16", "paged", 16, 1, 8, 128, 70), ("bf16", "contiguous", 0, 2, 8, 96, 12),
    ("f32", "contiguous", 0, 2, 8, 128, 12), ("f32", "paged", 16, 2, 4, 80, 20)])
def test_infinities_and_nan_of_the_prefix_behind_a_window(dt, layout, page, H, Hq, D, nodes, far):
    """Prefix tokens that the window hides from some nodes, or from all: only those that see them are touched.
    Positions lie near one another, `far` behind the prefix, or over 300 tokens (several tiles)."""
    t = Tree(dt, layout, 3, Hq, H, D, page, nodes, [nodes + 900, nodes + 433, nodes + 150], window=200, seed=51)
    prefix = t.lens - nodes
    if far == 300:
        t.at = (prefix[:, None] + t.rng.integers(0, far, (3, nodes))).astype(np.int32)
        t.at[:, 0] = prefix
    else:
        t.at = t.at + far
    t.at_d = torch.from_numpy(t.at).to(DEV)
    touched = 0
    for b in range(3):
        low = np.maximum(t.at[b].astype(np.int64) - 200, 0)  # each node's lowest prefix token
        for x in sorted({int(low.min()) - 1, int(low.min()), int(np.median(low)), int(low.max()) - 1}):
            if 0 <= x < min(int(low.max()), int(prefix[b])):  # hidden from some node
                t.token(1, b, x)[:, x % D] = float("inf") if x % 2 else float("nan")
                if x < low.min():
                    t.token(0, b, x)[:] = float("nan")
                    t.token(1, b, x)[:] = float("nan")
                touched += 1
        x = int(prefix[b]) - 200
        if 0 <= x < low.min():                               # seen by none, although a node at the prefix's end would
            t.token(0, b, x)[:] = float("nan")
            t.token(1, b, x)[:] = -float("inf")
            touched += 1
    assert touched >= 3
    t.call()
    t.check()


@pytest.mark.parametrize("dt,nodes,D", [("bf16", 12, 128), ("bf16", 64, 128), ("bf16", 9, 64), ("f32", 12, 128)])
def test_infinities_that_every_node_sees_stay_infinities(dt, nodes, D):
    """V of prefix tokens with infinities of one sign in an element: infinite outputs of that sign, not NaN, whatever
    the token's weight: the row's largest (a power of two), small ones, and equal ones."""
    for q_scale in (1.0, 0.0):
        t = Tree(dt, "contiguous", 2, 8, 2, D, 0, nodes, [nodes + 700, nodes + 40], seed=71)
        t.q.mul_(q_scale)
        for b in range(2):
            for x in range(0, int(t.lens[b]) - nodes, 3):
                t.token(1, b, x)[:, x % D] = float("inf") if x % D % 2 else -float("inf")
        t.call()
        t.check()
        assert bool(torch.isinf(t.out).any()) and not bool(torch.isnan(t.out).any())


def test_large_scores_and_equal_scores():
    t = Tree("bf16", "contiguous", 1, 4, 1, 128, 0, 6, [900], seed=4)
    t.q.mul_(16)                                     # weights concentrate: the running maximum moves often
    t.cache[0, :, :, :300].mul_(0.1)
    t.call()
    t.check()
    t.q.zero_()                                      # a plain mean
    t.out.fill_(-77.0)
    t.call()
    t.check()


def test_one_long_row_past_32_bit_offsets():
    """The last tokens of a cache of more than 2^31 elements."""
    H, D, C = 4, 128, 2200000                        # 2 * 4 * 2.2e6 * 128 = 2.25e9 elements
    cache = torch.zeros((2, 1, H, C, D), device=DEV, dtype=torch.bfloat16)
    gen = torch.Generator(device=DEV).manual_seed(3)
    n, nodes, window = C - 1, 5, 700
    live = window + nodes + 300
    for plane in (0, 1):
        cache[plane, 0, :, n - live: n] = torch.randn((H, live, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    q = torch.randn((1, 8, nodes, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    lens = np.array([n], np.int32)
    size = ol.ol_workspace_size_tree(1, 8, H, D, nodes)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    ol.ol_tree_attention(ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(cache), q, 8, nodes, lens, torch.from_numpy(lens).to(DEV),
                         None, None, None, None, 0.0, window, out, ol.OL_BF16, ws, size)
    ok = du.visible(live, nodes, None, None, window)
    for g in range(H):
        k, v = cache[0, 0, g, n - live: n], cache[1, 0, g, n - live: n]
        want, pv, _, s = du.tree_attention(q[0, 2 * g: 2 * g + 2], k, v, ok, D ** -0.5)
        tol = du.tree_tolerance(want, pv, s, D, live, torch.bfloat16, True)
        assert bool(((out[0, 2 * g: 2 * g + 2].double() - want).abs() <= tol).all())
    assert ol.ol_workspace_status(ws) == ol.OL_DEVICE_OK


@pytest.mark.parametrize("window", [-1, 100, 0])
@pytest.mark.parametrize("short", [0, 1, 31, 40])
def test_the_longest_row(short, window):
    """A contiguous cache of 2^31 - 1 tokens of one element: lengths at which a tile's end passes 2^31."""
    C, nodes = 2 ** 31 - 1, 5
    n = C - short
    cache = torch.zeros((2, 1, 1, C, 1), device=DEV, dtype=torch.bfloat16)
    gen = torch.Generator(device=DEV).manual_seed(7)
    last = 200
    for plane in (0, 1):
        cache[plane, 0, 0, n - last: n] = torch.randn((last, 1), generator=gen, device=DEV).to(torch.bfloat16)
        cache[plane, 0, 0, n:] = float("nan")
    if window < 0:  # what lies before counts by its number: keys of zero, weights of one, values of zero
        cache[0, 0, 0, n - last: n] *= 8
    q = torch.randn((1, 2, nodes, 1), generator=gen, device=DEV).to(torch.bfloat16) * 4
    out = torch.full((1, 2, nodes, 1), -77.0, device=DEV)
    lens = np.array([n], np.int32)
    sees, depth = du.random_trees(np.random.default_rng(3), 1, nodes)
    at = np.minimum(n - nodes + depth, 2 ** 31 - 1).astype(np.int32)
    size = ol.ol_workspace_size_tree(1, 2, 1, 1, nodes)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    ol.ol_tree_attention(ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(cache), q, 2, nodes, lens, torch.from_numpy(lens).to(DEV),
                         None, None, torch.from_numpy(du.pack_mask(sees)).to(DEV), torch.from_numpy(at).to(DEV), 1.0, window,
                         out, ol.OL_F32, ws, size)
    k, v = cache[0, 0, 0, n - last: n].double(), cache[1, 0, 0, n - last: n].double()
    ok = torch.from_numpy(du.visible(last, nodes, sees[0], at[0].astype(np.int64) - (n - last), window)).to(DEV)
    s = torch.where(ok, q[0].double() * k[:, 0], -torch.inf)           # [2, nodes, last]
    before = n - last if window < 0 else 0                             # tokens of score 0 and value 0
    top = torch.clamp(s.amax(-1, keepdim=True), min=0.0 if before else -torch.inf)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True) + before * torch.exp(-top)
    want, pv = (p * v[:, 0]).sum(-1) / total[..., 0], (p * v[:, 0].abs()).sum(-1) / total[..., 0]
    # sums of n positive terms in fp32 over some 600 CTAs of 16 threads a row, then their merge
    tol = du.tree_tolerance(want, pv, s[ok.expand_as(s)].abs().max(), 1, n / 9000 + 700, torch.float32, False)
    assert ol.ol_workspace_status(ws) == ol.OL_DEVICE_OK
    assert bool(((out[0, ..., 0].double() - want).abs() <= tol).all())
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_replays_follow_the_device_lengths(dt):
    """A captured call replays with the lengths, counts and masks on the device; two captured calls with workspaces
    of their own run side by side."""
    trees = [Tree(dt, layout, 3, 8, 2, 128, page, 10, [500, 77, 300], [10, 3, 0], seed=s)
             for layout, page, s in (("contiguous", 0, 5), ("paged", 16, 6))]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for t, s in zip(trees, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            t.call()
        graphs.append(g)
    for lens, counts in (([500, 77, 300], [10, 3, 0]), ([20, 60, 299], [0, 10, 9]), ([0, 1, 500 - 7], [0, 1, 4])):
        lens, counts = np.array(lens, np.int32), np.array(counts, np.int32)
        for t in trees:
            t.lens, t.counts = lens, counts
            for b in range(3):  # rows that grow keep finite tokens: fill what is new
                for plane in (0, 1):
                    x = t.row(plane, b, int(lens[b]))
                    t.put(plane, b, torch.where(torch.isnan(x), torch.ones_like(x), x))
            t.lens_d.copy_(torch.from_numpy(lens))
            t.counts_d.copy_(torch.from_numpy(counts))
            t.at = ((lens - counts)[:, None] + np.arange(10)).astype(np.int32)
            t.at_d.copy_(torch.from_numpy(t.at))
            t.out.fill_(-77.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for t in trees:
            t.check()


@pytest.mark.parametrize("D", [128, 64])
def test_non_finite_values_in_a_tree_that_crosses_tiles_and_segments(D):
    """Drafted tokens with infinities over several tiles, in units of two query tiles that several CTAs share."""
    t = Tree("bf16", "paged", 5, 16, 4, D, 64, 200, [3000, 200, 2111, 1000, 500], seed=17)
    for b in range(5):
        first = int(t.lens[b]) - 200
        for j in (0, 70, 130, 199):
            t.token(1, b, first + j)[:, j % D] = float("inf") if j % 20 else float("nan")
        t.sees[b, :, 130] = False                        # seen by a few nodes only
        t.sees[b, ::9, 130] = True
        t.sees[b, :, 0] = False
        t.sees[b, 5, 0] = True
    t.mask = torch.from_numpy(du.pack_mask(t.sees)).to(DEV)
    t.call()
    t.check()


def test_calls_in_a_row_share_a_workspace_and_repeat_bits():
    t = Tree("bf16", "contiguous", 2, 28, 4, 128, 0, 16, [3000, 400])
    t.call()
    torch.cuda.synchronize()
    first = t.out.clone()
    u = Tree("bf16", "contiguous", 1, 28, 4, 128, 0, 16, [2000], seed=8)
    u.ws, u.ws_bytes, u.ws_buf = t.ws, t.ws_bytes, t.ws_buf
    for _ in range(5):
        u.call()
        t.call()
    t.check()
    u.check()
    assert torch.equal(first, t.out)


@pytest.mark.parametrize("layout,page,nodes", [("paged", 64, 256), ("contiguous", 0, 70), ("paged", 16, 16)])
def test_repeated_calls_over_many_tiles_end_and_repeat_bits(layout, page, nodes):
    """Loads land in any order and segments of many lengths meet in a CTA: every call ends without a device status."""
    t = Tree("bf16", layout, 8, 28, 4, 128, page, nodes, [3893, 4047, 5021, 5802, 2139, 2576, 5292, 1000])
    t.call()
    t.check()
    first = t.out.clone()
    for _ in range(40):
        t.call()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK
    assert torch.equal(first, t.out)


def test_tree_decode_and_chunk_share_a_workspace():
    """Tickets of decode and chunked steps stay at zero under a tree's notes and slots, and the other way round."""
    t = Tree("bf16", "contiguous", 2, 28, 4, 128, 0, 16, [3000, 2000])
    chunk = 5
    size = max(t.ws_bytes, ol.ol_workspace_size(2, 28, 4, 128), ol.ol_workspace_size_chunk(2, 28, 4, 128, chunk))
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    q = torch.randn((2, 28, 128), generator=t.gen, device=DEV, dtype=torch.bfloat16)
    qc = torch.randn((2, 28, chunk, 128), generator=t.gen, device=DEV, dtype=torch.bfloat16)
    kv = torch.stack([torch.stack([t.row(p, b, int(t.lens[b]))[:, -chunk:] for b in range(2)]) for p in (0, 1)])
    desc = ol.kv_cache(t.cache)

    def decode(ws):
        out = torch.full_like(q, -77.0)
        ol.ol_decode_attention(desc, q, 28, t.lens, t.lens_d, 0.0, -1, out, ol.OL_BF16, ws, ws.numel())
        return out

    def chunked(ws):  # rewrites the last tokens with what they hold
        out = torch.full_like(qc, -77.0)
        ol.ol_chunk_step(t.code, desc, t.cache, qc, 28, chunk, kv.contiguous(), t.lens, t.lens_d, 0.0, -1, out,
                         ol.OL_BF16, ws, ws.numel())
        return out

    fresh = [f(torch.zeros_like(shared)) for f in (decode, chunked)]
    t.ws, t.ws_bytes = shared, size
    for f, want in zip((decode, chunked), fresh):
        t.out.fill_(-77.0)
        t.call()
        assert torch.equal(f(shared), want)
        shared.zero_()                               # chunked and decode steps have tickets in different places
    decode(shared)
    t.call()
    t.check()


@pytest.mark.parametrize("dt,nodes,chunk", [("bf16", 16, 16), ("f32", 16, 16), ("bf16", 40, 24)])
def test_a_workspace_alternates_between_trees_and_steps(dt, nodes, chunk):
    """Batches whose chunked steps' tickets reach past a decode step's: trees between chunked steps, then (zeroed once)
    trees between decode steps; the tickets stay zero and every result is that of a workspace of its own."""
    B, Hq, H, D = 16, 32, 8, 128
    t = Tree(dt, "contiguous", B, Hq, H, D, 0, nodes, [400 + 131 * b for b in range(B)], out=dt)
    size = max(t.ws_bytes, ol.ol_workspace_size_chunk(B, Hq, H, D, chunk))
    tickets = 256 + 4 * chunk * B * H  # behind the status word
    shared = torch.zeros(size, dtype=torch.uint8, device=DEV)
    q = torch.randn((B, Hq, D), generator=t.gen, device=DEV, dtype=t.dtype)
    qc = torch.randn((B, Hq, chunk, D), generator=t.gen, device=DEV, dtype=t.dtype)
    kv = torch.stack([torch.stack([t.row(p, b, int(t.lens[b]))[:, -chunk:] for b in range(B)]) for p in (0, 1)]).contiguous()
    desc = ol.kv_cache(t.cache)

    def decode(ws):
        out = torch.full_like(q, -77.0)
        ol.ol_decode_attention(desc, q, Hq, t.lens, t.lens_d, 0.0, -1, out, CODE[t.dtype], ws, ws.numel())
        return out

    def chunked(ws):  # rewrites the last tokens with what they hold
        out = torch.full_like(qc, -77.0)
        ol.ol_chunk_step(t.code, desc, t.cache, qc, Hq, chunk, kv, t.lens, t.lens_d, 0.0, -1, out, CODE[t.dtype], ws,
                         ws.numel())
        return out

    t.call()
    tree = t.out.clone()
    t.ws, t.ws_bytes = shared, size
    for step in (chunked, decode):
        want = step(torch.zeros_like(shared))
        shared.zero_()
        for _ in range(3):
            t.out.fill_(-77.0)
            t.call()
            assert torch.equal(t.out, tree)
            if step is chunked:
                assert not bool(shared[:tickets].any())
            assert torch.equal(step(shared), want)
    assert ol.ol_workspace_status(shared) == ol.OL_DEVICE_OK


def test_device_lengths_and_pages_that_disagree_are_recorded():
    t = Tree("bf16", "paged", 2, 8, 2, 128, 16, 4, [100, 50], [4, 4])
    t.lens_d.copy_(torch.tensor([100000, -5], dtype=torch.int32))  # clamped to the capacity, and to nothing
    t.counts_d.copy_(torch.tensor([4, 4], dtype=torch.int32))
    t.call()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_GUARD
    assert bool((t.out[1] == -77.0).all()) and canaries_intact(t.out_buf)
    t = Tree("bf16", "paged", 2, 8, 2, 128, 16, 4, [100, 50])
    t.table_d[0, 2] = 10 ** 6
    t.call()
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_GUARD
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK


# ------------------------------------------------------------- the accepted path

KEEPS = [
    # dt, layout, B, Hkv, D, page, nodes, capacity, starts, kept
    ("bf16", "contiguous", 3, 4, 128, 0, 8, 40, [0, 32, 9], [[0, 2, 5], [], [7]]),
    ("bf16", "paged", 3, 8, 128, 16, 16, 64, [15, 48, 0], [[0, 1, 2, 9, 15], list(range(16)), [3, 4]]),
    ("f32", "paged", 2, 2, 80, 5, 11, 40, [3, 29], [[1, 3, 5, 7, 9, 10], [10]]),
    ("bf16", "contiguous", 1, 1, 5, 0, 3, 5, [2], [[0, 2]]),
    ("f32", "contiguous", 2, 2, 256, 0, 512, 600, [88, 0], [list(range(1, 512, 2)), list(range(200, 512))]),
    ("bf16", "contiguous", 1, 2, 64, 0, 1, 4, [3], [[0]]),
    # more nodes than a CTA looks up at once
    ("bf16", "paged", 2, 2, 64, 16, 700, 1000, [100, 300], [list(range(3, 700)), list(range(0, 700, 3))]),
    ("f32", "contiguous", 1, 1, 128, 0, 600, 600, [0], [list(range(1, 600))]),
]


@pytest.mark.parametrize("case", KEEPS, ids=lambda c: "-".join(map(str, c[:8])))
def test_tree_keep(case):
    dt, layout, B, H, D, page, nodes, C, starts, kept = case
    t = Tree(dt, layout, B, H, H, D, page, 1, [C] * B, spare=0)
    before = t.cache.clone()
    want = t.cache.clone()
    desc = ol.kv_cache(t.cache) if layout == "contiguous" else ol.paged_kv(t.cache, t.table_d, t.table)
    lists = np.full((B, nodes), -9, np.int32)  # past a row's count: not read
    for b in range(B):
        lists[b, : len(kept[b])] = kept[b]
    starts_h = np.array(starts, np.int32)
    args = (t.code, desc, t.cache, nodes, starts_h, torch.from_numpy(starts_h).to(DEV),
            torch.from_numpy(lists).to(DEV), torch.tensor([len(k) for k in kept], dtype=torch.int32, device=DEV), t.ws)
    ol.ol_tree_keep(*args)
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK
    got, t.cache = t.cache, before
    for plane in (0, 1):
        for b in range(B):
            for j, k in enumerate(kept[b]):
                src = t.token(plane, b, starts[b] + k)
                at = (plane, b, slice(None), starts[b] + j) if t.table is None else \
                    (plane, int(t.table[b, (starts[b] + j) // page]), slice(None), (starts[b] + j) % page)
                want[at] = src
    bits = torch.int32 if dt == "f32" else torch.int16
    assert torch.equal(got.view(bits), want.view(bits))


@pytest.mark.parametrize("kept,count", [([0, 2, 2, 3], 4), ([0, 3, 1, 2], 3), ([0, 1, 2, 4], 4), ([-1, 1, 2, 3], 2),
                                        ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1)])
def test_tree_keep_leaves_a_row_whose_list_is_wrong(kept, count):
    t = Tree("bf16", "contiguous", 2, 2, 2, 64, 0, 1, [20, 20], spare=0)
    before = t.cache.clone()
    starts = np.array([3, 5], np.int32)
    lists = torch.tensor([kept, [1, 2, 0, 0]], dtype=torch.int32, device=DEV)
    ol.ol_tree_keep(t.code, ol.kv_cache(t.cache), t.cache, 4, starts, torch.from_numpy(starts).to(DEV), lists,
                    torch.tensor([count, 2], dtype=torch.int32, device=DEV), t.ws)
    torch.cuda.synchronize()
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_GUARD
    before[:, 1, :, 5:7] = before[:, 1, :, 6:8].clone()
    assert torch.equal(t.cache, before)


@pytest.mark.parametrize("dt,layout,page", [("bf16", "contiguous", 0), ("bf16", "paged", 16), ("f32", "paged", 8)])
def test_ragged_trees_at_the_end_of_their_cache(dt, layout, page):
    """Rows that drafted 0 to 6 of 6 nodes, two of them at the end of their cache, tables without pages past a row's
    tokens: appended, attended and kept."""
    B, Hq, H, D, T, C = 4, 8, 2, 64, 6, 48
    t = Tree(dt, layout, B, Hq, H, D, page, T, [C, C, 17, 16], [4, 6, 1, 0], spare=0, seed=61)
    start = t.lens - t.counts
    if page:
        for b in range(B):
            t.table[b, -(-int(t.lens[b]) // page):] = -1
        t.table_d.copy_(torch.from_numpy(t.table))
        desc = ol.paged_kv(t.cache, t.table_d, t.table)
    else:
        desc = ol.kv_cache(t.cache)
    start_d = torch.from_numpy(start).to(DEV)
    qkv = torch.randn((B, T, Hq + 2 * H, D), generator=t.gen, device=DEV, dtype=t.dtype).transpose(1, 2)
    q, k, v = qkv.split((Hq, H, H), dim=1)
    ol.ol_rope_append(t.code, desc, t.cache, ol.rope(D, device=DEV), T, k, v, Hq, q, t.q, start, start_d, t.counts,
                      t.counts_d, t.at_d)
    t.call()
    t.check()
    lists = np.full((B, T), 77, np.int32)
    lists[0, :2], lists[1, :3], lists[2, :1] = [1, 3], [0, 2, 5], [0]
    kept = torch.tensor([2, 3, 1, 0], dtype=torch.int32, device=DEV)
    lists_d = torch.from_numpy(lists).to(DEV)
    want = [[t.row(p, b, int(t.lens[b])).clone() for b in range(B)] for p in (0, 1)]
    before = t.cache.clone()
    ol.ol_tree_keep_counted(t.code, desc, t.cache, T, start, start_d, t.counts, t.counts_d, lists_d, kept, t.ws)
    for p in (0, 1):
        for b in range(B):
            n = int(kept[b])
            want[p][b][:, start[b]: start[b] + n] = want[p][b][:, start[b] + lists[b, :n]].clone()
            assert torch.equal(t.row(p, b, int(t.lens[b])), want[p][b])
    bits = torch.int32 if dt == "f32" else torch.int16
    changed = (t.cache.view(bits) != before.view(bits)).any(-1).sum()
    assert int(changed) <= 2 * H * (2 + 2) and ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK
    with pytest.raises(ol.OlError):  # without the counts: row 0 leaves its cache, or its table
        ol.ol_tree_keep(t.code, desc, t.cache, T, start, start_d, lists_d, kept, t.ws)
    # a list that names what the row did not draft, and a count on the device past `nodes`: the row stays
    before = t.cache.clone()
    lists_d[0, 1] = 4
    t.counts_d[1] = T + 1
    kept[2] = 2
    ol.ol_tree_keep_counted(t.code, desc, t.cache, T, start, start_d, t.counts, t.counts_d, lists_d, kept, t.ws)
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_GUARD
    assert torch.equal(t.cache.view(bits), before.view(bits))


# --------------------------------------------------------------- all of it together

@pytest.mark.parametrize("layout,page", [("contiguous", 0), ("paged", 16)])
def test_speculative_steps_give_the_plain_decode(layout, page):
    """Two rows: prompts appended with rotation, then rounds of drafted trees (append, attend, keep a path). Every
    node's output equals that of a plain decode of its path, and after the rounds ol_decode_attention over the cache
    equals the plain form over the accepted tokens."""
    B, Hq, H, D, T, G = 2, 8, 2, 128, 9, 4
    rng = np.random.default_rng(41)
    gen = torch.Generator(device=DEV).manual_seed(42)
    t = Tree("bf16", layout, B, Hq, H, D, page, T, [150, 150], seed=43)  # buffers; the tokens are replaced
    t.cache.fill_(float("nan"))
    desc = ol.kv_cache(t.cache) if layout == "contiguous" else ol.paged_kv(t.cache, t.table_d, t.table)
    freq = du.frequencies(D)
    rope = ol.rope(D, device=DEV)
    k_ref = [torch.zeros((H, 0, D), device=DEV, dtype=torch.float64) for _ in range(B)]  # rotated in 64 bits
    v_ref = [torch.zeros((H, 0, D), device=DEV, dtype=torch.float64) for _ in range(B)]

    def project(n):
        return torch.randn((B, n, Hq + 2 * H, D), generator=gen, device=DEV, dtype=torch.bfloat16).transpose(1, 2) \
            .split((Hq, H, H), dim=1)

    prompt = np.array([70, 33], np.int32)
    q, k, v = project(70)
    zero = np.zeros(B, np.int32)
    ol.ol_rope_append(t.code, desc, t.cache, rope, 70, k, v, 0, None, None, zero, torch.from_numpy(zero).to(DEV), prompt,
                      torch.from_numpy(prompt).to(DEV))
    for b in range(B):
        n = int(prompt[b])
        k_ref[b] = du.rotate(k[b, :, :n], torch.arange(n, device=DEV), freq, du.HALF)[0]
        v_ref[b] = v[b, :, :n].double()
    length = prompt.copy()
    for round_ in range(3):
        q, k, v = project(T)
        sees, depth = du.random_trees(rng, B, T)
        counts = np.array([T, T - 1 - round_], np.int32)
        counts_d = torch.from_numpy(counts).to(DEV)
        angles = torch.from_numpy((length[:, None] + depth).astype(np.int32)).to(DEV)
        q_rot = torch.zeros((B, Hq, T, D), device=DEV, dtype=torch.bfloat16)
        start_d = torch.from_numpy(length).to(DEV)
        ol.ol_rope_append(t.code, desc, t.cache, rope, T, k, v, Hq, q, q_rot, length, start_d, counts, counts_d, angles)
        lens = length + counts
        out = torch.zeros_like(q_rot)
        ol.ol_tree_attention(t.code, desc, q_rot, Hq, T, lens, torch.from_numpy(lens).to(DEV), counts, counts_d,
                             torch.from_numpy(du.pack_mask(sees)).to(DEV), angles, 0.0, -1, out, ol.OL_BF16, t.ws,
                             t.ws_bytes)
        kept = np.zeros((B, T), np.int32)
        n_kept = np.zeros(B, np.int32)
        for b in range(B):
            n = int(counts[b])
            at = torch.from_numpy(length[b] + depth[b, :n]).to(DEV)
            kr = du.rotate(k[b, :, :n], at, freq, du.HALF)[0]
            qr = du.rotate(q[b, :, :n], at, freq, du.HALF)[0]
            path = np.nonzero(sees[b, n - 1])[0]  # the last node's ancestors and itself
            for i in range(n):
                mine = torch.from_numpy(np.nonzero(sees[b, i])[0]).to(DEV)
                for g in range(H):
                    kk = torch.cat((k_ref[b][g], kr[g][mine]))
                    vv = torch.cat((v_ref[b][g], v[b, g].double()[mine]))
                    ok = np.ones((1, len(kk)), bool)
                    want = du.tree_attention(qr[g * G: (g + 1) * G, i: i + 1], kk, vv, ok, D ** -0.5)[0]
                    # q and K are rounded to bf16 after the rotation, which the plain form is not: two roundings of
                    # 2^-8 of each product, independent over D of them (a score moves by about 2^-8 of its spread, 1)
                    assert float((out[b, g * G: (g + 1) * G, i: i + 1].double() - want).abs().max()) < 0.05
            kept[b, : len(path)], n_kept[b] = path, len(path)
            pick = torch.from_numpy(path).to(DEV)
            k_ref[b] = torch.cat((k_ref[b], kr[:, pick]), 1)
            v_ref[b] = torch.cat((v_ref[b], v[b].double()[:, pick]), 1)
        ol.ol_tree_keep(t.code, desc, t.cache, T, length, start_d, torch.from_numpy(kept).to(DEV),
                        torch.from_numpy(n_kept).to(DEV), t.ws)
        length = length + n_kept
    assert ol.ol_workspace_status(t.ws) == ol.OL_DEVICE_OK
    for b in range(B):
        n = int(length[b])
        got = t.row(0, b, n).double()
        tol = 2.0 ** -8 * k_ref[b].abs() + 1e-5
        assert bool(((got - k_ref[b]).abs() <= tol).all())
        assert torch.equal(t.row(1, b, n).double(), v_ref[b])
    # the framework's decode attention reads what was kept
    q = torch.randn((B, Hq, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    n = ol.ol_workspace_size(B, Hq, H, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    ol.ol_workspace_init(ws, n)
    fn = ol.ol_decode_attention if layout == "contiguous" else ol.ol_paged_decode_attention
    fn(desc, q, Hq, length, torch.from_numpy(length).to(DEV), 0.0, -1, out, ol.OL_BF16, ws, n)
    for b in range(B):
        for g in range(H):
            rows = t.row(0, b, int(length[b]))[g], t.row(1, b, int(length[b]))[g]
            ok = np.ones((1, int(length[b])), bool)
            want = du.tree_attention(q[b, g * G: (g + 1) * G, None], *rows, ok, D ** -0.5)[0][:, 0]
            assert float((out[b, g * G: (g + 1) * G].double() - want).abs().max()) < 0.02
