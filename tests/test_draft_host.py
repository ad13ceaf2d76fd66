"""CPU tests of the operators around drafted tokens: the table of turns against
the scalings' formulas, and every refusal, on the host before any launch. Device
pointers are fake aligned addresses; valid requests are stopped right after
validation by the host fault-injection switch, so nothing reaches the GPU."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import place_kv_cache_gb300 as ol
from tests import draft_util as du

BASE = 0x7F0000000000
MB = 1 << 20


@pytest.fixture(autouse=True)
def _inject(monkeypatch):
    monkeypatch.setenv("OL_FAULT_INJECT", "after_validate")
    yield


def status_of(fn, *a, **k):
    try:
        fn(*a, **k)
    except ol.OlError as e:
        return e.status
    return ol.OL_OK


# ------------------------------------------------------------------------ turns

@pytest.mark.parametrize("rot", [2, 4, 64, 128, 250])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
def test_turns_are_the_formula(rot, scaling):
    if scaling == "ntk" and rot < 4:
        pytest.skip("no such base")
    kind = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}[scaling]
    got = np.zeros(rot // 2, np.uint64)
    ol.ol_rope_turns(kind, rot, 10000.0, 8.0, 4096.0, 1.0, 32.0, got)
    factor = 1.0 if scaling == "none" else 8.0
    want = du.frequencies(rot, scaling=scaling, factor=factor, original=4096.0) / (2 * math.pi)
    # pow, a product and the quotient in double: a few units of 2^-53; the table's own step is 2^-64
    assert np.all(np.abs(got.astype(np.float64) * 2.0 ** -64 - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -63)


def test_turns_by_parts_keeps_short_waves_and_stretches_long_ones():
    t = np.zeros(64, np.uint64)
    u = np.zeros(64, np.uint64)
    ol.ol_rope_turns(ol.OL_ROPE_BY_PARTS, 128, 10000.0, 4.0, 4096.0, 1.0, 32.0, t)
    ol.ol_rope_turns(ol.OL_ROPE_UNSCALED, 128, 10000.0, 1.0, 0.0, 0.0, 0.0, u)
    assert abs(int(t[0]) - int(u[0])) <= int(u[0]) >> 50
    assert abs(4 * int(t[-1]) - int(u[-1])) <= (int(u[-1]) >> 50) + 8


def test_turns_refusals():
    t = np.zeros(8, np.uint64)
    good = dict(scaling=3, rot_dim=16, base=1e4, factor=2.0, original_len=128.0, low=1.0, high=4.0)

    def st(**k):
        a = {**good, **k}
        return status_of(ol.ol_rope_turns, *(a[n] for n in good), a.get("out", t))
    assert st() == ol.OL_OK
    assert st(out=None) == ol.OL_ERR_NULL
    for bad in (dict(rot_dim=0), dict(rot_dim=15), dict(rot_dim=-2), dict(base=1.0), dict(base=math.inf),
                dict(base=math.nan), dict(factor=0.5), dict(factor=math.nan), dict(original_len=0.0), dict(low=-1.0),
                dict(low=4.0), dict(high=math.inf), dict(scaling=4), dict(scaling=-1), dict(scaling=2, rot_dim=2),
                dict(scaling=2, factor=1e300, rot_dim=4)):
        assert st(**bad) == ol.OL_ERR_SHAPE, bad


def test_rope_and_rows_helpers():
    r = ol.rope(16, base=1e4, device="cpu")
    assert r.rot_dim == 16 and r.turns and r.magnitude == 1.0
    x = torch.zeros(2, 5, 3, 8)
    v = ol.rows(x.transpose(1, 2)[:, 1:])
    assert (v.stride_batch, v.stride_head, v.stride_token) == (120, 8, 24) and v.data == x.data_ptr() + 32
    with pytest.raises(ValueError):
        ol.rows(x[0])
    with pytest.raises(ValueError):
        ol.rows(x.transpose(2, 3))


# ------------------------------------------------------------------------- views

B, HQ, HKV, C, D, T = 2, 8, 2, 64, 128, 4
TURNS = BASE + 500 * MB


def rope(rot=128, style=0, magnitude=1.0, turns=TURNS):
    return ol.Rope(turns, rot, style, magnitude)


def dense(at, heads=HQ, tokens=T, dim=D):
    return ol.Rows(at, heads * tokens * dim, tokens * dim, dim)


def rows_call(r=None, dtype=ol.OL_BF16, batch=B, heads=HQ, tokens=T, dim=D, src=None, dst=None,
              at=BASE + 30 * MB, per_token=True):
    return status_of(ol.ol_rope_rows, rope() if r is None else r, dtype, batch, heads, tokens, dim,
                     dense(BASE) if src is None else src, dense(BASE + 10 * MB) if dst is None else dst, at, per_token,
                     stream=0)


def test_rope_rows_passes_and_refuses():
    assert rows_call() == ol.OL_ERR_INJECTED
    assert rows_call(dst=dense(BASE)) == ol.OL_ERR_INJECTED                # in place
    assert rows_call(dst=dense(BASE + 256)) == ol.OL_ERR_ALIAS             # a shifted overlap
    assert rows_call(dst=ol.Rows(BASE, T * D, B * T * D, D)) == ol.OL_ERR_ALIAS  # same memory, other order
    assert rows_call(dst=ol.Rows(BASE + 10 * MB, HQ * T * D, 0, D)) == ol.OL_ERR_SHAPE   # vectors on one another
    assert rows_call(dst=ol.Rows(BASE + 10 * MB, HQ * T * D, T * D, D - 1)) == ol.OL_ERR_SHAPE
    assert rows_call(src=ol.Rows(BASE, 0, 0, 0)) == ol.OL_ERR_INJECTED     # a broadcast input
    assert rows_call(src=ol.Rows(BASE, -1, D, D)) == ol.OL_ERR_SHAPE
    assert rows_call(src=ol.Rows(BASE, 1 << 41, D, D)) == ol.OL_ERR_SHAPE
    assert rows_call(src=ol.Rows(BASE + 2, T * HQ * D, T * D, D)) == ol.OL_ERR_INJECTED  # element alignment
    assert rows_call(src=dense(BASE + 1)) == ol.OL_ERR_ALIGN
    assert rows_call(src=ol.Rows(None, 0, 0, 0)) == ol.OL_ERR_NULL
    assert rows_call(at=None) == ol.OL_ERR_NULL
    assert rows_call(at=BASE + 30 * MB + 4) == ol.OL_ERR_ALIGN
    assert rows_call(at=BASE + 10 * MB) == ol.OL_ERR_ALIAS                 # positions under the output
    assert rows_call(r=rope(turns=BASE + 10 * MB)) == ol.OL_ERR_ALIAS
    assert rows_call(dtype=2) == ol.OL_ERR_DTYPE
    assert rows_call(r=rope(turns=None)) == ol.OL_ERR_NULL
    for bad in (rope(rot=0), rope(rot=3), rope(rot=130), rope(style=2), rope(magnitude=0.0), rope(magnitude=math.nan),
                rope(magnitude=math.inf)):
        assert rows_call(r=bad) == ol.OL_ERR_SHAPE
    assert rows_call(heads=-1) == ol.OL_ERR_SHAPE
    assert rows_call(batch=-1) == ol.OL_ERR_SHAPE
    assert rows_call(dim=1026, r=rope(rot=2)) == ol.OL_ERR_UNSUPPORTED
    assert rows_call(batch=1 << 16, tokens=1 << 15, heads=1, src=ol.Rows(BASE, 0, 0, 0)) == ol.OL_ERR_UNSUPPORTED


def test_rope_rows_is_a_recorded_call():
    """As every call that passes its checks; one that does not leaves the record as it was."""
    ol.ol_reset_stats()
    assert append() == ol.OL_ERR_INJECTED
    assert ol.ol_last_call_stats()["storage_append_copied_bytes"] > 0
    assert rows_call() == ol.OL_ERR_INJECTED
    last, total = ol.ol_last_call_stats(), ol.ol_total_stats()
    assert last["calls"] == 1 and total["calls"] == 2
    assert all(v == 0 for k, v in last.items() if k != "calls")
    assert rows_call(heads=-1) == ol.OL_ERR_SHAPE
    assert ol.ol_total_stats() == total and ol.ol_last_call_stats() == last


# ------------------------------------------------------------------------- append

CACHE = BASE + 100 * MB


def contiguous(**k):
    return ol.kv_cache(CACHE, dims=(B, HKV, C, D), dtype=ol.OL_BF16, **k)


TABLE = np.arange(8, dtype=np.int32).reshape(2, 4)


def paged(table=TABLE, **k):
    return ol.paged_kv(CACHE, BASE + 90 * MB, table, dims=(8, HKV, 16, D), dtype=ol.OL_BF16, **k)


def append(desc=None, layout=ol.OL_LAYOUT_CONTIGUOUS, updated=CACHE, r=None, n=T, k="k", v="v", hq=HQ, q="q",
           q_out="out", pos=(3, 60), pos_dev=BASE + 91 * MB, counts=None, counts_dev=None, angles=None):
    views = {"q": dense(BASE), "out": dense(BASE + 10 * MB), "k": dense(BASE + 20 * MB, HKV),
             "v": dense(BASE + 30 * MB, HKV)}
    get = lambda x: views.get(x, x) if isinstance(x, str) else x  # noqa: E731
    return status_of(ol.ol_rope_append, layout, contiguous() if desc is None else desc, updated,
                     rope() if r is None else r, n, get(k), get(v), hq, get(q), get(q_out), np.array(pos, np.int32),
                     pos_dev, counts, counts_dev, angles, stream=0)


def test_rope_append_passes_and_refuses():
    assert append() == ol.OL_ERR_INJECTED
    assert append(desc=paged(), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_INJECTED
    assert append(hq=0, q=None, q_out=None) == ol.OL_ERR_INJECTED
    assert append(q_out="q") == ol.OL_ERR_INJECTED
    assert append(layout=ol.OL_LAYOUT_INT4) == ol.OL_ERR_UNSUPPORTED
    assert append(updated=CACHE + 16) == ol.OL_ERR_ALIAS
    assert append(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_READONLY
    assert append(pos=(3, 61)) == ol.OL_ERR_CAPACITY
    assert append(pos=(-1, 0)) == ol.OL_ERR_CAPACITY
    counts = np.array([4, 3], np.int32)
    dev = BASE + 92 * MB
    assert append(pos=(3, 61), counts=counts, counts_dev=dev) == ol.OL_ERR_INJECTED
    assert append(counts=counts) == ol.OL_ERR_NULL
    assert append(counts_dev=dev) == ol.OL_ERR_NULL
    assert append(counts=np.array([5, 0], np.int32), counts_dev=dev) == ol.OL_ERR_SHAPE
    assert append(counts=np.array([-1, 0], np.int32), counts_dev=dev) == ol.OL_ERR_SHAPE
    assert append(q=None) == ol.OL_ERR_NULL
    assert append(q_out=None) == ol.OL_ERR_NULL
    assert append(k=None) == ol.OL_ERR_NULL
    assert append(v=ol.Rows(None, 0, 0, 0)) == ol.OL_ERR_NULL
    assert append(hq=0) == ol.OL_ERR_SHAPE
    assert append(hq=3, q=None, q_out=None) == ol.OL_ERR_SHAPE
    assert append(pos_dev=None) == ol.OL_ERR_NULL
    assert append(pos_dev=BASE + 91 * MB + 8) == ol.OL_ERR_ALIGN
    assert append(angles=BASE + 93 * MB + 4) == ol.OL_ERR_ALIGN
    assert append(r=rope(rot=130)) == ol.OL_ERR_SHAPE
    for name in ("k", "v", "q", "q_out"):
        assert append(**{name: dense(CACHE + 64, HQ if name[0] == "q" else HKV)}) == ol.OL_ERR_ALIAS, name
    assert append(q_out=dense(BASE + 20 * MB)) == ol.OL_ERR_ALIAS          # q_out over k
    assert append(q_out=dense(BASE + 256)) == ol.OL_ERR_ALIAS              # q_out shifted over q
    assert append(angles=CACHE) == ol.OL_ERR_ALIAS
    assert append(pos_dev=BASE + 10 * MB) == ol.OL_ERR_ALIAS
    assert append(q_out=dense(BASE + 90 * MB), desc=paged(), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_ALIAS
    assert append(n=-1) == ol.OL_ERR_SHAPE


def test_rope_append_in_place_refuses_shared_elements():
    """q in place in one projection's output with k and v: taken where the vectors interleave, refused where they meet."""
    rng = np.random.default_rng(3)
    seen = set()
    for _ in range(400):
        order = rng.permutation(3)
        sizes, strides = np.array([B, HQ + 2 * HKV + int(rng.integers(0, 3)), T]), [0, 0, 0]
        step = D + int(rng.integers(0, 2)) * 8
        for i in order:                                  # batch, heads, tokens, in any order of nesting
            strides[i] = int(step)
            step = step * sizes[i]
        at = {"k": int(rng.integers(0, 12)), "v": int(rng.integers(0, 12))}
        shift = int(rng.choice([0, 0, 8, -8, D - 8]))
        view = lambda head, more=0: ol.Rows(BASE + 2 * (head * strides[1] + more), *strides)  # noqa: E731

        def elements(first, heads):
            i = np.indices((B, heads, T, D)).reshape(4, -1)
            return set((first + i[0] * strides[0] + i[1] * strides[1] + i[2] * strides[2] + i[3]).tolist())
        q = elements(0, HQ)
        k, v = elements(at["k"] * strides[1] + shift, HKV), elements(at["v"] * strides[1], HKV)
        want = ol.OL_ERR_ALIAS if q & (k | v) else ol.OL_ERR_INJECTED
        if at["k"] * strides[1] + shift < 0:
            continue
        got = append(q=view(0), q_out=view(0), k=view(at["k"], shift), v=view(at["v"]))
        assert got == want, (strides, at, shift)
        seen.add((got, shift))
    assert len(seen) > 5
    other = ol.Rows(BASE + 2 * HQ * D, 10 * T * D, D, 12 * D)  # no projection's output has q with other strides
    mine = ol.Rows(BASE, 12 * T * D, D, 12 * D)
    assert append(q=mine, q_out=mine, k=other) == ol.OL_ERR_ALIAS


def test_rope_append_checks_the_pages_it_writes():
    def st(table, **k):
        return append(desc=paged(np.array(table, np.int32)), layout=ol.OL_LAYOUT_PAGED, **k)
    assert st([[0, 1, 2, 3], [4, 5, 6, 7]], pos=(14, 60)) == ol.OL_ERR_INJECTED
    assert st([[0, 8, 2, 3], [4, 5, 6, 7]], pos=(14, 60)) == ol.OL_ERR_PAGE      # past the pool
    assert st([[0, -1, 2, 3], [4, 5, 6, 7]], pos=(14, 60)) == ol.OL_ERR_PAGE
    assert st([[0, 1, 2, 3], [4, 5, 6, 1]], pos=(14, 60)) == ol.OL_ERR_PAGE      # two rows, one page
    assert st([[0, 0, 2, 3], [4, 5, 6, 7]], pos=(14, 60)) == ol.OL_ERR_PAGE      # one row, twice
    assert st([[-1, 1, -1, 9], [4, 5, 6, 7]], pos=(20, 60)) == ol.OL_ERR_INJECTED  # entries it does not write
    assert st([[0, 1, 2, 3], [4, 5, 6, 1]], pos=(0, 60)) == ol.OL_ERR_INJECTED


def test_rope_append_respects_bindings():
    ol.ol_cache_bind(CACHE, 1 << 20, 9)
    try:
        assert append() == ol.OL_ERR_BUSY
        assert append(desc=contiguous(owner=9)) == ol.OL_ERR_INJECTED
        assert tree() == ol.OL_ERR_BUSY
        assert keep() == ol.OL_ERR_BUSY
    finally:
        ol.ol_cache_unbind(CACHE, 9)


# --------------------------------------------------------------------------- tree

WS = BASE + 200 * MB
WS_BYTES = ol.ol_workspace_size_tree(B, HQ, HKV, D, T)


def tree(desc=None, layout=ol.OL_LAYOUT_CONTIGUOUS, q=BASE, hq=HQ, nodes=T, lens=(10, 64), lens_dev=BASE + 91 * MB,
         counts=None, counts_dev=None, mask=BASE + 92 * MB, positions=BASE + 93 * MB, window=-1, out=BASE + 10 * MB,
         out_dtype=ol.OL_BF16, ws=WS, ws_bytes=WS_BYTES):
    return status_of(ol.ol_tree_attention, layout, contiguous() if desc is None else desc, q, hq, nodes,
                     np.array(lens, np.int32), lens_dev, counts, counts_dev, mask, positions, 0.0, window, out,
                     out_dtype, ws, ws_bytes, stream=0)


def test_tree_attention_passes_and_refuses():
    assert tree() == ol.OL_ERR_INJECTED
    assert tree(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_INJECTED
    assert tree(desc=paged(), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_INJECTED
    assert tree(mask=None, positions=None) == ol.OL_ERR_INJECTED
    assert tree(mask=None, positions=None, window=3) == ol.OL_ERR_INJECTED
    assert tree(positions=None, window=3) == ol.OL_ERR_NULL
    assert tree(layout=ol.OL_LAYOUT_INT4) == ol.OL_ERR_UNSUPPORTED
    assert tree(layout=ol.OL_LAYOUT_HPAGED) == ol.OL_ERR_UNSUPPORTED
    assert tree(nodes=513, lens=(64, 64), ws_bytes=1 << 40) == ol.OL_ERR_UNSUPPORTED
    assert tree(nodes=0) == ol.OL_ERR_SHAPE
    assert tree(hq=7) == ol.OL_ERR_SHAPE
    assert tree(lens=(10, 65)) == ol.OL_ERR_CAPACITY
    assert tree(lens=(-1, 5)) == ol.OL_ERR_CAPACITY
    assert tree(lens=(3, 5)) == ol.OL_ERR_CAPACITY                      # fewer tokens than nodes
    dev = BASE + 94 * MB
    assert tree(lens=(3, 5), counts=np.array([3, 0], np.int32), counts_dev=dev) == ol.OL_ERR_INJECTED
    assert tree(counts=np.array([5, 0], np.int32), counts_dev=dev) == ol.OL_ERR_SHAPE
    assert tree(counts=np.array([-1, 0], np.int32), counts_dev=dev) == ol.OL_ERR_SHAPE
    assert tree(counts=np.array([1, 1], np.int32)) == ol.OL_ERR_NULL
    for name in ("q", "lens_dev", "out", "ws"):
        assert tree(**{name: None}) == ol.OL_ERR_NULL, name
        assert tree(**{name: CACHE + 1024}) == ol.OL_ERR_ALIAS, name
    assert tree(q=BASE + 8) == ol.OL_ERR_ALIGN
    assert tree(mask=BASE + 92 * MB + 8) == ol.OL_ERR_ALIGN
    assert tree(out=BASE) == ol.OL_ERR_ALIAS
    assert tree(out=WS) == ol.OL_ERR_ALIAS
    assert tree(mask=WS + 512) == ol.OL_ERR_ALIAS
    assert tree(out_dtype=7) == ol.OL_ERR_DTYPE
    assert tree(ws_bytes=WS_BYTES - 1) == ol.OL_ERR_WORKSPACE


def test_tree_attention_counts_its_work_in_32_bits():
    """A cache of 2^31 rows is beyond the tensor-core kernel: tiles of 32 tokens of units of 64 (head, node) rows,
    2^31 of which are refused, and fewer are not."""
    def st(capacity, nodes):
        batch, far = 8, 1 << 45
        desc = ol.kv_cache(BASE - far, dims=(batch, HKV, capacity, D), dtype=ol.OL_BF16)
        return tree(desc=desc, nodes=nodes, lens=[nodes] * batch, mask=None, positions=None, ws_bytes=1 << 40,
                    ws=BASE + far)
    assert st((1 << 31) - 1, 32) == ol.OL_ERR_UNSUPPORTED               # 2^26 tiles, 8 rows, 2 heads, 2 units
    assert st((1 << 31) - 1, 16) == ol.OL_ERR_INJECTED                  # 1 unit
    assert st((1 << 30) - 200, 32) == ol.OL_ERR_INJECTED                # half the tiles


def test_a_rows_tiles_up_to_the_largest_length(tmp_path):
    """The work split's tiles of a row, against Python's integers: lengths up to 2^31 - 1, with and without a window."""
    cases = []
    for log2 in (5, 7):
        for length in [1, 2, 31, 32, 33, 128, 129] + [2 ** 31 - 1 - d for d in (0, 1, 30, 31, 32, 127, 128, 129, 300)]:
            for count in sorted({0, 1, min(length, 7), min(length, 512)}):
                for window in (-1, 0, 100, 2 ** 31 - 1):
                    cases.append((length, count, window, log2))
    source = tmp_path / "rows.cpp"
    source.write_text('#include <cstdio>\n#include "ol_draft.h"\nint main() {\n  int n, c, w, t;\n'
                      "  while (scanf(\"%d %d %d %d\", &n, &c, &w, &t) == 4) {\n"
                      "    const ol::TreeRow r = ol::tree_row(n, c, w, t);\n"
                      '    printf("%d %d %d\\n", r.prefix, r.start, r.ntiles);\n  }\n}\n')
    exe = str(tmp_path / "rows")
    csrc = os.path.join(os.path.dirname(ol.__file__), "csrc")
    cuda = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda") if d and os.path.isdir(d)), None)
    if cuda is None or shutil.which("g++") is None:
        pytest.skip("no host compiler or no CUDA headers")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, "-I", os.path.join(cuda, "include"), str(source), "-o", exe],
                   check=True)
    got = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.split("\n")
    for (length, count, window, log2), line in zip(cases, got):
        prefix = length - count
        start = (0 if window < 0 else max(0, prefix - window)) >> log2 << log2
        tiles = -(-(length - start) // 2 ** log2) if count else 0
        assert line == f"{prefix} {start} {tiles}", (length, count, window, log2)


def test_tree_attention_checks_the_pages_it_reads():
    def st(table, **k):
        return tree(desc=paged(np.array(table, np.int32)), layout=ol.OL_LAYOUT_PAGED, **k)
    assert st([[0, 1, 2, 3], [0, 1, 2, 3]], lens=(33, 64)) == ol.OL_ERR_INJECTED      # shared pages are read
    assert st([[0, 8, 2, 3], [4, 5, 6, 7]], lens=(33, 64)) == ol.OL_ERR_PAGE
    assert st([[0, 1, 2, -1], [4, 5, 6, 7]], lens=(33, 64)) == ol.OL_ERR_INJECTED     # past the row
    # with a window of 8 the lowest token is 64 - 4 - 8 = 52: pages below it are not read
    assert st([[0, 1, 2, 3], [-1, -1, -1, 7]], lens=(33, 64), window=8) == ol.OL_ERR_INJECTED
    assert st([[0, 1, 2, 3], [-1, -1, -1, 7]], lens=(33, 64), window=13) == ol.OL_ERR_PAGE


def test_tree_statistics_and_workspace():
    ol.ol_reset_stats()
    tree(lens=(10, 64), window=8)
    s = ol.ol_last_call_stats()
    # tokens that some node may see: [0, 10) and [52, 64)
    assert s["attended_tokens"] == (4 * 10 + 4 * 12) * HKV
    assert s["kv_payload_bytes_read"] == 2 * (10 + 12) * HKV * D * 2
    assert s["workspace_bytes"] == WS_BYTES
    assert ol.ol_workspace_size_tree(1, 7, 2, 128, 4) == 0
    assert ol.ol_workspace_size_tree(1, 8, 2, 128, 0) == 0
    assert ol.ol_workspace_size_tree(1, 8, 2, 128, 64) > ol.ol_workspace_size_tree(1, 8, 2, 128, 4)


# --------------------------------------------------------------------------- keep

def keep(desc=None, layout=ol.OL_LAYOUT_CONTIGUOUS, updated=CACHE, nodes=T, starts=(3, 60), starts_dev=BASE + 91 * MB,
         kept=BASE + 92 * MB, counts=BASE + 93 * MB, ws=None):
    return status_of(ol.ol_tree_keep, layout, contiguous() if desc is None else desc, updated, nodes,
                     np.array(starts, np.int32), starts_dev, kept, counts, ws, stream=0)


def test_tree_keep_passes_and_refuses():
    assert keep() == ol.OL_ERR_INJECTED
    assert keep(ws=WS) == ol.OL_ERR_INJECTED
    assert keep(desc=paged(), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_INJECTED
    assert keep(layout=ol.OL_LAYOUT_HPAGED) == ol.OL_ERR_UNSUPPORTED
    assert keep(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_READONLY
    assert keep(updated=BASE) == ol.OL_ERR_ALIAS
    assert keep(starts=(3, 61)) == ol.OL_ERR_CAPACITY
    assert keep(starts=(-1, 0)) == ol.OL_ERR_CAPACITY
    assert keep(nodes=0) == ol.OL_ERR_SHAPE
    for name in ("starts_dev", "kept", "counts"):
        assert keep(**{name: None}) == ol.OL_ERR_NULL
        assert keep(**{name: CACHE}) == ol.OL_ERR_ALIAS
        assert keep(**{name: BASE + 4}) == ol.OL_ERR_ALIGN
    assert keep(ws=CACHE) == ol.OL_ERR_ALIAS
    shared = np.array([[0, 1, 2, 3], [4, 5, 6, 0]], np.int32)
    assert keep(desc=paged(shared), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_PAGE
    outside = np.array([[8, 1, 2, 3], [4, 5, 6, 7]], np.int32)
    assert keep(desc=paged(outside), layout=ol.OL_LAYOUT_PAGED) == ol.OL_ERR_PAGE


def test_tree_keep_refuses_a_status_word_over_what_it_reads():
    """The kernel writes the status word while other CTAs read the lists."""
    for at in (BASE + 91 * MB, BASE + 92 * MB, BASE + 93 * MB):  # starts, kept, counts
        assert keep(ws=at) == ol.OL_ERR_ALIAS
        assert keep(ws=at + 16) == (ol.OL_ERR_ALIAS if at == BASE + 92 * MB else ol.OL_ERR_INJECTED)  # 32 bytes and 8
        assert keep(ws=at - 16) == keep(ws=at + 32) == ol.OL_ERR_INJECTED
    assert keep(desc=paged(), layout=ol.OL_LAYOUT_PAGED, ws=BASE + 90 * MB) == ol.OL_ERR_ALIAS


def keep_counted(counts, counts_dev=BASE + 94 * MB, desc=None, layout=ol.OL_LAYOUT_CONTIGUOUS, nodes=T, starts=(3, 60),
                 updated=CACHE):
    return status_of(ol.ol_tree_keep_counted, layout, contiguous() if desc is None else desc, updated, nodes,
                     np.array(starts, np.int32), BASE + 91 * MB, counts, counts_dev, BASE + 92 * MB, BASE + 93 * MB,
                     stream=0)


def test_tree_keep_counted_checks_the_tokens_that_rows_drafted():
    """A short row that ends at its capacity, or whose table names no page (or a shared one) past its tokens, passes."""
    n = lambda *x: np.array(x, np.int32)  # noqa: E731
    assert keep_counted(None, None) == ol.OL_ERR_INJECTED
    assert keep_counted(n(4, 4)) == ol.OL_ERR_INJECTED
    assert keep_counted(n(0, 0)) == ol.OL_ERR_INJECTED
    assert keep_counted(n(4, 1), starts=(3, 63)) == ol.OL_ERR_INJECTED
    assert keep_counted(n(4, 0), starts=(3, 64)) == ol.OL_ERR_INJECTED
    assert keep_counted(n(4, 2), starts=(3, 63)) == ol.OL_ERR_CAPACITY
    assert keep_counted(None, None, starts=(3, 63)) == ol.OL_ERR_CAPACITY
    assert keep_counted(n(4, 1), starts=(3, -1)) == ol.OL_ERR_CAPACITY
    assert keep_counted(n(5, 1)) == ol.OL_ERR_SHAPE
    assert keep_counted(n(4, -1)) == ol.OL_ERR_SHAPE
    assert keep_counted(n(4, 1), None) == ol.OL_ERR_NULL
    assert keep_counted(None) == ol.OL_ERR_NULL
    assert keep_counted(n(4, 1), CACHE) == ol.OL_ERR_ALIAS
    assert keep_counted(n(4, 1), BASE + 94 * MB + 4) == ol.OL_ERR_ALIGN
    assert keep_counted(n(4, 1), desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_READONLY
    assert keep_counted(n(4, 1), updated=BASE) == ol.OL_ERR_ALIAS

    def st(table, counts, starts=(14, 30)):
        return keep_counted(counts, desc=paged(np.array(table, np.int32)), layout=ol.OL_LAYOUT_PAGED, starts=starts)
    missing, padded = [[0, -1, -1, -1], [4, 5, -1, -1]], [[1, 0, 0, 0], [4, 5, 0, 0]]
    assert st(missing, n(2, 2)) == st(padded, n(2, 2)) == ol.OL_ERR_INJECTED
    assert st(missing, n(3, 2)) == ol.OL_ERR_PAGE
    assert st(padded, n(3, 3)) == ol.OL_ERR_PAGE                       # page 0 for two rows
    assert st([[0, 1, 2, 3], [4, 0, 6, 7]], n(2, 2)) == ol.OL_ERR_PAGE
