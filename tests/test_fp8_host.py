"""CPU tests of the E4M3 cache's operators and of the norms with their rotation:
every refusal, on the host before any launch, and the statistics of valid calls.
Device pointers are fake aligned addresses; valid requests are stopped right after
validation by the host fault-injection switch, so nothing reaches the GPU."""
import math

import numpy as np
import pytest
import torch

import place_kv_cache_gb300 as ol
from tests import fp8_util as fu

BASE = 0x7F0000000000
MB = 1 << 20
B, HQ, HKV, C, D, T, BLOCK = 2, 8, 2, 64, 128, 4, 16
CODES, SCALES, TABLE_DEV, WS = BASE + 100 * MB, BASE + 150 * MB, BASE + 90 * MB, BASE + 200 * MB
TURNS = BASE + 500 * MB
TABLE = np.arange(8, dtype=np.int32).reshape(2, 4)


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


def dense(at, heads=HKV, tokens=T, dim=D):
    return ol.Rows(at, heads * tokens * dim, tokens * dim, dim)


def contiguous(codes=CODES, scales=SCALES, block=BLOCK, dims=(B, HKV, C, D), **k):
    return ol.fp8_kv(codes, scales, block=block, dims=dims, **k)


def paged(table=TABLE, block=BLOCK, page=16, dim=D, **k):
    return ol.fp8_kv(CODES, SCALES, TABLE_DEV, table, block=block, dims=(8, HKV, page, dim), **k)


def i32(x):
    return None if x is None else np.array(x, np.int32)


def append(desc=None, updated=CODES, dtype=ol.OL_BF16, n=T, k="k", v="v", pos=(3, 60), pos_dev=BASE + 91 * MB,
           counts=None, counts_dev=None):
    views = {"k": dense(BASE), "v": dense(BASE + 10 * MB)}
    get = lambda x: views.get(x) if isinstance(x, str) else x  # noqa: E731
    return status_of(ol.ol_fp8kv_append, contiguous() if desc is None else desc, updated, dtype, n, get(k), get(v),
                     i32(pos), pos_dev, i32(counts), counts_dev, stream=0)


def read(desc=None, dtype=ol.OL_BF16, n=T, k="k", v="v", start=(3, 60), start_dev=BASE + 91 * MB, counts=None,
         counts_dev=None):
    views = {"k": dense(BASE), "v": dense(BASE + 10 * MB)}
    get = lambda x: views.get(x) if isinstance(x, str) else x  # noqa: E731
    return status_of(ol.ol_fp8kv_read, contiguous() if desc is None else desc, dtype, n, get(k), get(v), i32(start),
                     start_dev, i32(counts), counts_dev, stream=0)


WS_BYTES = ol.ol_workspace_size_fp8kv(B, HQ, HKV, D, T)


def attention(desc=None, dtype=ol.OL_BF16, q=BASE, hq=HQ, n=T, lens=(10, 64), lens_dev=BASE + 91 * MB, counts=None,
              counts_dev=None, window=-1, out=BASE + 10 * MB, out_dtype=ol.OL_BF16, ws=WS, ws_bytes=WS_BYTES):
    return status_of(ol.ol_fp8kv_attention, contiguous() if desc is None else desc, dtype, q, hq, n, i32(lens), lens_dev,
                     i32(counts), counts_dev, 0.0, window, out, out_dtype, ws, ws_bytes, stream=0)


CALLS = {"append": append, "read": read, "attention": attention}


# -------------------------------------------------------------------- descriptor

@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_descriptor_checks(call):
    assert call() == ol.OL_ERR_INJECTED
    assert call(desc=paged()) == ol.OL_ERR_INJECTED
    assert call(desc=contiguous(scales=None)) == ol.OL_ERR_NULL
    assert call(desc=contiguous(codes=CODES, scales=SCALES + 4)) == ol.OL_ERR_ALIGN
    assert call(desc=contiguous(scales=CODES + 1024)) == ol.OL_ERR_ALIAS
    for block in (0, 8, 24, 256, -16):
        assert call(desc=contiguous(block=block)) == ol.OL_ERR_SHAPE
    assert call(desc=paged(block=32)) == ol.OL_ERR_SHAPE                       # a page of half a block
    for dim in (8, 120, 272):
        assert call(desc=contiguous(dims=(B, HKV, C, dim))) == ol.OL_ERR_UNSUPPORTED
    for dims in ((-1, HKV, C, D), (B, 0, C, D), (B, HKV, -1, D), (B, HKV, C, 0)):
        assert call(desc=contiguous(dims=dims)) == ol.OL_ERR_SHAPE
    half = paged()
    half.block_table = None
    assert call(desc=half) == ol.OL_ERR_NULL
    mixed = paged()
    mixed.capacity = 64
    assert call(desc=mixed) == ol.OL_ERR_SHAPE
    mixed = contiguous()
    mixed.page_size = 16
    assert call(desc=mixed) == ol.OL_ERR_SHAPE
    odd = paged()
    odd.block_table = TABLE_DEV + 4
    assert call(desc=odd) == ol.OL_ERR_ALIGN
    ol.ol_cache_bind(SCALES, 16, 9)
    try:
        assert call() == ol.OL_ERR_BUSY
        assert call(desc=contiguous(owner=9)) == ol.OL_ERR_INJECTED
    finally:
        ol.ol_cache_unbind(SCALES, 9)


def test_descriptor_of_tensors():
    codes = torch.zeros(2, 3, 2, 40, 64, dtype=torch.uint8)
    scales = torch.zeros(2, 3, 2, 3)
    d = ol.fp8_kv(codes, scales, block=16)
    assert (d.batch, d.kv_heads, d.capacity, d.head_dim, d.num_pages, d.page_size, d.max_pages, d.block) == \
        (3, 2, 40, 64, 0, 0, 0, 16)
    pool = torch.zeros(2, 7, 2, 32, 64, dtype=torch.float8_e4m3fn)
    table = torch.zeros(3, 2, dtype=torch.int32)
    d = ol.fp8_kv(pool, scales, table, table, block=16)
    assert (d.batch, d.kv_heads, d.capacity, d.head_dim, d.num_pages, d.page_size, d.max_pages) == (3, 2, 0, 64, 7, 32, 2)


# ----------------------------------------------------------------- append and read

def places(call, dev_name):
    counts_dev = BASE + 92 * MB
    where = "pos" if call is append else "start"
    assert call(**{where: (3, 61)}) == ol.OL_ERR_CAPACITY
    assert call(**{where: (-1, 0)}) == ol.OL_ERR_CAPACITY
    assert call(**{where: (3, 61)}, counts=(4, 3), counts_dev=counts_dev) == ol.OL_ERR_INJECTED
    assert call(counts=(4, 3)) == ol.OL_ERR_NULL
    assert call(counts_dev=counts_dev) == ol.OL_ERR_NULL
    assert call(counts=(5, 0), counts_dev=counts_dev) == ol.OL_ERR_SHAPE
    assert call(counts=(-1, 0), counts_dev=counts_dev) == ol.OL_ERR_SHAPE
    assert call(**{where: None}) == ol.OL_ERR_NULL
    assert call(**{dev_name: None}) == ol.OL_ERR_NULL
    assert call(**{dev_name: BASE + 91 * MB + 8}) == ol.OL_ERR_ALIGN
    assert call(counts=(4, 3), counts_dev=counts_dev + 4) == ol.OL_ERR_ALIGN
    assert call(**{dev_name: CODES}) in (ol.OL_ERR_ALIAS, ol.OL_ERR_INJECTED)
    assert call(dtype=2) == ol.OL_ERR_DTYPE
    assert call(n=-1) == ol.OL_ERR_SHAPE
    assert call(k=ol.Rows(None, 0, 0, 0)) == ol.OL_ERR_NULL
    assert call(k=ol.Rows(BASE + 1, HKV * T * D, T * D, D)) == ol.OL_ERR_ALIGN
    assert call(k=ol.Rows(BASE + 2, HKV * T * D, T * D, D)) == ol.OL_ERR_INJECTED
    assert call(k=ol.Rows(BASE, -1, T * D, D)) == ol.OL_ERR_SHAPE
    for at in (CODES + 64, SCALES):
        assert call(k=dense(at)) == ol.OL_ERR_ALIAS
        assert call(v=dense(at)) == ol.OL_ERR_ALIAS

    def pages(table, *at):
        return call(desc=paged(np.array(table, np.int32)), **{where: at})
    assert pages([[0, 1, 2, 3], [4, 5, 6, 7]], 14, 60) == ol.OL_ERR_INJECTED
    assert pages([[0, 8, 2, 3], [4, 5, 6, 7]], 14, 60) == ol.OL_ERR_PAGE
    assert pages([[0, -1, 2, 3], [4, 5, 6, 7]], 14, 60) == ol.OL_ERR_PAGE
    assert pages([[-1, 1, -1, 9], [4, 5, 6, 7]], 20, 60) == ol.OL_ERR_INJECTED  # entries it does not reach
    return pages


def test_append_refuses():
    pages = places(append, "pos_dev")
    assert pages([[0, 1, 2, 3], [4, 5, 6, 1]], 14, 60) == ol.OL_ERR_PAGE        # two rows, one page
    assert pages([[0, 0, 2, 3], [4, 5, 6, 7]], 14, 60) == ol.OL_ERR_PAGE        # one row, twice
    assert append(updated=CODES + 16) == ol.OL_ERR_ALIAS
    assert append(updated=None) == ol.OL_ERR_NULL
    assert append(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_READONLY
    assert append(k=None) == ol.OL_ERR_NULL
    assert append(v=None) == ol.OL_ERR_NULL
    assert append(pos_dev=SCALES) == ol.OL_ERR_ALIAS
    assert append(k=ol.Rows(BASE, 0, 0, 0)) == ol.OL_ERR_INJECTED               # a broadcast input
    big = contiguous(dims=(1 << 16, 1 << 10, 1 << 20, 16))
    assert status_of(ol.ol_fp8kv_append, big, CODES, ol.OL_BF16, 1 << 20, ol.Rows(BASE, 0, 0, 0), ol.Rows(BASE, 0, 0, 0),
                     np.zeros(1 << 16, np.int32), BASE + 91 * MB, stream=0) in (ol.OL_ERR_UNSUPPORTED, ol.OL_ERR_ALIAS)


def test_read_refuses():
    pages = places(read, "start_dev")
    assert pages([[0, 1, 2, 3], [4, 5, 6, 1]], 14, 60) == ol.OL_ERR_INJECTED    # a shared page is read twice
    assert read(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_INJECTED
    assert read(k=None) == ol.OL_ERR_INJECTED
    assert read(v=None) == ol.OL_ERR_INJECTED
    assert read(k=None, v=None) == ol.OL_ERR_NULL
    assert read(k=ol.Rows(BASE, 0, 0, 0)) == ol.OL_ERR_SHAPE                    # vectors on one another
    assert read(v=dense(BASE + 256)) == ol.OL_ERR_ALIAS
    both = lambda at: ol.Rows(BASE + 2 * at * D, 2 * HKV * T * D, D, 2 * HKV * D)  # noqa: E731  K and V of a token in turn
    assert read(k=both(0), v=both(HKV)) == ol.OL_ERR_INJECTED
    assert read(k=both(0), v=both(HKV - 1)) == ol.OL_ERR_ALIAS
    assert read(start_dev=BASE) == ol.OL_ERR_ALIAS
    assert read(desc=paged(), k=dense(TABLE_DEV)) == ol.OL_ERR_ALIAS


def test_statistics():
    assert append() == ol.OL_ERR_INJECTED
    st = ol.ol_last_call_stats()
    # rows at 3 and 60, four tokens each: a block each
    assert st["storage_append_copied_bytes"] == 2 * HKV * (8 * D + 2 * 4) and st["storage_reuse_count"] == 2
    assert append(pos=(14, 60), counts=(4, 0), counts_dev=BASE + 92 * MB) == ol.OL_ERR_INJECTED
    assert ol.ol_last_call_stats()["storage_append_copied_bytes"] == 2 * HKV * (4 * D + 2 * 4)
    assert read(start=(14, 60), v=None) == ol.OL_ERR_INJECTED
    st = ol.ol_last_call_stats()
    assert st["dequantized_bytes"] == 4 * HKV * 8 * D and st["kv_payload_bytes_read"] == HKV * (8 * D + 3 * 4)
    assert attention() == ol.OL_ERR_INJECTED
    st = ol.ol_last_call_stats()
    assert st["attended_tokens"] == T * HKV * 74 and st["dequantized_bytes"] == 8 * HKV * 74 * D
    assert st["kv_payload_bytes_read"] == 2 * HKV * (74 * D + 5 * 4) and st["workspace_bytes"] == WS_BYTES
    assert attention(window=5) == ol.OL_ERR_INJECTED                           # tokens [1, 10) and [55, 64)
    assert ol.ol_last_call_stats()["kv_payload_bytes_read"] == 2 * HKV * (18 * D + 2 * 4)


# --------------------------------------------------------------------- attention

def test_attention_refuses():
    for bad in (dict(q=None), dict(out=None), dict(ws=None), dict(lens=None), dict(lens_dev=None), dict(counts=(1, 1)),
                dict(counts_dev=BASE + 92 * MB)):
        assert attention(**bad) == ol.OL_ERR_NULL, bad
    for bad in (dict(hq=0), dict(hq=7), dict(n=0), dict(counts=(5, 1), counts_dev=BASE + 92 * MB),
                dict(counts=(-1, 1), counts_dev=BASE + 92 * MB)):
        assert attention(**bad) == ol.OL_ERR_SHAPE, bad
    assert attention(dtype=2) == ol.OL_ERR_DTYPE
    assert attention(out_dtype=2) == ol.OL_ERR_DTYPE
    assert attention(n=513, ws_bytes=1 << 40) == ol.OL_ERR_UNSUPPORTED
    for bad in (dict(lens=(65, 4)), dict(lens=(-1, 4)), dict(lens=(3, 64))):
        assert attention(**bad) == ol.OL_ERR_CAPACITY, bad
    assert attention(lens=(3, 64), counts=(3, 4), counts_dev=BASE + 92 * MB) == ol.OL_ERR_INJECTED
    assert attention(lens=(0, 64), counts=(0, 4), counts_dev=BASE + 92 * MB) == ol.OL_ERR_INJECTED
    assert attention(ws_bytes=WS_BYTES - 1) == ol.OL_ERR_WORKSPACE
    for name, at in (("q", BASE), ("out", BASE + 10 * MB), ("ws", WS), ("lens_dev", BASE + 91 * MB)):
        assert attention(**{name: at + 8}) == ol.OL_ERR_ALIGN, name
        assert attention(**{name: CODES}) == ol.OL_ERR_ALIAS, name
        assert attention(**{name: SCALES}) == ol.OL_ERR_ALIAS, name
    assert attention(out=BASE) == ol.OL_ERR_ALIAS
    assert attention(out=WS) == ol.OL_ERR_ALIAS
    assert attention(q=WS) == ol.OL_ERR_ALIAS
    assert attention(desc=paged(), out=TABLE_DEV) == ol.OL_ERR_ALIAS
    assert attention(desc=contiguous(access=ol.OL_READ_ONLY)) == ol.OL_ERR_INJECTED

    def pages(table, **k):
        return attention(desc=paged(np.array(table, np.int32)), **k)
    assert pages([[0, 1, 2, 3], [0, 5, 6, 7]]) == ol.OL_ERR_INJECTED           # a shared page is read twice
    assert pages([[0, 9, 9, 9], [4, 5, 6, 7]]) == ol.OL_ERR_INJECTED           # entries past the row
    assert pages([[9, 1, 2, 3], [4, 5, 6, 7]]) == ol.OL_ERR_PAGE
    assert pages([[0, 1, 2, 3], [4, 5, 6, 8]]) == ol.OL_ERR_PAGE
    assert pages([[0, 1, 2, 3], [-1, -1, 6, 7]], window=20) == ol.OL_ERR_INJECTED  # entries below the window


def test_workspace_size():
    assert WS_BYTES >= 2 * (D + 2) * 4
    for bad in ((-1, 8, 2, 128, 1), (1, 8, 0, 128, 1), (1, 7, 2, 128, 1), (1, 8, 2, 0, 1), (1, 8, 2, 128, 0)):
        assert ol.ol_workspace_size_fp8kv(*bad) == 0


def test_two_rows_of_two_gigabytes_are_counted():
    """Work that does not fit 31 bits of tiles is refused."""
    big = contiguous(dims=(1 << 12, 1 << 8, 1 << 30, 16))
    lens = np.full(1 << 12, 4, np.int32)
    assert status_of(ol.ol_fp8kv_attention, big, ol.OL_BF16, 4096, 1 << 8, 1, lens, 1 << 30, None, None, 0.0, -1, 1 << 31,
                     ol.OL_BF16, 1 << 33, 1 << 40, stream=0) in (ol.OL_ERR_UNSUPPORTED, ol.OL_ERR_ALIAS)


# -------------------------------------------------------------- norms and rotation

def norm_rope(r="rope", norm=None, dtype=ol.OL_BF16, batch=B, tokens=T, dim=D, hq=HQ, q="q", q_out="qo", hk=HKV, k="k",
              k_out="ko", at=BASE + 30 * MB, per_token=True):
    views = {"q": dense(BASE, HQ), "qo": dense(BASE + 10 * MB, HQ), "k": dense(BASE + 20 * MB),
             "ko": dense(BASE + 25 * MB)}
    get = lambda x: views.get(x) if isinstance(x, str) else x  # noqa: E731
    rope = ol.Rope(TURNS, dim, 0, 1.0) if r == "rope" else r
    norm = ol.head_norm(BASE + 40 * MB, BASE + 41 * MB) if norm is None else norm
    return status_of(ol.ol_norm_rope_rows, rope, norm, dtype, batch, tokens, dim, hq, get(q), get(q_out), hk, get(k),
                     get(k_out), at, per_token, stream=0)


def test_norm_rope_passes_and_refuses():
    ok = ol.OL_ERR_INJECTED
    assert norm_rope() == ok
    assert norm_rope(r=None, at=None) == ok
    assert norm_rope(norm=ol.head_norm()) == ok
    assert norm_rope(hk=0, k=None, k_out=None) == ok
    assert norm_rope(hq=0, q=None, q_out=None) == ok
    assert norm_rope(q_out="q", k_out="k") == ok
    for bad in (dict(r=None), dict(at=None), dict(q=None), dict(q_out=None), dict(k=None), dict(k_out=None),
                dict(hq=0, hk=0, q=None, q_out=None, k=None, k_out=None), dict(r=ol.Rope(None, D, 0, 1.0)),
                dict(q=ol.Rows(None, 0, 0, 0))):
        assert norm_rope(**bad) == ol.OL_ERR_NULL, bad
    assert status_of(ol.ol_norm_rope_rows, None, None, ol.OL_BF16, 1, 1, 64, 1, dense(BASE), dense(BASE + MB), 0, None,
                     None, None, False, stream=0) == ol.OL_ERR_NULL
    for bad in (dict(hq=0), dict(hk=0), dict(hq=-1), dict(batch=-1), dict(tokens=-1), dict(dim=0, r=None, at=None),
                dict(hq=3, q=None, q_out=None), dict(norm=ol.head_norm(eps=0.0)), dict(norm=ol.head_norm(eps=-1.0)),
                dict(norm=ol.head_norm(eps=math.nan)), dict(norm=ol.head_norm(eps=math.inf)),
                dict(norm=ol.head_norm(weight_offset=math.nan)), dict(r=ol.Rope(TURNS, 130, 0, 1.0)),
                dict(r=ol.Rope(TURNS, 3, 0, 1.0)), dict(r=ol.Rope(TURNS, D, 2, 1.0)), dict(r=ol.Rope(TURNS, D, 0, 0.0)),
                dict(q=ol.Rows(BASE, -1, T * D, D)), dict(q_out=ol.Rows(BASE + 10 * MB, 0, 0, 0))):
        assert norm_rope(**bad) == ol.OL_ERR_SHAPE, bad
    assert norm_rope(dtype=2) == ol.OL_ERR_DTYPE
    assert norm_rope(dim=1026, r=ol.Rope(TURNS, 2, 0, 1.0)) == ol.OL_ERR_UNSUPPORTED
    assert norm_rope(dim=1026, r=None, at=None) == ol.OL_ERR_UNSUPPORTED
    for bad in (dict(at=BASE + 30 * MB + 4), dict(norm=ol.head_norm(BASE + 8)), dict(norm=ol.head_norm(None, BASE + 8)),
                dict(q=dense(BASE + 1, HQ)), dict(k_out=dense(BASE + 25 * MB + 1)), dict(r=ol.Rope(TURNS + 8, D, 0, 1.0))):
        assert norm_rope(**bad) == ol.OL_ERR_ALIGN, bad


def test_norm_rope_refuses_what_overlaps():
    bad = ol.OL_ERR_ALIAS
    assert norm_rope(q_out=dense(BASE + 256, HQ)) == bad                       # shifted over q
    assert norm_rope(q_out=dense(BASE + 20 * MB, HQ)) == bad                   # over k
    assert norm_rope(k_out=dense(BASE + 10 * MB)) == bad                       # over q_out
    assert norm_rope(k_out=dense(BASE)) == bad                                 # over q
    assert norm_rope(at=BASE + 10 * MB) == bad
    assert norm_rope(norm=ol.head_norm(BASE + 25 * MB)) == bad
    assert norm_rope(r=ol.Rope(BASE + 10 * MB, D, 0, 1.0)) == bad
    heads = HQ + 2 * HKV
    fused = lambda first: ol.Rows(BASE + 2 * first * D, T * heads * D, D, heads * D)  # noqa: E731
    q, k = fused(0), fused(HQ)
    assert norm_rope(q=q, q_out=q, k=k, k_out=k) == ol.OL_ERR_INJECTED         # in place in a projection's output
    assert norm_rope(q=q, q_out="qo", k=k, k_out="ko") == ol.OL_ERR_INJECTED
    assert norm_rope(q=q, q_out=q, k=k, k_out="ko") == ol.OL_ERR_INJECTED
    near = fused(HQ - 1)
    assert norm_rope(q=q, q_out=q, k=near, k_out=near) == bad                  # they share a head
    assert norm_rope(q=q, q_out=q, k=near, k_out="ko") == bad
    assert norm_rope(q=q, q_out="qo", k=k, k_out=fused(HQ + HKV)) == bad       # not in place, within the extent


# ------------------------------------------------- the tests' own definition, by hand

def test_e4m3_by_hand():
    x = torch.tensor([448.0, 449.0, 1e9, -465.0, 17.0, 18.0, 19.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 0.0],
                     dtype=torch.float64)
    assert fu.e4m3(x).tolist() == [448.0, 448.0, 448.0, -448.0, 16.0, 18.0, 20.0, 2.0 ** -9, 0.0, 2.0 ** -8, 0.0]
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[~torch.isnan(every)]
    assert torch.equal(fu.e4m3(every), every)


def test_block_by_hand():
    codes = torch.zeros(4, 1, dtype=torch.float64)
    codes, scale = fu.append_block(codes, 0.0, 0, torch.tensor([[448.0], [1.0]], dtype=torch.float64))
    assert scale == 1.0 and codes[:, 0].tolist() == [448.0, 1.0, 0.0, 0.0]
    codes, scale = fu.append_block(codes, scale, 2, torch.tensor([[1000.0]], dtype=torch.float64))
    assert scale == 4.0 and codes[:, 0].tolist() == [112.0, 0.25, 256.0, 0.0]  # 250 is a tie: to even
    codes, scale = fu.append_block(codes, scale, 3, torch.tensor([[math.inf]], dtype=torch.float64))
    assert math.isnan(scale) and codes[3, 0] == 0
