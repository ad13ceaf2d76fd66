"""The operators of a cache held in 8 bits, as they are measured: norms of queries
and keys with the position rotation in the same pass, the append that quantises
to E4M3 with a scale for each block of tokens and head, reading such a cache
back, and attention over it.

Every case runs in two forms on the same inputs: the plain form (elementary
torch operations in fp32, angles in fp64) and, where ``own`` is true, the
framework's own calls. ``exact`` computes the same outputs from the
definitions in fp64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HEADS = ((28, 4), (32, 8), (8, 8), (16, 2))
TOP = 448.0         # the largest E4M3 value
LEAST = 2.0 ** -80  # the smallest scale but 0
EPS = 1e-6


def listed():
    return [
        # one new token of 64 rows before its append: latency
        dict(name="norm_rope_decode_b64", op="norm_rope", dtype="bf16", batch=64, q_heads=32, kv_heads=8, tokens=1,
             head_dim=128, rot=128, style="half", far=131072),
        # four prompts of 4096 tokens
        dict(name="norm_rope_prompt_b4", op="norm_rope", dtype="bf16", batch=4, q_heads=32, kv_heads=8, tokens=4096,
             head_dim=128, rot=128, style="half", far=0),
        # prompts of odd length in fp32, half of each head rotated, interleaved pairs
        dict(name="norm_rope_f32_part", op="norm_rope", dtype="f32", batch=3, q_heads=28, kv_heads=4, tokens=2047,
             head_dim=96, rot=48, style="interleaved", far=60000),
        # a decode step's append to pages of 16: most tokens continue a block
        dict(name="append_decode_paged_b64", op="append", dtype="bf16", page=16, block=16, batch=64, kv_heads=8,
             head_dim=128, tokens=1, capacity=512, ragged=False),
        # four prompts of different lengths filled into a contiguous cache
        dict(name="append_prompt_b4", op="append", dtype="bf16", page=0, block=64, batch=4, kv_heads=8, head_dim=128,
             tokens=4096, capacity=8192, ragged=True),
        # 8 rows of up to 8192 tokens read back from pages of 16
        dict(name="read_paged_b8", op="read", dtype="bf16", page=16, block=16, batch=8, kv_heads=8, head_dim=128,
             tokens=8192, capacity=8192, ragged=True),
        # a few tokens of a contiguous cache in fp32, a head size of no power of two
        dict(name="read_f32_short", op="read", dtype="f32", page=0, block=32, batch=3, kv_heads=2, head_dim=80,
             tokens=37, capacity=100, ragged=True),
        # a decode step of the single-row shape: latency
        dict(name="attention_b1_gqa7", op="attention", dtype="bf16", page=0, block=128, batch=1, q_heads=28, kv_heads=4,
             head_dim=128, tokens=1, shortest=4097, longest=4097, ragged=False, window=-1),
        # a decode step of the paged shape (rows of 1 to 16384 tokens)
        dict(name="attention_paged_b64", op="attention", dtype="bf16", page=16, block=16, batch=64, q_heads=32,
             kv_heads=8, head_dim=128, tokens=1, shortest=1, longest=16384, ragged=False, window=-1),
        # chunks of 4 tokens over the ragged contiguous shape
        dict(name="attention_chunk4_b32", op="attention", dtype="bf16", page=0, block=64, batch=32, q_heads=32,
             kv_heads=8, head_dim=128, tokens=4, shortest=512, longest=8192, ragged=False, window=-1),
        # chunks of up to 64 tokens of a prompt over pages of 64
        dict(name="attention_chunk64_b8", op="attention", dtype="bf16", page=64, block=64, batch=8, q_heads=28,
             kv_heads=4, head_dim=128, tokens=64, shortest=2000, longest=6000, ragged=True, window=-1),
        # fp32 queries, a head size of no power of two, a left window
        dict(name="attention_f32_window", op="attention", dtype="f32", page=32, block=32, batch=6, q_heads=16,
             kv_heads=2, head_dim=80, tokens=5, shortest=100, longest=4000, ragged=True, window=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "read", "attention", "attention"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    q_heads, kv_heads = rng.choice(HEADS)
    batch = _log_int(rng, 1, 64)
    if op == "norm_rope":
        head_dim = rng.choice((64, 80, 96, 128, 128, 256))
        tokens = _log_int(rng, 1, max(1, 6000 // batch))
        return dict(op=op, dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads, tokens=tokens,
                    head_dim=head_dim, rot=rng.choice((head_dim, head_dim, head_dim // 2)),
                    style=rng.choice(("half", "interleaved")), far=rng.choice((0, 4096, 131072, 1000000)))
    page = rng.choice((0, 0, 16, 32, 64, 128))
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= (page or 128)])
    head_dim = rng.choice((64, 80, 128, 128, 128, 256))
    if op in ("append", "read"):
        tokens = _log_int(rng, 1, max(1, 8192 * 128 // (batch * head_dim)))
        capacity = tokens + rng.randint(1, 200)
        if page:
            capacity = -(-capacity // page) * page
        return dict(op=op, dtype=dtype, page=page, block=block, batch=batch, kv_heads=kv_heads, head_dim=head_dim,
                    tokens=tokens, capacity=capacity, ragged=rng.random() < 0.5)
    tokens = 1 if rng.random() < 0.5 else _log_int(rng, 1, 64)
    # no more K/V and no more scores than the listed cases have; fp32 and other heads stay smaller
    share = 32 if dtype == "f32" or head_dim not in (64, 128) else 1
    most = min(64 * 16384 * 8 * 128 // (2 * share * batch * kv_heads * head_dim),
               8 * 28 * 64 * 6000 // (share * batch * q_heads * tokens), 16384)
    longest = max(tokens + 1, _log_int(rng, 64, max(64, most)))
    window = rng.choice((-1, -1, -1, rng.randint(0, longest)))
    return dict(op=op, dtype=dtype, page=page, block=block, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, tokens=tokens, shortest=rng.randint(1, longest), longest=longest,
                ragged=rng.random() < 0.5, window=window)


# ------------------------------------------------------------------ inputs

def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _storage(case, gen, rng, state):
    """The cache: codes [2, B, Hkv, C, D] with scales [2, B, Hkv, C / block], or a pool of pages and its table."""
    batch, page, block, heads = case["batch"], case["page"], case["block"], case["kv_heads"]
    capacity = case["capacity"] if "capacity" in case else case["longest"]
    if page:
        per_row = -(-capacity // page)
        pages = batch * per_row + 3
        table = rng.permutation(pages)[: batch * per_row].astype(np.int32).reshape(batch, per_row)
        state["table_host"], state["table"] = table, _device(table)
        shape = (2, pages, heads, page, case["head_dim"])
    else:
        shape = (2, batch, heads, capacity, case["head_dim"])
    # N(0, 1) tokens whose block's largest element is about 3
    values = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(TOP / 3.2).clamp_(-TOP, TOP)
    state["codes"] = values.to(torch.float8_e4m3fn)
    spread = torch.rand((*shape[:3], -(-shape[3] // block)), generator=gen, device=DEV)
    state["scales"] = (spread + 2.5) / TOP


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dtype, batch, t, d = DTYPES[case["dtype"]], case["batch"], case["tokens"], case["head_dim"]
    state = {"case": case}
    counts = rng.integers(0, t + 1, size=batch).astype(np.int32) if case.get("ragged") else np.full(batch, t, np.int32)
    if case["op"] == "norm_rope":
        hq, hkv = case["q_heads"], case["kv_heads"]
        # a fused projection's output, token by token, with V behind
        qkv = torch.randn((batch, t, hq + 2 * hkv, d), generator=gen, device=DEV, dtype=dtype)
        state["q"], state["k"], _ = qkv.transpose(1, 2).split((hq, hkv, hkv), dim=1)
        state["qw"], state["kw"] = (1 + 0.1 * torch.randn((2, d), generator=gen, device=DEV)).to(dtype)
        first = rng.integers(0, case["far"] + 1, size=(batch, 1))
        state["positions"] = _device((first + np.arange(t)).astype(np.int32))
        state["inv_freq"] = _device(_frequencies(case))
        state["q_out"] = torch.zeros((batch, hq, t, d), device=DEV, dtype=dtype)
        state["k_out"] = torch.zeros((batch, hkv, t, d), device=DEV, dtype=dtype)
    elif case["op"] in ("append", "read"):
        start = np.array([rng.integers(0, case["capacity"] - n + 1) for n in counts], np.int32)
        state.update(counts_host=counts, counts=_device(counts), start_host=start, start=_device(start))
        _storage(case, gen, rng, state)
        if case["op"] == "append":
            kv = torch.randn((batch, t, 2 * case["kv_heads"], d), generator=gen, device=DEV, dtype=dtype)
            state["k"], state["v"] = kv.transpose(1, 2).chunk(2, dim=1)
        else:
            state["k_out"], state["v_out"] = torch.zeros((2, batch, case["kv_heads"], t, d), device=DEV, dtype=dtype)
    else:
        counts = np.maximum(counts, 1)
        lens = np.maximum(rng.integers(case["shortest"], case["longest"] + 1, size=batch), counts).astype(np.int32)
        state.update(counts_host=counts, counts=_device(counts), lens_host=lens, lens=_device(lens))
        state["q"] = torch.randn((batch, case["q_heads"], t, d), generator=gen, device=DEV, dtype=dtype)
        _storage(case, gen, rng, state)
        state["out"] = torch.zeros_like(state["q"])
    if own:
        state["handle"] = _handle(state)
    return state


def _frequencies(case):
    """Angle per position of each pair, radians, fp64 (numpy)."""
    return 10000.0 ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])


# ------------------------------------------------------- the framework's calls

def _handle(state):
    """What a program keeps between calls: the cache's descriptor, rotation and norms, views and the workspace."""
    import place_kv_cache_gb300 as ol
    case, h = state["case"], {"ol": ol}
    h["rows"] = {k: ol.rows(state[k]) for k in ("q", "k", "v", "q_out", "k_out", "v_out") if k in state}
    h["code"] = ol.OL_BF16 if case["dtype"] == "bf16" else ol.OL_F32
    if case["op"] == "norm_rope":
        h["rope"] = ol.rope(case["rot"], style=ol.OL_ROPE_HALF if case["style"] == "half" else ol.OL_ROPE_INTERLEAVED)
        h["norm"] = ol.head_norm(state["qw"], state["kw"], eps=EPS)
        return h
    h["kv"] = ol.fp8_kv(state["codes"], state["scales"], state.get("table"), state.get("table_host"),
                        block=case["block"])
    if case["op"] == "attention":
        n = ol.ol_workspace_size_fp8kv(case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"],
                                       case["tokens"])
        h["ws"], h["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device=DEV), n
        ol.ol_workspace_init(h["ws"], n)
    return h


def _run_own(state):
    case, h = state["case"], state["handle"]
    ol, r = h["ol"], h["rows"]
    if case["op"] == "norm_rope":
        ol.ol_norm_rope_rows(h["rope"], h["norm"], h["code"], case["batch"], case["tokens"], case["head_dim"],
                             case["q_heads"], r["q"], r["q_out"], case["kv_heads"], r["k"], r["k_out"],
                             state["positions"], True)
        return {"q": state["q_out"], "k": state["k_out"]}
    if case["op"] == "append":
        ol.ol_fp8kv_append(h["kv"], state["codes"], h["code"], case["tokens"], r["k"], r["v"], state["start_host"],
                           state["start"], state["counts_host"], state["counts"])
        return {"codes": state["codes"], "scales": state["scales"]}
    if case["op"] == "read":
        ol.ol_fp8kv_read(h["kv"], h["code"], case["tokens"], r["k_out"], r["v_out"], state["start_host"],
                         state["start"], state["counts_host"], state["counts"])
        return {"k": state["k_out"], "v": state["v_out"]}
    ol.ol_fp8kv_attention(h["kv"], h["code"], state["q"], case["q_heads"], case["tokens"], state["lens_host"],
                          state["lens"], state["counts_host"], state["counts"], 0.0, case["window"], state["out"],
                          h["code"], h["ws"], h["ws_bytes"])
    return state["out"]


# ------------------------------------------------------------ the plain forms

def _normed_rotated(state, x, weight):
    """x [B, H, T, D] over its root mean square, times the weights, its leading part rotated: fp32, angles in fp64."""
    case = state["case"]
    r = case["rot"]
    angle = state["positions"].double()[..., None] * state["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if case["style"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    return torch.cat((turned, x[..., r:]), dim=-1)


def _place(state, row, token):
    """Index of tokens behind the plane: codes[plane][index] is [..., Hkv, D] for row and token of any shape."""
    page = state["case"]["page"]
    if not page:
        return row, slice(None), token
    return state["table"][row, token // page].long(), slice(None), token % page


def _scale_place(state, row, token):
    """The same for the scales of the tokens' blocks."""
    page, block = state["case"]["page"], state["case"]["block"]
    if not page:
        return row, slice(None), token // block
    return state["table"][row, token // page].long(), slice(None), token % page // block


def _coded(x, s):
    """The E4M3 values of x / s, in fp32; 0 where there is no scale."""
    q = torch.where((s > 0) & (s < math.inf), x / s, 0.0)
    return q.clamp(-TOP, TOP).to(torch.float8_e4m3fn).float()


def _append_plane(state, plane, x):
    case = state["case"]
    b, t, block, d = case["batch"], case["tokens"], case["block"], case["head_dim"]
    blocks = (t + block - 2) // block + 1                             # that a row's tokens may lie in
    first = state["start"].long() // block * block                    # [B]
    cell = first[:, None] + torch.arange(blocks * block, device=DEV)  # [B, blocks * block]: tokens of the cache
    new = cell - state["start"][:, None]
    mine = (new >= 0) & (new < state["counts"][:, None])
    kept = (new < 0)[..., None, None]
    capacity = case["capacity"]
    row = torch.arange(b, device=DEV)[:, None].expand_as(cell)
    at = cell.clamp(max=capacity - 1)
    given = torch.gather(x.transpose(1, 2).float(), 1,
                         new.clamp(0, t - 1)[..., None, None].expand(-1, -1, case["kv_heads"], d))
    given = torch.where(mine[..., None, None], given, 0.0)            # [B, cells, Hkv, D]
    most = given.abs().unflatten(1, (blocks, block)).amax((2, 4))     # [B, blocks, Hkv]
    # (by a tensor: a quotient by a number is a product with its rounded inverse)
    fresh = torch.where(most > 0, (most / torch.full_like(most, TOP)).clamp(min=LEAST), 0.0)
    fresh = torch.where(most < math.inf, fresh, math.nan)
    head = cell[:, ::block]
    place = _scale_place(state, row[:, ::block], at[:, ::block])
    old = state["scales"][plane][place]                               # [B, blocks, Hkv]
    begun = (head < state["start"][:, None])[..., None]
    limit = TOP * old
    grown = torch.exp2(torch.ceil(torch.log2(most.double() / limit.double())).clamp(min=0)).float()
    grown = torch.where(most > limit * grown, grown * 2, grown)       # (a logarithm next to a whole number)
    grown = torch.where((grown > 1) & (most <= limit * grown * 0.5), grown * 0.5, grown)
    scale = torch.where(begun & (old != 0), torch.where(most < math.inf, old * grown, math.nan), fresh)
    wide = scale.repeat_interleave(block, 1)[..., None]               # [B, cells, Hkv, 1]
    before = state["codes"][plane].view(torch.uint8)[_place(state, row, at)].view(torch.float8_e4m3fn).float()
    shrunk = (before * (old / scale).repeat_interleave(block, 1)[..., None]).to(torch.float8_e4m3fn).float()
    grew = (begun & (old != 0) & (grown > 1) & (most < math.inf)).repeat_interleave(block, 1)[..., None]
    codes = torch.where(kept, torch.where(grew, shrunk, before), _coded(given, wide))
    touched = mine.unflatten(1, (blocks, block)).any(-1)              # [B, blocks]
    write = touched.repeat_interleave(block, 1) & (mine | kept[..., 0, 0])
    r, c = row[write], cell[write]
    state["codes"][plane].view(torch.uint8)[_place(state, r, c)] = \
        codes[write].to(torch.float8_e4m3fn).view(torch.uint8)
    r, c = row[:, ::block][touched], head[touched]
    state["scales"][plane][_scale_place(state, r, c)] = scale[touched]


def _gathered(state, plane, n):
    """The first n tokens of every row of a plane, [B, Hkv, n, D] in fp32."""
    case = state["case"]
    if not case["page"]:
        codes, scales = state["codes"][plane][:, :, :n].float(), state["scales"][plane]
    else:
        index = state["table"][:, : -(-n // case["page"])].long()
        codes = state["codes"][plane].view(torch.uint8)[index].view(torch.float8_e4m3fn).float()
        codes = codes.transpose(1, 2).flatten(2, 3)[:, :, :n]
        scales = state["scales"][plane][index].transpose(1, 2).flatten(2, 3)
    return codes * scales.repeat_interleave(case["block"], 2)[:, :, :n, None]


def _run_plain(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        state["q_out"].copy_(_normed_rotated(state, state["q"], state["qw"]))
        state["k_out"].copy_(_normed_rotated(state, state["k"], state["kw"]))
        return {"q": state["q_out"], "k": state["k_out"]}
    if case["op"] == "append":
        _append_plane(state, 0, state["k"])
        _append_plane(state, 1, state["v"])
        return {"codes": state["codes"], "scales": state["scales"]}
    t = case["tokens"]
    if case["op"] == "read":
        token = torch.arange(t, device=DEV)[None].expand(case["batch"], -1)
        row, token = torch.nonzero(token < state["counts"][:, None], as_tuple=True)
        at = state["start"][row].long() + token
        place, scale = _place(state, row, at), _scale_place(state, row, at)
        k = state["codes"][0].view(torch.uint8)[place].view(torch.float8_e4m3fn).float() * state["scales"][0][scale][..., None]
        v = state["codes"][1].view(torch.uint8)[place].view(torch.float8_e4m3fn).float() * state["scales"][1][scale][..., None]
        state["k_out"][row, :, token] = k.to(state["k_out"].dtype)
        state["v_out"][row, :, token] = v.to(state["v_out"].dtype)
        return {"k": state["k_out"], "v": state["v_out"]}
    group, n = case["q_heads"] // case["kv_heads"], int(state["lens_host"].max())
    at = (state["lens"] - state["counts"])[:, None] + torch.arange(t, device=DEV)  # [B, T]: the queries' positions
    key = torch.arange(n, device=DEV)[None, None]
    seen = key <= at[..., None]
    if case["window"] >= 0:
        seen &= key >= at[..., None] - case["window"]
    q = state["q"].float().view(case["batch"], case["kv_heads"], group * t, -1)
    scores = q @ _gathered(state, 0, n).transpose(2, 3) * case["head_dim"] ** -0.5
    scores = scores.view(case["batch"], case["kv_heads"], group, t, n).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weight = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = weight.sum(-1, keepdim=True)
    got = weight.view(case["batch"], case["kv_heads"], group * t, n) @ _gathered(state, 1, n)
    got = got.view(case["batch"], case["kv_heads"], group, t, -1) / torch.where(total == 0, 1.0, total)
    got = got.view(case["batch"], case["q_heads"], t, -1).to(state["out"].dtype)
    live = torch.arange(t, device=DEV) < state["counts"][:, None]
    state["out"].copy_(torch.where(live[:, None, :, None], got, state["out"]))
    return state["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------- work and definition

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    batch, t, d = case["batch"], case["tokens"], case["head_dim"]
    share = 0.5 if case.get("ragged") else 1.0  # counts are uniform in [0, tokens]
    if case["op"] == "norm_rope":
        vectors = batch * (case["q_heads"] + case["kv_heads"]) * t
        return {"bytes": vectors * d * size * 2 + batch * t * 4 + 2 * d * size,
                "flops": vectors * (4 * d + 3 * case["rot"])}
    if case["op"] in ("append", "read"):
        elements = 2 * batch * case["kv_heads"] * t * share * d
        scales = 4 * elements / (d * case["block"])
        return {"bytes": elements * (size + 1) + scales, "flops": elements * (2 if case["op"] == "append" else 1)}
    seen = (case["shortest"] + case["longest"]) / 2
    if case["window"] >= 0:
        seen = min(seen, case["window"] + t * share)
    kv = 2 * batch * case["kv_heads"] * seen * (d + 4 / case["block"])
    return {"bytes": kv + 2 * batch * case["q_heads"] * t * share * d * size,
            "flops": 4 * batch * case["q_heads"] * t * share * seen * d}


def _turned_exactly(case, positions, x):
    """x [..., D] fp64 at positions [...]: the rotation as a product of complex numbers."""
    r = case["rot"]
    angle = positions.double()[..., None] * torch.from_numpy(_frequencies(case)).to(DEV)
    turn = torch.polar(torch.ones_like(angle), angle)
    head = x[..., :r]
    pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["style"] == "half" else head.unflatten(-1, (-1, 2))
    got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    got = got.transpose(-1, -2).flatten(-2) if case["style"] == "half" else got.flatten(-2)
    return torch.cat((got, x[..., r:]), -1)


def _e4m3(x):
    """fp64 values rounded to E4M3, nearest even, by arithmetic: 4 significant bits, steps of 2^-9 at least."""
    step = torch.exp2((torch.frexp(x)[1].double() - 4).clamp(min=-9.0))
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _row_view(state, what, plane, b):
    """All of row b's tokens (or blocks) of a plane as a new tensor [Hkv, n, ...], fp64."""
    if not state["case"]["page"]:
        return what[plane, b].double()
    pages = [what[plane, p].double() for p in state["table_host"][b].tolist()]
    return torch.cat(pages, 1)


def _put_row(state, what, plane, b, value):
    """The inverse: row b's tokens (or blocks) put into an fp64 copy of the cache."""
    if not state["case"]["page"]:
        what[plane, b] = value
        return
    for i, p in enumerate(state["table_host"][b].tolist()):
        n = what.shape[3]
        what[plane, p] = value[:, i * n: (i + 1) * n]


def _append_exactly(case, state):
    codes, scales, block = state["codes"].double(), state["scales"].double(), case["block"]
    for plane, x in ((0, state["k"]), (1, state["v"])):
        for b in range(case["batch"]):
            n, start = int(state["counts_host"][b]), int(state["start_host"][b])
            if n == 0:
                continue
            c, s = _row_view(state, codes, plane, b), _row_view(state, scales, plane, b)
            for at in range(start // block, (start + n - 1) // block + 1):
                lo, hi = max(start, at * block), min(start + n, at * block + block)
                part = x[b, :, lo - start: hi - start].double()
                most = part.abs().amax((1, 2))
                one = (most / torch.full_like(most, TOP)).float().double().clamp(min=LEAST) * (most > 0)
                if lo > at * block:
                    was = s[:, at]
                    limit = (was * TOP).float().double()
                    times = torch.ones_like(was)
                    for _ in range(300):
                        times = torch.where(most > limit * times, times * 2, times)
                    c[:, at * block: lo] = torch.where((times > 1)[:, None, None],
                                                       _e4m3(c[:, at * block: lo] / times[:, None, None]),
                                                       c[:, at * block: lo])
                    one = torch.where(was == 0, one, was * times)
                s[:, at] = one
                safe = torch.where(one == 0, 1.0, one)[:, None, None]
                c[:, lo: hi] = _e4m3((part / safe).float().double()) * (one != 0)[:, None, None]
            _put_row(state, codes, plane, b, c)
            _put_row(state, scales, plane, b, s)
    return {"codes": codes, "scales": scales}


def _values(case, state, plane, b, first, n):
    """Tokens [first, first + n) of row b of a plane, [Hkv, n, D]: code times scale."""
    c = _row_view(state, state["codes"], plane, b)[:, first: first + n]
    s = _row_view(state, state["scales"], plane, b)
    return c * s[:, torch.arange(first, first + n, device=DEV) // case["block"]][..., None]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm_rope":
        got = {}
        for name, weight in (("q", "qw"), ("k", "kw")):
            x = state[name].double()
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["head_dim"] + EPS) * state[weight].double()
            got[name] = _turned_exactly(case, state["positions"][:, None].expand(-1, x.shape[1], -1), x)
        return got
    if case["op"] == "append":
        return _append_exactly(case, state)
    if case["op"] == "read":
        k, v = state["k_out"].double(), state["v_out"].double()
        for b in range(case["batch"]):
            n, start = int(state["counts_host"][b]), int(state["start_host"][b])
            k[b, :, :n] = _values(case, state, 0, b, start, n)
            v[b, :, :n] = _values(case, state, 1, b, start, n)
        return {"k": k, "v": v}
    out = torch.zeros_like(state["out"], dtype=torch.float64)
    group = case["q_heads"] // case["kv_heads"]
    for b in range(case["batch"]):
        n, t = int(state["lens_host"][b]), int(state["counts_host"][b])
        at = torch.arange(n - t, n, device=DEV)[:, None]
        key = torch.arange(n, device=DEV)[None]
        hidden = key > at
        if case["window"] >= 0:
            hidden |= key < at - case["window"]
        k, v = _values(case, state, 0, b, 0, n), _values(case, state, 1, b, 0, n)
        q = state["q"][b].double()
        for g in range(case["kv_heads"]):
            s = torch.einsum("htd,nd->htn", q[g * group: (g + 1) * group, :t], k[g]) / math.sqrt(case["head_dim"])
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            out[b, g * group: (g + 1) * group, :t] = torch.einsum("htn,nd->htd", p, v[g])
    return out
