"""The operators around drafted tokens, as they are measured: rotary positions,
the rotating append to a cache, attention of a tree of drafted tokens over a
cache, and the accepted path moved to its place.

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


def listed():
    return [
        # one new token of 64 rows before a fused decode step: q and k heads of a projection, by-parts scaling
        dict(name="rope_decode_b64", op="rope", dtype="bf16", batch=64, heads=40, tokens=1, head_dim=128, rot=128,
             style="half", scaling="by_parts", factor=8.0, far=131072),
        # prompts of odd length, half of each head rotated, interleaved pairs
        dict(name="rope_prompt_f32_part", op="rope", dtype="f32", batch=3, heads=36, tokens=2047, head_dim=96, rot=48,
             style="interleaved", scaling="linear", factor=4.0, far=60000),
        # a decode step's append to pages of 16, q rotated on the way
        dict(name="append_decode_paged_b64", op="append", dtype="bf16", layout="paged", page=16, batch=64, q_heads=32,
             kv_heads=8, head_dim=128, rot=128, style="half", scaling="by_parts", factor=8.0, tokens=1, capacity=512,
             ragged=False, tree=False, far=131072),
        # four prompts of different lengths filled into a contiguous cache
        dict(name="append_prompt_b4", op="append", dtype="bf16", layout="contiguous", page=0, batch=4, q_heads=32,
             kv_heads=8, head_dim=128, rot=128, style="half", scaling="none", factor=1.0, tokens=4096, capacity=8192,
             ragged=True, tree=False, far=0),
        # drafted trees of up to 16 nodes: positions by depth, rows with fewer nodes, part of the head interleaved
        dict(name="append_tree_paged_b32", op="append", dtype="bf16", layout="paged", page=16, batch=32, q_heads=28,
             kv_heads=4, head_dim=128, rot=64, style="interleaved", scaling="ntk", factor=2.0, tokens=16, capacity=1024,
             ragged=True, tree=True, far=0),
        # the single-row shape verifying a tree of 8: latency
        dict(name="tree8_b1_gqa7", op="tree", dtype="bf16", layout="contiguous", page=0, batch=1, q_heads=28, kv_heads=4,
             head_dim=128, nodes=8, shortest=4097, longest=4097, ragged=False, window=-1),
        # the paged shape (rows of 1 to 16384 tokens) verifying trees of 16
        dict(name="tree16_paged_b64", op="tree", dtype="bf16", layout="paged", page=16, batch=64, q_heads=32, kv_heads=8,
             head_dim=128, nodes=16, shortest=1, longest=16384, ragged=True, window=-1),
        # the ragged contiguous shape with wide trees
        dict(name="tree64_b32", op="tree", dtype="bf16", layout="contiguous", page=0, batch=32, q_heads=32, kv_heads=8,
             head_dim=128, nodes=64, shortest=512, longest=8192, ragged=False, window=-1),
        # the widest trees: products dominate
        dict(name="tree256_gqa7_b8", op="tree", dtype="bf16", layout="paged", page=64, batch=8, q_heads=28, kv_heads=4,
             head_dim=128, nodes=256, shortest=2000, longest=6000, ragged=False, window=-1),
        # fp32 cache, a head size of no power of two, a left window
        dict(name="tree5_f32_window", op="tree", dtype="f32", layout="contiguous", page=0, batch=6, q_heads=16,
             kv_heads=2, head_dim=80, nodes=5, shortest=100, longest=4000, ragged=True, window=1000),
        # accepted paths of 64 rows, pages of 16
        dict(name="keep16_paged_b64", op="keep", dtype="bf16", layout="paged", page=16, batch=64, kv_heads=8,
             head_dim=128, nodes=16, capacity=512),
        # wide trees in a large batch of fp32 rows
        dict(name="keep64_f32_b128", op="keep", dtype="f32", layout="contiguous", page=0, batch=128, kv_heads=8,
             head_dim=128, nodes=64, capacity=256),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rotation(rng, head_dim):
    scaling = rng.choice(("none", "linear", "ntk", "by_parts"))
    return dict(rot=rng.choice((head_dim, head_dim, head_dim // 2)), style=rng.choice(("half", "interleaved")),
                scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0)))


def draw(rng):
    op = rng.choice(("rope", "append", "tree", "tree", "keep"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    layout = rng.choice(("contiguous", "paged"))
    page = rng.choice((16, 32, 64, 128)) if layout == "paged" else 0
    q_heads, kv_heads = rng.choice(HEADS)
    if op == "rope":
        head_dim = rng.choice((64, 80, 96, 128, 256))
        batch = _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, max(1, 6000 // batch))
        return dict(op=op, dtype=dtype, batch=batch, heads=rng.randint(1, 40), tokens=tokens, head_dim=head_dim,
                    far=rng.choice((0, 4096, 131072, 1000000)), **_rotation(rng, head_dim))
    if op == "append":
        head_dim = rng.choice((64, 96, 128, 256))
        batch = _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, max(1, 8192 * 128 // (batch * head_dim)))
        tree = tokens <= 256 and rng.random() < 0.5
        capacity = tokens + rng.randint(1, 200)
        if page:
            capacity = -(-capacity // page) * page
        return dict(op=op, dtype=dtype, layout=layout, page=page, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                    head_dim=head_dim, tokens=tokens, capacity=capacity, ragged=rng.random() < 0.5, tree=tree,
                    far=0 if tree else rng.choice((0, 131072)), **_rotation(rng, head_dim))
    if op == "tree":
        head_dim = rng.choice((64, 128, 128, 80)) if dtype == "f32" else rng.choice((64, 128, 128, 128, 96))
        batch = _log_int(rng, 1, 64)
        nodes = _log_int(rng, 1, 64 if dtype == "f32" else 256)
        # no more K/V and no more scores than the listed cases have; fp32 and small heads stay smaller
        share = 32 if dtype == "f32" or head_dim not in (64, 128) else 1
        most = min(64 * 16384 * 8 * 128 // (2 * share * batch * kv_heads * head_dim),
                   64 * 32 * 16 * 16384 // (2 * share * batch * q_heads * nodes), 16384)
        longest = max(nodes + 1, _log_int(rng, 64, max(64, most)))
        window = rng.choice((-1, -1, -1, rng.randint(0, longest)))
        return dict(op=op, dtype=dtype, layout=layout, page=page, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
                    head_dim=head_dim, nodes=nodes, shortest=rng.randint(1, longest), longest=longest,
                    ragged=rng.random() < 0.5, window=window)
    head_dim = rng.choice((64, 80, 128, 256))
    nodes = _log_int(rng, 1, 128)
    batch = _log_int(rng, 1, max(1, 128 * 64 * 128 // (2 * nodes * head_dim)))
    batch = min(batch, 128)
    capacity = nodes + rng.randint(1, 200)
    if page:
        capacity = -(-capacity // page) * page
    return dict(op=op, dtype=dtype, layout=layout, page=page, batch=batch, kv_heads=kv_heads, head_dim=head_dim,
                nodes=nodes, capacity=capacity)


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """Angle per position of each pair, radians, fp64 (numpy): the definition of the scalings."""
    r, s = case["rot"], case["factor"]
    base = 10000.0
    if case["scaling"] == "ntk":
        base *= s ** (r / (r - 2))
    f = base ** (-2.0 * np.arange(r // 2) / r)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "by_parts":
        turns = ORIGINAL * f / (2 * math.pi)
        keep = np.clip((turns - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = f / s * (1 - keep) + f * keep
    return f


ORIGINAL, LOW, HIGH = 8192.0, 1.0, 32.0


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0


def _trees(rng, batch, nodes):
    """Random trees in topological order: ancestor bits [B, T, W] (each node's own bit too) and depths [B, T]."""
    words = -(-nodes // 64)
    bits = np.zeros((batch, nodes, words), np.uint64)
    depth = np.zeros((batch, nodes), np.int32)
    rows = np.arange(batch)
    for i in range(nodes):
        parent = rng.integers(max(-1, i // 2 - 1), max(i, 1), size=batch) if i else np.full(batch, -1)
        root = parent < 0
        above = bits[rows, np.maximum(parent, 0)].copy()
        above[root] = 0
        above[:, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        bits[:, i] = above
        depth[:, i] = np.where(root, 0, depth[rows, np.maximum(parent, 0)] + 1)
    return bits, depth


def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _storage(case, gen, rng, state):
    """The cache: contiguous [2, B, Hkv, C, D], or a pool of pages and its table."""
    dtype, batch, page = DTYPES[case["dtype"]], case["batch"], case["page"]
    capacity = case["capacity"] if "capacity" in case else case["longest"]
    if case["layout"] == "contiguous":
        shape = (2, batch, case["kv_heads"], capacity, case["head_dim"])
    else:
        per_row = -(-capacity // page)
        pages = batch * per_row + 3
        table = rng.permutation(pages)[: batch * per_row].astype(np.int32).reshape(batch, per_row)
        state["table_host"], state["table"] = table, _device(table)
        shape = (2, pages, case["kv_heads"], page, case["head_dim"])
    state["cache"] = torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dtype, batch = DTYPES[case["dtype"]], case["batch"]
    state = {"case": case}
    if case["op"] in ("rope", "append"):
        state["inv_freq"] = _device(_frequencies(case))
    if case["op"] == "rope":
        shape = (batch, case["tokens"], case["heads"], case["head_dim"])  # a projection's output, token by token
        state["x"] = torch.randn(shape, generator=gen, device=DEV, dtype=dtype).transpose(1, 2)
        first = rng.integers(0, case["far"] + 1, size=(batch, 1))
        state["positions"] = _device((first + np.arange(case["tokens"])).astype(np.int32))
        state["out"] = torch.zeros((batch, case["heads"], case["tokens"], case["head_dim"]), device=DEV, dtype=dtype)
    elif case["op"] == "append":
        t, hq, hkv = case["tokens"], case["q_heads"], case["kv_heads"]
        qkv = torch.randn((batch, t, hq + 2 * hkv, case["head_dim"]), generator=gen, device=DEV, dtype=dtype)
        state["q"], state["k"], state["v"] = qkv.transpose(1, 2).split((hq, hkv, hkv), dim=1)
        counts = rng.integers(0, t + 1, size=batch).astype(np.int32) if case["ragged"] else np.full(batch, t, np.int32)
        start = np.array([rng.integers(0, case["capacity"] - n + 1) for n in counts], np.int32)
        where = start[:, None] + np.arange(t)
        if case["tree"]:
            where = start[:, None] + _trees(rng, batch, t)[1]
        elif case["far"]:  # a window of a longer context: the cache's slots are not the positions
            where = where + rng.integers(0, case["far"] + 1, size=(batch, 1))
        state.update(counts_host=counts, counts=_device(counts), start_host=start, start=_device(start),
                     positions=_device(where.astype(np.int32)))
        live = np.nonzero(np.arange(t)[None] < counts[:, None])
        state["live"] = tuple(_device(a) for a in live)  # the (row, token) pairs that are appended
        _storage(case, gen, rng, state)
        state["out"] = torch.zeros((batch, hq, t, case["head_dim"]), device=DEV, dtype=dtype)
    elif case["op"] == "tree":
        t = case["nodes"]
        counts = rng.integers(1, t + 1, size=batch).astype(np.int32) if case["ragged"] else np.full(batch, t, np.int32)
        lens = np.maximum(rng.integers(case["shortest"], case["longest"] + 1, size=batch), counts).astype(np.int32)
        bits, depth = _trees(rng, batch, t)
        state.update(counts_host=counts, counts=_device(counts), lens_host=lens, lens=_device(lens),
                     mask=_device(bits.view(np.int64)),
                     positions=_device(((lens - counts)[:, None] + depth).astype(np.int32)))
        state["q"] = torch.randn((batch, case["q_heads"], t, case["head_dim"]), generator=gen, device=DEV, dtype=dtype)
        _storage(case, gen, rng, state)
        state["out"] = torch.zeros_like(state["q"])
    else:
        t = case["nodes"]
        start = rng.integers(0, case["capacity"] - t + 1, size=batch).astype(np.int32)
        counts = rng.integers(0, t + 1, size=batch).astype(np.int32)
        kept = np.argsort(rng.random((batch, t)), axis=1)
        kept = np.sort(np.where(np.arange(t)[None] < counts[:, None], kept, t), axis=1).astype(np.int32)
        state.update(start_host=start, start=_device(start), kept=_device(kept), kept_counts=_device(counts))
        _storage(case, gen, rng, state)
    if own:
        state["handle"] = _handle(state)
    return state


# ------------------------------------------------------- the framework's calls

def _handle(state):
    """What a program keeps between calls: the cache's descriptor, the rotation, views and the workspace."""
    import place_kv_cache_gb300 as ol
    case, h = state["case"], {"ol": ol}
    if case["op"] in ("rope", "append"):
        h["rope"] = ol.rope(case["rot"], style=ol.OL_ROPE_HALF if case["style"] == "half" else ol.OL_ROPE_INTERLEAVED,
                            base=10000.0, scaling={"none": ol.OL_ROPE_UNSCALED, "linear": ol.OL_ROPE_LINEAR,
                                                   "ntk": ol.OL_ROPE_NTK, "by_parts": ol.OL_ROPE_BY_PARTS}[case["scaling"]],
                            factor=case["factor"], original_len=ORIGINAL, low=LOW, high=HIGH,
                            magnitude=_magnitude(case))
        h["rows"] = {k: ol.rows(state[k]) for k in ("x", "q", "k", "v", "out") if k in state}
    if "cache" in state:
        if case["layout"] == "contiguous":
            h["layout"], h["desc"] = ol.OL_LAYOUT_CONTIGUOUS, ol.kv_cache(state["cache"])
        else:
            h["layout"], h["desc"] = ol.OL_LAYOUT_PAGED, ol.paged_kv(state["cache"], state["table"], state["table_host"])
    if case["op"] == "tree":
        n = ol.ol_workspace_size_tree(case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["nodes"])
        h["ws"], h["ws_bytes"] = torch.empty(n, dtype=torch.uint8, device=DEV), n
        ol.ol_workspace_init(h["ws"], n)
    return h


def _run_own(state):
    case, h = state["case"], state["handle"]
    ol = h["ol"]
    code = ol.OL_BF16 if case["dtype"] == "bf16" else ol.OL_F32
    if case["op"] == "rope":
        ol.ol_rope_rows(h["rope"], code, case["batch"], case["heads"], case["tokens"], case["head_dim"], h["rows"]["x"],
                        h["rows"]["out"], state["positions"], True)
        return state["out"]
    if case["op"] == "append":
        r = h["rows"]
        ol.ol_rope_append(h["layout"], h["desc"], state["cache"], h["rope"], case["tokens"], r["k"], r["v"],
                          case["q_heads"], r["q"], r["out"], state["start_host"], state["start"],
                          state["counts_host"], state["counts"], state["positions"])
        return {"q": state["out"], "cache": state["cache"]}
    if case["op"] == "tree":
        ol.ol_tree_attention(h["layout"], h["desc"], state["q"], case["q_heads"], case["nodes"], state["lens_host"],
                             state["lens"], state["counts_host"], state["counts"], state["mask"], state["positions"],
                             0.0, case["window"], state["out"], code, h["ws"], h["ws_bytes"])
        return state["out"]
    ol.ol_tree_keep(h["layout"], h["desc"], state["cache"], case["nodes"], state["start_host"], state["start"],
                    state["kept"], state["kept_counts"])
    return state["cache"]


# ------------------------------------------------------------ the plain forms

def _rotated(state, x):
    """x [B, H, T, D] with its leading part rotated to the positions: fp32, angles in fp64."""
    case = state["case"]
    r = case["rot"]
    angle = state["positions"].double()[..., None] * state["inv_freq"]
    cos = (angle.cos() * _magnitude(case)).float()[:, None]
    sin = (angle.sin() * _magnitude(case)).float()[:, None]
    x = x.float()
    if case["style"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    return torch.cat((turned, x[..., r:]), dim=-1)


def _slots(state, row, token):
    """Index of cache tokens (row, token) behind the plane: the views cache[plane][index] are [n, Hkv, D]."""
    if state["case"]["layout"] == "contiguous":
        return row, slice(None), token
    page = state["case"]["page"]
    return state["table"][row, token // page].long(), slice(None), token % page


def _gathered(state, plane, n):
    """The first n tokens of every row of a plane, [B, Hkv, n, D] in fp32."""
    case = state["case"]
    if case["layout"] == "contiguous":
        return state["cache"][plane][:, :, :n].float()
    pages = state["cache"][plane][state["table"][:, : -(-n // case["page"])].long()]
    return pages.transpose(1, 2).flatten(2, 3)[:, :, :n].float()


def _run_plain(state):
    case = state["case"]
    if case["op"] == "rope":
        state["out"].copy_(_rotated(state, state["x"]))
        return state["out"]
    if case["op"] == "append":
        row, token = state["live"]
        place = _slots(state, row, state["start"][row].long() + token)
        state["out"][row, :, token] = _rotated(state, state["q"])[row, :, token].to(state["out"].dtype)
        state["cache"][0][place] = _rotated(state, state["k"])[row, :, token].to(state["cache"].dtype)
        state["cache"][1][place] = state["v"][row, :, token]
        return {"q": state["out"], "cache": state["cache"]}
    if case["op"] == "keep":
        t = torch.arange(case["nodes"], device=DEV)[None]
        taken = torch.where(t < state["kept_counts"][:, None], state["kept"], t)
        row = torch.arange(case["batch"], device=DEV)[:, None].expand_as(taken)
        source = _slots(state, row, state["start"][:, None].long() + taken)
        place = _slots(state, row, state["start"][:, None].long() + t)
        state["cache"][0][place] = state["cache"][0][source]
        state["cache"][1][place] = state["cache"][1][source]
        return state["cache"]
    t, group = case["nodes"], case["q_heads"] // case["kv_heads"]
    n = int(state["lens_host"].max())
    first = (state["lens"] - state["counts"])[:, None, None]                      # [B, 1, 1]: tokens before the tree
    key = torch.arange(n, device=DEV)[None, None]
    drafted = (key - first).clamp(0, t - 1)                                        # [B, 1, n]
    word = torch.gather(state["mask"], 2, (drafted // 64).expand(-1, t, -1))
    seen = ((word >> (drafted % 64)) & 1 != 0) & (key >= first) & (key < state["lens"][:, None, None])
    seen |= key < first
    if case["window"] >= 0:
        at = torch.gather(state["positions"], 1, drafted[:, 0].long())[:, None]
        at = torch.where(key < first, key, at)
        seen &= state["positions"][..., None] - at <= case["window"]
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
    batch, d = case["batch"], case["head_dim"]
    if case["op"] == "rope":
        vectors = batch * case["heads"] * case["tokens"]
        return {"bytes": vectors * d * size * 2 + batch * case["tokens"] * 4, "flops": vectors * case["rot"] * 3}
    if case["op"] == "append":
        tokens = batch * case["tokens"] * (0.5 if case["ragged"] else 1.0)  # counts are uniform in [0, tokens]
        heads = case["q_heads"] + 2 * case["kv_heads"]
        return {"bytes": tokens * heads * d * size * 2,
                "flops": tokens * (case["q_heads"] + case["kv_heads"]) * case["rot"] * 3}
    if case["op"] == "keep":
        tokens = batch * case["nodes"] * 0.5  # counts are uniform in [0, nodes]
        return {"bytes": tokens * 2 * case["kv_heads"] * d * size * 2 + tokens * 4, "flops": 0}
    nodes = case["nodes"] * (0.5 if case["ragged"] else 1.0)
    seen = (case["shortest"] + case["longest"]) / 2
    if case["window"] >= 0:
        seen = min(seen, case["window"] + nodes)
    kv = 2 * batch * case["kv_heads"] * seen * d * size
    return {"bytes": kv + 2 * batch * case["q_heads"] * nodes * d * size,
            "flops": 4 * batch * case["q_heads"] * nodes * seen * d}


def _turned_exactly(case, positions, x):
    """x [..., D] fp64 at positions [...]: the rotation as a product of complex numbers."""
    r = case["rot"]
    angle = positions.double()[..., None] * torch.from_numpy(_frequencies(case)).to(DEV)
    turn = torch.polar(torch.full_like(angle, _magnitude(case)), angle)
    head = x[..., :r]
    pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["style"] == "half" else head.unflatten(-1, (-1, 2))
    got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    got = got.transpose(-1, -2).flatten(-2) if case["style"] == "half" else got.flatten(-2)
    return torch.cat((got, x[..., r:]), -1)


def _row_of(state, plane, b, n):
    """Tokens [0, n) of row b of a plane, [Hkv, n, D]: a copy, token after token."""
    if state["case"]["layout"] == "contiguous":
        return state["cache"][plane, b, :, :n].double()
    page = state["case"]["page"]
    return torch.cat([state["cache"][plane, p] for p in state["table_host"][b, : -(-n // page)].tolist()], 1)[:, :n].double()


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _turned_exactly(case, state["positions"][:, None].expand(-1, case["heads"], -1), state["x"].double())
    if case["op"] in ("append", "keep"):
        cache = state["cache"].double()
        out = torch.zeros_like(state["out"], dtype=torch.float64) if case["op"] == "append" else None
        for b in range(case["batch"]):
            start = int(state["start_host"][b])
            if case["op"] == "append":
                n = int(state["counts_host"][b])
                if n == 0:
                    continue
                at = state["positions"][b, :n][None]
                out[b, :, :n] = _turned_exactly(case, at.expand(case["q_heads"], -1), state["q"][b, :, :n].double())
                new = (_turned_exactly(case, at.expand(case["kv_heads"], -1), state["k"][b, :, :n].double()),
                       state["v"][b, :, :n].double())
            else:
                n = int(state["kept_counts"][b])
                if n == 0:
                    continue
                rows = state["kept"][b, :n].long() + start
                reach = start + case["nodes"]
                new = tuple(_row_of(state, plane, b, reach)[:, rows] for plane in (0, 1))
            if case["layout"] == "contiguous":
                cache[0, b, :, start: start + n], cache[1, b, :, start: start + n] = new
            else:
                slot = torch.arange(start, start + n, device=DEV)
                pages = state["table"][b][slot // case["page"]].long()
                for plane in (0, 1):
                    cache[plane].index_put_((pages[:, None], torch.arange(case["kv_heads"], device=DEV)[None],
                                             (slot % case["page"])[:, None]), new[plane].transpose(0, 1).contiguous())
        return {"q": out, "cache": cache} if case["op"] == "append" else cache
    out = torch.zeros_like(state["out"], dtype=torch.float64)
    group = case["q_heads"] // case["kv_heads"]
    bits = state["mask"].cpu().numpy().view(np.uint64)
    for b in range(case["batch"]):
        n, t = int(state["lens_host"][b]), int(state["counts_host"][b])
        first = n - t
        allowed = np.ones((t, n), bool)
        for j in range(t):
            allowed[:, first + j] = (bits[b, :t, j // 64] >> np.uint64(j % 64)) & np.uint64(1)
        at = state["positions"][b, :t].cpu().numpy()
        if case["window"] >= 0:
            where = np.concatenate((np.arange(first), at))
            allowed &= at[:, None] - where[None] <= case["window"]
        hidden = ~_device(allowed)
        k, v = _row_of(state, 0, b, n), _row_of(state, 1, b, n)
        q = state["q"][b].double()
        for g in range(case["kv_heads"]):
            s = torch.einsum("htd,nd->htn", q[g * group: (g + 1) * group, :t], k[g]) / math.sqrt(case["head_dim"])
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            out[b, g * group: (g + 1) * group, :t] = torch.nan_to_num(torch.einsum("htn,nd->htd", p, v[g]), nan=0.0)
    return out
