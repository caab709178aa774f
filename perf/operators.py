"""What the cache operators cost: rotary positions, appending rows to a KV cache, reading
rows back, and attention over a cache held in 4 bits.

Every case runs either in its plain form (elementary torch operations in 32 bits) or, with
`own` set, through the library's entry points, on the same inputs.

The 4-bit format both forms read and write: 16 consecutive slots of one key/value head are a
block of 9 * dh bytes, first 16 rows of dh/2 bytes (element 2i in the low nibble of byte i,
2i + 1 in the high one, each a sign and an e2m1 magnitude), then 16 rows of dh/16 scales in
e4m3, one for each 16 elements.  An element stands for e2m1 * scale * g, g one number for all
keys and one for all values.  Contiguous caches are [B][Hkv][capacity/16] blocks, paged ones
[pages][Hkv][page/16].
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
K_SCALE, V_SCALE = 0.5, 0.25       # powers of two: what is held stays exact in bf16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's 65 tree nodes, queries and keys out of one projection's rows
        {"name": "rope_tree", "op": "rope", "rows": 65, "hq": 32, "hk": 32, "dh": 128, "rot": 128,
         "layout": "half", "scaling": "plain", "dtype": "bf16", "max_pos": 4096},
        # two long prompts of a model with shared key heads, half of each head rotated,
        # positions stretched to long contexts
        {"name": "rope_prompt", "op": "rope", "rows": 16381, "hq": 32, "hk": 8, "dh": 128, "rot": 64,
         "layout": "interleaved", "scaling": "ramp", "dtype": "bf16", "max_pos": 131072},
        # serving: one new token in each of 16 sequences, paged cache
        {"name": "append_tokens", "op": "append", "B": 16, "hk": 8, "dh": 128, "fmt": "bf16",
         "dtype": "bf16", "page": 16, "before": "1000-4000", "new": "1-1", "rot": 128,
         "layout": "half", "lens": 1},
        # a small batch of short ragged prompts in full precision
        {"name": "append_short_f32", "op": "append", "B": 6, "hk": 4, "dh": 128, "fmt": "f32",
         "dtype": "f32", "page": 0, "before": "0-40", "new": "1-300", "rot": 128,
         "layout": "half", "lens": 2},
        # prompts of a batch of 8 into a 4-bit cache, and the whole cache read back
        {"name": "append_prompts_kv4", "op": "append", "B": 8, "hk": 40, "dh": 128, "fmt": "kv4",
         "dtype": "bf16", "page": 0, "before": "0-0", "new": "2048-4096", "rot": 128,
         "layout": "half", "lens": 3},
        # one sequence's prefix taken out of a 4-bit cache
        {"name": "read_one", "op": "read", "B": 1, "hk": 32, "dh": 128, "page": 0, "len": "1024-1024",
         "dtype": "bf16", "lens": 4},
        # the prefixes of a whole paged batch taken out
        {"name": "read_batch", "op": "read", "B": 16, "hk": 8, "dh": 128, "page": 16,
         "len": "4100-8192", "dtype": "bf16", "lens": 5},
        # plain decoding of one sequence: one query row for each key head
        {"name": "attn_token", "op": "attention", "B": 1, "hq": 32, "hk": 32, "dh": 128, "n1": 1,
         "len": "1024-1024", "page": 0, "dtype": "bf16", "lens": 6},
        # plain decoding of a batch with long prefixes, 4 query heads to a key head
        {"name": "attn_tokens_gqa", "op": "attention", "B": 16, "hq": 32, "hk": 8, "dh": 128, "n1": 1,
         "len": "4100-8192", "page": 16, "dtype": "bf16", "lens": 7},
        # verification of a 64-candidate tree in a batch of 8
        {"name": "attn_tree", "op": "attention", "B": 8, "hq": 40, "hk": 40, "dh": 128, "n1": 65,
         "len": "2048-4096", "page": 0, "dtype": "bf16", "lens": 8},
        # verification of a 42-candidate tree, long paged prefixes, 4 query heads to a key head
        {"name": "attn_tree_gqa", "op": "attention", "B": 16, "hq": 32, "hk": 8, "dh": 128, "n1": 43,
         "len": "8192-8192", "page": 16, "dtype": "bf16", "lens": 9},
        # short ragged prefixes in full precision
        {"name": "attn_small_f32", "op": "attention", "B": 3, "hq": 8, "hk": 2, "dh": 64, "n1": 31,
         "len": "0-300", "page": 16, "dtype": "f32", "lens": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["rope", "append", "read", "attention", "attention"])
    for _ in range(1000):
        hk = rng.choice([1, 2, 4, 8, 32, 40])
        hq = hk * rng.choice([n for n in (1, 1, 2, 4, 7, 8) if n == 1 or hk * n <= 64])
        dh = rng.choice([32, 64, 128, 128, 128])
        page = rng.choice([0, 16, 16, 32, 48])
        B = _log(rng, 1, 32)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        lens = rng.randrange(1 << 30)
        hi = _log(rng, 1, 8192)
        lo = rng.choice([0, hi // 2, hi])
        rot = rng.choice([dh, dh, dh // 2, dh // 4 * 2 + 8 if dh > 32 else 16])
        layout = rng.choice(["half", "interleaved"])
        if op == "rope":
            case = {"op": op, "rows": _log(rng, 1, 16384), "hq": hq, "hk": hk, "dh": dh, "rot": rot,
                    "layout": layout, "scaling": rng.choice(["plain", "linear", "banded", "ramp"]),
                    "dtype": dtype, "max_pos": _log(rng, 512, 131072), "lens": lens}
        elif op == "append":
            new = _log(rng, 1, 4096)
            fmt = rng.choice([dtype, "kv4"])
            case = {"op": op, "B": B, "hk": hk, "dh": dh, "fmt": fmt, "dtype": dtype, "page": page,
                    "before": "0-%d" % rng.choice([0, _log(rng, 1, 2048)]),
                    "new": "%d-%d" % (rng.choice([0, new]), new), "rot": rot, "layout": layout,
                    "lens": lens}
        elif op == "read":
            case = {"op": op, "B": B, "hk": hk, "dh": dh, "page": page, "len": "%d-%d" % (lo, hi),
                    "dtype": dtype, "lens": lens}
        else:
            n1 = rng.choice([1, 1, _log(rng, 2, 200), rng.randrange(2, 70)])
            case = {"op": op, "B": B, "hq": hq, "hk": hk, "dh": dh, "n1": n1,
                    "len": "%d-%d" % (lo, hi), "page": page, "dtype": dtype, "lens": lens}
        if _cost(case) <= most[op]:
            return case
    return dict(case, B=1, rows=1) if op == "rope" else dict(case, B=1)


def _range(case, key):
    """The lengths of a case's sequences: drawn evenly from its range, its ends among them."""
    lo, hi = (int(x) for x in case[key].split("-"))
    r = np.random.RandomState((case["lens"] + len(key)) % (1 << 31))
    n = r.randint(lo, hi + 1, case["B"])
    n[-1] = hi
    if case["B"] > 1:
        n[0] = lo
    return [int(x) for x in n]


def _capacity(case, longest):
    unit = case["page"] or 16
    return (max(1, longest) + unit - 1) // unit * unit


def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    op, dh = case["op"], case["dh"]
    if op == "rope":
        n = case["rows"] * (case["hq"] + case["hk"]) * dh
        table = min(case["rows"], case["max_pos"]) * case["rot"] * 4
        return {"bytes": 2 * n * e + table, "flops": 3 * n * case["rot"] / dh}
    if op == "append":
        before, new = _range(case, "before"), _range(case, "new")
        n = 2 * sum(new) * case["hk"] * dh
        if case["fmt"] == "kv4":       # written once, and everything read back
            total = 2 * (sum(new) + sum(before)) * case["hk"] * dh
            return {"bytes": n * (e + 9 / 16) + total * (9 / 16 + 2), "flops": 6 * n}
        return {"bytes": n * (e + (4 if case["fmt"] == "f32" else 2)), "flops": 3 * n / 2}
    if op == "read":
        n = 2 * sum(_range(case, "len")) * case["hk"] * dh
        return {"bytes": n * (9 / 16 + e), "flops": 2 * n}
    total, n1 = sum(_range(case, "len")), case["n1"]
    rows = case["B"] * n1
    return {"bytes": 2 * total * case["hk"] * dh * 9 / 16 + 2 * rows * case["hq"] * dh * e
            + 2 * rows * case["hk"] * dh * e,
            "flops": 4.0 * dh * case["hq"] * (n1 * total + rows * min(n1, 8))}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _keys(g, shape):
    """Values as projections give them: a few channels of each head much larger."""
    gain = 1 + 3 * (torch.rand(shape[-2:], generator=g, device="cuda") < 0.05).float()
    return torch.randn(shape, generator=g, device="cuda") * gain


def _rope_case(case):
    """What a rotation needs beside the rows."""
    r = {"rot": case["rot"], "layout": case["layout"], "scaling": case.get("scaling", "plain"),
         "base": 10000.0, "factor": 1.0, "orig": 0, "low": 1.0, "high": 32.0, "attn": 1.0}
    if r["scaling"] != "plain":
        r.update(factor=8.0, orig=4096)
    if r["scaling"] == "banded":
        r.update(low=1.0, high=4.0)
    if r["scaling"] == "ramp":
        r.update(attn=0.1 * math.log(8.0) + 1.0)
    return r


def _frequencies(r):
    """f_i of every rotated pair, in 64 bits."""
    h = r["rot"] // 2
    f = [r["base"] ** (-2.0 * i / r["rot"]) for i in range(h)]
    if r["scaling"] == "plain":
        return f
    if r["scaling"] == "linear":
        return [x / r["factor"] for x in f]
    if r["scaling"] == "banded":
        keep = [(r["orig"] * x / (2 * math.pi) - r["low"]) / (r["high"] - r["low"]) for x in f]
    else:
        def pair(turns):
            return r["rot"] * math.log(r["orig"] / (2 * math.pi * turns)) / (2 * math.log(r["base"]))
        a = max(0.0, math.floor(pair(r["high"])))
        b = min(r["rot"] - 1.0, math.ceil(pair(r["low"])))
        keep = [1 - (i - a) / max(b - a, 0.001) for i in range(h)]
    keep = [min(1.0, max(0.0, k)) for k in keep]
    return [k * x + (1 - k) * x / r["factor"] for k, x in zip(keep, f)]


def _table(r, max_pos):
    """cos and sin for every position, [max_pos][rot/2] in 32 bits, from angles in 64."""
    f = torch.tensor(_frequencies(r), dtype=torch.float64, device="cuda")
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return ((a.cos() * r["attn"]).float(), (a.sin() * r["attn"]).float())


def _e2m1(a):
    """Code of the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to a >= 0, ties to the even code."""
    return ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())


def _quantise(x, g):
    """[..., dh] in 32 bits -> packed codes [..., dh/2] and scales [..., dh/16], as bytes."""
    y = x.unflatten(-1, (-1, 16))
    top = y.abs().amax(-1)
    # a true quotient (dividing by a number may multiply by its rounded reciprocal)
    s8 = (top / torch.full_like(top, 6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = (s8.float() * g).unsqueeze(-1)
    code = torch.where(s > 0, _e2m1(torch.where(s > 0, y.abs() / s, s)), 0)
    code = (code + 8 * (y < 0).int()).flatten(-2).to(torch.uint8)
    return code[..., 0::2] + code[..., 1::2] * 16, s8.view(torch.uint8)


def _blocks(pool, dh):
    """Views of a pool [blocks][9 dh]: codes [blocks][16][dh/2], scales [blocks][16][dh/16]."""
    return pool[:, :8 * dh].unflatten(1, (16, dh // 2)), pool[:, 8 * dh:].unflatten(1, (16, dh // 16))


def _values(codes, scales, g, mag):
    """What packed codes [..., dh/2] and scales [..., dh/16] stand for, in 32 bits; `mag`:
    the 16 codes' values."""
    v = torch.stack((mag[(codes & 15).int()], mag[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * g
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _pages(case, B, capacity, seed):
    """A page table whose pages lie in no order, with some pages that no sequence has."""
    n = capacity // case["page"]
    total = B * n + 3
    p = np.random.RandomState((seed * 7 + 1) % (1 << 31)).permutation(total)[:B * n].reshape(B, n)
    return _ints(p), total


def _pool(g, slots, hk, dh, k_scale):
    """A 4-bit pool of `slots` slots of hk heads, filled with quantised values."""
    pool = torch.empty(slots // 16 * hk, 9 * dh, dtype=torch.uint8, device="cuda")
    part = max(1, (1 << 26) // (16 * dh))
    gain = None
    for i in range(0, pool.shape[0], part):
        n = min(part, pool.shape[0] - i)
        if gain is None:
            gain = 1 + 3 * (torch.rand(dh, generator=g, device="cuda") < 0.05).float()
        codes, scales = _quantise(torch.randn(n, 16, dh, generator=g, device="cuda") * gain, k_scale)
        pool[i:i + n] = torch.cat((codes.flatten(1), scales.flatten(1)), 1)
    return pool


def _starts(n):
    return _ints([0] + list(np.cumsum(n)))


def _binding():
    from medusa_head_speculative_gb300 import binding
    return binding


def _rope_handle(r, max_pos):
    b = _binding()
    return b.Rope(r["rot"], max_pos, layout=r["layout"], base=r["base"], scaling=r["scaling"],
                  factor=r["factor"], orig_pos=r["orig"], low=r["low"], high=r["high"], attn=r["attn"])


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case, "mag": torch.tensor(_MAG + tuple(-m for m in _MAG), device="cuda")}
    dh = case["dh"]
    dt = _DT[case["dtype"]]
    if case["op"] == "rope":
        rows, hq, hk = case["rows"], case["hq"], case["hk"]
        r = _rope_case(case)
        # q and k as a projection leaves them: parts of rows that hold q, k and v
        qkv = torch.randn(rows, hq + 2 * hk, dh, generator=g, device="cuda").to(dt)
        # two runs of positions, the second one up to the last position there is
        n2 = min(rows // 2, case["max_pos"])
        n1 = rows - n2
        pos = torch.cat((torch.arange(n1) % case["max_pos"], torch.arange(n2) + case["max_pos"] - n2))
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], pos=pos.int().cuda(), rope=r,
                  q_out=torch.empty(rows, hq, dh, dtype=dt, device="cuda"),
                  k_out=torch.empty(rows, hk, dh, dtype=dt, device="cuda"))
        st["cos"], st["sin"] = _table(r, case["max_pos"])
        if own:
            st["handle"] = _rope_handle(r, case["max_pos"])
        return st
    B, hk, page = case["B"], case["hk"], case["page"]
    if case["op"] == "append":
        before, new = _range(case, "before"), _range(case, "new")
        after = [x + y for x, y in zip(before, new)]
        rows = sum(new)
        capacity = _capacity(case, max(after))
        src = _keys(g, (rows, 2 * hk, dh)).to(dt)
        st.update(k=src[:, :hk], v=src[:, hk:], rope=_rope_case(case), start=_starts(new), rows=rows)
    else:
        after = _range(case, "len")
        capacity = _capacity(case, max(after))
    st.update(capacity=capacity, pages=None, n_pages=0)
    if page:
        st["pages"], st["n_pages"] = _pages(case, B, capacity, seed)
    slots = st["n_pages"] * page if page else B * capacity
    fmt = case.get("fmt", "kv4")
    if fmt == "kv4":
        st["kc"], st["vc"] = _pool(g, slots, hk, dh, K_SCALE), _pool(g, slots, hk, dh, V_SCALE)
    else:
        shape = (st["n_pages"], page, hk, dh) if page else (B, capacity, hk, dh)
        st["kc"], st["vc"] = (torch.randn(shape, generator=g, device="cuda", dtype=_DT[fmt]) for _ in "kv")
    st["after"] = _ints(after)
    total = sum(after)
    if case["op"] == "append":
        st["len"] = _ints(before)
        st["len_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["cos"], st["sin"] = _table(st["rope"], capacity)
        out_dt = torch.bfloat16
    else:
        st["len"], out_dt = st["after"], dt
    if case["op"] == "read" or (case["op"] == "append" and fmt == "kv4"):
        st["all"], st["all_rows"] = _starts(after), total
        st["k_rows"], st["v_rows"] = (torch.empty(total, hk, dh, dtype=out_dt, device="cuda") for _ in "kv")
    n1 = case.get("n1", 1)
    if case["op"] == "attention":
        hq = case["hq"]
        st["q"] = torch.randn(B, n1, hq, dh, generator=g, device="cuda").to(dt)
        st["tk"] = _keys(g, (B, n1, hk, dh)).to(dt)
        st["tv"] = torch.randn(B, n1, hk, dh, generator=g, device="cuda").to(dt)
        st["o"] = torch.empty(B, n1, hq, dh, dtype=dt, device="cuda")
        # a candidate tree: every node under one of the nodes before it, at most 5 deep
        r = np.random.RandomState((seed * 3 + 2) % (1 << 31))
        see, depth = np.zeros((n1, 256), bool), [0] * n1
        see[0, 0] = True
        for n in range(1, n1):
            p = int(r.randint(0, n))
            while depth[p] >= 5:
                p = int(r.randint(0, n))
            depth[n] = depth[p] + 1
            see[n] = see[p]
            see[n, n] = True
        st["see"] = torch.from_numpy(see[:, :n1].copy()).cuda()
        bits = np.packbits(see, axis=1, bitorder="little").view(np.uint32)
        st["mask"] = torch.from_numpy(bits.view(np.int32).copy()).cuda()
    if own:
        b = _binding()
        st["cache"] = b.Cache(B, case.get("hq", hk), hk, dh, {"f32": b.F32, "bf16": b.BF16, "kv4": b.KV4}[fmt],
                              capacity, page_size=page, num_pages=st["n_pages"], max_nodes=n1)
        st["kv"] = b.kv_struct(st["kc"], st["vc"], st["len"], st.get("len_out"), st["pages"])
        if case["op"] == "append":
            st["handle"] = _rope_handle(st["rope"], capacity)
            st["kv_after"] = b.kv_struct(st["kc"], st["vc"], st["len_out"], None, st["pages"])
        if case["op"] == "attention":
            st["ws"] = torch.empty(st["cache"].workspace_size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, rot, layout):
    """x [rows][heads][dh] in 32 bits turned by its rows' angles."""
    c, s = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _sequences(start, rows):
    """The sequence of each packed row and its place there."""
    i = torch.arange(rows, device="cuda")
    b = torch.searchsorted(start[1:].long(), i, right=True)
    return b, i - start.long()[b]


def _slots(st, b, t):
    """Row of the cache ([slots][hk][dh]) that holds slot t of sequence b."""
    page = st["case"]["page"]
    if not page:
        return b * st["capacity"] + t
    return st["pages"][b, t // page].long() * page + t % page


def _kv4_place(st, b, t):
    """(block, row in it) for [rows][hk] of slot t of sequence b in a 4-bit cache."""
    hk, page = st["case"]["hk"], st["case"]["page"]
    per = (page or st["capacity"]) // 16
    first = st["pages"][b, t // page].long() if page else b
    t = t % page if page else t
    return (first[:, None] * hk + torch.arange(hk, device="cuda")) * per + (t // 16)[:, None], (t % 16)[:, None]


def _read_plain(st, pool, g, dt):
    b, t = _sequences(st["all"], st["all_rows"])
    at, row = _kv4_place(st, b, t)
    codes, scales = _blocks(pool, st["case"]["dh"])
    return _values(codes[at, row], scales[at, row], g, st["mag"]).to(dt)


def _append_plain(st):
    case = st["case"]
    b, i = _sequences(st["start"], st["rows"])
    t = st["len"].long()[b] + i
    k = _turn(st["k"].float(), st["cos"][t], st["sin"][t], case["rot"], case["layout"])
    v = st["v"].float()
    st["len_out"].copy_(st["len"] + (st["start"][1:] - st["start"][:-1]))
    if case["fmt"] != "kv4":
        at = _slots(st, b, t)
        st["kc"].flatten(0, 1)[at] = k.to(st["kc"].dtype)
        st["vc"].flatten(0, 1)[at] = v.to(st["vc"].dtype)
        return {"k": st["kc"], "v": st["vc"], "len": st["len_out"]}
    at, row = _kv4_place(st, b, t)
    for pool, x, g in ((st["kc"], k, K_SCALE), (st["vc"], v, V_SCALE)):
        codes, scales = _blocks(pool, case["dh"])
        codes[at, row], scales[at, row] = _quantise(x, g)
    return {"k": _read_plain(st, st["kc"], K_SCALE, torch.bfloat16),
            "v": _read_plain(st, st["vc"], V_SCALE, torch.bfloat16), "len": st["len_out"]}


def _prefix(st, pool, g):
    """A 4-bit cache's values as [B][hk][capacity][dh]."""
    case = st["case"]
    B, hk, dh, page = case["B"], case["hk"], case["dh"], case["page"]
    codes, scales = _blocks(pool, dh)
    v = _values(codes, scales, g, st["mag"]).flatten(0, 1)              # [blocks * 16][dh]
    if not page:
        return v.view(B, hk, st["capacity"], dh)
    v = v.view(st["n_pages"], hk, page, dh)[st["pages"].long()]      # [B][n][hk][page][dh]
    return v.transpose(1, 2).reshape(B, hk, st["capacity"], dh)


def _attention_plain(st):
    case = st["case"]
    B, hq, hk, dh, n1 = case["B"], case["hq"], case["hk"], case["dh"], case["n1"]
    K, V = _prefix(st, st["kc"], K_SCALE), _prefix(st, st["vc"], V_SCALE)
    q = st["q"].float().view(B, n1, hk, hq // hk, dh).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, dh)
    past = torch.arange(st["capacity"], device="cuda") < st["len"][:, None]
    V = torch.where(past[:, None, :, None], V, 0.0)
    s = torch.cat((torch.where(past[:, None, None], q @ K.transpose(-1, -2), -math.inf),
                   torch.where(st["see"].repeat_interleave(hq // hk, 0),
                               q @ st["tk"].float().permute(0, 2, 3, 1), -math.inf)), -1) / math.sqrt(dh)
    p = (s - s.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    o = p[..., :st["capacity"]] @ V + p[..., st["capacity"]:] @ st["tv"].float().transpose(1, 2)
    return o.view(B, hk, n1, hq // hk, dh).permute(0, 2, 1, 3, 4).reshape(B, n1, hq, dh).to(st["q"].dtype)


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        if op == "rope":
            c, s = st["cos"][st["pos"]], st["sin"][st["pos"]]
            return [_turn(x.float(), c, s, case["rot"], case["layout"]).to(x.dtype) for x in (st["q"], st["k"])]
        if op == "append":
            return _append_plain(st)
        if op == "read":
            return {"k": _read_plain(st, st["kc"], K_SCALE, st["k_rows"].dtype),
                    "v": _read_plain(st, st["vc"], V_SCALE, st["v_rows"].dtype)}
        return _attention_plain(st)
    b = _binding()
    if op == "rope":
        b.rope_apply(st["handle"], st["pos"], ((st["q"], st["q_out"]), (st["k"], st["k_out"])))
        return [st["q_out"], st["k_out"]]
    if op == "append":
        b.kv_append(st["cache"], st["kv"], st["k"], st["v"], start=st["start"], rope=st["handle"],
                    k_scale=K_SCALE, v_scale=V_SCALE)
        if case["fmt"] != "kv4":
            return {"k": st["kc"], "v": st["vc"], "len": st["len_out"]}
        b.kv_read(st["cache"], st["kv_after"], st["k_rows"], st["v_rows"], start=st["all"],
                  k_scale=K_SCALE, v_scale=V_SCALE)
        return {"k": st["k_rows"], "v": st["v_rows"], "len": st["len_out"]}
    if op == "read":
        b.kv_read(st["cache"], st["kv"], st["k_rows"], st["v_rows"], start=st["all"],
                  k_scale=K_SCALE, v_scale=V_SCALE)
        return {"k": st["k_rows"], "v": st["v_rows"]}
    b.kv4_attention(st["cache"], st["kv"], st["q"], st["o"], st["ws"], tree_k=st["tk"], tree_v=st["tv"],
                    mask=st["mask"], k_scale=K_SCALE, v_scale=V_SCALE)
    return st["o"]


# ------------------------------------------------------------------ 64 bits
def _exact_turn(x, pos, r):
    """Pairs as complex numbers, multiplied by e^(i angle)."""
    f = torch.tensor(_frequencies(r), dtype=torch.float64, device="cuda")
    a = pos.double()[:, None] * f
    w = torch.polar(torch.full_like(a, r["attn"]), a)[:, None]
    h, y = r["rot"] // 2, x.double().clone()
    if r["layout"] == "half":
        z = torch.complex(y[..., :h], y[..., h:2 * h]) * w
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * h:2], y[..., 1:2 * h:2]) * w
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = z.real, z.imag
    return y


def _two_to(e):
    """2^e in 64 bits for whole e in -64..63, without a power function's rounding."""
    return torch.tensor([math.ldexp(1.0, i) for i in range(-64, 64)], dtype=torch.float64, device="cuda")[e.long() + 64]


def _exact_held(x, g):
    """What a 4-bit cache holds of x, from the definition of its two number formats."""
    y = x.unflatten(-1, (-1, 16)) / g
    top = y.abs().amax(-1, keepdim=True) / 6
    e = torch.frexp(top.clamp(min=2.0 ** -9))[1] - 1
    step = _two_to(e.clamp(min=-6, max=60) - 3)
    s = (torch.round(top / step) * step).clamp(max=448.0)
    a = torch.where(s > 0, y.abs() / torch.where(s > 0, s, 1.0), 0.0)
    mid = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
    down, up = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    code = torch.where(down % 2 == 0, down, up)
    code = torch.where(down == up, down, code)
    m = torch.tensor(_MAG, dtype=torch.float64, device="cuda")[code]
    return (torch.where(y < 0, -m, m) * s * g).flatten(-2)


def _exact_cache(pool, case, st, g):
    """A 4-bit pool's values in 64 bits, [B][capacity][hk][dh], nibble by nibble."""
    dh, hk, page = case["dh"], case["hk"], case["page"]
    unit = page or st["capacity"]
    p = pool.view(-1, hk, unit // 16, 9 * dh)
    c, s = p[..., :8 * dh].reshape(-1, hk, unit, dh // 2).long(), p[..., 8 * dh:].reshape(-1, hk, unit, dh // 16).long()
    e, m = (s >> 3) & 15, s & 7
    s = torch.where(e > 0, (8 + m).double() * _two_to(e - 10), m.double() * 2.0 ** -9) * g
    n = torch.stack((c % 16, c // 16), -1).flatten(-2)
    ne, nm = (n >> 1) & 3, n & 1
    v = torch.where(ne > 0, (2 + nm).double() * _two_to(ne - 2), nm.double() / 2)
    v = torch.where(n >= 8, -v, v) * s.repeat_interleave(16, -1)
    v = v.transpose(1, 2)                                          # [pages or B][unit][hk][dh]
    return v[st["pages"].long()].flatten(1, 2) if page else v


def exact(case, seed):
    st = prepare(case, seed)
    op, dh = case["op"], case["dh"]
    if op == "rope":
        return [_exact_turn(x, st["pos"], st["rope"]) for x in (st["q"], st["k"])]
    if op == "append":
        before, new = _range(case, "before"), _range(case, "new")
        kv4 = case["fmt"] == "kv4"
        if kv4:
            K, V = _exact_cache(st["kc"], case, st, K_SCALE), _exact_cache(st["vc"], case, st, V_SCALE)
        else:
            K, V = st["kc"].double(), st["vc"].double()
        at = 0
        for b, (t0, n) in enumerate(zip(before, new)):
            if n == 0:
                continue
            pos = torch.arange(t0, t0 + n, device="cuda")
            k, v = _exact_turn(st["k"][at:at + n], pos, st["rope"]), st["v"][at:at + n].double()
            at += n
            if kv4:
                K[b, t0:t0 + n], V[b, t0:t0 + n] = _exact_held(k, K_SCALE), _exact_held(v, V_SCALE)
            elif case["page"]:
                where = st["pages"][b].long()[pos // case["page"]], pos % case["page"]
                K[where], V[where] = k, v
            else:
                K[b, t0:t0 + n], V[b, t0:t0 + n] = k, v
        n = [x + y for x, y in zip(before, new)]
        if kv4:
            K, V = (torch.cat([x[b, :m] for b, m in enumerate(n)]) for x in (K, V))
        return {"k": K, "v": V, "len": _ints(n)}
    n = _range(case, "len")
    K, V = _exact_cache(st["kc"], case, st, K_SCALE), _exact_cache(st["vc"], case, st, V_SCALE)
    if op == "read":
        return {x: torch.cat([c[b, :m] for b, m in enumerate(n)]) for x, c in (("k", K), ("v", V))}
    group = case["hq"] // case["hk"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, m in enumerate(n):
        k = torch.cat((K[b, :m], st["tk"][b].double())).permute(1, 2, 0)            # [hk][dh][keys]
        v = torch.cat((V[b, :m], st["tv"][b].double())).transpose(0, 1)
        q = st["q"][b].double().unflatten(1, (-1, group)).permute(1, 0, 2, 3).flatten(1, 2)
        s = torch.bmm(q, k) * dh ** -0.5
        hide = torch.cat((torch.zeros(case["n1"], m, dtype=torch.bool, device="cuda"), ~st["see"]), 1)
        s.masked_fill_(hide.repeat_interleave(group, 0), -math.inf)
        o = torch.bmm(torch.softmax(s, -1), v)
        out[b] = o.unflatten(1, (case["n1"], group)).permute(1, 0, 2, 3).flatten(1, 2)
    return out
