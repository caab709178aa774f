"""What the projections in 8 bits and attention over a shared prefix cost: rounding rows and
weights to 8 bits and reading them back, products of such rows and weights, the gated pair of
products of a feed-forward block, and attention of a batch whose sequences begin with the same
tokens.

Every case runs either in its plain form (elementary torch operations in 32 bits) or, with
`own` set, through the library's entry points, on the same inputs.

The 8-bit format both forms read and write: elements are e4m3, and an element stands for its
code times a float scale.  A row has one scale for each 128 consecutive elements, a weight
matrix one for each 128 x 128 block; the last ones may be shorter.  Rounding takes 2^e for the
smallest whole e >= -126 with max|x| <= 448 * 2^e over the elements (1 where all are zero), and
the nearest code to x / 2^e, ties to even.  A product takes any scales.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_E4M3 = torch.float8_e4m3fn
GROUP = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the hidden states of a batch of 8 trees of 65 nodes, a part of wider rows
        {"name": "round_rows", "op": "round", "rows": 520, "k": 5120, "block": 1, "dtype": "bf16", "wide": 1},
        # loading: one projection's weights out of a checkpoint in full precision
        {"name": "round_weights", "op": "round", "rows": 13824, "k": 5120, "block": 128, "dtype": "f32", "wide": 0},
        # decoding one token: an attention layer's output projection on the row as it is
        {"name": "linear_token", "op": "linear", "rows": 1, "n": 4096, "k": 4096, "x": "bf16", "y": "bf16", "add": 0},
        # a small batch, odd sizes, full precision and a residual
        {"name": "linear_odd_f32", "op": "linear", "rows": 37, "n": 997, "k": 1040, "x": "f32", "y": "f32", "add": 1},
        # queries, keys and values of a batch of 8 trees of 65 nodes
        {"name": "linear_tree", "op": "linear", "rows": 520, "n": 15360, "k": 5120, "x": "codes", "y": "bf16", "add": 0},
        # two long prompts: a feed-forward block's last projection
        {"name": "linear_prompt", "op": "linear", "rows": 8192, "n": 5120, "k": 13824, "x": "codes", "y": "bf16",
         "add": 1},
        # decoding: a feed-forward block's two first projections for a batch of 8 tokens
        {"name": "gated_tokens", "op": "gated", "rows": 8, "n": 13824, "k": 5120, "x": "bf16", "y": "bf16"},
        # the same for 16 trees of 43 nodes
        {"name": "gated_tree", "op": "gated", "rows": 688, "n": 14336, "k": 4096, "x": "codes", "y": "bf16"},
        # decoding 32 sequences that begin with the same long instructions, own tokens paged
        {"name": "prefix_tokens", "op": "prefix", "B": 32, "hq": 32, "hk": 8, "dh": 128, "n1": 1, "prefix": 16384,
         "len": "100-1000", "page": 16, "prefix_page": 16, "dtype": "bf16", "lens": 1},
        # verification of 64-candidate trees in a batch of 8, a key head for each query head
        {"name": "prefix_tree", "op": "prefix", "B": 8, "hq": 40, "hk": 40, "dh": 128, "n1": 65, "prefix": 2048,
         "len": "0-1024", "page": 0, "prefix_page": 0, "dtype": "bf16", "lens": 2},
        # verification of 42-candidate trees, long prefix, 4 query heads to a key head
        {"name": "prefix_tree_gqa", "op": "prefix", "B": 16, "hq": 32, "hk": 8, "dh": 128, "n1": 43, "prefix": 8192,
         "len": "64-512", "page": 16, "prefix_page": 0, "dtype": "bf16", "lens": 3},
        # short ragged sequences in full precision
        {"name": "prefix_small_f32", "op": "prefix", "B": 3, "hq": 8, "hk": 2, "dh": 64, "n1": 31, "prefix": 777,
         "len": "0-100", "page": 16, "prefix_page": 0, "dtype": "f32", "lens": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15 * (10 if case.get("dtype") == "f32" and case["op"] == "prefix" else 1)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["round", "linear", "linear", "gated", "prefix", "prefix"])
    for _ in range(1000):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = rng.choice([_log(rng, 1, 16), _log(rng, 1, 8192), _log(rng, 1, 8192)])
        n, k = _log(rng, 16, 32000), 16 * _log(rng, 2, 1024)
        if op == "round":
            block = rng.choice([1, 128])
            case = {"op": op, "rows": _log(rng, 1, 16384), "k": k, "block": block, "dtype": dtype,
                    "wide": rng.choice([0, 1])}
        elif op == "linear":
            case = {"op": op, "rows": rows, "n": n, "k": k, "x": rng.choice(["codes", dtype]), "y": dtype,
                    "add": rng.choice([0, 0, 1])}
        elif op == "gated":
            case = {"op": op, "rows": rows, "n": n, "k": k, "x": rng.choice(["codes", dtype]), "y": dtype}
        else:
            hk = rng.choice([1, 2, 4, 8, 32, 40])
            hq = hk * rng.choice([g for g in (1, 1, 2, 4, 5, 7, 8) if g == 1 or hk * g <= 64])
            hi = _log(rng, 1, 2048)
            case = {"op": op, "B": _log(rng, 1, 64), "hq": hq, "hk": hk, "dh": rng.choice([32, 64, 128, 128, 128]),
                    "n1": rng.choice([1, 1, _log(rng, 2, 200), rng.randrange(2, 70)]),
                    "prefix": _log(rng, 1, 32768), "len": "%d-%d" % (rng.choice([0, hi // 2, hi]), hi),
                    "page": rng.choice([0, 16, 16, 32, 48, 20]), "prefix_page": rng.choice([0, 0, 16, 48]),
                    "dtype": dtype, "lens": rng.randrange(1 << 30)}
        if _cost(case) <= most[op]:
            return case
    return dict(case, B=1, n1=1) if op == "prefix" else dict(case, rows=1)


def _lengths(case):
    """The lengths of a case's sequences: drawn evenly from its range, its ends among them."""
    lo, hi = (int(x) for x in case["len"].split("-"))
    n = np.random.RandomState(case["lens"] % (1 << 31)).randint(lo, hi + 1, case["B"])
    n[-1] = hi
    if case["B"] > 1:
        n[0] = lo
    return [int(x) for x in n]


def _size(t):
    return {"f32": 4, "bf16": 2, "codes": 1 + 4 / GROUP}[t]


def work(case):
    op = case["op"]
    if op == "round":                                 # rounded, and read back
        e, n = _size(case["dtype"]), case["rows"] * case["k"]
        return {"bytes": n * (2 * e + 2 * (1 + 4 / (GROUP * case["block"]))), "flops": 3 * n}
    if op in ("linear", "gated"):
        rows, n, k = case["rows"], case["n"], case["k"]
        w = n * k * (1 + 4 / GROUP ** 2)
        if op == "gated":
            return {"bytes": 2 * w + rows * (k * _size(case["x"]) + n * _size(case["y"])), "flops": 4.0 * rows * n * k}
        return {"bytes": w + rows * (k * _size(case["x"]) + (1 + case["add"]) * n * _size(case["y"])),
                "flops": 2.0 * rows * n * k}
    e, rows, dh, n1 = _size(case["dtype"]), case["B"] * case["n1"], case["dh"], case["n1"]
    slots = case["prefix"] + sum(_lengths(case))
    return {"bytes": e * dh * (2 * slots * case["hk"] + 2 * rows * (case["hq"] + case["hk"])),
            "flops": 4.0 * dh * case["hq"] * (rows * (case["prefix"] + min(n1, 4)) + n1 * sum(_lengths(case)))}


# ------------------------------------------------------------------ 8 bits
def _groups(x, block):
    """[rows][k] as [rows/block][block][k/128][128], zeros behind the last ones."""
    r, k = x.shape
    br, bk = -(-r // block), -(-k // GROUP)
    y = torch.zeros(br * block, bk * GROUP, dtype=x.dtype, device=x.device)
    y[:r, :k] = x
    return y.view(br, block, bk, GROUP)


def _spread(scales, rows, k, block):
    """The scale of every element."""
    return scales.repeat_interleave(block, 0)[:rows].repeat_interleave(GROUP, 1)[:, :k]


def _round(x, block):
    """Codes and scales (powers of two) of x in 32 bits."""
    top = _groups(x, block).abs().amax((1, 3))
    m, e = torch.frexp(top)                           # top = m 2^e, m in [.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), 1.0)
    return (x / _spread(s, *x.shape, block)).to(_E4M3), s


def _values(codes, scales, block):
    return codes.float() * _spread(scales, *codes.shape, block)


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _hidden(g, rows, k):
    """Hidden states: a few channels much larger than the others, rows of different sizes."""
    gain = 1 + 15 * (torch.rand(k, generator=g, device="cuda") < 0.01).float()
    size = 0.25 + torch.rand(rows, 1, generator=g, device="cuda")
    return torch.randn(rows, k, generator=g, device="cuda") * gain * size


def _weights(g, n, k):
    """Weights as a checkpoint holds them: the largest element of a block is 448 scales."""
    w = torch.randn(n, k, generator=g, device="cuda") * (2.0 / k) ** 0.5
    s = _groups(w, GROUP).abs().amax((1, 3)) / 448.0
    return (w / _spread(s, n, k, GROUP)).clamp(-448, 448).to(_E4M3), s


def _keys(g, shape):
    """Values as projections give them: a few channels of each head much larger."""
    gain = 1 + 3 * (torch.rand(shape[-2:], generator=g, device="cuda") < 0.05).float()
    return torch.randn(shape, generator=g, device="cuda") * gain


def _binding():
    from medusa_head_speculative_gb300 import binding
    return binding


def _pool(g, B, slots, page, hk, dh, dt, seed):
    """Keys, values, page table and pages of a cache whose sequences have room for `slots`."""
    unit = page or 16
    capacity = (max(1, slots) + unit - 1) // unit * unit
    if not page:
        k, v = (_keys(g, (B, capacity, hk, dh)).to(dt) for _ in "kv")
        return {"k": k, "v": v, "pages": None, "n_pages": 0, "capacity": capacity}
    n = capacity // page
    total = B * n + 3                                 # in no order, some of them nobody's
    p = np.random.RandomState((seed * 7 + page) % (1 << 31)).permutation(total)[:B * n].reshape(B, n)
    k, v = (_keys(g, (total, page, hk, dh)).to(dt) for _ in "kv")
    return {"k": k, "v": v, "pages": _ints(p), "n_pages": total, "capacity": capacity}


def _tree(n1, seed):
    """Which nodes a node sees: every node under one of those before it, at most 5 deep."""
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
    bits = np.packbits(see, axis=1, bitorder="little").view(np.uint32)
    return torch.from_numpy(see[:, :n1].copy()).cuda(), torch.from_numpy(bits.view(np.int32).copy()).cuda()


def _prepare_prefix(case, g, seed, st):
    B, hq, hk, dh, n1, dt = case["B"], case["hq"], case["hk"], case["dh"], case["n1"], _DT[case["dtype"]]
    n = _lengths(case)
    st["own"] = _pool(g, B, max(n), case["page"], hk, dh, dt, seed)
    st["shared"] = _pool(g, 1, case["prefix"], case["prefix_page"], hk, dh, dt, seed + 1)
    st["len"], st["prefix_len"] = _ints(n), _ints([case["prefix"]])
    st["q"] = torch.randn(B, n1, hq, dh, generator=g, device="cuda").to(dt)
    st["tk"] = _keys(g, (B, n1, hk, dh)).to(dt)
    st["tv"] = torch.randn(B, n1, hk, dh, generator=g, device="cuda").to(dt)
    st["o"] = torch.empty(B, n1, hq, dh, dtype=dt, device="cuda")
    st["see"], st["mask"] = _tree(n1, seed)
    if own:
        b = _binding()
        fmt = b.F32 if case["dtype"] == "f32" else b.BF16
        for name, count, page, length in (("own", B, case["page"], st["len"]),
                                          ("shared", 1, case["prefix_page"], st["prefix_len"])):
            c = st[name]
            c["cache"] = b.Cache(count, hq, hk, dh, fmt, c["capacity"], page_size=page, num_pages=c["n_pages"],
                                 max_nodes=n1)
            c["kv"] = b.kv_struct(c["k"], c["v"], length, None, c["pages"])
        size = b.prefix_workspace_size(st["own"]["cache"], st["shared"]["cache"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    op = case["op"]
    if op == "prefix":
        return _prepare_prefix(case, g, seed, st)
    rows, k = case["rows"], case["k"]
    if op == "round":
        dt, block = _DT[case["dtype"]], case["block"]
        x = _hidden(g, rows, k + 64 * case["wide"]) if block == 1 else \
            torch.randn(rows, k + 64 * case["wide"], generator=g, device="cuda") * (2.0 / k) ** 0.5
        st["x"] = x.to(dt)[:, 64 * case["wide"]:]
        st["codes"] = torch.empty(rows, k, dtype=_E4M3, device="cuda")
        st["scales"] = torch.empty(-(-rows // block), -(-k // GROUP), device="cuda")
        st["values"] = torch.empty(rows, k, dtype=dt, device="cuda")
        if own:
            b = _binding()
            st["fp8"] = b.Fp8(n=rows, k=k, max_rows=rows) if block > 1 else b.Fp8(n=GROUP, k=k, max_rows=rows)
        return st
    n, dt = case["n"], _DT[case["y"]]
    x = _hidden(g, rows, k)
    if case["x"] == "codes":
        st["x"], st["scales"] = _round(x, 1)
    else:
        st["x"], st["scales"] = x.to(_DT[case["x"]]), None
    st["w"], st["w_scales"] = _weights(g, n, k)
    st["up"], st["up_scales"] = _weights(g, n, k) if op == "gated" else (None, None)
    st["add"] = torch.randn(rows, n, generator=g, device="cuda").to(dt) if case.get("add") else None
    st["y"] = torch.empty(rows, n, dtype=dt, device="cuda")
    if own:
        b = _binding()
        st["fp8"] = b.Fp8(n=n, k=k, max_rows=rows, gated=op == "gated")
        st["ws"] = torch.empty(st["fp8"].workspace_size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _gather(c, B):
    """A cache's keys and values as [B][hk][capacity][dh] in 32 bits."""
    out = []
    for x in (c["k"], c["v"]):
        x = x if c["pages"] is None else x[c["pages"].long()].flatten(1, 2)
        out.append(x.float().transpose(1, 2))
    return out


def _prefix_plain(st):
    case = st["case"]
    B, hq, hk, dh, n1 = case["B"], case["hq"], case["hk"], case["dh"], case["n1"]
    group, P = hq // hk, case["prefix"]
    (K, V), (pk, pv) = _gather(st["own"], B), _gather(st["shared"], 1)
    q = st["q"].float().view(B, n1, hk, group, dh).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, dh)
    past = torch.arange(K.shape[2], device="cuda") < st["len"][:, None]
    V = torch.where(past[:, None, :, None], V, 0.0)
    every = q.transpose(0, 1).reshape(hk, -1, dh)                # all rows of a key head, for the shared keys
    s = torch.cat(((every @ pk[0, :, :P].transpose(-1, -2)).view(hk, B, -1, P).transpose(0, 1),
                   torch.where(past[:, None, None], q @ K.transpose(-1, -2), -math.inf),
                   torch.where(st["see"].repeat_interleave(group, 0),
                               q @ st["tk"].float().permute(0, 2, 3, 1), -math.inf)), -1) / math.sqrt(dh)
    p = (s - s.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    a, b, c = p.split((P, K.shape[2], n1), -1)
    o = (a.transpose(0, 1).reshape(hk, -1, P) @ pv[0, :, :P]).view(hk, B, -1, dh).transpose(0, 1)
    o = o + b @ V + c @ st["tv"].float().transpose(1, 2)
    return o.view(B, hk, n1, group, dh).permute(0, 2, 1, 3, 4).reshape(B, n1, hq, dh).to(st["q"].dtype)


def _product_plain(st, w, scales):
    if st["scales"] is None:
        x = _values(*_round(st["x"].float(), 1), 1)
    else:
        x = _values(st["x"], st["scales"], 1)
    return x @ _values(w, scales, GROUP).T


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        return _run_own(st)
    if op == "prefix":
        return _prefix_plain(st)
    if op == "round":
        codes, scales = _round(st["x"].float(), case["block"])
        return {"values": _values(codes, scales, case["block"]).to(st["x"].dtype), "scales": scales}
    y = _product_plain(st, st["w"], st["w_scales"])
    if op == "gated":
        y = y / (1 + torch.exp(-y)) * _product_plain(st, st["up"], st["up_scales"])
    elif st["add"] is not None:
        y = y + st["add"].float()
    return y.to(st["y"].dtype)


def _run_own(st):
    b, case, op = _binding(), st["case"], st["case"]["op"]
    if op == "prefix":
        b.prefix_attention(st["own"]["cache"], st["own"]["kv"], st["shared"]["cache"], st["shared"]["kv"], st["q"],
                           st["o"], st["ws"], tree_k=st["tk"], tree_v=st["tv"], mask=st["mask"])
        return st["o"]
    if op == "round":
        b.fp8_round(st["fp8"], st["x"], st["codes"], st["scales"], block=case["block"])
        b.fp8_read(st["fp8"], st["codes"], st["scales"], st["values"], block=case["block"])
        return {"values": st["values"], "scales": st["scales"]}
    b.fp8_linear(st["fp8"], st["x"], st["w"], st["w_scales"], st["y"], st["ws"], x_scales=st["scales"], up=st["up"],
                 up_scales=st["up_scales"], add=st["add"])
    return st["y"]


# ------------------------------------------------------------------ 64 bits
def _exact_scales(x, block):
    """The scale of every element of x in 64 bits: the first power of two that is large enough."""
    r, k = x.shape
    out = torch.empty_like(x)
    small = torch.empty(-(-r // block), -(-k // GROUP), dtype=torch.float64, device="cuda")
    two = torch.tensor([math.ldexp(1.0, e) for e in range(-126, 128)], dtype=torch.float64, device="cuda")
    for i in range(0, k, GROUP):
        part = x[:, i:i + GROUP].abs().amax(1)
        if block > 1:
            full = torch.zeros(small.shape[0] * block, dtype=torch.float64, device="cuda")
            full[:r] = part
            part = full.view(-1, block).amax(1)
        s = two[torch.searchsorted(two * 448.0, part)]
        small[:, i // GROUP] = torch.where(part > 0, s, 1.0)
        out[:, i:i + GROUP] = small[:, i // GROUP].repeat_interleave(block)[:r, None]
    return out, small


def _exact_codes(y):
    """The nearest e4m3 numbers (ties to even) to |y| <= 448 in 64 bits, from the format's definition."""
    e = torch.frexp(y)[1].clamp(min=-5) - 4           # steps of 2^-9 below 2^-6, of an eighth of the power of two above
    two = torch.tensor([math.ldexp(1.0, i) for i in range(-9, 7)], dtype=torch.float64, device="cuda")
    step = two[(e + 9).clamp(0, 15).long()]
    return torch.round(y / step) * step


def _exact_rows(codes, scales):
    bits = codes.view(torch.uint8).long()
    m, e = bits & 7, (bits >> 3) & 15
    two = torch.tensor([math.ldexp(1.0, i) for i in range(-10, 6)], dtype=torch.float64, device="cuda")
    v = torch.where(e > 0, (8 + m).double() * two[e], m.double() * 2.0 ** -9)
    return torch.where(bits > 127, -v, v), scales.double()


def _exact_product(x, xs, w, ws):
    """sum over blocks of 128 of (codes times codes) * scale * scale, in 64 bits."""
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    n = torch.arange(w.shape[0], device="cuda") // GROUP
    for j, i in enumerate(range(0, x.shape[1], GROUP)):
        y += (x[:, i:i + GROUP] @ w[:, i:i + GROUP].T) * xs[:, j, None] * ws[n, j]
    return y


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "round":
        x = st["x"].double()
        s, small = _exact_scales(x, case["block"])
        return {"values": _exact_codes(x / s) * s, "scales": small}
    if op in ("linear", "gated"):
        if st["scales"] is None:
            x = st["x"].double()
            s, xs = _exact_scales(x, 1)
            x = _exact_codes(x / s)
        else:
            x, xs = _exact_rows(st["x"], st["scales"])
        y = _exact_product(x, xs, *_exact_rows(st["w"], st["w_scales"]))
        if op == "gated":
            y = y * torch.sigmoid(y) * _exact_product(x, xs, *_exact_rows(st["up"], st["up_scales"]))
        return y if st.get("add") is None else y + st["add"].double()
    group, P = case["hq"] // case["hk"], case["prefix"]

    def taken(c, b, n):
        """The first n keys and values of sequence b, slot by slot."""
        t = torch.arange(n, device="cuda")
        if c["pages"] is None:
            return c["k"][b, t].double(), c["v"][b, t].double()
        page = c["k"].shape[1]
        at = c["pages"][b].long()[t // page], t % page
        return c["k"][at].double(), c["v"][at].double()

    pk, pv = taken(st["shared"], 0, P)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, m in enumerate(_lengths(case)):
        k, v = taken(st["own"], b, m)
        k = torch.cat((pk, k, st["tk"][b].double())).permute(1, 2, 0)
        v = torch.cat((pv, v, st["tv"][b].double())).transpose(0, 1)
        q = st["q"][b].double().unflatten(1, (-1, group)).permute(1, 0, 2, 3).flatten(1, 2)
        s = torch.bmm(q, k) * case["dh"] ** -0.5
        hide = torch.cat((torch.zeros(case["n1"], P + m, dtype=torch.bool, device="cuda"), ~st["see"]), 1)
        s.masked_fill_(hide.repeat_interleave(group, 0), -math.inf)
        o = torch.bmm(torch.softmax(s, -1), v)
        out[b] = o.unflatten(1, (case["n1"], group)).permute(1, 0, 2, 3).flatten(1, 2)
    return out
