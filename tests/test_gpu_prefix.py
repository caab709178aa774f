"""Attention over a shared prefix against the 64-bit form in prefix_ref.py (whose comment derives the bound),
through the public binding; and a layer that uses it together with 8-bit projections and the caches."""
import numpy as np
import pytest
import torch

import fp8_ref as F
import prefix_ref as A
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FMT = {"f32": Bnd.F32, "bf16": Bnd.BF16}
H = {"f32": U, "bf16": 2.0 ** -8}
PHALF = {"f32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def pool(r, B, lens, page, hk, dh, dtype, spare):
    """Keys, values (NaN where no sequence has a slot), page table, pages and capacity."""
    unit = page or 1
    cap = -(-(max(max(lens), 1) + spare) // unit) * unit
    if page:
        n = cap // page
        table = r.permutation(B * n + 2)[:B * n].reshape(B, n)
        shape = (B * n + 2, page, hk, dh)
    else:
        table, shape = None, (B, cap, hk, dh)
    k, v = (torch.from_numpy(r.standard_normal(shape)).to(DT[dtype]) for _ in "kv")
    held = np.zeros(shape[:2], bool)
    for b, n in enumerate(lens):
        t = np.arange(n)
        if page:
            held[table[b, t // page], t % page] = True
        else:
            held[b, :n] = True
    hole = torch.from_numpy(~held)
    k[hole], v[hole] = float("nan"), float("nan")
    return dict(k=k.cuda(), v=v.cuda(), table=table, page=page, cap=cap, pages=shape[0] if page else 0, lens=lens)


def tree_mask(r, n1, kind):
    """sees [n1][n1] and mask words (None: causal)."""
    see = np.zeros((n1, n1), bool)
    for n in range(n1):
        if kind == "causal":
            see[n, :n + 1] = True
        elif kind == "tree":
            if n:
                see[n] = see[r.integers(0, n)]
            see[n, n] = True
        elif kind == "holes":                     # some rows see nothing, some all
            see[n] = r.random(n1) < r.choice([0.0, 0.3, 1.0])
    if kind == "causal":
        return see, None
    full = np.zeros((n1, 256), bool)
    full[:, :n1] = see
    full[:, n1:] = True                           # bits of no row
    return see, i32(np.packbits(full, axis=1, bitorder="little").view(np.int32))


class Case:
    def __init__(self, seed, B, hq, hk, dh, n1, P, lens, page, ppage, dtype, kind, max_nodes=None, spare=5):
        r = np.random.default_rng(seed)
        self.dims, self.dtype, self.kind = (B, hq, hk, dh, n1), dtype, kind
        self.own_pool, self.shared_pool = pool(r, B, lens, page, hk, dh, dtype, spare), pool(r, 1, [P], ppage, hk, dh, dtype, spare)
        self.handles = []
        for p, count in ((self.own_pool, B), (self.shared_pool, 1)):
            c = Bnd.Cache(count, hq, hk, dh, FMT[dtype], p["cap"], page_size=p["page"], num_pages=p["pages"],
                          max_nodes=max_nodes or n1)
            self.handles.append((c, Bnd.kv_struct(p["k"], p["v"], self.keep(p, "len", i32(p["lens"])), None,
                                                  self.keep(p, "pt", None if p["table"] is None else i32(p["table"])))))
        self.q = torch.from_numpy(r.standard_normal((B, n1, hq, dh))).to(DT[dtype]).cuda()
        self.tk, self.tv, self.mask, self.see = None, None, None, None
        if kind:
            self.tk, self.tv = (torch.from_numpy(r.standard_normal((B, n1, hk, dh))).to(DT[dtype]).cuda() for _ in "kv")
            self.see, self.mask = tree_mask(r, n1, kind)
        self.ws = torch.full((Bnd.prefix_workspace_size(self.handles[0][0], self.handles[1][0]),), 255, dtype=torch.uint8, device="cuda")
        self.scale = 0.0

    @staticmethod
    def keep(p, name, t):
        p[name] = t
        return t

    def run(self, q=None, o=None, ws=None, stream=None):
        q = self.q if q is None else q
        o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if o is None else o
        (own, okv), (shared, skv) = self.handles
        Bnd.prefix_attention(own, okv, shared, skv, q, o, self.ws if ws is None else ws, tree_k=self.tk, tree_v=self.tv,
                             mask=self.mask, scale=self.scale, stream=stream)
        return o

    def want(self, lens=None):
        B, hq, hk, dh, n1 = self.dims
        lens = self.own_pool["lens"] if lens is None else lens
        o, tol = np.zeros((B, n1, hq, dh)), np.zeros((B, n1, hq, dh))
        q = f64(self.q)
        sk, sv = ([A.slots(f64(p), self.shared_pool["table"], self.shared_pool["page"], 0, self.shared_pool["lens"][0])
                   for p in (self.shared_pool["k"], self.shared_pool["v"])])
        ok, ov = f64(self.own_pool["k"]), f64(self.own_pool["v"])
        for b in range(B):
            parts = [(sk, sv), tuple(A.slots(x, self.own_pool["table"], self.own_pool["page"], b, lens[b]) for x in (ok, ov))]
            if self.tk is not None:
                parts.append((f64(self.tk[b]), f64(self.tv[b])))
            o[b], tol[b] = A.attention(q[b], parts, self.see, self.scale or dh ** -0.5, PHALF[self.dtype])
        return o, tol + H[self.dtype] * (np.abs(o) + tol)

    def check(self, o):
        want, tol = self.want()
        err = np.abs(f64(o) - want)
        assert (err <= tol).all(), (err - tol).max()
        assert [c.status() for c, _ in self.handles] == [0, 0]


CASES = [
    # B, hq, hk, dh, n1, P, lens, page, ppage, kind
    (1, 1, 1, 32, 1, 1, [0], 0, 0, None),
    (1, 4, 4, 64, 1, 0, [0], 0, 0, "causal"),
    (1, 4, 2, 64, 1, 0, [1], 0, 0, None),
    (2, 2, 2, 128, 1, 128, [0, 0], 0, 0, None),
    (3, 8, 2, 64, 31, 777, [0, 57, 100], 16, 0, "tree"),
    (4, 8, 1, 128, 1, 300, [3, 128, 129, 255], 16, 16, "causal"),
    (2, 5, 1, 128, 7, 130, [40, 0], 20, 48, "tree"),
    (5, 14, 2, 64, 3, 129, [1, 2, 3, 4, 500], 0, 16, "holes"),
    (2, 7, 1, 128, 37, 257, [300, 20], 48, 0, "tree"),
    (3, 4, 4, 128, 65, 200, [64, 0, 127], 0, 0, "tree"),
    (2, 8, 2, 128, 43, 512, [130, 256], 16, 0, "tree"),
    (2, 2, 1, 128, 200, 100, [0, 33], 32, 16, "causal"),
    (1, 2, 2, 64, 256, 140, [5], 0, 0, "holes"),
    (9, 3, 3, 32, 5, 66, [0, 1, 2, 3, 4, 5, 64, 65, 130], 3, 1, "tree"),
    (40, 2, 2, 64, 2, 64, list(range(40)), 0, 0, None),
    (70, 1, 1, 128, 1, 5, [0] * 69 + [200], 16, 0, "causal"),
    (2, 40, 8, 32, 9, 90, [10, 11], 0, 0, "holes"),
    (2, 4, 1, 64, 1, 5000, [2000, 3000], 16, 20, None),
    (3, 64, 1, 128, 5, 150, [7, 0, 200], 0, 0, "tree"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention(case, dtype):
    *dims, kind = case
    c = Case(sum(dims[:6]), *dims, dtype, kind)
    o = c.run()
    c.check(o)
    assert torch.equal(o.view(torch.uint8), c.run().view(torch.uint8))        # the same bits again


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [32, 64, 128])
def test_strides_scale_and_smaller_calls(dtype, dh):
    """Queries out of wider rows, results into wider ones, a scale, fewer rows than max_nodes."""
    c = Case(5, 3, 6, 2, dh, 4, 150, [9, 0, 140], 16, 0, dtype, "causal", max_nodes=17)
    wide_q = torch.zeros(3, 4, 9, dh + 8, dtype=DT[dtype], device="cuda")
    wide_o = torch.full((3, 4, 10, dh), 7.0, dtype=DT[dtype], device="cuda")
    q = wide_q[:, :, 1:7, :dh]
    q.copy_(c.q)
    c.scale = 0.3
    c.run(q=q, o=wide_o[:, :, 2:8])
    c.check(wide_o[:, :, 2:8])
    assert (wide_o[:, :, :2] == 7).all() and (wide_o[:, :, 8:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_are_not_seen_may_hold_anything(dtype):
    """Infinities and NaN in the call's rows reach only the rows that see them."""
    c = Case(6, 2, 4, 2, 64, 40, 100, [30, 0], 0, 0, dtype, "tree")
    want, tol = c.want()
    c.tk[0, 39], c.tv[0, 38] = float("nan"), float("inf")
    c.tv[1, 37, 0, 5] = float("nan")
    g = f64(c.run())
    hit = np.zeros((2, 40, 4), bool)
    hit[0, c.see[:, 39]] = hit[0, c.see[:, 38]] = True
    hit[1, c.see[:, 37], :2] = True
    keep = ~hit
    assert np.isfinite(g[keep]).all() and (np.abs(g - want)[keep] <= tol[keep]).all()
    nan = np.zeros((2, 40, 4), bool)
    nan[0, c.see[:, 39]] = True
    assert np.isnan(g[nan]).all() and not np.isfinite(g[hit]).all(-1).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_query_that_is_nan_or_far_from_the_others(dtype):
    c = Case(7, 2, 2, 1, 128, 3, 300, [140, 10], 0, 16, dtype, "causal")
    c.q[0, 0, 0] *= 60                            # one key takes nearly all
    c.q[1, 2] *= 1e-6
    c.check(c.run())
    c.q[0, 1, 1, 3] = float("nan")
    g = f64(c.run())
    assert np.isnan(g[0, 1, 1]).all() and np.isnan(g).any(-1).sum() == 1


def test_lengths_out_of_range_and_bad_pages():
    for dtype in ("f32", "bf16"):
        c = Case(8, 3, 2, 2, 64, 2, 40, [16, 20, 32], 16, 8, dtype, "causal", spare=0)
        want, tol = c.want(lens=[0, 20, 32])
        c.own_pool["len"].copy_(i32([-5, 20, 1 << 30]))
        g = f64(c.run())
        assert (np.abs(g - want) <= tol).all() and c.handles[0][0].status() == 0
        c.own_pool["pt"][1, 0] = 999
        c.run()
        assert (c.handles[0][0].status(), c.handles[1][0].status()) == (Bnd.FLAG_PAGE_RANGE, 0)
        c.own_pool["pt"][1, 0] = 0
        c.shared_pool["pt"][0, 4] = -1
        c.run()
        assert (c.handles[0][0].status(), c.handles[1][0].status()) == (0, Bnd.FLAG_PAGE_RANGE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_and_replays_with_other_lengths(dtype):
    c = Case(9, 4, 4, 2, 128, 6, 260, [100, 7, 30, 200], 16, 0, dtype, "tree")
    other = torch.empty_like(c.ws)
    outs = [torch.zeros_like(c.q), torch.zeros_like(c.q)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st, o, ws in zip(streams, outs, (c.ws, other)):
        with torch.cuda.stream(st):
            for _ in range(3):
                c.run(o=o, ws=ws)
    torch.cuda.synchronize()
    for o in outs:
        c.check(o)
    g, o = torch.cuda.CUDAGraph(), torch.zeros_like(c.q)
    with torch.cuda.graph(g):
        c.run(o=o)
    lens = [0, 150, 30, 64]                       # within what the pool holds of each
    full = [100, 7, 30, 200]
    lens = [min(a, b) for a, b in zip(lens, full)]
    c.own_pool["len"].copy_(i32(lens))
    g.replay()
    want, tol = c.want(lens=lens)
    assert (np.abs(f64(o) - want) <= tol).all()


def test_library_refusals():
    c = Case(10, 2, 4, 2, 64, 3, 50, [5, 6], 0, 0, "bf16", "causal")
    (own, okv), (shared, skv) = c.handles
    o = torch.empty_like(c.q)
    cache = lambda **kw: Bnd.Cache(**dict(dict(B=1, Hq=4, Hkv=2, dh=64, format=Bnd.BF16, capacity=64), **kw))  # noqa: E731

    def call(own=own, okv=okv, shared=shared, skv=skv, q=c.q, o=o, ws=c.ws, **kw):
        Bnd.prefix_attention(own, okv, shared, skv, q, o, ws, **dict(dict(tree_k=c.tk, tree_v=c.tv, mask=c.mask), **kw))

    call()
    for other in (cache(B=2), cache(Hq=2), cache(Hkv=4), cache(dh=32), cache(format=Bnd.F32), cache(format=Bnd.KV4)):
        assert Bnd.prefix_workspace_size(own, other) == 0
        with pytest.raises(Bnd.MedusaError) as e:
            call(shared=other)
        assert e.value.code == -1
    kv4 = [cache(B=2, format=Bnd.KV4), cache(format=Bnd.KV4)]
    with pytest.raises(Bnd.MedusaError) as e:
        call(own=kv4[0], shared=kv4[1])
    assert e.value.code == -2 and Bnd.prefix_workspace_size(*kv4) == 0
    bad = Bnd.kv_struct(c.own_pool["k"], c.own_pool["v"], None, None, None)
    off = torch.zeros(c.q.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view(c.q.shape)
    for kw, code in ((dict(ws=c.ws[:-1]), -6), (dict(ws=c.ws[16:]), -6), (dict(okv=bad), -1), (dict(skv=bad), -1),
                     (dict(q=off), -1), (dict(o=off), -1), (dict(scale=-1.0), -1), (dict(tree_k=None, tree_v=None, mask=i32([0] * 24)), -1),
                     (dict(q=c.q.float(), o=o.float(), tree_k=c.tk.float(), tree_v=c.tv.float()), -1),
                     (dict(q=torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16, device="cuda"),
                           o=torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16, device="cuda"), tree_k=None, tree_v=None), -1),
                     (dict(o=torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16, device="cuda").expand(2, 3, 4, 64)), -1)):
        with pytest.raises(Bnd.MedusaError) as e:
            call(**kw)
        assert e.value.code == code, kw
    assert own.status() == 0 and shared.status() == 0


def test_a_layer_of_8_bit_projections_over_a_shared_prefix():
    """Hidden states -> queries, keys, values (8-bit products) -> the prompt's part into the shared cache and the
    sequences' into their own -> attention -> output projection onto the residual -> gated feed-forward block, each
    stage compared with the 64-bit form of the same stage's inputs."""
    r = np.random.default_rng(11)
    B, P, d, hq, hk, dh, f = 3, 70, 256, 4, 2, 64, 384
    bf = torch.bfloat16

    def w8(n, k):
        h = Bnd.Fp8(n=n, k=k, max_rows=n)
        x = torch.from_numpy(r.standard_normal((n, k)) * (2 / k) ** 0.5).float().cuda()
        c, s = torch.empty(n, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(-(-n // 128), -(-k // 128), device="cuda")
        Bnd.fp8_round(h, x, c, s, block=128)
        return c, s

    def linear(x, w, add=None, up=None):
        n, k = w[0].shape
        h = Bnd.Fp8(n=n, k=k, max_rows=x.shape[0], gated=up is not None)
        y = torch.empty(x.shape[0], n, dtype=bf, device="cuda")
        ws = torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda")
        Bnd.fp8_linear(h, x, w[0], w[1], y, ws, add=add, up=None if up is None else up[0], up_scales=None if up is None else up[1])
        xv = F.values(*F.round8(f64(x), 1), 1)
        val = lambda p: F.values(p[0].view(torch.uint8).cpu().numpy(), f64(p[1]), 128)  # noqa: E731
        a, da = xv @ val(w).T, 2 * U * (132 + h.kb) * (np.abs(xv) @ np.abs(val(w)).T)
        want, tol = a, da
        if up is not None:
            b, db = xv @ val(up).T, 2 * U * (132 + h.kb) * (np.abs(xv) @ np.abs(val(up)).T)
            want, tol = F.silu(a) * b, 1.1 * da * np.abs(b) + (np.abs(F.silu(a)) + 1.1 * da) * db + 8 * U * np.abs(F.silu(a) * b)
        if add is not None:
            want = want + f64(add)
            tol = tol + U * np.abs(want)
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        assert (np.abs(f64(y) - want) <= tol).all()
        return y

    wqkv, wo, w1, w3, w2 = w8((hq + 2 * hk) * dh, d), w8(d, hq * dh), w8(f, d), w8(f, d), w8(d, f)
    own = Bnd.Cache(B, hq, hk, dh, Bnd.BF16, 48, page_size=16, num_pages=10, max_nodes=1)
    shared = Bnd.Cache(1, hq, hk, dh, Bnd.BF16, 80)
    rope = Bnd.Rope(dh, 256)
    kv = {}
    for name, shape, n, table in (("own", (10, 16, hk, dh), B, i32(r.permutation(9).reshape(3, 3))), ("shared", (1, 80, hk, dh), 1, None)):
        k, v = (torch.full(shape, float("nan"), dtype=bf, device="cuda") for _ in "kv")
        length = torch.zeros(n, dtype=torch.int32, device="cuda")
        kv[name] = (k, v, length, table, Bnd.kv_struct(k, v, length, length, table))

    def split(y):
        z = y.view(-1, hq + 2 * hk, dh)
        return z[:, :hq], z[:, hq:hq + hk], z[:, hq + hk:]

    _, k, v = split(linear(torch.from_numpy(r.standard_normal((P, d))).to(bf).cuda(), wqkv))
    Bnd.kv_append(shared, kv["shared"][4], k, v, rope=rope)
    ws = torch.empty(Bnd.prefix_workspace_size(own, shared), dtype=torch.uint8, device="cuda")
    for step in range(18):                        # past a page
        x = torch.from_numpy(r.standard_normal((B, d))).to(bf).cuda()
        q, k, v = split(linear(x, wqkv))
        pos = i32([P + step] * B)
        Bnd.rope_apply(rope, pos, [(q, q)])
        Bnd.kv_append(own, kv["own"][4], k, v, pos=pos, rope=rope)
        o = torch.empty(B, 1, hq, dh, dtype=bf, device="cuda")
        Bnd.prefix_attention(own, kv["own"][4], shared, kv["shared"][4], q.unsqueeze(1), o, ws)
        if step in (0, 17):
            for b in range(B):
                parts = [tuple(f64(t)[0, :P] for t in kv["shared"][:2]),
                         tuple(A.slots(f64(t), kv["own"][3].cpu().numpy(), 16, b, step + 1) for t in kv["own"][:2])]
                want, tol = A.attention(f64(q[b:b + 1]), parts, None, dh ** -0.5, 2.0 ** -8)
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                assert (np.abs(f64(o[b]) - want) <= tol).all()
        y = linear(o.view(B, hq * dh), wo, add=x)
        y = linear(linear(y, w1, up=w3), w2, add=y)
        assert torch.isfinite(y).all()
    assert own.status() == 0 and shared.status() == 0
