"""Rotary positions, appending to and reading from KV caches, and attention over 4-bit caches,
against the 64-bit forms in kv4_ref.py, through the public binding.

Tolerances.  u = 2^-24 is half a step of float32 relative to the value, H(t) of dtype t
(bf16 2^-8).  A rotated element is a*c - b*s from a float32 table (entries off by u relative,
plus the error of the double angle: p < 2^17, so below 2^-35), two products and one sum:
off by at most 4u (|a||c| + |b||s|) <= 4u attn (|a| + |b|), then one rounding to the dtype.
Attention bounds are made in attn_bound()."""
import numpy as np
import pytest
import torch

import kv4_ref as R
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = {"f32": 0.0, "bf16": 2.0 ** -8}
FMT = {"f32": Bnd.F32, "bf16": Bnd.BF16, "kv4": Bnd.KV4}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def rnd(seed, shape, dtype, gain=1.0):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * gain)
    return x.to(DT[dtype])


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary positions
RAMP = dict(scaling="ramp", factor=8.0, orig_pos=512, low=1.0, high=32.0, attn=1.2)
BANDED = dict(scaling="banded", factor=4.0, orig_pos=256, low=1.0, high=4.0)
ROPES = [
    # dtype, dh, rot, layout, heads, rows, scaling
    ("bf16", 128, 128, "half", (4, 2), 37, {}),
    ("bf16", 128, 64, "half", (3, 1), 5, dict(scaling="linear", factor=2.5)),
    ("bf16", 128, 64, "interleaved", (8, 2), 129, RAMP),
    ("bf16", 64, 40, "half", (2, 2), 9, BANDED),
    ("bf16", 64, 40, "interleaved", (1,), 300, BANDED),
    ("f32", 128, 128, "half", (5,), 1, {}),
    ("f32", 32, 32, "interleaved", (2, 1, 3), 66, RAMP),
    ("f32", 96, 18, "half", (7, 1), 11, {}),
    ("f32", 33, 2, "interleaved", (2,), 3, {}),
    ("bf16", 128, 96, "half", (40, 40), 65, {}),
    ("bf16", 256, 256, "half", (2, 1), 17, RAMP),
    ("bf16", 128, 72, "half", (32, 8), 520, {}),           # halves of 36: 8-byte units, two heads a thread
    ("bf16", 128, 100, "interleaved", (32, 8), 515, {}),
    ("bf16", 128, 128, "interleaved", (31, 7), 600, {}),
]


@pytest.mark.parametrize("dtype,dh,rot,layout,heads,rows,kw", ROPES)
@pytest.mark.parametrize("form", ["new", "place", "odd", "inverse"])
def test_rope(dtype, dh, rot, layout, heads, rows, kw, form):
    max_pos = 1000
    rope = Bnd.Rope(rot, max_pos, layout=layout, **kw)
    pos = np.random.default_rng(rows).integers(0, max_pos, rows)
    pos[-1] = max_pos - 1
    pos[0] = 0
    xs, ys = [], []
    fused = rnd(1, (rows, sum(heads) + 3, dh), dtype).cuda()
    at = 0
    for n in heads:
        x = fused[:, at:at + n]
        at += n
        if form == "odd":                    # neither 16-byte pointers nor 16-byte strides
            buf = torch.zeros(rows * (n * (dh + 1) + 5) + 3, dtype=DT[dtype], device="cuda")
            v = torch.as_strided(buf, (rows, n, dh), (n * (dh + 1) + 5, dh + 1, 1), 1)
            v.copy_(x)
            x = v
        xs.append(x)
        ys.append(x if form == "place" else torch.full((rows, n, dh), 7.0, dtype=DT[dtype], device="cuda"))
    want = [R.rope(f64(x), pos, rot, layout, inverse=form == "inverse", **kw) for x in xs]
    src = [f64(x) for x in xs]
    rest = f64(fused[:, at:])
    Bnd.rope_apply(rope, i32(pos), list(zip(xs, ys)), inverse=form == "inverse")
    for x, y, w in zip(src, ys, want):
        g = f64(y)
        np.testing.assert_array_equal(g[..., rot:], x[..., rot:])
        i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                else (slice(0, rot, 2), slice(1, rot, 2)))
        m = np.zeros(x.shape)
        m[..., i] = m[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
        tol = 4 * U * kw.get("attn", 1.0) * m
        tol = tol + H[dtype] * (np.abs(w) + tol)
        assert (np.abs(g - w) <= tol).all(), np.abs(g - w).max()
    np.testing.assert_array_equal(f64(fused[:, at:]), rest)
    assert rope.status() == 0


def test_rope_positions_outside_the_table_pass_through():
    rope = Bnd.Rope(64, 10)
    x = rnd(2, (4, 2, 64), "bf16").cuda()
    y = torch.zeros_like(x)
    Bnd.rope_apply(rope, i32([3, -1, 10, 2**31 - 1]), [(x, y)])
    assert torch.equal(y[1:], x[1:]) and not torch.equal(y[0], x[0])
    assert rope.status() == Bnd.FLAG_POS_RANGE and rope.status() == 0
    Bnd.rope_apply(rope, i32([]), [(x[:0], y[:0])])
    assert rope.status() == 0


def test_rope_far_positions():
    """The angle of a far position keeps double precision: one table entry per position."""
    far = 1 << 17
    rope = Bnd.Rope(128, far)
    x = rnd(3, (3, 1, 128), "f32").cuda()
    y = torch.empty_like(x)
    pos = [far - 1, far // 2 + 1, 99999]
    Bnd.rope_apply(rope, i32(pos), [(x, y)])
    w = R.rope(f64(x), pos, 128)
    m = np.abs(f64(x))
    tol = 4 * U * (m + np.roll(m, 64, -1))
    assert (np.abs(f64(y) - w) <= tol).all()


def test_rope_refusals():
    rope = Bnd.Rope(64, 10)
    x = rnd(4, (4, 2, 64), "bf16").cuda()
    with pytest.raises(TypeError):
        Bnd.rope_apply(rope, i32([0] * 4), [(x, x.float())])
    with pytest.raises(TypeError):
        Bnd.rope_apply(rope, i32([0] * 4), [(x.half(), x.half())])
    with pytest.raises(ValueError):
        Bnd.rope_apply(rope, i32([0] * 4), [(x, x[:, :1])])
    with pytest.raises(ValueError):
        Bnd.rope_apply(rope, torch.zeros(4, dtype=torch.int64, device="cuda"), [(x, x)])
    with pytest.raises(ValueError):
        Bnd.rope_apply(rope, i32([0] * 5), [(x, x)])
    with pytest.raises(Bnd.MedusaError) as e:                      # heads narrower than the rotation
        Bnd.rope_apply(rope, i32([0] * 4), [(x[..., :32], x[..., :32])])
    assert e.value.code == Bnd.MEDUSA_ERR_INVALID
    with pytest.raises(Bnd.MedusaError):                           # in place with other strides
        Bnd.rope_apply(rope, i32([0, 0]), [(x[:2], torch.as_strided(x, (2, 2, 64), (64, 64, 1)))])
    with pytest.raises(Bnd.MedusaError):
        Bnd.rope_apply(rope, i32([0] * 4), [(x, x)] * 5)


# ------------------------------------------------------------------ caches
class Case:
    """A cache with known contents on both sides."""

    def __init__(self, fmt, B, Hkv, dh, capacity, page=0, Hq=None, gk=0.5, gv=0.25, max_nodes=1, seed=0,
                 spare=2):
        self.fmt, self.B, self.Hkv, self.dh, self.capacity, self.page = fmt, B, Hkv, dh, capacity, page
        self.gk, self.gv = gk, gv
        rng = np.random.default_rng(seed)
        self.pages = self.table = None
        n_pages = 0
        if page:
            per = capacity // page
            n_pages = B * per + spare
            self.pages = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
            self.table = torch.from_numpy(self.pages).cuda()
        self.cache = Bnd.Cache(B, Hq or Hkv, Hkv, dh, FMT[fmt], capacity, page_size=page,
                               num_pages=n_pages, max_nodes=max_nodes)
        slots = n_pages * page if page else B * capacity
        self.view = R.Pool(fmt, B, Hkv, dh, capacity, page, self.pages)
        self.pool = []
        for g in (gk, gv):
            if fmt == "kv4":
                # every byte value may lie in slots nobody has written: NaN scales among them
                raw = rng.integers(0, 256, self.cache.pool_bytes, dtype=np.uint8)
                self.pool.append(torch.from_numpy(raw).cuda())
            else:
                self.pool.append(rnd(seed + 1, (slots, Hkv, dh), fmt).cuda())
            n = self.pool[-1].numel() * self.pool[-1].element_size()
            assert n == self.cache.pool_bytes

    def kv(self, length, len_out=None):
        self.keep = length, len_out              # the struct holds addresses only
        return Bnd.kv_struct(self.pool[0], self.pool[1], length, len_out, self.table)

    def host(self, which):
        p = self.pool[which]
        return p.cpu().numpy().copy() if self.fmt == "kv4" else p.float().cpu().numpy().copy()

    def fill(self, lens, seed=5, gain=1.0):
        """Writes the first lens[b] slots with encoded random values (4-bit caches)."""
        rng = np.random.default_rng(seed)
        for which, g in ((0, self.gk), (1, self.gv)):
            raw = self.host(which)
            for b, n in enumerate(lens):
                codes, scales = R.encode(rng.standard_normal((n, self.Hkv, self.dh)) * gain, g)
                for t in range(n):
                    c, s = self.view.slot(raw, b, t)
                    c[:], s[:] = codes[t], scales[t]
            self.pool[which].copy_(torch.from_numpy(raw))


def want_rows(case, x, g, dtype_out):
    """What the cache holds of rows x (float32 values as float64)."""
    if case.fmt == "kv4":
        return R.decode(*R.encode(x, g), g)
    return x if case.fmt == "f32" else f64(torch.from_numpy(x).float().bfloat16())


APPENDS = [
    # fmt, src, Hkv, dh, capacity, page, before, new
    ("bf16", "bf16", 2, 64, 96, 0, (0, 17, 80), (5, 0, 16)),
    ("bf16", "f32", 1, 32, 100, 5, (3, 50), (97, 1)),
    ("f32", "f32", 3, 128, 64, 16, (0, 0, 63, 10), (0, 64, 1, 7)),
    ("kv4", "bf16", 2, 128, 96, 0, (0, 17, 79), (33, 0, 17)),
    ("kv4", "bf16", 3, 64, 96, 16, (15, 1), (1, 95)),
    ("kv4", "f32", 1, 32, 144, 48, (0, 47, 100), (48, 2, 44)),
    ("kv4", "bf16", 40, 128, 32, 32, (7,), (1,)),
]


@pytest.mark.parametrize("fmt,src,Hkv,dh,capacity,page,before,new", APPENDS)
@pytest.mark.parametrize("turn", [None, "half", "interleaved", "partial"])
@pytest.mark.parametrize("alias", [False, True])
def test_append_packed(fmt, src, Hkv, dh, capacity, page, before, new, turn, alias):
    B = len(before)
    case = Case(fmt, B, Hkv, dh, capacity, page)
    rot = dh if turn in ("half", "interleaved") else (dh // 4 * 2 - 4)
    layout = "interleaved" if turn == "interleaved" else "half"
    rope = Bnd.Rope(rot, capacity, layout=layout) if turn else None
    total, lead, tail = sum(new), 2, 3         # places before start[0] and behind start[B]
    fused = rnd(9, (lead + total + tail, 2 * Hkv, dh), src).cuda()
    k, v = fused[:, :Hkv], fused[:, Hkv:]
    start = i32(np.concatenate(([0], np.cumsum(new))) + lead)
    length = i32(before)
    len_out = length if alias else torch.full_like(length, -5)
    old = case.host(0), case.host(1)
    Bnd.kv_append(case.cache, case.kv(length, len_out), k, v, start=start, rope=rope,
                  k_scale=case.gk, v_scale=case.gv)
    assert len_out.tolist() == [x + n for x, n in zip(before, new)]
    assert case.cache.status() == 0
    got = case.host(0), case.host(1)
    at = lead
    for b in range(B):
        for j in range(new[b]):
            t = before[b] + j
            kr, vr = f64(k[at]), f64(v[at])
            at += 1
            np.testing.assert_array_equal(case.view.value(got[1], b, t, case.gv),
                                          want_rows(case, vr, case.gv, fmt))
            held = case.view.value(got[0], b, t, case.gk)
            if not turn:
                np.testing.assert_array_equal(held, want_rows(case, kr, case.gk, fmt))
                continue
            w = R.rope(kr[None], [t], rot, layout)[0]
            m = np.abs(kr) + 4 * np.abs(kr).max()        # no smaller than |a| + |b| of any pair
            tol = 4 * U * m
            if fmt == "kv4":
                # the scale of the rounded maximum, or its neighbour where the maximum lies at
                # the border; each element at the code nearest to it under that scale
                codes, scales = case.view.slot(got[0], b, t)
                near = [R.encode(w * f, case.gk)[1] for f in (1 - 2 ** -20, 1 + 2 ** -20)]
                assert ((scales == near[0]) | (scales == near[1])).all()
                s = np.repeat(R.E4M3[scales], 16, -1) * case.gk
                best = np.abs(R.E2M1[:, None, None] * s - w).min(0)
                assert (np.abs(held - w) <= best + 2 * tol + 4 * U * 6 * s).all()
            else:
                tol = tol + H[fmt] * (np.abs(w) + tol)
                assert (np.abs(held - w) <= tol).all()
            # slots written, now blank them on both sides for the comparison below
        for j in range(new[b]):
            for which in (0, 1):
                for p in (old[which], got[which]):
                    s = case.view.slot(p, b, before[b] + j)
                    for x in (s if isinstance(s, tuple) else (s,)):
                        x[...] = 0
    np.testing.assert_array_equal(old[0].view(np.uint8), got[0].view(np.uint8))   # nothing else moved
    np.testing.assert_array_equal(old[1].view(np.uint8), got[1].view(np.uint8))


@pytest.mark.parametrize("fmt,page", [("bf16", 16), ("kv4", 16), ("kv4", 0), ("f32", 0)])
def test_append_accepted_path(fmt, page):
    """Padded batches with an index: the accepted nodes of a tree, as medusa_verify names them,
    the same node twice included; keys as they are."""
    B, K1, n1, Hkv, dh = 4, 4, 9, 2, 64
    case = Case(fmt, B, Hkv, dh, 64, page)
    tk, tv = rnd(1, (B, n1, Hkv, dh), "bf16").cuda(), rnd(2, (B, n1, Hkv, dh), "bf16").cuda()
    path = [[0, 3, 8, -1], [0, -1, -1, -1], [0, 5, 5, 2], [0, 1, 2, 3]]
    n_acc, length = [3, 1, 4, 0], i32([0, 31, 60, 7])
    out = torch.zeros_like(length)
    Bnd.kv_append(case.cache, case.kv(length, out), tk.view(-1, Hkv, dh), tv.view(-1, Hkv, dh), per_seq=K1,
                  count=i32(n_acc), index=i32(path), index_rows=n1, k_scale=case.gk, v_scale=case.gv)
    assert out.tolist() == [3, 32, 64, 7] and case.cache.status() == 0
    got = case.host(0), case.host(1)
    for b in range(B):
        for j in range(n_acc[b]):
            t, n = int(length[b]) + j, path[b][j]
            np.testing.assert_array_equal(case.view.value(got[0], b, t, case.gk),
                                          want_rows(case, f64(tk[b, n]), case.gk, fmt))
            np.testing.assert_array_equal(case.view.value(got[1], b, t, case.gv),
                                          want_rows(case, f64(tv[b, n]), case.gv, fmt))


def test_append_equals_the_step_compaction():
    """medusa_kv_compact and an append with the path as index leave the same bf16 cache."""
    B, n1, Hkv, dh, K = 2, 7, 2, 64, 3
    parent, rank = Bnd.tree_cartesian((2, 2, 1))
    n1 = len(parent)
    plan = Bnd.Plan(B, 128, 500, K, 4, Hkv, dh, Bnd.BF16, 64, (2, 2, 1), parent, rank)
    case = Case("bf16", B, Hkv, dh, 64)
    k2, v2 = case.pool[0].clone(), case.pool[1].clone()
    tk, tv = rnd(1, (B, n1, Hkv, dh), "bf16").cuda(), rnd(2, (B, n1, Hkv, dh), "bf16").cuda()
    path, n_acc, length = i32([[0, 2, 5, -1], [0, 1, -1, -1]]), i32([3, 2]), i32([10, 0])
    out, out2 = torch.zeros_like(length), torch.zeros_like(length)
    Bnd.kv_append(case.cache, case.kv(length, out), tk.view(-1, Hkv, dh), tv.view(-1, Hkv, dh),
                  per_seq=K + 1, count=n_acc, index=path, index_rows=n1)
    Bnd.kv_compact(plan, Bnd.kv_struct(k2, v2, length, out2), tk, tv, path, n_acc)
    assert torch.equal(out, out2) and torch.equal(case.pool[0], k2) and torch.equal(case.pool[1], v2)


@pytest.mark.parametrize("fmt", ["bf16", "kv4"])
def test_append_reports_what_it_cannot_place(fmt):
    case = Case(fmt, 3, 1, 32, 48, 16)
    case.table[1, 2] = 1 << 20                     # outside the pool, in the way of sequence 1
    rows = rnd(3, (9, 1, 32), "bf16").cuda()
    length = i32([46, 30, 60])                     # sequence 0 runs over, 2 lies past the capacity
    out = torch.zeros_like(length)
    old = case.host(0)
    Bnd.kv_append(case.cache, case.kv(length, out), rows, rows, per_seq=3, k_scale=case.gk, v_scale=case.gv)
    assert out.tolist() == [48, 33, 48]
    assert case.cache.status() == Bnd.FLAG_KV_CAPACITY | Bnd.FLAG_PAGE_RANGE
    got = case.host(0)
    case.view.table = case.pages
    for b, t, i in ((0, 46, 0), (0, 47, 1), (1, 30, 3), (1, 31, 4)):
        np.testing.assert_array_equal(case.view.value(got, b, t, case.gk), want_rows(case, f64(rows[i]), case.gk, fmt))
        for p in (old, got):
            s = case.view.slot(p, b, t)
            for x in (s if isinstance(s, tuple) else (s,)):
                x[...] = 0
    np.testing.assert_array_equal(old.view(np.uint8), got.view(np.uint8))
    # an index outside its rows, and a position outside the table
    Bnd.kv_append(case.cache, case.kv(i32([0, 0, 0]), out), rows, rows, per_seq=1, index=i32([0, 3, -1]), index_rows=3)
    assert case.cache.status() == Bnd.FLAG_ROW_RANGE
    Bnd.kv_append(case.cache, case.kv(i32([0, 0, 0]), out), rows[:3], rows[:3], per_seq=1,
                  pos=i32([0, 8, 3]), rope=Bnd.Rope(32, 8))
    assert case.cache.status() == Bnd.FLAG_POS_RANGE
    assert out.tolist() == [1, 1, 1]


def test_append_extreme_values():
    """Zeros, the format's ends, infinities and NaN in a 4-bit cache."""
    case = Case("kv4", 1, 1, 64, 16, gk=1.0, gv=1.0)
    x = torch.zeros(4, 1, 64)
    x[1, 0, :16] = torch.linspace(-2688, 2688, 16)              # the largest scale, 448
    x[1, 0, 16:32] = 1e30                                       # beyond: saturates
    x[1, 0, 32:48] = 2.0 ** -11                                 # below the smallest scale: zero
    x[2, 0, 3] = float("inf")
    x[2, 0, 20] = float("nan")
    x[3, 0, :16] = -0.0
    x = x.cuda()
    out = i32([0])
    Bnd.kv_append(case.cache, case.kv(i32([0]), out), x, x, per_seq=4)
    assert case.cache.status() == Bnd.FLAG_NONFINITE
    got = case.view.prefix(case.host(1), 0, 4)
    assert (got[0] == 0).all() and (got[3] == 0).all()
    np.testing.assert_array_equal(got[1, 0, :16], R.decode(*R.encode(f64(x[1, 0, :16]), 1.0), 1.0))
    assert (got[1, 0, 16:32] == 2688).all() and (got[1, 0, 32:48] == 0).all()
    assert np.isnan(got[2, 0, :32]).all() and (got[2, 0, 32:] == 0).all()


@pytest.mark.parametrize("fmt,dtype", [("kv4", "bf16"), ("kv4", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("dh,page", [(32, 0), (64, 48), (128, 16), (128, 0)])
def test_read(fmt, dtype, dh, page):
    B, Hkv, capacity = 3, 2, 96
    case = Case(fmt, B, Hkv, dh, capacity, page)
    lens, first, n = [96, 40, 7], [0, 11, 7], [96, 29, 0]
    if fmt == "kv4":
        case.fill(lens)
    start = i32([1, 97, 126, 126])
    out = [torch.full((130, Hkv + 1, dh), 3.0, dtype=DT[dtype], device="cuda") for _ in "kv"]
    k, v = out[0][:, 1:], out[1][:, :Hkv]
    Bnd.kv_read(case.cache, case.kv(i32(lens)), k, v, start=start, first=i32(first), k_scale=case.gk,
                v_scale=case.gv)
    assert case.cache.status() == 0
    for which, x, g in ((0, k, case.gk), (1, v, case.gv)):
        raw, at = case.host(which), 1
        for b in range(B):
            for j in range(n[b]):
                w = case.view.value(raw, b, first[b] + j, g)
                np.testing.assert_array_equal(f64(x[at]), f64(torch.from_numpy(w).float().to(DT[dtype])))
                at += 1
        assert (x[0] == 3).all() and (x[126:] == 3).all()
    assert (out[0][:, 0] == 3).all() and (out[1][:, Hkv] == 3).all()
    # slots past a length stay as they were, and are reported
    Bnd.kv_read(case.cache, case.kv(i32(lens)), k, v, per_seq=8, first=i32([90, 38, 0]), count=i32([8, 8, 8]),
                k_scale=case.gk, v_scale=case.gv, rows=24)
    assert case.cache.status() == Bnd.FLAG_KV_CAPACITY


def test_cache_refusals():
    case = Case("kv4", 2, 2, 64, 32, Hq=4, max_nodes=4)
    length, out = i32([0, 0]), i32([0, 0])
    rows = rnd(1, (4, 2, 64), "bf16").cuda()
    kv = case.kv(length, out)

    def refused(code, fn, *a, **kw):
        with pytest.raises(Bnd.MedusaError) as e:
            fn(*a, **kw)
        assert e.value.code == code

    refused(-1, Bnd.kv_append, case.cache, case.kv(length, None), rows, rows, per_seq=2)
    refused(-1, Bnd.kv_append, case.cache, kv, rows, rows, per_seq=2, k_scale=0.0)
    refused(-1, Bnd.kv_append, case.cache, kv, rows, rows, per_seq=2, v_scale=float("nan"))
    refused(-1, Bnd.kv_append, case.cache, kv, rows, rows, per_seq=2, rope=Bnd.Rope(128, 8))
    refused(-1, Bnd.kv_append, case.cache, kv, rows, rows, per_seq=0)
    refused(-1, Bnd.kv_append, case.cache, Bnd.kv_struct(case.pool[0][1:], case.pool[1], length, out), rows, rows,
            per_seq=2)
    refused(-1, Bnd.kv_append, case.cache, kv, rows, rows, per_seq=2, index=i32([0] * 4), index_rows=0)
    with pytest.raises(ValueError):
        Bnd.kv_append(case.cache, kv, rows[:, :1], rows, per_seq=2)
    with pytest.raises(TypeError):
        Bnd.kv_append(case.cache, kv, rows, rows.float(), per_seq=2)
    with pytest.raises(ValueError):
        Bnd.kv_append(case.cache, kv, rows, rows, start=i32([0, 4]))
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    q = rnd(2, (2, 3, 4, 64), "bf16").cuda()
    o, t = torch.empty_like(q), rnd(3, (2, 3, 2, 64), "bf16").cuda()
    refused(-6, Bnd.kv4_attention, case.cache, kv, q, o, ws[:16])
    refused(-1, Bnd.kv4_attention, case.cache, kv, q, o, ws, tree_k=t)
    refused(-1, Bnd.kv4_attention, case.cache, kv, q, o, ws, mask=i32([1] * 24))
    refused(-1, Bnd.kv4_attention, case.cache, kv, q, o, ws, scale=float("inf"))
    five = rnd(2, (2, 5, 4, 64), "bf16").cuda()
    refused(-1, Bnd.kv4_attention, case.cache, kv, five, torch.empty_like(five), ws)     # past max_nodes
    with pytest.raises(TypeError):
        Bnd.kv4_attention(case.cache, kv, q, o.float(), ws)
    with pytest.raises(ValueError):
        Bnd.kv4_attention(case.cache, kv, q, o, ws, tree_k=t[:, :2], tree_v=t[:, :2])
    plain = Case("bf16", 2, 2, 64, 32, Hq=4)
    refused(-2, Bnd.kv4_attention, plain.cache, plain.kv(length), q[:, :1], o[:, :1], ws)
    assert case.cache.status() == 0


# ------------------------------------------------------------------ attention
def attn_bound(dtype, o, spread, reach, dh, keys, vmax):
    """How far a float32 softmax-weighted sum may be from the 64-bit one.

    Scores: the queries keep 22 bits (f32; exact for bf16 up to 2^-25 of the row's largest), dh
    products are summed in float32 in some order, and the base-2 exponential's argument and
    result round: a score moves by at most reach (2^-21 + dh u + 4u) + 2^-22, a probability by
    that relative, numerator and denominator both.  Probabilities keep 22 bits (f32) or 11 (bf16:
    2^-12 relative, 2^-25 absolute below the normal halves), sums over the keys round once
    each key."""
    d = reach * (2.0 ** -21 + (dh + 4) * U) + 2.0 ** -22
    if dtype == "f32":
        return spread * (2 * d + 2.0 ** -21 + 2 * keys * U) + keys * 2.0 ** -36 * vmax
    e = spread * (2 * d + 2.0 ** -12 + 2 * keys * U) + keys * 2.0 ** -25 * vmax
    return e + H["bf16"] * (np.abs(o) + e)


def see_matrix(n1, kind, seed=0):
    rng = np.random.default_rng(seed)
    see = np.zeros((n1, n1), bool)
    for n in range(n1):
        if kind == "chain":
            see[n, :n + 1] = True
        elif kind == "tree":
            if n:
                see[n] = see[rng.integers(0, n)]
            see[n, n] = True
        else:                                  # any bits, some rows none
            see[n] = rng.random(n1) < 0.4
            if n % 3 == 0:
                see[n] = False
    return see


def mask_of(see):
    full = np.zeros((see.shape[0], 256), bool)
    full[:, :see.shape[1]] = see
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def run_attention(dtype, Hq, Hkv, dh, n1, lens, page, kind, scale=0.0, gain=1.0, qgain=1.0, seed=0,
                  capacity=None, strided=False, stream=None):
    B = len(lens)
    unit = page or 16
    capacity = capacity or (max(max(lens), 1) + unit - 1) // unit * unit
    case = Case("kv4", B, Hkv, dh, capacity, page, Hq=Hq, max_nodes=n1, seed=seed)
    case.fill(lens, seed + 1, gain)
    q = rnd(seed + 2, (B, n1, Hq + (3 if strided else 0), dh), dtype, qgain).cuda()[:, :, :Hq]
    tk = tv = see = None
    if kind is not None:
        see = see_matrix(n1, kind, seed)
        tk, tv = rnd(seed + 3, (B, n1, Hkv, dh), dtype).cuda(), rnd(seed + 4, (B, n1, Hkv, dh), dtype).cuda()
    o = torch.full((B, n1, Hq, dh), float("nan"), dtype=DT[dtype], device="cuda")
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)
    mask = None if kind in (None, "chain") else mask_of(see)
    length = i32(lens)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    Bnd.kv4_attention(case.cache, case.kv(length), q, o, ws, tree_k=tk, tree_v=tv, mask=mask, scale=scale,
                      k_scale=case.gk, v_scale=case.gv, stream=stream)
    torch.cuda.synchronize()
    assert case.cache.status() == 0
    raw = case.host(0), case.host(1)
    for b in range(B):
        K, V = (case.view.prefix(raw[i], b, lens[b], g) for i, g in ((0, case.gk), (1, case.gv)))
        w, spread, reach = R.attention(f64(q[b]), K, V, None if tk is None else f64(tk[b]),
                                       None if tv is None else f64(tv[b]), see, scale or dh ** -0.5)
        keys = lens[b] + n1
        vmax = max(np.abs(V).max() if len(V) else 0, np.abs(f64(tv[b])).max() if tv is not None else 0)
        tol = attn_bound(dtype, w, spread, reach, dh, keys, vmax)
        g = f64(o[b])
        assert np.isfinite(g).all(), (b, lens[b])
        assert (np.abs(g - w) <= tol).all(), (b, lens[b], np.abs(g - w).max(), (np.abs(g - w) / (tol + 1e-30)).max())


ATTENTION = [
    # Hq, Hkv, dh, n1, lens, page, kind
    (4, 4, 128, 1, (0, 1, 15, 16, 17), 0, "chain"),
    (4, 4, 128, 1, (0, 5, 64, 129), 16, None),
    (8, 2, 128, 1, (300, 63, 64, 65), 16, "chain"),
    (7, 1, 64, 1, (127, 128, 200), 48, "chain"),
    (16, 2, 32, 1, (33, 500), 0, None),
    (32, 1, 128, 1, (100,), 16, "chain"),                  # 32 rows of one KV head
    (2, 1, 128, 9, (40, 0, 700), 16, "tree"),
    (8, 2, 64, 31, (1, 45, 300), 16, "tree"),
    (4, 4, 128, 65, (200, 128, 0), 0, "tree"),
    (4, 1, 128, 43, (257, 16), 16, "tree"),                # 172 rows
    (2, 2, 32, 66, (70, 130), 32, "any"),
    (3, 3, 64, 150, (129, 1), 0, "any"),
    (1, 1, 128, 256, (140,), 0, "chain"),
    (28, 4, 128, 20, (333, 0), 48, "any"),                 # groups of 7: 140 rows
    (64, 8, 128, 40, (90,), 0, None),                      # 320 rows
]


@pytest.mark.parametrize("Hq,Hkv,dh,n1,lens,page,kind", ATTENTION)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention(Hq, Hkv, dh, n1, lens, page, kind, dtype):
    run_attention(dtype, Hq, Hkv, dh, n1, lens, page, kind, seed=n1 + dh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n1", [1, 20, 70])
def test_attention_sharp_and_flat(dtype, n1):
    """Scores far apart (one key takes all), all alike, and far from a half's range."""
    run_attention(dtype, 4, 2, 64, n1, (100, 257), 16, "tree", gain=30.0, qgain=20.0, seed=3)
    run_attention(dtype, 4, 2, 64, n1, (100, 257), 16, "tree", scale=1e-6, seed=4)
    run_attention(dtype, 4, 2, 64, n1, (90,), 0, "tree", qgain=1e6, scale=1e-7, seed=5)
    run_attention(dtype, 4, 2, 64, n1, (90,), 0, "tree", qgain=1e-6, scale=1e5, seed=6)


@pytest.mark.parametrize("n1,Hq,Hkv", [(1, 2, 2), (1, 8, 1), (65, 1, 1), (43, 4, 1)])
def test_attention_long_and_ragged(n1, Hq, Hkv):
    """Prefixes that are shared out over many blocks, beside empty and short ones, in a cache
    with room left."""
    run_attention("bf16", Hq, Hkv, 128, n1, (3000, 0, 1, 129, 2047), 16, "tree", capacity=4096, strided=True)
    run_attention("f32", Hq, Hkv, 64, n1, (2500, 7), 0, "chain", capacity=4096)


@pytest.mark.parametrize("capacity", [8192, 8208])
@pytest.mark.parametrize("dtype,dh,n1", [("bf16", 128, 1), ("bf16", 64, 9), ("f32", 32, 5), ("f32", 128, 12)])
def test_attention_few_rows_in_short_and_long_caches(capacity, dtype, dh, n1):
    """Small calls share a head out over a fixed number of blocks, in long caches over all: with
    fewer chunks than blocks, one short of and one past a multiple, empty and full ones."""
    run_attention(dtype, 2, 2, dh, n1, (1025, 0, 1, 1023, 130), 16, "tree", capacity=capacity, strided=True)
    run_attention(dtype, 3, 1, dh, n1, (0, 8192), 0, None, capacity=capacity)


def test_attention_many_sequences():
    lens = [int(x) for x in np.random.default_rng(2).integers(0, 90, 70)]
    run_attention("bf16", 2, 1, 64, 1, lens, 16, "chain")
    run_attention("bf16", 2, 1, 64, 17, lens[:40], 16, "tree")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n1,capacity", [(1, 512), (1, 8208), (9, 512), (40, 512), (160, 512)])
def test_attention_not_a_number(dtype, n1, capacity):
    """A NaN that a row sees (in its query, a key, a value, a call's own row) makes that row's head
    NaN and nothing else; one that it does not see changes nothing."""
    B, H, dh = 6, 2, 64
    case = Case("kv4", B, H, dh, capacity, 16, max_nodes=n1)
    lens = [1, 300, 300, 300, 300, 0]
    case.fill(lens)
    ws = torch.full((case.cache.workspace_size,), 0xff, dtype=torch.uint8, device="cuda")
    q = rnd(1, (B, n1, H, dh), dtype).cuda()
    tk, tv = rnd(2, (B, n1, H, dh), dtype).cuda(), rnd(3, (B, n1, H, dh), dtype).cuda()
    see = np.eye(n1, dtype=bool)                       # each node sees itself
    last = see.copy()
    last[n1 - 1] = False                               # the last one nothing

    def run(see):
        o = torch.empty_like(q)
        Bnd.kv4_attention(case.cache, case.kv(i32(lens)), q, o, ws, tree_k=tk, tree_v=tv, mask=mask_of(see),
                          k_scale=case.gk, v_scale=case.gv)
        assert case.cache.status() == 0
        return o

    good, hidden = run(see), run(last)
    assert torch.isfinite(good.float()).all() and torch.isfinite(hidden.float()).all()
    assert (hidden[5, n1 - 1] == 0).all()
    # the scale of the first 16 elements of head 1: slot 0 of sequence 0 (keys), slot 299 of 1 (keys), of 2 (values)
    for pool, b, t in ((0, 0, 0), (0, 1, 299), (1, 2, 299)):
        block = (int(case.pages[b, t // 16]) * H + 1) * 9 * dh
        case.pool[pool][block + 8 * dh + t % 16 * (dh // 16)] = 0x7f
    q[3, n1 - 1, 0, 5] = float("nan")
    tk[4, n1 - 1, 1, 7] = float("nan")
    tv[5, n1 - 1, 0, 7] = float("nan")
    bad, hidden2 = run(see).float(), run(last).float()
    want = torch.zeros(B, n1, H, dh, dtype=torch.bool, device="cuda")
    want[0, :, 1] = want[1, :, 1] = True
    want[2, :, 1, :16] = True
    want[3, n1 - 1, 0] = True
    unseen = want.clone()
    want[4, n1 - 1, 1] = True
    want[5, n1 - 1, 0, 7] = True
    assert torch.equal(bad.isnan(), want)
    assert torch.equal(bad[~want], good.float()[~want])
    assert torch.equal(hidden2.isnan(), unseen)
    assert torch.equal(hidden2[~unseen], hidden.float()[~unseen])


@pytest.mark.parametrize("Hq,Hkv,dh,n1", [(32, 8, 128, 43), (32, 8, 64, 43), (64, 8, 128, 40), (24, 24, 128, 65),
                                           (32, 8, 64, 20)])
def test_attention_blocks_that_do_many_heads(Hq, Hkv, dh, n1):
    """More (sequence, head) pairs than there are blocks on the GPU: each goes from head to head."""
    lens = [int(x) for x in np.random.default_rng(n1).integers(1, 420, 24)]
    lens[3] = 0
    run_attention("bf16", Hq, Hkv, dh, n1, lens, 16, "tree", seed=n1)


@pytest.mark.parametrize("Hq,Hkv,dh,n1,B,most,page", [
    (32, 8, 64, 43, 24, 420, 16), (32, 8, 128, 43, 24, 420, 16), (64, 8, 64, 40, 24, 420, 16),
    (24, 24, 64, 65, 24, 420, 0), (40, 40, 128, 65, 8, 4000, 0), (40, 40, 64, 65, 8, 2000, 16),
    (32, 8, 128, 43, 16, 4000, 16), (40, 40, 128, 8, 8, 1000, 0)])
def test_attention_repeats_bit_for_bit(Hq, Hkv, dh, n1, B, most, page):
    """The same call gives the same bits every time: blocks that go from head to head, with odd
    and even numbers of chunks, wait for what they read."""
    rng = np.random.default_rng(n1)
    lens = [int(x) for x in rng.integers(1, most, B)]
    capacity = (max(lens) + 15) // 16 * 16
    case = Case("kv4", B, Hkv, dh, capacity, page, Hq=Hq, max_nodes=n1)
    for pool in case.pool:                             # any codes, scales from 0.5 to 1.875
        scales = pool.view(-1, 9 * dh)[:, 8 * dh:]
        scales.copy_(torch.randint(0x30, 0x40, scales.shape, dtype=torch.uint8, device="cuda"))
    q = rnd(1, (B, n1, Hq, dh), "bf16").cuda()
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    kv, outs = case.kv(i32(lens)), []
    for _ in range(60):
        o = torch.empty_like(q)
        Bnd.kv4_attention(case.cache, kv, q, o, ws, k_scale=case.gk, v_scale=case.gv)
        outs.append(o)
    assert case.cache.status() == 0
    assert torch.isfinite(outs[0].float()).all()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_attention_on_another_stream_and_repeated():
    run_attention("bf16", 8, 2, 128, 20, (300, 100), 16, "tree", stream=torch.cuda.Stream())
    case = Case("kv4", 3, 2, 128, 512, 16, Hq=8, max_nodes=43)
    case.fill([500, 100, 511])
    q = rnd(1, (3, 43, 8, 128), "bf16").cuda()
    outs = []
    for n in (43, 1):
        for _ in range(3):
            o = torch.empty(3, n, 8, 128, dtype=torch.bfloat16, device="cuda")
            ws = torch.randint(0, 256, (case.cache.workspace_size,), dtype=torch.uint8, device="cuda")
            Bnd.kv4_attention(case.cache, case.kv(i32([500, 100, 511])), q[:, :n].contiguous(), o, ws,
                              k_scale=case.gk, v_scale=case.gv)
            outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])      # bit for bit
    assert torch.equal(outs[3], outs[4]) and torch.equal(outs[3], outs[5])


def test_two_streams_and_two_graphs_with_one_handle():
    """Calls on one cache handle at the same time, each with its own workspace and outputs, eager
    and as two captured graphs replayed side by side."""
    case = Case("kv4", 4, 4, 128, 1024, 16, Hq=8, max_nodes=40)
    lens = [1000, 3, 517, 1024]
    case.fill(lens)
    length = i32(lens)
    kv = case.kv(length)
    q = [rnd(i, (4, n1, 8, 128), "bf16").cuda() for i, n1 in enumerate((40, 1))]
    o = [torch.empty_like(x) for x in q]
    ws = [torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda") for _ in q]
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    rows = [torch.empty(2, sum(lens), 4, 128, dtype=torch.bfloat16, device="cuda") for _ in q]

    def call(i, stream=None):
        Bnd.kv4_attention(case.cache, kv, q[i], o[i], ws[i], k_scale=case.gk, v_scale=case.gv, stream=stream)
        Bnd.kv_read(case.cache, kv, rows[i][0], rows[i][1], start=start, k_scale=case.gk, v_scale=case.gv, stream=stream)

    for i in (0, 1):
        call(i)
    torch.cuda.synchronize()
    want = [x.clone() for x in o + rows]
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(20):
        for i in (0, 1):
            call(i, streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, o + rows))
    graphs = [torch.cuda.CUDAGraph() for _ in q]
    for i in (0, 1):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            call(i)
    for x in o + rows:
        x.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, o + rows))
    assert case.cache.status() == 0


def test_attention_bad_lengths_and_pages_are_reported():
    case = Case("kv4", 2, 1, 64, 64, 16, Hq=2, max_nodes=30)
    case.fill([64, 64])
    case.table[1, 1] = -7
    for n1 in (1, 30):
        q = rnd(1, (2, n1, 2, 64), "bf16").cuda()
        o = torch.empty_like(q)
        ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
        Bnd.kv4_attention(case.cache, case.kv(i32([64, 64])), q, o, ws)
        assert case.cache.status() == Bnd.FLAG_PAGE_RANGE
        # lengths outside 0..capacity count as the nearer end
        Bnd.kv4_attention(case.cache, case.kv(i32([99, -3])), q, o, ws)
        assert case.cache.status() == 0
        assert torch.isfinite(o[0].float()).all() and (o[1] == 0).all()


def test_decode_loop_captured():
    """A graph of rotate, append, attend and read, replayed: a cache that grows in place."""
    B, Hq, Hkv, dh, cap = 2, 4, 2, 64, 64
    case = Case("kv4", B, Hkv, dh, cap, 16, Hq=Hq)
    rope = Bnd.Rope(dh, cap)
    length, kv = i32([0, 20]), None
    case.fill([0, 20])
    kv = case.kv(length, length)
    x = torch.empty(B, Hq + 2 * Hkv, dh, dtype=torch.bfloat16, device="cuda")
    qr, o = torch.empty(B, 1, Hq, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, Hq, dh, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")

    def step():
        Bnd.rope_apply(rope, length, [(x[:, :Hq], qr[:, 0])])
        Bnd.kv_append(case.cache, kv, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], per_seq=1, rope=rope, k_scale=case.gk,
                      v_scale=case.gv)
        Bnd.kv4_attention(case.cache, kv, qr, o, ws, k_scale=case.gk, v_scale=case.gv)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x.copy_(rnd(50, x.shape, "bf16"))
    with torch.cuda.stream(s):
        step()
        length.sub_(1)                     # the warm-up token is written again
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(30):
        xi = rnd(100 + i, x.shape, "bf16")
        x.copy_(xi)
        g.replay()
        lens = [i + 1, 21 + i]
        assert length.tolist() == lens
        raw = case.host(0), case.host(1)
        for b in range(B):
            K, V = (case.view.prefix(raw[j], b, lens[b], sc) for j, sc in ((0, case.gk), (1, case.gv)))
            np.testing.assert_array_equal(V[-1], R.decode(*R.encode(f64(xi[b, Hq + Hkv:]), case.gv), case.gv))
            w, spread, reach = R.attention(f64(qr[b]), K, V, None, None, None, dh ** -0.5)
            assert (np.abs(f64(o[b]) - w) <= attn_bound("bf16", w, spread, reach, dh, lens[b], np.abs(V).max())).all()
    assert case.cache.status() == 0 and rope.status() == 0


def test_step_on_a_four_bit_cache():
    """The stages of a decode step with the cache in 4 bits: prompt appended, tree projected by
    the step's own stage, attention over the 4-bit prefix, output stage, acceptance, and the
    accepted nodes appended; attention against the 64-bit form of the same rows, the cache
    against the 64-bit encoding of the kept nodes."""
    import synthetic as S
    w = S.Workload("kv4", B=2, d=256, V=500, Hq=4, Hkv=2, dh=64, K=3, dtype="bf16", lengths=(37, 90),
                   tree="cartesian", s=(3, 2, 2), N=21, page_size=16)
    from harness import accept_of, spec_for
    parent, rank, spec = spec_for(w)
    B, n1 = w.B, w.N + 1
    plan = Bnd.Plan(B, w.d, w.V, w.K, w.Hq, w.Hkv, w.dh, Bnd.BF16, w.capacity, w.s, parent, rank, page_size=16,
                    num_pages=B * w.pages_per_seq)
    wts = {k: v.cuda() for k, v in S.weights(w).items()}
    ws = torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    W, h = Bnd.weights_struct(wts), S.hidden(w).cuda()
    case = Case("kv4", B, w.Hkv, w.dh, w.capacity, 16, Hq=w.Hq, max_nodes=n1)
    rows = sum(w.lengths)
    pk, pv = rnd(7, (rows, w.Hkv, w.dh), "bf16").cuda(), rnd(8, (rows, w.Hkv, w.dh), "bf16").cuda()
    length = i32([0, 0])
    kv = case.kv(length, length)
    Bnd.kv_append(case.cache, kv, pk, pv, start=i32([0, 37, 127]), rope=Bnd.Rope(w.dh, w.capacity),
                  k_scale=case.gk, v_scale=case.gv)
    assert length.tolist() == list(w.lengths)
    i = dict(dtype=torch.int32, device="cuda")
    ttok, root = torch.empty(B, w.K, 16, **i), torch.empty(B, **i)
    tval = torch.empty(B, w.K, 16, device="cuda")
    Bnd.heads(plan, h, None, W, None, ttok, tval, root, ws)
    tok, pos, mask = torch.empty(B, n1, **i), torch.empty(B, n1, **i), torch.empty(n1, 8, **i)
    retr = torch.empty(n1, w.K + 1, **i)
    Bnd.tree_build(plan, ttok, root, length, tok, pos, mask, retr)
    q = torch.empty(B, n1, w.Hq, w.dh, device="cuda")
    tk, tv = (torch.empty(B, n1, w.Hkv, w.dh, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    Bnd.layer_qkv(plan, W, tok, pos, q, tk, tv, ws)
    # in float32 from the stage's queries and the tree's keys, so that o feeds the next stage
    o = torch.empty_like(q)
    aws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    tk32, tv32 = tk.float(), tv.float()
    Bnd.kv4_attention(case.cache, kv, q, o, aws, tree_k=tk32, tree_v=tv32, mask=mask, k_scale=case.gk,
                      v_scale=case.gv)
    see = np.zeros((n1, n1), bool)
    for n in range(n1):
        j = n
        while j >= 0:
            see[n, j] = True
            j = spec.parent[j]
    raw = case.host(0), case.host(1)
    for b in range(B):
        K, V = (case.view.prefix(raw[x], b, w.lengths[b], g) for x, g in ((0, case.gk), (1, case.gv)))
        want, spread, reach = R.attention(f64(q[b]), K, V, f64(tk[b]), f64(tv[b]), see, w.dh ** -0.5)
        tol = attn_bound("f32", want, spread, reach, w.dh, w.lengths[b] + n1, np.abs(V).max())
        assert (np.abs(f64(o[b]) - want) <= tol).all()
    hp, am, stats = torch.empty(B, n1, w.d, device="cuda"), torch.empty(B, n1, **i), torch.empty(B, n1, 4, device="cuda")
    Bnd.layer_out(plan, W, tok, o, hp, ws)
    acc = Bnd.accept_struct(**accept_of(w))
    Bnd.verify_logits(plan, W, hp, tok, acc, None, am, stats, ws)
    out_tok, path, n_acc = torch.empty(B, w.K + 1, **i), torch.empty(B, w.K + 1, **i), torch.empty(B, **i)
    outs = Bnd.outputs_struct(out_tok, n_acc, path, torch.empty(B, w.d, device="cuda"), torch.empty(B, **i))
    Bnd.verify(plan, tok, am, stats, retr, hp, acc, outs)
    Bnd.kv_append(case.cache, kv, tk.view(-1, w.Hkv, w.dh), tv.view(-1, w.Hkv, w.dh), per_seq=w.K + 1, count=n_acc,
                  index=path, index_rows=n1, k_scale=case.gk, v_scale=case.gv)
    assert length.tolist() == [x + int(n) for x, n in zip(w.lengths, n_acc)]
    raw = case.host(0), case.host(1)
    for b in range(B):
        for j in range(int(n_acc[b])):
            node, t = int(path[b, j]), w.lengths[b] + j
            np.testing.assert_array_equal(case.view.value(raw[0], b, t, case.gk), R.decode(*R.encode(f64(tk[b, node]), case.gk), case.gk))
            np.testing.assert_array_equal(case.view.value(raw[1], b, t, case.gv), R.decode(*R.encode(f64(tv[b, node]), case.gv), case.gv))
    assert case.cache.status() == 0 and plan.status() == 0


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: its last pages are written, read and attended over."""
    Hkv, dh, page = 8, 128, 16
    pages = (1 << 32) // (Hkv * 9 * dh) + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * pages * Hkv * 9 * dh:
        pytest.skip("not enough device memory")
    cache = Bnd.Cache(1, 8, Hkv, dh, Bnd.KV4, 64, page_size=page, num_pages=pages)
    k, v = (torch.empty(cache.pool_bytes, dtype=torch.uint8, device="cuda") for _ in "kv")
    table, length, out = i32([[pages - 1, 3, pages - 7, pages // 2]]), i32([0]), i32([0])
    rows = rnd(1, (64, Hkv, dh), "bf16").cuda()
    vals = rnd(2, (64, Hkv, dh), "bf16").cuda()
    Bnd.kv_append(cache, Bnd.kv_struct(k, v, length, out, table), rows, vals, per_seq=64)
    kv = Bnd.kv_struct(k, v, out, None, table)
    gk, gv = torch.empty_like(rows), torch.empty_like(rows)
    Bnd.kv_read(cache, kv, gk, gv, per_seq=64)
    K, V = (R.decode(*R.encode(f64(x), 1.0), 1.0) for x in (rows, vals))
    np.testing.assert_array_equal(f64(gk), K)
    np.testing.assert_array_equal(f64(gv), V)
    q = rnd(3, (1, 1, 8, dh), "bf16").cuda()
    o = torch.empty_like(q)
    ws = torch.empty(cache.workspace_size, dtype=torch.uint8, device="cuda")
    Bnd.kv4_attention(cache, kv, q, o, ws)
    w, spread, reach = R.attention(f64(q[0]), K, V, None, None, None, dh ** -0.5)
    assert (np.abs(f64(o[0]) - w) <= attn_bound("bf16", w, spread, reach, dh, 64, np.abs(V).max())).all()
    assert cache.status() == 0
