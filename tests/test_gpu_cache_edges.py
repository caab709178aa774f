"""Edges of the cache operators' documented ranges, against the 64-bit forms in kv4_ref.py.
Tolerances as in test_gpu_cache.py, or exact."""
import time

import numpy as np
import pytest
import torch

import kv4_ref as R
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd
from test_gpu_cache import DT, H, U, Case, attn_bound, f64, i32, mask_of, rnd, see_matrix, want_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def off_by_one(x):
    """The same rows one element off every 16-byte boundary."""
    n, h, d = x.shape
    buf = torch.zeros(n * h * (d + 1) + 1, dtype=x.dtype, device=x.device)
    v = torch.as_strided(buf, (n, h, d), (h * (d + 1), d + 1, 1), 1)
    return v.copy_(x)


# ------------------------------------------------------------------ values past the 4-bit scales
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("g", [1e-20, 1e-3, 0.05, 1.0, 1e20])
def test_append_beyond_the_largest_scale(g, aligned, src):
    """Finite groups whose largest element passes 6 * 448 g, up to a float's end: scale 448, elements
    beyond it the largest code of their sign, the others (none nearer than 8 % to a border between two codes, bf16
    rounding moves them by 0.4 %) their nearest code.  Nothing of it is not finite."""
    g = float(np.float32(g))
    case = Case("kv4", 1, 1, 64, 16, gk=g, gv=g)
    codes = [.1, -.4, .6, -.9, 1.1, -1.4, 1.6, -1.9, 2.2, -2.8, 3.2, -3.9, 4.4, -5.5]
    x = np.zeros((4, 1, 64))
    for i, big in enumerate((3.3e38, min(2e39 * g, 1e38), 2800 * g, 1e5 * g)):
        for part, ends in enumerate(((big, -big), (-big, 0.0), (0.0, big), (-big, -big))):
            x[i, 0, 16 * part:16 * part + 16] = [448 * g * c for c in codes] + list(ends)
    x = torch.from_numpy(x.astype(np.float32)).to(DT[src]).cuda()
    k = x if aligned else off_by_one(x)
    out = i32([0])
    Bnd.kv_append(case.cache, case.kv(i32([0]), out), k, k, per_seq=4, k_scale=g, v_scale=g)
    assert case.cache.status() == 0 and out.tolist() == [4]
    want_codes, want_scales = R.encode(f64(x), g)
    assert (want_scales == 0x7e).all()
    for which in (0, 1):
        raw = case.host(which)
        for t in range(4):
            got_codes, got_scales = case.view.slot(raw, 0, t)
            np.testing.assert_array_equal(got_scales, want_scales[t])
            np.testing.assert_array_equal(got_codes, want_codes[t])
    rk, rv = (torch.empty(4, 1, 64, device="cuda") for _ in "kv")
    Bnd.kv_read(case.cache, case.kv(out), rk, rv, per_seq=4, k_scale=g, v_scale=g)
    held = R.decode(want_codes, want_scales, g)
    assert (np.abs(f64(rk) - held) <= 4 * U * np.abs(held)).all() and torch.equal(rk, rv)


# ------------------------------------------------------------------ scores at the ends of a float's range
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n1", [1, 20, 70])
@pytest.mark.parametrize("kind", [None, "tree"])
@pytest.mark.parametrize("qgain,scale,g,kvgain", [
    (1e-30, 1e-10, 1e-20, 1e-18),          # scale, k_scale and the row's largest query multiply to 0 in float
    (1e-38, 1e27, 1e14, 1e14),             # scale * k_scale alone passes a float's range, the scores do not
    (1e30, 1e-20, 1e-20, 1e-18),
])
def test_attention_factors_outside_a_float(qgain, scale, g, kvgain, kind, n1, dtype):
    Hq, Hkv, dh, lens, page, capacity = 4, 2, 64, (90, 257, 16), 16, 512
    g = float(np.float32(g))
    case = Case("kv4", len(lens), Hkv, dh, capacity, page, Hq=Hq, max_nodes=n1, gk=g, gv=g)
    case.fill(lens, 1, kvgain)
    q = rnd(2, (3, n1, Hq, dh), dtype, qgain).cuda()
    tk = tv = see = mask = None
    if kind:
        see = see_matrix(n1, kind)
        tk, tv = rnd(3, (3, n1, Hkv, dh), dtype, kvgain).cuda(), rnd(4, (3, n1, Hkv, dh), dtype, kvgain).cuda()
        mask = mask_of(see)
    ws = torch.full((case.cache.workspace_size,), 0xff, dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    Bnd.kv4_attention(case.cache, case.kv(i32(lens)), q, o, ws, tree_k=tk, tree_v=tv, mask=mask, scale=scale, k_scale=g,
                      v_scale=g)
    assert case.cache.status() == 0
    raw = case.host(0), case.host(1)
    for b, n in enumerate(lens):
        K, V = (case.view.prefix(raw[i], b, n, g) for i in (0, 1))
        w, spread, reach = R.attention(f64(q[b]), K, V, None if tk is None else f64(tk[b]),
                                       None if tv is None else f64(tv[b]), see, float(np.float32(scale)))
        vmax = max(np.abs(V).max(), 0 if tv is None else np.abs(f64(tv[b])).max())
        got = f64(o[b])
        assert np.isfinite(got).all()
        assert (np.abs(got - w) <= attn_bound(dtype, w, spread, reach, dh, n + n1, vmax)).all()


def test_attention_scales_at_the_end_of_a_float():
    """scale * log2(e) past a float's range made scores of 0 NaN: such scales are refused, the largest others work."""
    case = Case("kv4", 1, 1, 64, 16, max_nodes=1)
    case.fill([0])
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    t, o = rnd(1, q.shape, "bf16").cuda(), torch.empty_like(q)
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    kv = case.kv(i32([0]))
    for scale in (3e38, -1.0, float("nan"), float("inf")):
        with pytest.raises(Bnd.MedusaError) as e:
            Bnd.kv4_attention(case.cache, kv, q, o, ws, tree_k=t, tree_v=t, scale=scale)
        assert e.value.code == Bnd.MEDUSA_ERR_INVALID
    Bnd.kv4_attention(case.cache, kv, q, o, ws, tree_k=t, tree_v=t, scale=1e38)
    assert torch.equal(o, t)                           # one row seen, with a score of 0


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("dtype,Hq,Hkv,dh,n1,capacity,page", [
    ("bf16", 4, 4, 128, 1, 512, 16), ("f32", 4, 2, 64, 9, 512, 0),         # few rows, short caches
    ("bf16", 8, 2, 128, 1, 8208, 16), ("f32", 4, 4, 32, 20, 8208, 0),      # and long ones
    ("bf16", 4, 4, 128, 65, 4096, 16), ("bf16", 2, 2, 64, 20, 512, 0),     # one tile of rows
    ("bf16", 8, 2, 128, 43, 4096, 16), ("bf16", 4, 1, 64, 100, 512, 0),    # two tiles, several of them
])
def test_expired_wait_is_reported_and_nothing_else_is_lost(dtype, Hq, Hkv, dh, n1, capacity, page):
    """A bounded wait of the attention kernels is made to run out: the call returns with
    MEDUSA_FLAG_TIMEOUT, whatever the workspace held, and the next one is as before."""
    B = 3
    case = Case("kv4", B, Hkv, dh, capacity, page, Hq=Hq, max_nodes=n1)
    lens = [min(capacity, 1500), 0, 129]
    for pool in case.pool:                             # any codes, scales from 0.5 to 1.875
        pool.view(-1, 9 * dh)[:, 8 * dh:] = 0x35
    q = rnd(1, (B, n1, Hq, dh), dtype).cuda()
    tk, tv = rnd(2, (B, n1, Hkv, dh), dtype).cuda(), rnd(3, (B, n1, Hkv, dh), dtype).cuda()
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    kv = case.kv(i32(lens))

    def call():
        ws.fill_(0x7f)                                 # what another program may have left there
        o = torch.empty_like(q)
        t0 = time.perf_counter()
        Bnd.kv4_attention(case.cache, kv, q, o, ws, tree_k=tk, tree_v=tv, k_scale=case.gk, v_scale=case.gv)
        torch.cuda.synchronize()
        return o, time.perf_counter() - t0

    clean, _ = call()
    assert case.cache.status() == 0 and torch.isfinite(clean.float()).all()
    case.cache.expire_wait_once(2_000_000)
    assert call()[1] < 30.0
    assert case.cache.status() == Bnd.FLAG_TIMEOUT
    assert case.cache.status() == 0
    again, _ = call()
    assert case.cache.status() == 0 and torch.equal(again, clean)


def test_expire_wait_argument_checks():
    case = Case("kv4", 1, 1, 64, 16)
    for ns in (0, 10**10 + 1):
        with pytest.raises(Bnd.MedusaError) as e:
            case.cache.expire_wait_once(ns)
        assert e.value.code == Bnd.MEDUSA_ERR_INVALID
    with pytest.raises(Bnd.MedusaError) as e:
        Case("bf16", 1, 1, 64, 16).cache.expire_wait_once(1000)
    assert e.value.code == Bnd.MEDUSA_ERR_UNSUPPORTED


# ------------------------------------------------------------------ offsets, counts and row numbers
@pytest.mark.parametrize("fmt", ["bf16", "kv4"])
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("start,rows,items", [
    ([0, 3, 9], 5, (range(0, 3), range(3, 5))),            # past the last row
    ([-2, 2, 4], 5, (range(0, 2), range(2, 4))),           # before the first
    ([7, 9, 12], 5, ((), ())),                             # nothing there at all
    ([-2**31, 2, 2**31 - 1], 5, (range(0, 2), range(2, 5))),
    ([4, 2, 5], 5, ((), range(2, 5))),                     # not ascending: the first has no items
])
def test_packed_offsets_out_of_range(start, rows, items, aligned, alias, fmt):
    """Only items there are count: len_out grows by what was written, and the offsets are reported."""
    case = Case(fmt, 2, 1, 32, 32)
    x = rnd(1, (rows, 1, 32), "bf16").cuda()
    if not aligned:
        x = off_by_one(x)
    length = i32([1, 6])
    out = length if alias else torch.zeros_like(length)
    Bnd.kv_append(case.cache, case.kv(length, out), x, x, start=i32(start), k_scale=case.gk, v_scale=case.gv)
    assert out.tolist() == [1 + len(items[0]), 6 + len(items[1])]
    assert case.cache.status() == Bnd.FLAG_ROW_RANGE
    raw = case.host(1)
    for b, at in ((0, 1), (1, 6)):
        for j, i in enumerate(items[b]):
            np.testing.assert_array_equal(case.view.value(raw, b, at + j, case.gv), want_rows(case, f64(x[i]), case.gv, fmt))
    if fmt == "kv4":
        case.fill([8, 8])
    lens = i32([8, 8])
    k, v = (torch.full((rows, 1, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    Bnd.kv_read(case.cache, case.kv(lens), k, v, start=i32(start), k_scale=case.gk, v_scale=case.gv)
    assert case.cache.status() == Bnd.FLAG_ROW_RANGE
    raw, seen = case.host(1), set()
    for b in (0, 1):
        for j, i in enumerate(items[b]):
            seen.add(i)
            np.testing.assert_array_equal(f64(v[i]), case.view.value(raw, b, j, case.gv))
    for i in set(range(rows)) - seen:
        assert (v[i] == 7).all() and (k[i] == 7).all()


@pytest.mark.parametrize("alias", [False, True])
def test_counts_out_of_range(alias):
    case = Case("bf16", 3, 1, 32, 32)
    x = rnd(1, (6, 1, 32), "bf16").cuda()
    length = i32([0, 4, 8])
    out = length if alias else torch.zeros_like(length)
    Bnd.kv_append(case.cache, case.kv(length, out), x, x, per_seq=2, count=i32([5, -1, 1]))
    assert out.tolist() == [2, 4, 9] and case.cache.status() == Bnd.FLAG_ROW_RANGE
    k, v = torch.zeros_like(x), torch.zeros_like(x)
    Bnd.kv_read(case.cache, case.kv(out), k, v, per_seq=2, count=i32([1, 3, 2]), first=i32([0, 0, 7]))
    assert case.cache.status() == Bnd.FLAG_ROW_RANGE
    Bnd.kv_read(case.cache, case.kv(out), k, v, per_seq=2, count=i32([1, 2, 0]))
    assert case.cache.status() == 0


def test_append_of_two_thousand_million_places():
    """Row counts up to a 32-bit integer's end: the last places of all are found."""
    rows = 2**31 - 1
    case = Case("bf16", 2, 1, 32, 32)
    x = rnd(1, (1, 1, 32), "bf16").cuda()
    length, out = i32([3, 0]), i32([0, 0])
    Bnd.kv_append(case.cache, case.kv(length, out), x.expand(rows, 1, 32), x.expand(rows, 1, 32),
                  start=i32([rows - 5, rows - 1, rows]))
    assert out.tolist() == [7, 1] and case.cache.status() == 0
    raw = case.host(0)
    for b, t in ((0, 3), (0, 4), (0, 5), (0, 6), (1, 0)):
        np.testing.assert_array_equal(case.view.value(raw, b, t), f64(x[0]))


def test_rows_that_are_no_equal_shares_are_refused():
    case = Case("bf16", 4, 1, 32, 16)
    rows, length, out = rnd(1, (10, 1, 32), "bf16").cuda(), i32([0] * 4), i32([-5] * 4)
    with pytest.raises(ValueError):
        Bnd.kv_append(case.cache, case.kv(length, out), rows, rows)
    with pytest.raises(ValueError):
        Bnd.kv_read(case.cache, case.kv(i32([3] * 4)), rows, rows.clone())
    assert out.tolist() == [-5] * 4
    Bnd.kv_append(case.cache, case.kv(length, out), rows[:8], rows[:8])
    Bnd.kv_append(case.cache, case.kv(length, out), rows, rows, per_seq=2)      # the rows behind are the caller's
    assert out.tolist() == [2] * 4


# ------------------------------------------------------------------ results that lie on one another
def strided(shape, strides, dtype=torch.bfloat16):
    n = 1 + sum((a - 1) * b for a, b in zip(shape, strides))
    return torch.as_strided(torch.full((n,), 7.0, dtype=dtype, device="cuda"), shape, strides)


@pytest.mark.parametrize("rows,heads,row,head,ok", [
    (6, 2, 0, 64, False), (6, 2, 128, 0, False), (6, 2, 128, 40, False), (6, 2, 64, 64, False),
    (6, 2, 128, 64, True), (6, 2, 64, 6 * 64, True), (6, 2, 64, 5 * 64, False),
    (2, 3, 192, 128, True), (3, 4, 192, 128, False), (6, 2, 136, 72, True),
    (2, 3, 200, 128, False),                   # row 1, head 0 has 200..263, row 0, head 2 256..319
])
def test_results_that_share_elements_are_refused(rows, heads, row, head, ok):
    """Rotated rows, slots read and attention's results written more than once, in any order."""
    dh = 64
    shape, strides = (rows, heads, dh), (row, head, 1)
    refused = pytest.raises(Bnd.MedusaError)
    rope, x = Bnd.Rope(dh, 16), rnd(1, shape, "bf16").cuda()
    y, want = strided(shape, strides), torch.empty_like(x)
    pos = i32(list(range(rows)))

    def attempt(call):
        if ok:
            return call()
        with refused as e:
            call()
        assert e.value.code == Bnd.MEDUSA_ERR_INVALID

    attempt(lambda: Bnd.rope_apply(rope, pos, [(x, y)]))
    Bnd.rope_apply(rope, pos, [(x, want)])
    assert torch.equal(y, want) or not ok
    case = Case("kv4", 1, heads, dh, 16, max_nodes=rows)
    case.fill([rows])
    kv = case.kv(i32([rows]))
    k, v, want = strided(shape, strides), torch.empty_like(x), torch.empty_like(x)
    attempt(lambda: Bnd.kv_read(case.cache, kv, k, v, per_seq=rows))
    attempt(lambda: Bnd.kv_read(case.cache, kv, v, k, per_seq=rows))
    Bnd.kv_read(case.cache, kv, v, want, per_seq=rows)
    assert torch.equal(k, want) or not ok
    q, o, want = x[None], strided((1,) + shape, (0,) + strides), torch.empty_like(x[None])
    ws = torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda")
    attempt(lambda: Bnd.kv4_attention(case.cache, kv, q, o, ws))
    Bnd.kv4_attention(case.cache, kv, q, want, ws)
    assert torch.equal(o, want) or not ok


def test_rows_turned_in_place_more_than_once_are_refused():
    rope, x = Bnd.Rope(64, 16), rnd(1, (1, 2, 64), "bf16").cuda()
    same = x.expand(4, 2, 64)
    with pytest.raises(Bnd.MedusaError):
        Bnd.rope_apply(rope, i32([0, 1, 2, 3]), [(same, same)])
    y = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    Bnd.rope_apply(rope, i32([0, 1, 2, 3]), [(same, y)])               # read more than once: as often as wanted
    assert torch.equal(y[0], x[0]) and not torch.equal(y[1], x[0])


# ------------------------------------------------------------------ many rows, and rotations of a part
def held(case, raw, seq, slot):
    """What pool raw has at (sequence, slot) pairs: [n][Hkv][dh] elements, or 4-bit codes and scales."""
    per = case.page or case.capacity
    unit = seq if not case.page else case.pages[seq, slot // per]
    at = slot % per
    if case.fmt != "kv4":
        return raw.reshape(-1, per, case.Hkv, case.dh)[unit, at]
    n, dh = len(seq), case.dh
    blocks = raw.reshape(-1, case.Hkv, per // 16, 9 * dh)[unit, :, at // 16]
    return (blocks[..., :8 * dh].reshape(n, case.Hkv, 16, dh // 2)[np.arange(n), :, at % 16],
            blocks[..., 8 * dh:].reshape(n, case.Hkv, 16, dh // 16)[np.arange(n), :, at % 16])


def rest(case, raw, seq, slot):
    """The pool with those slots blanked."""
    raw, per = raw.copy(), case.page or case.capacity
    unit = seq if not case.page else case.pages[seq, slot // per]
    at = slot % per
    if case.fmt != "kv4":
        raw.reshape(-1, per, case.Hkv, case.dh)[unit, at] = 0
        return raw
    dh, blocks = case.dh, raw.reshape(-1, case.Hkv, per // 16, 9 * case.dh)
    for u, t in zip(unit, at):
        r = t % 16
        blocks[u, :, t // 16, r * dh // 2:(r + 1) * dh // 2] = 0
        blocks[u, :, t // 16, 8 * dh + r * dh // 16:8 * dh + (r + 1) * dh // 16] = 0
    return raw


def check_turned(fmt, got, x, pos, rot, layout, g):
    """Keys x [n][Hkv][dh] as held after their rotation; bounds as in test_append_packed."""
    w = R.rope(x, pos, rot, layout)
    tol = 4 * U * (np.abs(x) + 4 * np.abs(x).max(-1, keepdims=True))
    tol[..., rot:] = 0                                     # passes through
    if fmt != "kv4":
        tol = np.where(tol > 0, tol + H[fmt] * (np.abs(w) + tol), H[fmt] * np.abs(w))
        assert (np.abs(got - w) <= tol).all()
        return
    codes, scales = got
    near = [R.encode(w * f, g)[1] for f in (1 - 2 ** -20, 1 + 2 ** -20)]
    assert ((scales == near[0]) | (scales == near[1])).all()
    s = np.repeat(R.E4M3[scales], 16, -1) * g
    best = np.abs(R.E2M1[R.e2m1_nearest(np.abs(w) / np.where(s > 0, s, 1))] * s - np.abs(w))
    assert (np.abs(R.decode(codes, scales, g) - w) <= best + 2 * tol + 4 * U * 6 * s).all()


MANY = [
    # fmt, src, Hkv, dh, rows, page, layout, rot (a warp takes several rows from 7296 on, 8192 elements of them)
    ("kv4", "bf16", 8, 32, 20001, 16, "half", 32), ("bf16", "bf16", 8, 32, 20001, 0, "half", 32),
    ("kv4", "f32", 8, 32, 7297, 0, None, 0), ("f32", "bf16", 8, 32, 7301, 5, "interleaved", 16),
    ("kv4", "bf16", 19, 64, 7301, 48, "interleaved", 48), ("bf16", "f32", 19, 64, 7301, 0, "half", 32),
    ("kv4", "bf16", 21, 128, 7303, 16, "half", 64), ("f32", "f32", 21, 128, 7296, 0, "interleaved", 48),
    # part of a head turned, whole units: pairs, then what passes through; a row over several warps
    ("kv4", "bf16", 2, 128, 37, 0, "half", 32), ("kv4", "f32", 40, 128, 37, 16, "half", 96),
    ("bf16", "bf16", 3, 128, 41, 5, "half", 64), ("f32", "f32", 2, 64, 37, 0, "half", 32),
    ("kv4", "bf16", 2, 128, 37, 16, "interleaved", 16), ("kv4", "bf16", 1, 64, 300, 0, "interleaved", 48),
    ("bf16", "f32", 5, 64, 37, 16, "interleaved", 16), ("f32", "bf16", 2, 128, 41, 0, "interleaved", 112),
    ("bf16", "bf16", 2, 128, 37, 0, "interleaved", 48),
]


@pytest.mark.parametrize("fmt,src,Hkv,dh,rows,page,layout,rot", MANY)
@pytest.mark.parametrize("given", [False, True])
def test_append_and_read_many_rows(fmt, src, Hkv, dh, rows, page, layout, rot, given):
    """Packed sequences, empty ones among them, and places that belong to none; positions from the slots or given."""
    lead, tail, B = 5, 9, 7
    n = rows - lead - tail
    new = [0, n // 9, 0, 3, n // 2, 0]
    new.append(n - sum(new))
    before = [3, 0, 7, 20, 1, 0, 33]
    unit = page or 16
    capacity = (max(new) + 40 + unit - 1) // unit * unit
    case = Case(fmt, B, Hkv, dh, capacity, page)
    rng = np.random.default_rng(rows)
    x = rnd(rows, (rows, 2 * Hkv, dh), src).cuda()
    k, v = x[:, :Hkv], x[:, Hkv:]
    start = np.concatenate(([0], np.cumsum(new))) + lead
    seq = np.repeat(np.arange(B), new)
    slot = np.concatenate([before[b] + np.arange(new[b]) for b in range(B)])
    rope = Bnd.Rope(rot, capacity, layout=layout) if layout else None
    pos = rng.integers(0, capacity, rows) if given else None
    out, old = i32([-1] * B), (case.host(0), case.host(1))
    Bnd.kv_append(case.cache, case.kv(i32(before), out), k, v, start=i32(start), rope=rope,
                  pos=None if pos is None else i32(pos), k_scale=case.gk, v_scale=case.gv)
    lens = [a + b for a, b in zip(before, new)]
    assert out.tolist() == lens and case.cache.status() == 0
    raw = case.host(0), case.host(1)
    for which in (0, 1):
        np.testing.assert_array_equal(rest(case, old[which], seq, slot).view(np.uint8),
                                      rest(case, raw[which], seq, slot).view(np.uint8))
    src_k, src_v = f64(k[lead:lead + n]), f64(v[lead:lead + n])
    for which, rows_in, g in ((1, src_v, case.gv),) + (() if layout else ((0, src_k, case.gk),)):
        got = held(case, raw[which], seq, slot)
        if fmt == "kv4":
            for a, b in zip(got, R.encode(rows_in, g)):
                np.testing.assert_array_equal(a, b)
        else:
            np.testing.assert_array_equal(got.astype(np.float64), want_rows(case, rows_in, g, fmt))
    if layout:
        check_turned(fmt, held(case, raw[0], seq, slot), src_k, slot if pos is None else pos[lead:lead + n], rot, layout,
                     case.gk)
    # and back: the same slots, from a place of each sequence on
    first = [int(b) for b in before]
    wide = [torch.full((rows, Hkv + 1, dh), 3.0, dtype=DT[src], device="cuda") for _ in "kv"]
    rk, rv = wide[0][:, 1:], wide[1][:, :Hkv]
    Bnd.kv_read(case.cache, case.kv(out), rk, rv, start=i32(start), first=i32(first), k_scale=case.gk, v_scale=case.gv)
    assert case.cache.status() == 0
    for which, y, g in ((0, rk, case.gk), (1, rv, case.gv)):
        got = held(case, raw[which], seq, slot)
        want = R.decode(*got, g) if fmt == "kv4" else got.astype(np.float64)
        np.testing.assert_array_equal(f64(y[lead:lead + n]), f64(torch.from_numpy(want).float().to(DT[src])))
        assert (y[:lead] == 3).all() and (y[lead + n:] == 3).all()
    assert (wide[0][:, 0] == 3).all() and (wide[1][:, Hkv] == 3).all()


# ------------------------------------------------------------------ calls at the same time
@pytest.mark.parametrize("dtype,Hq,Hkv,dh,n1,page", [
    ("bf16", 8, 8, 128, 20, 0), ("bf16", 8, 8, 128, 43, 256), ("bf16", 8, 8, 128, 100, 0), ("bf16", 8, 8, 64, 65, 0),
    ("bf16", 32, 8, 128, 43, 0), ("bf16", 8, 8, 64, 150, 48), ("bf16", 32, 8, 128, 1, 0), ("f32", 8, 8, 128, 9, 0),
])
def test_series_on_two_streams_repeat_bit_for_bit(dtype, Hq, Hkv, dh, n1, page):
    """Series of calls on two streams, each with its own workspace and result: blocks of one kernel start where
    those of another end, and staged codes wait for their readers.  The same bits every time."""
    B, capacity = 33, 9216
    rng = np.random.default_rng(1)
    lens = [int(rng.choice([0, 1, 9000, rng.integers(0, 9000), rng.integers(0, 70) * 128])) for _ in range(B)]
    case = Case("kv4", B, Hkv, dh, capacity, page, Hq=Hq, max_nodes=n1)
    for pool in case.pool:                             # any codes, scales from 0.5 to 1.875
        scales = pool.view(-1, 9 * dh)[:, 8 * dh:]
        scales.copy_(torch.randint(0x30, 0x40, scales.shape, dtype=torch.uint8, device="cuda"))
    q = rnd(1, (B, n1, Hq, dh), dtype).cuda()
    kv = case.kv(i32(lens))
    calls = 12 if q.numel() * q.element_size() < 1 << 25 else 6
    ws = [torch.empty(case.cache.workspace_size, dtype=torch.uint8, device="cuda") for _ in range(calls)]
    o = [torch.empty_like(q) for _ in range(calls)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    want = None
    for _ in range(300 if dtype == "bf16" else 60):
        for i in range(calls):
            Bnd.kv4_attention(case.cache, kv, q, o[i], ws[i], k_scale=case.gk, v_scale=case.gv, stream=streams[i % 2])
        torch.cuda.synchronize()
        if want is None:
            want = o[0].clone()
            assert torch.isfinite(want.float()).all()
        assert all(torch.equal(x, want) for x in o)
    assert case.cache.status() == 0
