"""Rounding to 8 bits and products of 8-bit rows and weights against fp8_ref.py, through the public binding.

Tolerances.  u = 2^-24.  Codes, scales and values read back are exact (reading rounds once to the dtype).  A
product's sum over a group of 128 is made of exact products added in float, each addition off by at most
2u of the partial sum (tensor cores may cut instead of rounding); scales multiply (u), and the kb groups are
added (2u each): |error| <= 2u (128 + kb + 4) sum |x||w| =: d.  silu(a) b of sums a, b with errors da, db: |silu'| <=
1.1, so 1.1 da |b| + (|silu(a)| + 1.1 da) db, and 8u of the result for the exponential and the quotient.  Adding
rounds once more (u).  The result is rounded once to the dtype (bf16 2^-8, float u)."""
import numpy as np
import pytest
import torch

import fp8_ref as F
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def rows_of(seed, rows, k, dtype, wide=0):
    """Rows whose groups differ much in size, some zero; a part of wider rows where asked for."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, k)) * np.exp(r.uniform(-20, 20, (rows, 1)))
    x *= 1 + 30 * (r.random((1, k)) < 0.02)
    if rows > 2:
        x[1] = 0
    buf = torch.zeros(rows, k + wide, dtype=DT[dtype])
    buf[:, wide:] = torch.from_numpy(x).to(DT[dtype])
    return buf.cuda()[:, wide:]


def weights(seed, n, k):
    """Weights as a checkpoint holds them: any scales."""
    r = np.random.default_rng(seed)
    codes, scales = F.round8(r.standard_normal((n, k)), 128)
    scales = r.uniform(0.5, 3, scales.shape).astype(np.float32)
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda(), torch.from_numpy(scales).cuda()


ROUNDS = [(1, 16, 1), (3, 128, 1), (37, 1040, 1), (129, 272, 1), (5, 5120, 1), (2000, 144, 1), (1, 16, 128),
          (128, 128, 128), (130, 272, 128), (997, 1040, 128)]


@pytest.mark.parametrize("rows,k,block", ROUNDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [0, 64, 3])
def test_round_and_read(rows, k, block, dtype, wide):
    h = Bnd.Fp8(n=rows, k=k, max_rows=rows)
    x = rows_of(rows + k, rows, k, dtype, wide)
    codes = torch.zeros(rows, k, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(-(-rows // block), -(-k // 128), device="cuda")
    Bnd.fp8_round(h, x, codes, scales, block=block)
    c, s = F.round8(f64(x), block)
    np.testing.assert_array_equal(f64(scales), s)
    np.testing.assert_array_equal(bits(codes), c)
    out = torch.full((rows, k + wide), 7.0, dtype=DT[dtype], device="cuda")
    Bnd.fp8_read(h, codes, scales, out[:, wide:], block=block)
    want = torch.from_numpy(F.values(c, s, block)).float().to(DT[dtype])      # (codes times powers of two: exact in float)
    assert torch.equal(out[:, wide:].cpu(), want) and (out[:, :wide] == 7).all()
    assert h.status() == 0


def test_round_at_borders():
    """448 * 2^e exactly and one step above, subnormal and largest floats, ties, and a -0."""
    x = torch.zeros(8, 128)
    x[0, 3] = 448.0
    x[1, 3] = float(np.nextafter(np.float32(448), np.float32(1000)))
    x[2, 0] = 1e-45
    x[3, 0], x[3, 1] = 3.4028234e38, -1e38
    x[4] = torch.arange(128) * 0.5
    x[5, 0], x[5, 1] = 2.0 ** -126 * 448, 2.0 ** -149
    x[6, 0], x[6, 1] = -0.0, 2.0 ** -140
    x = x.cuda()
    h = Bnd.Fp8(n=8, k=128, max_rows=8)
    codes, scales = torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, device="cuda")
    Bnd.fp8_round(h, x, codes, scales)
    c, s = F.round8(f64(x), 1)
    np.testing.assert_array_equal(f64(scales), s)
    np.testing.assert_array_equal(F.decode(codes.cpu().numpy()), F.decode(c))
    assert h.status() == 0


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_become_nan_in_their_group(block, dtype):
    x = rows_of(3, 130, 272, dtype)
    x[0, 5], x[129, 271] = float("inf"), float("nan")
    h = Bnd.Fp8(n=130, k=272, max_rows=130)
    codes = torch.zeros(130, 272, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(-(-130 // block), 3, device="cuda")
    Bnd.fp8_round(h, x, codes, scales, block=block)
    c, s = F.round8(f64(x), block)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    np.testing.assert_array_equal(f64(scales), s)
    assert h.status() == Bnd.FLAG_NONFINITE and h.status() == 0
    y = torch.zeros(130, 272, device="cuda")
    Bnd.fp8_read(h, codes, scales, y, block=block)
    np.testing.assert_array_equal(np.isnan(f64(y)), np.isnan(F.decode(c)))


# rows, n, k, x, y, add, gated
LINEAR = [
    (1, 16, 16, "bf16", "bf16", 0, 0), (1, 4096, 4096, "bf16", "bf16", 0, 0), (1, 129, 144, "f32", "f32", 1, 0),
    (2, 300, 2048, "codes", "bf16", 1, 0), (7, 1, 128, "codes", "f32", 0, 0), (8, 640, 1040, "bf16", "f32", 0, 1),
    (16, 997, 5120, "f32", "bf16", 0, 1), (31, 256, 272, "codes", "f32", 1, 0), (37, 997, 1040, "f32", "f32", 1, 0),
    (64, 128, 8192, "codes", "bf16", 0, 0), (65, 272, 128, "bf16", "bf16", 0, 1), (127, 130, 400, "codes", "f32", 0, 0),
    (128, 1000, 256, "codes", "bf16", 1, 0), (129, 257, 384, "f32", "f32", 0, 1), (300, 700, 1296, "codes", "bf16", 0, 1),
    (520, 2050, 512, "codes", "bf16", 1, 0), (1000, 33, 16, "bf16", "f32", 0, 0), (33, 24000, 64, "codes", "f32", 0, 0),
    (700, 5000, 640, "codes", "f32", 0, 0), (1300, 4100, 144, "codes", "bf16", 0, 1), (3, 20000, 272, "bf16", "bf16", 0, 1),
]


def product(seed, rows, n, k, x, y, add, gated, pad=0, h=None):
    """Inputs, the result's 64-bit value and bound."""
    X = rows_of(seed, rows, k, "f32" if x == "codes" else x, pad if x != "codes" else 0)
    X = X / X.abs().amax(1, keepdim=True).clamp(min=1e-30) if x != "codes" else X
    if x != "codes":
        X = X.to(DT[x])
    c, s = F.round8(f64(X), 1)
    if x == "codes":                              # scales that are no powers of two as well
        s = (s * np.random.default_rng(seed).uniform(1, 2, s.shape)).astype(np.float32).astype(float)
        s /= max(np.abs(s).max(), 1e-30)
        s = s.astype(np.float32).astype(float)
    w, ws = weights(seed + 1, n, k)
    up, us = weights(seed + 2, n, k) if gated else (None, None)
    A = torch.from_numpy(np.random.default_rng(seed + 3).standard_normal((rows, n))).to(DT[y]).cuda() if add else None
    xv, kb = F.values(c, s, 1), -(-k // 128)

    def sums(w, ws):
        wv = F.values(bits(w), f64(ws), 128)
        return xv @ wv.T, 2 * U * (128 + kb + 4) * (np.abs(xv) @ np.abs(wv).T)
    a, da = sums(w, ws)
    want, tol = a, da
    if gated:
        b, db = sums(up, us)
        want = F.silu(a) * b
        tol = 1.1 * da * np.abs(b) + (np.abs(F.silu(a)) + 1.1 * da) * db + 8 * U * np.abs(want)
    if add:
        want = want + f64(A)
        tol = tol + U * (np.abs(want) + tol)
    tol = tol + H[y] * (np.abs(want) + tol) + 1e-37
    if x == "codes":
        X = torch.from_numpy(c).view(torch.float8_e4m3fn).cuda()
        xs = torch.from_numpy(s.astype(np.float32)).cuda()
    else:
        xs = None
    return dict(x=X, x_scales=xs, w=w, w_scales=ws, up=up, up_scales=us, add=A), want, tol


def check(got, want, tol):
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("rows,n,k,x,y,add,gated", LINEAR)
def test_linear(rows, n, k, x, y, add, gated):
    h = Bnd.Fp8(n=n, k=k, max_rows=rows, gated=bool(gated))
    args, want, tol = product(rows + n + k, rows, n, k, x, y, add, gated)
    ws = torch.full((h.workspace_size,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((rows + 1, n), 7.0, dtype=DT[y], device="cuda")
    Bnd.fp8_linear(h, y=out[:rows], ws=ws, **args)
    check(out[:rows], want, tol)
    assert (out[rows] == 7).all() and h.status() == 0
    first = out.clone()
    Bnd.fp8_linear(h, y=out[:rows], ws=ws, **args)            # the same bits again
    assert torch.equal(out.view(torch.uint8), first.view(torch.uint8))


@pytest.mark.parametrize("rows,n,k", [(5, 130, 272), (200, 391, 400)])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_linear_strides_and_in_place_residual(rows, n, k, y):
    h = Bnd.Fp8(n=n, k=k, max_rows=rows + 3)
    for x in ("bf16", "codes"):
        args, want, tol = product(9, rows, n, k, x, y, 1, 0, pad=3)
        wide = torch.full((rows, n + 5), 7.0, dtype=DT[y], device="cuda")
        out = wide[:, 3:3 + n]
        out.copy_(args["add"])
        args["add"] = out
        if x == "codes":
            c = torch.zeros(rows, k + 16, dtype=torch.float8_e4m3fn, device="cuda")
            c.view(torch.uint8)[:, :k] = args["x"].view(torch.uint8)
            args["x"] = c[:, :k]
        Bnd.fp8_linear(h, y=out, ws=torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda"), **args)
        check(out, want, tol)
        assert (wide[:, :3] == 7).all() and (wide[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("rows", [3, 130])
def test_nan_stays_in_its_row_or_column(rows):
    n, k = 260, 400
    h = Bnd.Fp8(n=n, k=k, max_rows=rows)
    args, want, tol = product(5, rows, n, k, "codes", "f32", 0, 0)
    args["x"].view(torch.uint8)[2, 399] = 127
    args["w"].view(torch.uint8)[131, 0] = 255
    y = torch.zeros(rows, n, device="cuda")
    Bnd.fp8_linear(h, y=y, ws=torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda"), **args)
    g = f64(y)
    assert np.isnan(g[2]).all() and np.isnan(g[:, 131]).all()
    keep = np.ones((rows, n), bool)
    keep[2], keep[:, 131] = False, False
    assert (np.abs(g - want)[keep] <= tol[keep]).all()


def test_calls_are_captured_and_replayed_with_new_inputs():
    rows, n, k = 19, 384, 656
    h = Bnd.Fp8(n=n, k=k, max_rows=rows, gated=True)
    args, _, _ = product(1, rows, n, k, "bf16", "bf16", 0, 1)
    y, ws = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"), torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda")
    other = torch.empty_like(ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], [y, torch.zeros_like(y)]
    with torch.cuda.stream(st):
        for out, w in zip(outs, (ws, other)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                Bnd.fp8_linear(h, y=out, ws=w, **args)
            graphs.append(g)
    for seed in (1, 2):
        new, want, tol = product(seed, rows, n, k, "bf16", "bf16", 0, 1)
        for name, t in new.items():
            if t is not None:
                args[name].copy_(t)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(st):
            graphs[1].replay()
        torch.cuda.synchronize()
        for out in outs:
            check(out, want, tol)


def test_library_refusals():
    h = Bnd.Fp8(n=130, k=144, max_rows=4)
    args, _, _ = product(1, 5, 130, 144, "codes", "f32", 0, 0)
    ws = torch.empty(h.workspace_size + 16, dtype=torch.uint8, device="cuda")
    y = torch.zeros(5, 130, device="cuda")

    def call(rows=4, ws=ws[:-16], h=h, **kw):
        a = dict(args, **kw)
        a["x"], a["x_scales"] = a["x"][:rows], a["x_scales"][:rows]
        out = a.pop("y", y[:rows])
        Bnd.fp8_linear(h, y=out, ws=ws, **a)

    call()
    call(rows=0)
    off = torch.zeros(130 * 144 + 8, dtype=torch.uint8, device="cuda")[8:].view(130, 144)
    odd = torch.zeros(5, 152, dtype=torch.uint8, device="cuda")[:, :144]
    for kw, code in ((dict(rows=5), -1), (dict(ws=ws[:-17]), -6), (dict(ws=ws[16:]), -6), (dict(up=args["w"], up_scales=args["w_scales"]), -1),
                     (dict(w=off), -1), (dict(x=odd), -1), (dict(y=torch.zeros(130, device="cuda").expand(4, 130)), -1)):
        with pytest.raises(Bnd.MedusaError) as e:
            call(**kw)
        assert e.value.code == code, kw
    x = torch.zeros(4, 144, device="cuda")
    codes, scales = torch.zeros(4, 144, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda")
    for call in (lambda: Bnd.fp8_round(h, x, codes, torch.zeros(1, 2, device="cuda"), block=128),   # not n rows
                 lambda: Bnd.fp8_round(h, x, codes, torch.zeros(2, 2, device="cuda"), block=2),
                 lambda: Bnd.fp8_read(h, codes, scales, torch.zeros(144, device="cuda").expand(4, 144)),
                 lambda: Bnd.fp8_round(h, torch.zeros(5, 144, device="cuda"), torch.zeros(5, 144, dtype=torch.uint8, device="cuda"),
                                       torch.zeros(5, 2, device="cuda"))):
        with pytest.raises(Bnd.MedusaError) as e:
            call()
        assert e.value.code == -1
    assert h.status() == 0
