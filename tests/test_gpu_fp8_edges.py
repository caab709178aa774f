"""8-bit products where a factor leaves the range of normal floats, against fp8_ref.py in 64 bits, and waits that run out.

The bounds are those that test_gpu_fp8.py derives, with what each test adds to them beside it."""
import time

import numpy as np
import pytest
import torch

import fp8_ref as F
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MOST = float(np.finfo(np.float32).max)
TINY = 2.0 ** -149                                # a step of floats below 2^-126


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def f64(t):
    return t.detach().double().cpu().numpy()


def codes_of(r, rows, k):
    return F.round8(r.standard_normal((rows, k)), 128)[0]


def dev(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda()


def scales(r, shape, of):
    return np.float32(r.choice(np.float32(of), shape))


def run(rows, n, k, x, xs, w, ws, up=None, us=None):
    h = Bnd.Fp8(n=n, k=k, max_rows=rows, gated=up is not None)
    y = torch.zeros(rows, n, device="cuda")
    g = lambda s: None if s is None else torch.from_numpy(s).cuda()  # noqa: E731
    Bnd.fp8_linear(h, x, dev(w), g(ws), y, torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda"), x_scales=g(xs),
                   up=None if up is None else dev(up), up_scales=g(us))
    assert h.status() == 0
    return f64(y)


def product(x, w, ws, kb):
    """x (64 bits) times weights: the value, and the bound of the library's sums.  Of its 2u (128 + kb + 4) the last 4 are for
    the scales, one rounding each; where a result is below 2^-126 each group's addition is off by up to half a TINY."""
    wv = F.values(w, ws.astype(float), 128)
    return x @ wv.T, 2 * U * (128 + kb + 4) * (np.abs(x) @ np.abs(wv).T) + kb * TINY


ROW_SCALES = [2.0 ** -126, 2.0 ** -122, 1.3 * 2.0 ** -118, 1.0, 0.0, -2.0 ** -120, 2.0 ** 20]
WEIGHT_SCALES = [2.0 ** -24, 1.3 * 2.0 ** -24, 7.3e-4, 1.3e-6, -1e-3, 3 * 2.0 ** -149]


@pytest.mark.parametrize("rows,n,k,gated", [(5, 700, 272, 0), (200, 770, 400, 0), (37, 641, 5120, 0), (33, 700, 400, 1), (150, 670, 144, 1)])
def test_scales_whose_product_is_no_normal_float(rows, n, k, gated):
    """Row scales as rounding tiny rows gives them times small weight scales: their product has lost bits, or is 0, where the
    result is a normal float.  A row and a block of weights have one scale each; rows of other scales lie between them, so that
    a warp has both kinds."""
    r = np.random.default_rng(rows + n)
    kb, nb = -(-k // 128), -(-n // 128)
    x, w = codes_of(r, rows, k), codes_of(r, n, k)
    xs = np.float32(np.repeat(np.float32(ROW_SCALES)[np.arange(rows) % 7, None], kb, 1))
    ws = np.float32(np.repeat(np.float32(WEIGHT_SCALES)[np.arange(nb) % 6, None], kb, 1))
    xv = F.values(x, xs.astype(float), 1)
    a, da = product(xv, w, ws, kb)
    assert ((np.abs(a) < 1e-30) & (np.abs(a) > 1e-37)).mean() > 0.1
    if not gated:
        want, tol = a, da
        got = run(rows, n, k, dev(x), xs, w, ws)
    else:                                         # large factors beside tiny ones
        up, us = codes_of(r, n, k), scales(r, (nb, kb), [1e24, -3e23])
        b, db = product(xv, up, us, kb)
        s = F.silu(a)
        want, tol = s * b, 1.1 * da * np.abs(b) + (np.abs(s) + 1.1 * da) * db + 8 * U * np.abs(s * b) + TINY * np.abs(b)
        got = run(rows, n, k, dev(x), xs, w, ws, up, us)
    tol = tol + U * np.abs(want) + TINY
    far = np.abs(want) - tol > MOST               # a gated result past the range of floats is an infinity
    assert (got[far] == np.copysign(np.inf, want[far])).all()
    near = ~far & (np.abs(want) + tol <= MOST)
    assert (near | far).mean() > 0.95             # (where a sum is large its bound may pass the range, whatever the result is)
    err = np.abs(got - want)[near]
    assert (err <= tol[near]).all(), (err / tol[near]).max()


@pytest.mark.parametrize("size", [1e-37, 3e-36])
def test_tiny_rows_times_small_weights(size):
    """The same through the rounding of the call itself."""
    rows, n, k = 9, 260, 656
    r = np.random.default_rng(4)
    x = torch.from_numpy(r.standard_normal((rows, k)) * size).float()
    c, s = F.round8(f64(x), 1)
    assert s.max() <= 2.0 ** -120
    w, ws = codes_of(r, n, k), scales(r, (3, 6), [7.3e-4, 1.3e-6])
    want, tol = product(F.values(c, s, 1), w, ws, 6)
    err = np.abs(run(rows, n, k, x.cuda(), None, w, ws) - want)
    tol = tol + U * np.abs(want) + TINY
    assert (err <= tol).all(), (err / tol).max()


def test_a_gate_far_below_zero():
    """silu(a) b with a down to -300 and b up to 3e38.  Rows hold one 1 for each matrix, so that sums are exact: a = -scale, b = scale
    * up's scale * code, one rounding.  silu(a) b: four exponentials (a unit in the last place each, 2u), five products, or one, a sum
    and a quotient (two units): 16u of it with b's and the last rounding."""
    a = -np.float32([0.5, 20, 63, 63.9, 64, 64.1, 70, 80, 87, 87.3, 87.4, 88, 88.7, 88.8, 95, 103, 110, 120, 150, 170, 180, 200, 300])
    rows, n, k = len(a), 24, 16
    x, w, up = (np.zeros((m, k), np.uint8) for m in (rows, n, n))
    x[:, :2], w[:, 0] = 0x38, 0xb8                # 1, -1
    up[:, 1] = F.encode(np.r_[1.0:13.0, -1.0, -3.5, 448, 0.5, 0, 0, 2.0 ** -9, 7, 9, 16, 20, 24])
    for us in (1e-30, 1.0, 1e30, 2e33, 3e38 / 448 / 300):
        b = np.float32(-a * np.float32(us)).astype(float)[:, None] * F.decode(up[:, 1])[None]
        want = F.silu(a.astype(float))[:, None] * b
        got = run(rows, n, k, dev(x), -a[:, None], w, np.ones((1, 1), np.float32), up, np.full((1, 1), us, np.float32))
        err, tol = np.abs(got - want), 16 * U * np.abs(want) + TINY
        assert (err <= tol).all(), (err / tol).max()


# rows, n, k, gated: shares of a few columns, whole tiles, tiles of 256 columns in shares, a pair
@pytest.mark.parametrize("rows,n,k,gated", [(1, 4096, 4096, 0), (5, 130, 16, 0), (300, 700, 8192, 0), (700, 5000, 640, 0), (40, 3000, 2048, 1)])
@pytest.mark.parametrize("x", ["codes", "bf16"])
def test_expired_wait_is_reported_and_nothing_else_is_lost(rows, n, k, gated, x):
    """A bounded wait is made to run out: the call returns with MEDUSA_FLAG_TIMEOUT, whatever the workspace held, and the next one
    on the same workspace is as before."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    codes = lambda m: torch.randint(0, 119, (m, k), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    h = Bnd.Fp8(n=n, k=k, max_rows=rows, gated=bool(gated))
    kb, nb = h.kb, h.nb
    y, ws = torch.zeros(rows, n, device="cuda"), torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda")
    args = dict(x=codes(rows), x_scales=torch.rand(rows, kb, device="cuda", generator=g) * 1e-3) if x == "codes" else \
        dict(x=torch.randn(rows, k, device="cuda", generator=g).bfloat16())
    args.update(w=codes(n), w_scales=torch.rand(nb, kb, device="cuda", generator=g) * 1e-6)
    if gated:
        args.update(up=codes(n), up_scales=torch.rand(nb, kb, device="cuda", generator=g) * 1e-6)

    def call():
        ws.fill_(0x7f)
        y.fill_(7.0)
        t0 = time.perf_counter()
        Bnd.fp8_linear(h, y=y, ws=ws, **args)
        torch.cuda.synchronize()
        return y.clone(), time.perf_counter() - t0

    clean, _ = call()
    assert h.status() == 0 and torch.isfinite(clean).all()
    h.expire_wait_once(2_000_000)
    assert call()[1] < 30.0
    assert h.status() == Bnd.FLAG_TIMEOUT
    again, _ = call()
    assert h.status() == 0 and torch.equal(again, clean)


def test_expire_wait_argument_checks():
    h = Bnd.Fp8(n=16, k=16, max_rows=1)
    for ns in (0, 10**10 + 1):
        with pytest.raises(Bnd.MedusaError) as e:
            h.expire_wait_once(ns)
        assert e.value.code == Bnd.MEDUSA_ERR_INVALID


@pytest.mark.parametrize("rows", [5, 200])
def test_rows_and_residuals_that_are_one_row(rows):
    """Row strides of 0: one row of inputs for all, one row of residuals (a bias) for all."""
    n, k = 300, 656
    r = np.random.default_rng(rows)
    w, ws = codes_of(r, n, k), scales(r, (3, 6), [0.5, 3.0])
    x = torch.from_numpy(r.standard_normal((rows, k))).float().cuda()
    bias = torch.from_numpy(r.standard_normal(n)).float().cuda()
    h = Bnd.Fp8(n=n, k=k, max_rows=rows)
    work, s = torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda"), torch.from_numpy(ws).cuda()
    for one in (False, True):
        xin = x[:1].expand(rows, k) if one else x
        y = torch.zeros(rows, n, device="cuda")
        Bnd.fp8_linear(h, xin, dev(w), s, y, work, add=bias.expand(rows, n))
        want, tol = product(F.values(*F.round8(f64(xin), 1), 1), w, ws, 6)
        want = want + f64(bias)
        tol = tol + 2 * U * (np.abs(want) + tol)
        assert (np.abs(f64(y) - want) <= tol).all()
        if one:
            codes = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
            sc = torch.zeros(rows, 6, device="cuda")
            Bnd.fp8_round(h, xin, codes, sc)
            assert (codes == codes[0]).all() and (sc == sc[0]).all()
    assert h.status() == 0
