"""8-bit products of many rows whose last tiles are shared by several blocks: partial sums of 256 columns, joined in the first and
the later rows of tiles, beside and without whole tiles, and more rows of tiles than are dealt out at a time.  Every case says which
of these it is, and asks the library whether it still is.  The 64-bit value is computed on the GPU; the bound is the one that
test_gpu_fp8.py derives (its two roundings a group cover the additions of partial sums too: these are no more than groups)."""
import pytest
import torch

from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
H = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def eight(g, rows, k, block, lo, hi):
    """Codes of numbers of size 1, any scales in lo..hi; and the values they stand for."""
    c = torch.randn(rows, k, device="cuda", generator=g).to(torch.float8_e4m3fn)
    s = lo + (hi - lo) * torch.rand(-(-rows // block), -(-k // 128), device="cuda", generator=g)
    return c, s, c.double() * s.double().repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :k]


# rows, n, k, dtype of the result, residual, gated, columns, whole tiles (0: none), shared tiles (0: none)
CASES = [
    (300, 700, 8192, "f32", 1, 0, 256, 0, 9),                 # 3 x 3 tiles, all shared, the last ones ragged both ways
    (300, 700, 8192, "bf16", 0, 0, 256, 0, 9),
    (130, 257, 16384, "f32", 1, 0, 256, 0, 4),                # last row and column of tiles nearly empty
    (200, 391, 8192, "bf16", 0, 1, 128, 0, 8),                # pairs
    (300, 13700, 8192, "bf16", 1, 0, 256, 152, 10),           # whole tiles, then shares
    (270, 6800, 8192, "f32", 0, 1, 128, 152, 10),
    (2500, 2300, 8192, "f32", 1, 0, 256, 152, 28),            # 20 rows of tiles: 16, then 4
    (2300, 1400, 640, "bf16", 1, 0, 256, 108, 0),             # 18 rows of tiles, all whole
    (4200, 700, 400, "f32", 0, 1, 128, 198, 0),               # 33 rows of tiles: 16, 16 and 1
    (1, 700, 8192, "f32", 1, 0, 128, 0, 6),                   # one row
    (128, 24000, 4096, "bf16", 0, 0, None, None, None),
]


@pytest.mark.parametrize("rows,n,k,y,add,gated,columns,whole,shared", CASES)
def test_tiles_of_one_and_of_several_blocks(rows, n, k, y, add, gated, columns, whole, shared):
    h = Bnd.Fp8(n=n, k=k, max_rows=rows + 5, gated=bool(gated))
    if columns and torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert h.tiles(rows, bool(gated)) == (columns, whole, shared)
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x, xs, xv = eight(g, rows, k, 1, 0.1, 1)
    terms = 2 * U * (128 + h.kb + 4)
    pair = [eight(g, n, k, 128, 0.01, 0.03) for _ in range(1 + gated)]
    sums = [(xv @ wv.T, terms * (xv.abs() @ wv.abs().T)) for _, _, wv in pair]
    want, tol = sums[0]
    if gated:
        (a, da), (b, db) = sums
        s = a * torch.sigmoid(a)
        want, tol = s * b, 1.1 * da * b.abs() + (s.abs() + 1.1 * da) * db + 8 * U * (s * b).abs()
    wide = torch.full((rows + 1, n + 3), 7.0, dtype=DT[y], device="cuda")
    out = wide[:rows, 3:]
    residual = None
    if add:
        residual = out                                       # in place, in rows that are not aligned
        out.copy_(torch.randn(rows, n, device="cuda", generator=g))
        want = want + out.double()
        tol = tol + U * (want.abs() + tol)
    tol = tol + H[y] * (want.abs() + tol) + 1e-37
    ws = torch.full((h.workspace_size,), 255, dtype=torch.uint8, device="cuda")
    Bnd.fp8_linear(h, x, pair[0][0], pair[0][1], out, ws, x_scales=xs, add=residual, up=pair[1][0] if gated else None,
                   up_scales=pair[1][1] if gated else None)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert (wide[:, :3] == 7).all() and (wide[rows] == 7).all() and h.status() == 0


@pytest.mark.parametrize("rows", [1, 64, 128])
def test_columns_of_a_tile_go_by_how_many_blocks_have_one(rows):
    """One row of tiles: 128 columns while tiles of 256 are for less than half of the blocks."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for n, columns in ((16, 128), (256 * (-(-sms // 2) - 1), 128), (256 * (-(-sms // 2) - 1) + 1, 256), (64000, 256)):
        assert Bnd.Fp8(n=n, k=256, max_rows=200).tiles(rows)[0] == columns, n
        assert Bnd.Fp8(n=n, k=256, max_rows=200).tiles(129)[0] == 256


@pytest.mark.parametrize("rows,n,k,y", [(1, 20480, 4096, "f32"), (128, 24000, 2048, "bf16"), (77, 19457, 400, "f32"), (9, 39000, 656, "bf16")])
def test_wide_weights_for_one_row_of_tiles(rows, n, k, y):
    test_tiles_of_one_and_of_several_blocks(rows, n, k, y, 1, 0, None, None, None)
