"""8-bit products and attention over a shared prefix give the same bits at every call, also beside work on another stream that takes
SMs from them: sums are added up in an order that does not depend on which block comes first."""
import pytest
import torch

import test_gpu_prefix as T
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu

CALLS = 40


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def same_bits_beside_others(call, out, status):
    other, junk = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda").bfloat16()
    call()
    first = out.clone()
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(CALLS):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                junk @ junk
        out.fill_(7.0)
        call()
        differ += (out.view(torch.uint8) != first.view(torch.uint8)).any()
    torch.cuda.synchronize()
    assert differ.item() == 0 and not any(status())


# shares of few columns; whole tiles; shares of 256 columns; whole tiles and shares; pairs of either kind
@pytest.mark.parametrize("rows,n,k,gated", [(1, 4096, 4096, 0), (37, 997, 1040, 0), (64, 24000, 1024, 0), (700, 5000, 640, 0), (300, 700, 8192, 0),
                                            (300, 13700, 8192, 0), (8, 4096, 5120, 1), (200, 391, 8192, 1)])
@pytest.mark.parametrize("x", ["bf16", "codes"])
def test_products(rows, n, k, gated, x):
    g = torch.Generator(device="cuda").manual_seed(n)
    eight = lambda m: torch.randn(m, k, device="cuda", generator=g).to(torch.float8_e4m3fn)  # noqa: E731
    h = Bnd.Fp8(n=n, k=k, max_rows=rows, gated=bool(gated))
    scales = lambda m: torch.rand(m, h.kb, device="cuda", generator=g)  # noqa: E731
    y, ws = torch.empty(rows, n, device="cuda"), torch.empty(h.workspace_size, dtype=torch.uint8, device="cuda")
    kw = dict(x=eight(rows), x_scales=scales(rows)) if x == "codes" else dict(x=torch.randn(rows, k, device="cuda", generator=g).bfloat16())
    kw.update(w=eight(n), w_scales=scales(h.nb))
    if gated:
        kw.update(up=eight(n), up_scales=scales(h.nb))
    same_bits_beside_others(lambda: Bnd.fp8_linear(h, y=y, ws=ws, **kw), y, lambda: [h.status()])


@pytest.mark.parametrize("case", [
    # B, hq, hk, dh, n1, P, lens, page, ppage, kind: one tile of rows, pages or not; two tiles; the CUDA cores
    (9, 8, 2, 128, 1, 3000, [700, 0, 129, 1, 2, 3, 64, 500, 900], 16, 16, None),
    (4, 8, 8, 64, 65, 1000, [700, 0, 129, 40], 0, 0, "tree"),
    (6, 8, 2, 128, 43, 2000, [512, 0, 129, 64, 65, 300], 16, 0, "tree"),
    (2, 2, 1, 128, 200, 100, [0, 33], 32, 16, "causal"),
    (3, 8, 2, 32, 31, 777, [0, 57, 100], 16, 0, "tree"),
], ids=lambda c: "-".join(str(x) for x in c[:6]))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention(case, dtype):
    *dims, kind = case
    c = T.Case(1, *dims, dtype, kind)
    o = torch.empty_like(c.q)
    same_bits_beside_others(lambda: c.run(o=o), o, lambda: [h.status() for h, _ in c.handles])
