"""Attention over a shared prefix: waits that run out, and operands that are one row or one cache."""
import time

import pytest
import torch

import test_gpu_prefix as T
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("case", [
    # B, hq, hk, dh, n1, P, lens, page, ppage, kind
    (3, 8, 2, 128, 1, 5000, [700, 0, 129], 0, 0, None),              # one tile of rows, chunks by the copy engine
    (3, 8, 8, 64, 17, 3000, [1500, 0, 40], 16, 16, "tree"),          # one tile, pages
    (2, 2, 2, 128, 30, 130, [5, 0], 0, 0, "causal"),                 # fewer chunks than stages
    (3, 8, 2, 128, 43, 2000, [1500, 0, 129], 0, 0, "tree"),          # two tiles
    (2, 4, 1, 64, 100, 600, [300, 20], 16, 0, "holes"),              # two tiles, the last half empty
], ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_expired_wait_is_reported_and_nothing_else_is_lost(case):
    """A bounded wait is made to run out: the call returns with MEDUSA_FLAG_TIMEOUT in own's status, whatever the workspace
    held, and the next one on the same workspace is as before."""
    *dims, kind = case
    c = T.Case(3, *dims, "bf16", kind)
    own, shared = c.handles[0][0], c.handles[1][0]

    def call():
        c.ws.fill_(0x7f)
        t0 = time.perf_counter()
        o = c.run()
        torch.cuda.synchronize()
        return o, time.perf_counter() - t0

    clean, _ = call()
    c.check(clean)
    own.prefix_expire_wait_once(2_000_000)
    assert call()[1] < 30.0
    assert (own.status(), shared.status()) == (Bnd.FLAG_TIMEOUT, 0)
    again, _ = call()
    assert torch.equal(again.view(torch.uint8), clean.view(torch.uint8)) and (own.status(), shared.status()) == (0, 0)


def test_expire_wait_argument_checks():
    cache = lambda **kw: Bnd.Cache(**dict(dict(B=1, Hq=2, Hkv=1, dh=64, format=Bnd.BF16, capacity=16), **kw))  # noqa: E731
    for ns in (0, 10**10 + 1):
        with pytest.raises(Bnd.MedusaError) as e:
            cache().prefix_expire_wait_once(ns)
        assert e.value.code == Bnd.MEDUSA_ERR_INVALID
    for kw in (dict(format=Bnd.F32), dict(dh=32), dict(format=Bnd.KV4)):
        with pytest.raises(Bnd.MedusaError) as e:
            cache(**kw).prefix_expire_wait_once(1000)
        assert e.value.code == Bnd.MEDUSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_that_are_one_row_and_caches_that_are_one(dtype):
    """Row and head strides of 0 for the queries; and a sequence whose own cache is the shared one too (each key twice)."""
    c = T.Case(12, 1, 6, 2, 64, 5, 200, [200], 0, 0, dtype, None)
    q = c.q[:, :1, :1].expand_as(c.q)
    o = c.run(q=q)
    assert torch.equal(o[:, 1:].contiguous(), o[:, :1].expand(1, 4, 6, 64).contiguous())     # rows alike; heads of a key head too
    assert torch.equal(o[:, :, 0], o[:, :, 2]) and not torch.equal(o[:, :, 0], o[:, :, 3])
    (own, okv), _ = c.handles
    ws = torch.empty(Bnd.prefix_workspace_size(own, own), dtype=torch.uint8, device="cuda")
    twice, once = torch.empty_like(c.q), torch.empty_like(c.q)
    c.shared_pool["len"].zero_()
    c.shared_pool["lens"] = [0]
    c.run(o=once)
    Bnd.prefix_attention(own, okv, own, okv, c.q, twice, ws)
    want, tol = c.want()                          # doubled weights of equal keys: the same mean, over twice as many terms
    assert (abs(T.f64(once) - want) <= tol).all() and (abs(T.f64(twice) - want) <= 2 * tol).all() and own.status() == 0
