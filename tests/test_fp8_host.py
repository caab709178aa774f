"""8-bit projections and attention over a shared prefix: what creation and the bindings refuse, and the
references' own pins (CPU)."""
import ctypes as C
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import fp8_ref as F
import prefix_ref as A
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd

NO_STREAM = SimpleNamespace(cuda_stream=None)


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def unopened(cls, **kw):
    """A handle object without a handle: calls that pass the binding's own checks are refused by the library."""
    h = cls.__new__(cls)
    h.handle = None
    for name, value in dict(dict(device=-1), **kw).items():  # a CPU tensor's device
        setattr(h, name, value)
    return h


@pytest.mark.parametrize("bad,code", [
    (dict(n=0), -1), (dict(k=0), -1), (dict(k=24), -1), (dict(k=8), -1), (dict(max_rows=0), -1), (dict(n=-5), -1),
    (dict(n=(1 << 24) + 1), -2), (dict(k=(1 << 20) + 16), -2), (dict(max_rows=(1 << 24) + 1), -2),
    (dict(n=1 << 20, k=1 << 19), -2), (dict(max_rows=1 << 24, k=1 << 15), -2), (dict(max_rows=1 << 24, n=1 << 15), -2),
])
def test_fp8_creation_refuses(bad, code):
    with pytest.raises(Bnd.MedusaError) as e:
        Bnd.Fp8(**dict(dict(n=64, k=128, max_rows=4), **bad))
    assert e.value.code == code


def test_calls_without_a_handle_are_refused():
    L = Bnd.lib()
    out = C.c_void_p()
    assert L.medusa_fp8_create(None, None) == -1
    assert L.medusa_fp8_create(None, C.byref(out)) == -1 and not out
    assert L.medusa_fp8_workspace_size(None) == 0 and L.medusa_prefix_workspace_size(None, None) == 0
    assert L.medusa_fp8_get_status(None, None, None) == -1
    assert L.medusa_fp8_round(None, None, 0, 0, 0, None, None, 1, None) == -1
    assert L.medusa_fp8_read(None, None, None, 0, 1, None, 0, 0, None) == -1
    assert C.sizeof(Bnd.Fp8Product) == Bnd._PRODUCT.size
    assert L.medusa_fp8_linear(None, bytes(Bnd._PRODUCT.size), None, 0, None) == -1
    assert L.medusa_prefix_attention(None, Bnd.KV(), None, Bnd.KV(), Bnd.KV4Query(), None, 0, None) == -1
    L.medusa_fp8_destroy(None)


def test_bindings_refuse_shapes_types_and_devices():
    h = unopened(Bnd.Fp8, n=130, k=144, kb=2, nb=2)
    x, codes, scales = torch.zeros(5, 144), torch.zeros(5, 144, dtype=torch.uint8), torch.zeros(5, 2)
    w, ws, y = torch.zeros(130, 144, dtype=torch.float8_e4m3fn), torch.zeros(2, 2), torch.zeros(5, 130)
    work = torch.zeros(256, dtype=torch.uint8)
    kw = dict(stream=NO_STREAM)
    good = [lambda: Bnd.fp8_round(h, x, codes, scales, **kw), lambda: Bnd.fp8_read(h, codes, scales, x, **kw),
            lambda: Bnd.fp8_linear(h, x, w, ws, y, work, add=y, **kw),
            lambda: Bnd.fp8_linear(h, codes, w, ws, y, work, x_scales=scales, up=w, up_scales=ws, **kw)]
    for call in good:
        with pytest.raises(Bnd.MedusaError):                 # as far as the library
            call()
    for call in (lambda: Bnd.fp8_round(h, x[:, :128], codes, scales, **kw),
                 lambda: Bnd.fp8_round(h, x, codes.t().contiguous().t(), scales, **kw),
                 lambda: Bnd.fp8_round(h, x, codes, scales[:4], **kw),
                 lambda: Bnd.fp8_round(h, x, codes, scales, block=128, **kw),
                 lambda: Bnd.fp8_read(h, codes[:4], scales, x, **kw),
                 lambda: Bnd.fp8_linear(h, x, w[:129], ws, y, work, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws[:1], y, work, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws, y[:4], work, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws, y, work, up=w, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws, y, work, add=y[:3], **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws, y, work[::2], **kw)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: Bnd.fp8_round(h, x.double(), codes, scales, **kw),
                 lambda: Bnd.fp8_round(h, x, codes.short(), scales, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws.double(), y, work, **kw),
                 lambda: Bnd.fp8_linear(h, x, w, ws, y, work, add=y.bfloat16(), **kw),
                 lambda: Bnd.fp8_linear(h, codes, w, ws, y, work, **kw)):
        with pytest.raises(TypeError):
            call()
    h.device = 0
    for call in good:
        with pytest.raises(ValueError, match="device"):
            call()


def test_prefix_bindings_refuse():
    own, shared = (unopened(Bnd.Cache, B=b, Hq=4, Hkv=2, dh=32, format=Bnd.F32) for b in (2, 1))
    q, ws, ints = torch.zeros(2, 3, 4, 32), torch.zeros(256, dtype=torch.uint8), torch.zeros(24, dtype=torch.int32)
    tree = torch.zeros(2, 3, 2, 32)

    def call(q=q, ws=ws, **kw):
        Bnd.prefix_attention(own, Bnd.KV(), shared, Bnd.KV(), q, torch.empty_like(q), ws, stream=NO_STREAM, **kw)

    for kw in (dict(), dict(tree_k=tree, tree_v=tree, mask=ints)):
        with pytest.raises(Bnd.MedusaError):
            call(**kw)
    for kw in (dict(q=q[:1]), dict(q=q[..., :16]), dict(ws=ws[::2]), dict(tree_k=tree[:1], tree_v=tree),
               dict(tree_k=tree, tree_v=tree, mask=ints[:23])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(tree_k=tree.bfloat16(), tree_v=tree)
    shared.device = 0
    with pytest.raises(ValueError, match="one device"):
        call()


def test_reference_format():
    assert F.decode(0x7e) == 448 and F.decode(1) == 2.0 ** -9 and F.decode(0x80) == 0 and np.isnan(F.decode(0x7f))
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(F.decode(np.arange(256)), t)
    for i in range(126):                      # every code, every midpoint
        assert F.encode(F.decode(i)) == i and F.encode((F.decode(i) + F.decode(i + 1)) / 2) % 2 == 0
    x = np.random.default_rng(0).standard_normal((3, 300))
    x[1, :128] = 0
    codes, scales = F.round8(x, 1)
    assert (scales[1, 0], scales.shape) == (1.0, (3, 3)) and (np.abs(F.values(codes, scales, 1) - x) <=
                                                             np.maximum(np.abs(x) / 16, np.repeat(scales, 128, 1)[:, :300] * 2.0 ** -10)).all()


def test_reference_attention_is_a_mean():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((2, 2, 8)), r.standard_normal((5, 1, 8)), r.standard_normal((5, 1, 8))
    one = np.ones((5, 1, 8))
    o, _ = A.attention(q, [(k[:3], one[:3]), (k[3:], one[3:])], np.array([[1, 0], [1, 1]], bool), 0.3, 0)
    assert np.abs(o - 1).max() < 1e-12
    a, _ = A.attention(q, [(k, v)], None, 0.3, 0)
    b, _ = A.attention(q, [(k[2:], v[2:]), (k[:2], v[:2])], np.ones((2, 2), bool), 0.3, 0)
    assert np.abs(a - b).max() < 1e-12


def test_prefix_expire_wait_needs_a_cache():
    assert Bnd.lib().medusa_prefix_expire_wait_once(None, 1000) == Bnd.MEDUSA_ERR_INVALID


def test_fp8_expire_wait_needs_a_handle():
    assert Bnd.lib().medusa_fp8_expire_wait_once(None, 1000) == Bnd.MEDUSA_ERR_INVALID


def test_fp8_tiles_needs_a_handle():
    out = C.c_int()
    assert Bnd.lib().medusa_fp8_tiles(None, 1, 0, out, out, out) == Bnd.MEDUSA_ERR_INVALID
