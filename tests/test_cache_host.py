"""Rotary and cache handles: what creation refuses, and the 4-bit reference's own pins (CPU)."""
import ctypes as C
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv4_ref as R
from harness import ensure_built
from medusa_head_speculative_gb300 import binding as Bnd


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("bad,code", [
    (dict(rot=0), -1), (dict(rot=7), -1), (dict(max_pos=0), -1), (dict(base=1.0), -1),
    (dict(base=float("nan")), -1), (dict(scaling="linear", factor=0.0), -1),
    (dict(scaling="banded", orig_pos=0, factor=2.0), -1),
    (dict(scaling="ramp", orig_pos=64, factor=2.0, low=4.0, high=4.0), -1),
    (dict(attn=-1.0), -1), (dict(attn=float("inf")), -1), (dict(rot=2048), -2),
])
def test_rope_creation_refuses(bad, code):
    kw = dict(rot=64, max_pos=16)
    kw.update(bad)
    with pytest.raises(Bnd.MedusaError) as e:
        Bnd.Rope(**kw)
    assert e.value.code == code


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), -1), (dict(Hq=3), -1), (dict(Hkv=0), -1), (dict(format=3), -1), (dict(format=-1), -1),
    (dict(capacity=0), -1), (dict(page_size=-1), -1), (dict(page_size=16, num_pages=0), -1),
    (dict(page_size=16, num_pages=4, capacity=40), -1), (dict(max_nodes=0), -1),
    (dict(max_nodes=257), -2), (dict(dh=48), -2), (dict(dh=256), -2), (dict(capacity=40), -2),
    (dict(page_size=8, num_pages=8, capacity=64), -2),
])
def test_cache_creation_refuses(bad, code):
    kw = dict(B=2, Hq=4, Hkv=2, dh=64, format=Bnd.KV4, capacity=64)
    kw.update(bad)
    with pytest.raises(Bnd.MedusaError) as e:
        Bnd.Cache(**kw)
    assert e.value.code == code


@pytest.mark.parametrize("kw", [
    dict(B=1 << 22, Hq=65535, Hkv=65535, dh=128, format=Bnd.BF16, capacity=1 << 24),
    dict(B=1, Hq=65535, Hkv=65535, dh=128, format=Bnd.KV4, capacity=1 << 24, page_size=1 << 24, num_pages=(1 << 31) - 1),
    dict(B=1 << 22, Hq=65535, Hkv=1, dh=128, format=Bnd.KV4, capacity=16, max_nodes=256),
])
def test_caches_whose_sizes_pass_64_bits_are_refused(kw):
    with pytest.raises(Bnd.MedusaError) as e:
        Bnd.Cache(**kw)
    assert e.value.code == -2


def test_calls_without_a_handle_are_refused():
    L = Bnd.lib()
    kv, rows, places, q = Bnd.KV(), Bnd.KVRows(), Bnd.KVPlaces(), Bnd.KV4Query()
    assert L.medusa_rope_apply(None, 0, 64, 1, None, bytes(56), 1, 0, None) == -1
    assert L.medusa_kv_append(None, kv, rows, None, 1.0, 1.0, None) == -1
    assert L.medusa_kv_read(None, kv, places, 1.0, 1.0, None) == -1
    assert L.medusa_kv4_attention(None, kv, q, None, 0, None) == -1
    assert L.medusa_rope_create(None, None) == -1 and L.medusa_cache_create(None, None) == -1
    out = C.c_void_p()
    assert L.medusa_rope_create(None, C.byref(out)) == -1 and not out
    assert L.medusa_cache_create(None, C.byref(out)) == -1 and not out
    assert L.medusa_cache_pool_bytes(None) == 0 and L.medusa_cache_workspace_size(None) == 0
    L.medusa_rope_destroy(None)
    L.medusa_cache_destroy(None)


def test_reference_formats():
    assert R.E4M3[0x7e] == 448 and R.E4M3[1] == 2.0 ** -9 and np.isnan(R.E4M3[0x7f])
    for i in range(126):                      # every e4m3 and every midpoint
        assert R.e4m3_nearest(R.E4M3[i]) == i
        assert R.e4m3_nearest((R.E4M3[i] + R.E4M3[i + 1]) / 2) % 2 == 0
    assert list(R.e2m1_nearest(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 9]))) == [0, 2, 2, 4, 4, 6, 6, 7]
    x = np.random.default_rng(0).standard_normal((5, 3, 64))
    codes, scales = R.encode(x, 0.5)
    y = R.decode(codes, scales, 0.5)
    # the widest gap between codes is 2, and a scale rounded down clips less than that
    assert (np.abs(y - x) <= np.repeat(R.E4M3[scales], 16, -1) * 0.5).all()


def test_reference_rotation_depends_on_distance_only():
    r = np.random.default_rng(1)
    q, k = r.standard_normal((1, 1, 32)), r.standard_normal((1, 1, 32))
    for layout in ("half", "interleaved"):
        a = (R.rope(q, [9], 32, layout) * R.rope(k, [4], 32, layout)).sum()
        b = (R.rope(q, [105], 32, layout) * R.rope(k, [100], 32, layout)).sum()
        assert abs(a - b) < 1e-12
        back = R.rope(R.rope(q, [77], 24, layout), [77], 24, layout, inverse=True)
        assert np.abs(back - q).max() < 1e-14


def unopened(cls, **kw):
    """A handle object without a handle: calls that pass the binding's own checks are refused by the library."""
    h = cls.__new__(cls)
    h.handle = None
    for name, value in dict(kw, device=-1).items():          # a CPU tensor's device
        setattr(h, name, value)
    return h


NO_STREAM = SimpleNamespace(cuda_stream=None)


def test_rows_that_are_no_equal_shares_are_refused():
    cache = unopened(Bnd.Cache, B=4, Hq=1, Hkv=1, dh=32, format=Bnd.BF16)
    rows, ints = torch.zeros(10, 1, 32), torch.zeros(12, dtype=torch.int32)
    for call in (lambda **kw: Bnd.kv_append(cache, Bnd.KV(), rows, rows, stream=NO_STREAM, **kw),
                 lambda **kw: Bnd.kv_append(cache, Bnd.KV(), rows, rows, index=ints[:10], index_rows=2, stream=NO_STREAM, **kw),
                 lambda **kw: Bnd.kv_read(cache, Bnd.KV(), rows, rows, stream=NO_STREAM, **kw)):
        with pytest.raises(ValueError, match="equal shares"):
            call()
        with pytest.raises(Bnd.MedusaError):                 # as far as the library
            call(per_seq=2)
        with pytest.raises(Bnd.MedusaError):
            call(rows=8)


@pytest.mark.parametrize("device,error", [(0, ValueError), (-1, Bnd.MedusaError)])
def test_tensors_on_another_device_are_refused(device, error):
    """Their addresses would go to the kernels.  Tensors of the CPU with handles of a GPU, and (which the library
    alone refuses) with handles whose device is theirs."""
    x, ints = torch.zeros(4, 2, 32), torch.zeros(64, dtype=torch.int32)
    q, tree, ws = torch.zeros(2, 2, 2, 32), torch.zeros(2, 2, 2, 32), torch.zeros(256, dtype=torch.uint8)
    cache, rope = unopened(Bnd.Cache, B=2, Hq=2, Hkv=2, dh=32, format=Bnd.KV4), unopened(Bnd.Rope)
    cache.device = rope.device = device

    def attend(ws):
        Bnd.kv4_attention(cache, Bnd.KV(), q, torch.empty_like(q), ws, tree_k=tree, tree_v=tree, mask=ints,
                          stream=NO_STREAM)

    for call in (lambda: Bnd.rope_apply(rope, ints[:4], [(x, x)], stream=NO_STREAM),
                 lambda: Bnd.kv_append(cache, Bnd.KV(), x, x, pos=ints[:4], stream=NO_STREAM),
                 lambda: Bnd.kv_read(cache, Bnd.KV(), x, x, first=ints[:2], stream=NO_STREAM), lambda: attend(ws)):
        with pytest.raises(error):
            call()
    elsewhere = SimpleNamespace(device="elsewhere", get_device=lambda: 7, data_ptr=lambda: 256, numel=lambda: 256,
                                element_size=lambda: 1, is_contiguous=lambda: True)
    for bad in (elsewhere, ws[::2]):
        with pytest.raises(ValueError):
            attend(bad)


def test_closed_rotation_is_refused():
    """Appending with a Rope that has been closed must not leave the keys unturned."""
    cache, rope = unopened(Bnd.Cache, B=2, Hq=2, Hkv=2, dh=32, format=Bnd.KV4), unopened(Bnd.Rope)
    rope.close()
    x = torch.zeros(4, 2, 32)
    with pytest.raises(ValueError, match="closed"):
        Bnd.kv_append(cache, Bnd.KV(), x, x, rope=rope, stream=NO_STREAM)
    with pytest.raises(Bnd.MedusaError):
        Bnd.rope_apply(rope, torch.zeros(4, dtype=torch.int32), [(x, x)], stream=NO_STREAM)
