"""ctypes binding of libmedusa.so: the same entry points as include/medusa.h.

Argument marshalling only.  Torch tensors supply device memory and the stream; every step
of the computation runs in the library's CUDA kernels.  There is no fallback: if the
library is missing, loading raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmedusa.so")

MEDUSA_OK, MEDUSA_ERR_INVALID, MEDUSA_ERR_UNSUPPORTED = 0, -1, -2
MEDUSA_ERR_CUDA, MEDUSA_ERR_DEVICE, MEDUSA_ERR_WORKSPACE = -3, -4, -6
F32, BF16, KV4 = 0, 1, 2
GREEDY, TYPICAL, REJECT = 0, 1, 2
MAX_HEADS, MAX_TOPS, MAX_NODES = 8, 16, 256
FLAG_TOKEN_RANGE, FLAG_KV_CAPACITY, FLAG_PAGE_RANGE, FLAG_NONFINITE, FLAG_TIMEOUT = 1, 2, 4, 8, 16
FLAG_POS_RANGE, FLAG_ROW_RANGE = 32, 64
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "banded": 2, "ramp": 3}
STATUS_NAMES = {0: "OK", -1: "INVALID", -2: "UNSUPPORTED", -3: "CUDA", -4: "DEVICE", -6: "WORKSPACE"}


class MedusaError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code} ({STATUS_NAMES.get(code, '?')})")
        self.code = code


class Dims(C.Structure):
    _fields_ = [("B", C.c_int), ("d", C.c_int), ("V", C.c_int), ("K", C.c_int), ("Hq", C.c_int),
                ("Hkv", C.c_int), ("dh", C.c_int), ("dtype", C.c_int), ("rope_base", C.c_float),
                ("capacity", C.c_int), ("page_size", C.c_int), ("num_pages", C.c_int)]


class TreeSpec(C.Structure):
    _fields_ = [("K", C.c_int), ("s", C.c_int * MAX_HEADS), ("N", C.c_int),
                ("parent", C.POINTER(C.c_int32)), ("rank", C.POINTER(C.c_int32))]


class Weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w1", "w2", "lm", "emb", "wq", "wk", "wv", "wo")]


class Layer(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("wq", "wk", "wv", "wo", "k", "v")]


class KV(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_table", C.c_void_p),
                ("len", C.c_void_p), ("len_out", C.c_void_p)]


class Accept(C.Structure):
    _fields_ = [("mode", C.c_int), ("temperature", C.c_float), ("eps", C.c_float),
                ("delta", C.c_float), ("uniforms", C.c_void_p)]


class KernelTime(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("launches", C.c_int), ("total_ms", C.c_double)]


class Outputs(C.Structure):
    _fields_ = [("out_tok", C.c_void_p), ("n_acc", C.c_void_p), ("path_nodes", C.c_void_p),
                ("h_next", C.c_void_p), ("root_next", C.c_void_p)]


class RopeDesc(C.Structure):
    _fields_ = [("rot", C.c_int), ("layout", C.c_int), ("max_pos", C.c_int), ("scaling", C.c_int),
                ("base", C.c_double), ("factor", C.c_double), ("orig_pos", C.c_double),
                ("low", C.c_double), ("high", C.c_double), ("attn", C.c_double)]


class CacheDims(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("B", "Hq", "Hkv", "dh", "format", "capacity", "page_size",
                                       "num_pages", "max_nodes")]


class KVRows(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int), ("k_row", C.c_longlong),
                ("k_head", C.c_longlong), ("v_row", C.c_longlong), ("v_head", C.c_longlong),
                ("rows", C.c_int), ("start", C.c_void_p), ("per_seq", C.c_int), ("count", C.c_void_p),
                ("index", C.c_void_p), ("index_rows", C.c_int), ("pos", C.c_void_p)]


class KVPlaces(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int), ("k_row", C.c_longlong),
                ("k_head", C.c_longlong), ("v_row", C.c_longlong), ("v_head", C.c_longlong),
                ("rows", C.c_int), ("start", C.c_void_p), ("per_seq", C.c_int), ("count", C.c_void_p),
                ("first", C.c_void_p)]


class KV4Query(C.Structure):
    _fields_ = [("q", C.c_void_p), ("o", C.c_void_p), ("dtype", C.c_int), ("n1", C.c_int),
                ("q_row", C.c_longlong), ("q_head", C.c_longlong), ("o_row", C.c_longlong),
                ("o_head", C.c_longlong), ("tree_k", C.c_void_p), ("tree_v", C.c_void_p),
                ("mask", C.c_void_p), ("scale", C.c_float), ("k_scale", C.c_float),
                ("v_scale", C.c_float)]


_lib = None
P = C.c_void_p
SZ = C.c_size_t
I = C.c_int


def lib():
    """Load libmedusa.so (built by medusa_head_speculative_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m medusa_head_speculative_gb300.build`")
    L = C.CDLL(LIB_PATH)
    sigs = {
        "medusa_plan_create": (I, [C.POINTER(Dims), C.POINTER(TreeSpec), C.POINTER(P)]),
        "medusa_plan_destroy": (None, [P]),
        "medusa_workspace_size": (SZ, [P]),
        "medusa_get_status": (I, [P, P, C.POINTER(C.c_uint32)]),
        "medusa_step": (I, [P, P, P, C.POINTER(Weights), C.POINTER(KV), Accept,
                            C.POINTER(Outputs), P, SZ, P]),
        "medusa_workspace_size_layers": (SZ, [P, I]),
        "medusa_step_layers": (I, [P, P, P, C.POINTER(Weights), C.POINTER(Layer), I, C.POINTER(KV),
                                   Accept, C.POINTER(Outputs), P, SZ, P]),
        "medusa_heads": (I, [P, P, P, C.POINTER(Weights), P, P, P, P, P, SZ, P]),
        "medusa_heads_noalloc": (I, [P, P, P, C.POINTER(Weights), P, P, P, P]),
        "medusa_tree_build": (I, [P, P, P, P, P, P, P, P, P]),
        "medusa_layer_qkv": (I, [P, C.POINTER(Weights), P, P, P, P, P, P, SZ, P]),
        "medusa_tree_attention": (I, [P, P, C.POINTER(KV), P, P, P, P, P, SZ, P]),
        "medusa_layer_out": (I, [P, C.POINTER(Weights), P, P, P, P, SZ, P]),
        "medusa_verify_logits": (I, [P, C.POINTER(Weights), P, P, Accept, P, P, P, P, SZ, P]),
        "medusa_verify": (I, [P, P, P, P, P, P, P, Accept, C.POINTER(Outputs), P]),
        "medusa_kv_compact": (I, [P, C.POINTER(KV), P, P, P, P, P]),
        "medusa_profile_start": (I, [P, I]),
        "medusa_profile_stop": (I, [P, P, C.POINTER(KernelTime), I, C.POINTER(I), C.POINTER(I)]),
        "medusa_tree_cartesian": (I, [I, C.POINTER(C.c_int), I, C.POINTER(C.c_int32),
                                      C.POINTER(C.c_int32)]),
        "medusa_tree_greedy": (I, [I, C.POINTER(C.c_int), I, C.POINTER(C.c_double), I,
                                   C.POINTER(C.c_int32), C.POINTER(C.c_int32)]),
        "medusa_tree_greedy_device": (I, [I, C.POINTER(C.c_int), I, P, I, P, P, P, P]),
        "medusa_tree_size_choose": (I, [C.POINTER(C.c_double), I, C.POINTER(C.c_int),
                                        C.POINTER(C.c_double), I]),
        "medusa_loop_create": (I, [P, C.POINTER(Weights), C.POINTER(KV), Accept, P, P, P, P, I, P,
                                   SZ, C.POINTER(P)]),
        "medusa_loop_run": (I, [P, I, P]),
        "medusa_loop_steps": (I, [P, P, C.POINTER(C.c_longlong)]),
        "medusa_loop_destroy": (None, [P]),
        "medusa_plan_expire_wait_once": (I, [P, C.c_ulonglong]),
        "medusa_rope_create": (I, [C.POINTER(RopeDesc), C.POINTER(P)]),
        "medusa_rope_destroy": (None, [P]),
        "medusa_rope_get_status": (I, [P, P, C.POINTER(C.c_uint32)]),
        "medusa_rope_apply": (I, [P, I, I, I, P, C.c_char_p, I, I, P]),   # medusa_rope_rows as bytes
        "medusa_cache_create": (I, [C.POINTER(CacheDims), C.POINTER(P)]),
        "medusa_cache_destroy": (None, [P]),
        "medusa_cache_pool_bytes": (SZ, [P]),
        "medusa_cache_workspace_size": (SZ, [P]),
        "medusa_cache_get_status": (I, [P, P, C.POINTER(C.c_uint32)]),
        "medusa_cache_expire_wait_once": (I, [P, C.c_ulonglong]),
        "medusa_kv_append": (I, [P, C.POINTER(KV), C.POINTER(KVRows), P, C.c_float, C.c_float, P]),
        "medusa_kv_read": (I, [P, C.POINTER(KV), C.POINTER(KVPlaces), C.c_float, C.c_float, P]),
        "medusa_kv4_attention": (I, [P, C.POINTER(KV), C.POINTER(KV4Query), P, SZ, P]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(fn, code):
    if code != MEDUSA_OK:
        raise MedusaError(fn, code)


def ptr(t):
    """Device (or host) address of a tensor, or None."""
    return None if t is None else t.data_ptr()


_current = None     # address of the current device's current stream


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    global _current
    if _current is None:
        import torch
        try:        # a Stream object takes longer to make than a kernel to launch
            raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            _current = lambda: raw(device())  # noqa: E731
            torch.cuda.current_stream()       # (initialises CUDA)
            _current()
        except (AttributeError, TypeError):
            _current = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current()


# ------------------------------------------------------------------ host tree builders
def tree_cartesian(s):
    K = len(s)
    sa = (C.c_int * K)(*s)
    cap = MAX_NODES
    parent = (C.c_int32 * cap)()
    rank = (C.c_int32 * cap)()
    n1 = lib().medusa_tree_cartesian(K, sa, cap, parent, rank)
    if n1 < 0:
        raise MedusaError("medusa_tree_cartesian", n1)
    return np.array(parent[:n1], dtype=np.int32), np.array(rank[:n1], dtype=np.int32)


def tree_greedy(s, a, N):
    a = np.ascontiguousarray(a, dtype=np.float64)
    K, smax = a.shape
    sa = (C.c_int * K)(*s)
    parent = (C.c_int32 * (N + 1))()
    rank = (C.c_int32 * (N + 1))()
    n1 = lib().medusa_tree_greedy(K, sa, smax, a.ctypes.data_as(C.POINTER(C.c_double)), N,
                                  parent, rank)
    if n1 < 0:
        raise MedusaError("medusa_tree_greedy", n1)
    return np.array(parent[:n1], dtype=np.int32), np.array(rank[:n1], dtype=np.int32)


def tree_greedy_device(s, a_dev, N, parent, rank, expected=None, stream=None):
    """medusa_tree_greedy_device: a_dev a [K][smax] float64 CUDA tensor; parent, rank int32
    CUDA tensors of N+1 entries, expected float64 (N+1) or None."""
    K, smax = a_dev.shape
    sa = (C.c_int * K)(*s)
    _check("medusa_tree_greedy_device",
           lib().medusa_tree_greedy_device(K, sa, smax, ptr(a_dev), N, ptr(parent), ptr(rank),
                                           ptr(expected), _stream(stream)))


def tree_size_choose(expected, sizes, step_ms):
    """medusa_tree_size_choose: index into sizes of the best expected tokens per time."""
    e = np.ascontiguousarray(expected, dtype=np.float64)
    sz = (C.c_int * len(sizes))(*sizes)
    ms = np.ascontiguousarray(step_ms, dtype=np.float64)
    i = lib().medusa_tree_size_choose(e.ctypes.data_as(C.POINTER(C.c_double)), len(e) - 1, sz,
                                      ms.ctypes.data_as(C.POINTER(C.c_double)), len(sizes))
    if i < 0:
        raise MedusaError("medusa_tree_size_choose", i)
    return i


# ------------------------------------------------------------------ plan
class Plan:
    """Owns a medusa_plan: validated sizes and the uploaded tree spec."""

    def __init__(self, B, d, V, K, Hq, Hkv, dh, dtype, capacity, s, parent, rank,
                 rope_base=10000.0, page_size=0, num_pages=0):
        self.dims = Dims(B, d, V, K, Hq, Hkv, dh, dtype, rope_base, capacity, page_size, num_pages)
        parent = np.ascontiguousarray(parent, dtype=np.int32)
        rank = np.ascontiguousarray(rank, dtype=np.int32)
        self.spec = TreeSpec()
        self.spec.K = K
        for k in range(MAX_HEADS):
            self.spec.s[k] = int(s[k]) if k < len(s) else 0
        self.spec.N = len(parent) - 1
        self._keep = (parent, rank)
        self.spec.parent = parent.ctypes.data_as(C.POINTER(C.c_int32))
        self.spec.rank = rank.ctypes.data_as(C.POINTER(C.c_int32))
        h = P()
        _check("medusa_plan_create", lib().medusa_plan_create(C.byref(self.dims), C.byref(self.spec),
                                                              C.byref(h)))
        self.handle = h
        self.B, self.d, self.V, self.K, self.N = B, d, V, K, len(parent) - 1
        self.Hq, self.Hkv, self.dh, self.dtype = Hq, Hkv, dh, dtype
        self.n1 = self.N + 1
        self.parent, self.rank = parent, rank

    @property
    def workspace_size(self):
        return lib().medusa_workspace_size(self.handle)

    def workspace_size_layers(self, n_layers):
        return lib().medusa_workspace_size_layers(self.handle, n_layers)

    def status(self, stream=None):
        flags = C.c_uint32(0)
        code = lib().medusa_get_status(self.handle, _stream(stream), C.byref(flags))
        if code not in (MEDUSA_OK, MEDUSA_ERR_DEVICE):
            raise MedusaError("medusa_get_status", code)
        return flags.value

    def expire_wait_once(self, ns):
        """Failure-path testing: the next verification-logit GEMM's wait runs out after ns."""
        _check("medusa_plan_expire_wait_once", lib().medusa_plan_expire_wait_once(self.handle, int(ns)))

    def profile_start(self, max_launches):
        _check("medusa_profile_start", lib().medusa_profile_start(self.handle, max_launches))

    def profile_stop(self, stream=None):
        """Per-kernel {name: (launches, total_ms)} in first-launch order, and the launch count."""
        out = (KernelTime * 64)()
        n, launches = C.c_int(0), C.c_int(0)
        _check("medusa_profile_stop", lib().medusa_profile_stop(self.handle, _stream(stream), out, 64,
                                                                C.byref(n), C.byref(launches)))
        return {out[i].name.decode(): (out[i].launches, out[i].total_ms) for i in range(n.value)}, \
            launches.value

    def close(self):
        if getattr(self, "handle", None):
            lib().medusa_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def weights_struct(w):
    return Weights(*(ptr(w.get(n)) for n in ("w1", "w2", "lm", "emb", "wq", "wk", "wv", "wo")))


def layers_array(layers):
    """ctypes array of Layer from dicts with wq, wk, wv, wo, k, v (device tensors)."""
    arr = (Layer * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = Layer(*(ptr(L[n]) for n in ("wq", "wk", "wv", "wo", "k", "v")))
    return arr


def kv_struct(k, v, length, len_out=None, page_table=None):
    return KV(ptr(k), ptr(v), ptr(page_table), ptr(length), ptr(len_out))


def accept_struct(mode="greedy", temperature=0.0, eps=0.09, delta=0.3, uniforms=None):
    code = {"typical": TYPICAL, "reject": REJECT}.get(mode, GREEDY)
    return Accept(code, temperature, eps, delta, ptr(uniforms))


def outputs_struct(out_tok, n_acc, path_nodes, h_next, root_next):
    return Outputs(ptr(out_tok), ptr(n_acc), ptr(path_nodes), ptr(h_next), ptr(root_next))


# ------------------------------------------------------------------ entry points
def step(plan, h, root_in, wts, kv, accept, outs, ws, stream=None):
    _check("medusa_step", lib().medusa_step(plan.handle, ptr(h), ptr(root_in), C.byref(wts),
                                            C.byref(kv), accept, C.byref(outs), ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)))


def step_layers(plan, h, root_in, wts, layers, kv, accept, outs, ws, stream=None):
    """medusa_step_layers; `layers` from layers_array."""
    _check("medusa_step_layers",
           lib().medusa_step_layers(plan.handle, ptr(h), ptr(root_in), C.byref(wts), layers,
                                    len(layers), C.byref(kv), accept, C.byref(outs), ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)))


def heads(plan, h, root_in, wts, logits, topk_tok, topk_val, root, ws, stream=None):
    _check("medusa_heads", lib().medusa_heads(plan.handle, ptr(h), ptr(root_in), C.byref(wts),
                                              ptr(logits), ptr(topk_tok), ptr(topk_val), ptr(root),
                                              ptr(ws), ws.numel() * ws.element_size(),
                                              _stream(stream)))


def heads_noalloc(plan, h, root_in, wts, topk_tok, topk_val, root, stream=None):
    """Heads stage with no workspace: scratch in the library's fixed device array."""
    _check("medusa_heads_noalloc", lib().medusa_heads_noalloc(plan.handle, ptr(h), ptr(root_in),
                                                              C.byref(wts), ptr(topk_tok),
                                                              ptr(topk_val), ptr(root),
                                                              _stream(stream)))


def tree_build(plan, topk_tok, root, length, tok, pos, mask, retrieve, stream=None):
    _check("medusa_tree_build", lib().medusa_tree_build(plan.handle, ptr(topk_tok), ptr(root),
                                                        ptr(length), ptr(tok), ptr(pos), ptr(mask),
                                                        ptr(retrieve), _stream(stream)))


def layer_qkv(plan, wts, tok, pos, q, tk, tv, ws, stream=None):
    _check("medusa_layer_qkv", lib().medusa_layer_qkv(plan.handle, C.byref(wts), ptr(tok), ptr(pos),
                                                      ptr(q), ptr(tk), ptr(tv), ptr(ws),
                                                      ws.numel() * ws.element_size(),
                                                      _stream(stream)))


def tree_attention(plan, q, kv, tk, tv, mask, o, ws, stream=None):
    _check("medusa_tree_attention",
           lib().medusa_tree_attention(plan.handle, ptr(q), C.byref(kv), ptr(tk), ptr(tv), ptr(mask),
                                       ptr(o), ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)))


def layer_out(plan, wts, tok, o, hprime, ws, stream=None):
    _check("medusa_layer_out", lib().medusa_layer_out(plan.handle, C.byref(wts), ptr(tok), ptr(o),
                                                      ptr(hprime), ptr(ws),
                                                      ws.numel() * ws.element_size(),
                                                      _stream(stream)))


def verify_logits(plan, wts, hprime, tok, accept, logits, am, stats, ws, stream=None):
    _check("medusa_verify_logits",
           lib().medusa_verify_logits(plan.handle, C.byref(wts), ptr(hprime), ptr(tok), accept,
                                      ptr(logits), ptr(am), ptr(stats), ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)))


def verify(plan, tok, am, stats, retrieve, hprime, accept, outs, stream=None, logits=None):
    _check("medusa_verify", lib().medusa_verify(plan.handle, ptr(tok), ptr(am), ptr(stats),
                                                ptr(logits), ptr(retrieve), ptr(hprime), accept,
                                                C.byref(outs), _stream(stream)))


def kv_compact(plan, kv, tk, tv, path_nodes, n_acc, stream=None):
    _check("medusa_kv_compact", lib().medusa_kv_compact(plan.handle, C.byref(kv), ptr(tk), ptr(tv),
                                                        ptr(path_nodes), ptr(n_acc),
                                                        _stream(stream)))


class Loop:
    """Owns a medusa_loop: one medusa_step with its state carried in place (h, root, cache
    lengths) plus the append to the token rings, captured once as a CUDA graph.  The
    tensors passed here must outlive the loop (its replays use their addresses)."""

    def __init__(self, plan, wts, kv, accept, h, root, tokens, n_acc, ws):
        self._keep = (plan, wts, kv, h, root, tokens, n_acc, ws)
        self.max_steps = tokens.shape[0]
        out = P()
        _check("medusa_loop_create",
               lib().medusa_loop_create(plan.handle, C.byref(wts), C.byref(kv), accept, ptr(h),
                                        ptr(root), ptr(tokens), ptr(n_acc), self.max_steps,
                                        ptr(ws), ws.numel() * ws.element_size(), C.byref(out)))
        self.handle = out

    def run(self, n_steps, stream=None):
        _check("medusa_loop_run", lib().medusa_loop_run(self.handle, int(n_steps), _stream(stream)))

    def steps(self, stream=None):
        n = C.c_longlong(0)
        _check("medusa_loop_steps", lib().medusa_loop_steps(self.handle, _stream(stream), C.byref(n)))
        return n.value

    def close(self):
        if getattr(self, "handle", None):
            lib().medusa_loop_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass



# ------------------------------------------------------------------ rotary positions, KV caches
def _status(fn, handle, stream):
    flags = C.c_uint32(0)
    code = getattr(lib(), fn)(handle, _stream(stream), C.byref(flags))
    if code not in (MEDUSA_OK, MEDUSA_ERR_DEVICE):
        raise MedusaError(fn, code)
    return flags.value


# These calls are made once a layer and token, where the host's part is what takes time: each
# tensor is asked once for its shape, strides, dtype and device.
_DTYPES = {}        # torch dtype -> F32 or BF16; _INT32: torch.int32
_INT32 = None


def _load_dtypes():
    global _INT32
    import torch
    _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16})
    _INT32 = torch.int32


def _dtype(x):
    if not _DTYPES:
        _load_dtypes()
    t = _DTYPES.get(x.dtype)
    if t is None:
        raise TypeError(f"float32 or bfloat16 is needed, got {x.dtype}")
    return t


def _same(x, *others):
    """The others (None: none) have x's dtype and device."""
    t, d = x.dtype, x.get_device()
    for y in others:
        if y is not None and (y.dtype != t or y.get_device() != d):
            raise TypeError(f"tensors of one dtype on one device are needed: {t} on {x.device}, "
                            f"{y.dtype} on {y.device}")


def _device():
    """The current device, where a handle's memory is made."""
    import torch
    return torch.cuda.current_device()


def _elsewhere(handle, *tensors):
    """Not all tensors are on the handle's device, and the kernels take their addresses as they are."""
    raise ValueError(f"tensors on cuda:{handle.device}, the handle's device, are needed, got "
                     + ", ".join(str(t.device) for t in tensors))


def _ints(what, t, n, device):
    """Address of an int32 tensor of at least n entries in order, or None."""
    if t is None:
        return None
    if _INT32 is None:
        _load_dtypes()
    if t.dtype is not _INT32 or t.numel() < n or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: a contiguous int32 tensor of at least {n} entries on the handle's "
                         f"device is needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(what, x, rows, heads, dh):
    """(row, head) strides of [rows][heads][dh] whose elements lie together."""
    shape, strides = x.shape, x.stride()
    if len(shape) != 3 or shape[0] < rows or shape[1] != heads or shape[2] != dh or strides[2] != 1:
        raise ValueError(f"{what}: [{rows}][{heads}][{dh}] with elements in order is needed, got "
                         f"shape {tuple(shape)}, strides {strides}")
    return strides[0], strides[1]


class Rope:
    """Owns a medusa_rope: the cosine/sine table of one rotation, on the current device.  Keep it as
    long as CUDA graphs that captured calls with it: they use its memory."""

    def __init__(self, rot, max_pos, layout="half", base=10000.0, scaling="plain", factor=1.0,
                 orig_pos=0, low=1.0, high=32.0, attn=1.0):
        self.desc = RopeDesc(rot, ROPE_LAYOUTS[layout], max_pos, ROPE_SCALINGS[scaling], base, factor,
                             orig_pos, low, high, attn)
        out = P()
        _check("medusa_rope_create", lib().medusa_rope_create(C.byref(self.desc), C.byref(out)))
        self.handle, self.device = out, _device()

    def status(self, stream=None):
        return _status("medusa_rope_get_status", self.handle, stream)

    def close(self):
        if getattr(self, "handle", None):
            lib().medusa_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# n medusa_rope_rows as bytes: x, y, heads, x_row, x_head, y_row, y_head
_ROPE_ROWS = {n: struct.Struct("PPiqqqq" * n) for n in range(1, 5)}


def rope_apply(rope, pos, parts, inverse=False, stream=None):
    """medusa_rope_apply: `parts` holds (x, y) pairs of [rows][heads][dh] tensors (any strides
    between rows and heads); y may be x."""
    rows, first = pos.numel(), parts[0][0]
    dh, dtype, t, device = first.shape[-1], _dtype(first), first.dtype, rope.device
    if first.get_device() != device:
        _elsewhere(rope, first)
    args = []
    for x, y in parts:
        xs, xt, ys, yt = x.shape, x.stride(), y.shape, y.stride()
        if len(xs) != 3 or xs != ys or xs[0] < rows or xs[2] != dh or xt[2] != 1 or yt[2] != 1:
            raise ValueError(f"x, y: [{rows}][heads][{dh}] with elements in order is needed, got shapes "
                             f"{tuple(xs)}, {tuple(ys)}, strides {xt}, {yt}")
        if x.dtype is not t or y.dtype is not t or x.get_device() != device or y.get_device() != device:
            _same(first, x, y)
        args += (x.data_ptr(), y.data_ptr(), xs[1], xt[0], xt[1], yt[0], yt[1])
    n = len(parts)
    code = MEDUSA_ERR_INVALID
    if n in _ROPE_ROWS:
        code = lib().medusa_rope_apply(rope.handle, dtype, dh, rows, _ints("pos", pos, rows, device),
                                       _ROPE_ROWS[n].pack(*args), n, 1 if inverse else 0, _stream(stream))
    _check("medusa_rope_apply", code)


class Cache:
    """Owns a medusa_cache: the sizes and format of a KV cache whose pools the caller holds.  Keep it
    as long as CUDA graphs that captured calls with it: they use its status word."""

    def __init__(self, B, Hq, Hkv, dh, format, capacity, page_size=0, num_pages=0, max_nodes=1):
        self.dims = CacheDims(B, Hq, Hkv, dh, format, capacity, page_size, num_pages, max_nodes)
        out = P()
        _check("medusa_cache_create", lib().medusa_cache_create(C.byref(self.dims), C.byref(out)))
        self.handle, self.device = out, _device()
        self.B, self.Hq, self.Hkv, self.dh, self.format = B, Hq, Hkv, dh, format
        self.pool_bytes = lib().medusa_cache_pool_bytes(out)
        self.workspace_size = lib().medusa_cache_workspace_size(out)

    def status(self, stream=None):
        return _status("medusa_cache_get_status", self.handle, stream)

    def expire_wait_once(self, ns):
        """Failure-path testing: see medusa_cache_expire_wait_once."""
        _check("medusa_cache_expire_wait_once", lib().medusa_cache_expire_wait_once(self.handle, int(ns)))

    def close(self):
        if getattr(self, "handle", None):
            lib().medusa_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _items(cache, n, start, rows, per_seq, count, device):
    """rows, start, per_seq and count of medusa_kv_rows / medusa_kv_places; n: places there are."""
    if rows is None:
        rows = n
    if start is not None:
        return rows, _ints("start", start, cache.B + 1, device), 0, None
    if per_seq is None:
        per_seq, rest = divmod(rows, cache.B)
        if rest:
            raise ValueError(f"{rows} rows are no equal shares of {cache.B} sequences: per_seq or start is needed")
    return cache.B * per_seq, None, per_seq, _ints("count", count, cache.B, device)


def kv_append(cache, kv, k, v, start=None, per_seq=None, count=None, index=None, index_rows=0,
              pos=None, rope=None, k_scale=1.0, v_scale=1.0, rows=None, stream=None):
    """medusa_kv_append: k, v [rows][Hkv][dh] (any strides between rows and heads).  Packed
    batches give `start`, padded ones `per_seq` (default: an equal share of the rows) and
    `count`; with `index` the item places are index's and k, v the rows they name."""
    if rope is not None and not rope.handle:
        raise ValueError("rope: closed")               # (the library turns nothing for NULL)
    device = cache.device
    if k.get_device() != device:
        _elsewhere(cache, k)
    n, start, per_seq, count = _items(cache, k.shape[0] if index is None else index.numel(), start,
                                      rows, per_seq, count, device)
    need = n if index is None else cache.B * index_rows
    kr, kh = _rows("k", k, need, cache.Hkv, cache.dh)
    vr, vh = _rows("v", v, need, cache.Hkv, cache.dh)
    _same(k, v)
    r = KVRows(k.data_ptr(), v.data_ptr(), _dtype(k), kr, kh, vr, vh, n, start, per_seq, count,
               _ints("index", index, n, device), index_rows, _ints("pos", pos, n, device))
    _check("medusa_kv_append",
           lib().medusa_kv_append(cache.handle, kv, r, None if rope is None else rope.handle,
                                  k_scale, v_scale, _stream(stream)))


def kv_read(cache, kv, k, v, start=None, per_seq=None, count=None, first=None, k_scale=1.0,
            v_scale=1.0, rows=None, stream=None):
    """medusa_kv_read into k, v [rows][Hkv][dh]; batches as in kv_append."""
    device = cache.device
    if k.get_device() != device:
        _elsewhere(cache, k)
    n, start, per_seq, count = _items(cache, k.shape[0], start, rows, per_seq, count, device)
    kr, kh = _rows("k", k, n, cache.Hkv, cache.dh)
    vr, vh = _rows("v", v, n, cache.Hkv, cache.dh)
    _same(k, v)
    r = KVPlaces(k.data_ptr(), v.data_ptr(), _dtype(k), kr, kh, vr, vh, n, start, per_seq, count,
                 _ints("first", first, cache.B, device))
    _check("medusa_kv_read",
           lib().medusa_kv_read(cache.handle, kv, r, k_scale, v_scale, _stream(stream)))


def kv4_attention(cache, kv, q, o, ws, tree_k=None, tree_v=None, mask=None, scale=0.0, k_scale=1.0,
                  v_scale=1.0, stream=None):
    """medusa_kv4_attention: q, o [B][n1][Hq][dh] (rows evenly spaced), tree_k, tree_v
    [B][n1][Hkv][dh] contiguous or None, mask int32 [n1][8] or None."""
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.B or shape[2] != cache.Hq or shape[3] != cache.dh or o.shape != shape:
        raise ValueError(f"q, o: [{cache.B}][n1][{cache.Hq}][{cache.dh}] is needed, got {tuple(shape)}, "
                         f"{tuple(o.shape)}")
    B, n1 = shape[0], shape[1]
    at = 0 if n1 == 1 else 1
    qs, os_ = q.stride(), o.stride()
    for s in (qs, os_):
        if s[3] != 1 or (at and B > 1 and s[0] != n1 * s[1]):
            raise ValueError(f"q, o: elements in order and evenly spaced rows are needed, got strides {s}")
    device = cache.device
    if q.get_device() != device or ws.get_device() != device:
        _elsewhere(cache, q, ws)
    _same(q, o, tree_k, tree_v)
    if not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor is needed")
    for t in (tree_k, tree_v):
        if t is not None and (t.shape != (B, n1, cache.Hkv, cache.dh) or not t.is_contiguous()):
            raise ValueError(f"tree_k, tree_v: contiguous [{B}][{n1}][{cache.Hkv}][{cache.dh}] is needed")
    a = KV4Query(q.data_ptr(), o.data_ptr(), _dtype(q), n1, qs[at], qs[2], os_[at], os_[2],
                 None if tree_k is None else tree_k.data_ptr(), None if tree_v is None else tree_v.data_ptr(),
                 _ints("mask", mask, 8 * n1, device), scale, k_scale, v_scale)
    _check("medusa_kv4_attention",
           lib().medusa_kv4_attention(cache.handle, kv, a, ws.data_ptr(), ws.numel() * ws.element_size(),
                                      _stream(stream)))
