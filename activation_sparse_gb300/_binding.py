"""ctypes binding of ``libsi.so`` (declared in ``include/si.h``).

Argument marshalling only: torch tensors supply device pointers, the current
CUDA stream is passed through, status codes become exceptions. Every step of
the method runs in the library's CUDA kernels; there is no fallback. When the
library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes as C
import os

from . import _build

SI_OK, SI_ERR_INVALID_ARG, SI_ERR_CUDA, SI_ERR_OOM, SI_ERR_UNSUPPORTED, SI_ERR_DEVICE = range(6)
SI_DEVERR_WAIT_TIMEOUT, SI_DEVERR_COUNT, SI_DEVERR_RANGE, SI_DEVERR_CACHE = 1, 2, 4, 8

# every symbol include/si.h declares, with (restype, argtypes)
_vp, _i, _d, _ll, _u32p = C.c_void_p, C.c_int, C.c_double, C.c_longlong, C.POINTER(C.c_uint32)
_ip = C.POINTER(C.c_int)
SIGNATURES = {
    "si_last_error_string": (C.c_char_p, []),
    "si_abi_version": (_i, []),
    "si_count": (_ll, [_d, _ll]),
    "si_counts": (_i, [_i, _d, _d, _d, _ip, _ip, _ip, _ip]),
    "si_packed_bytes": (_ll, [_i, _i]),
    "si_sparse_layers": (_i, [_i, _i, _i, _vp, _ip]),
    "si_device_error": (_i, [_u32p, _i]),
    "si_profile_scores": (_i, [_vp, _vp, _i, _i, _vp, _i, _vp, _vp]),
    "si_merge_scores": (_i, [C.POINTER(_vp), C.POINTER(_ll), _i, _i, _vp, _vp]),
    "si_scores_save": (_i, [C.c_char_p, _vp, _i, _ll]),
    "si_scores_load": (_i, [C.c_char_p, _vp, _i, _ip, C.POINTER(_ll)]),
    "si_pack_loaded": (_i, [_vp, _vp, _vp, _i, _i, _vp, _vp, _d, _d, C.POINTER(_vp), _vp]),
    "si_layer_info": (_i, [_vp, _ip, _ip, _ip, _ip, _ip]),
    "si_layer_buffers": (_i, [_vp, C.POINTER(_vp), C.POINTER(_vp), C.POINTER(_vp)]),
    "si_layer_destroy": (_i, [_vp]),
    "si_select_dynamic": (_i, [_vp, _vp, _i, _i, _i, _d, _vp, _vp, _vp]),
    "si_prefill_absact": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "si_set_gemm_tile": (_i, [_i]),
    "si_layer_set_salience": (_i, [_vp, _i]),
    "si_layer_norms": (_i, [_vp, C.POINTER(_vp)]),
    "si_gemm_tile_for": (_i, [_i, _i, _ip]),
    "si_select_from_absact": (_i, [_vp, _vp, _i, _i, _i, _i, _d, _vp, _vp, _vp, _vp]),
    "si_decode_plan": (_i, [_vp, _vp, _i, _i, _vp]),
    "si_expand_clusters": (_i, [_vp, _vp, _i, _i, _vp, _ip, _vp]),
    "si_sparse_ffn_decode": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    "si_sparse_ffn_decode_residual": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    "si_sparse_ffn_decode_noalloc": (_i, [_vp, _i, _i, _vp, _i, _vp, _vp, _vp]),
    "si_stack_create": (_i, [C.POINTER(_vp), _i, C.POINTER(_vp)]),
    "si_stack_plan": (_i, [_vp, C.POINTER(_vp), _ip, _vp]),
    "si_sparse_ffn_decode_stack": (_i, [_vp, _vp, _vp, _vp]),
    "si_stack_destroy": (_i, [_vp]),
    "spax_encode": (_i, [_vp, _i, _i, _i, _i, C.POINTER(_vp), _vp]),
    "spax_layer_info": (_i, [_vp, _ip, _ip, _ip, _ip, _ip]),
    "spax_layer_buffers": (_i, [_vp, C.POINTER(_vp), C.POINTER(_vp), C.POINTER(_vp)]),
    "spax_layer_destroy": (_i, [_vp]),
    "spax_dense_act": (_i, [_vp, _vp, _i, _i, _vp, _vp, _vp]),
    "spax_tiered_down": (_i, [_vp, _vp, _d, _d, _vp, _vp, _vp, _vp]),
    "spax_ffn_decode": (_i, [_vp, _vp, _vp, _vp, _d, _d, _vp, _vp, _vp]),
    "spax_select_decode": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _d, _d, _vp, _vp, _vp]),
    "spax_gate_up": (_i, [_vp, _vp, _vp, _d, _d, _vp, _vp, _vp, _vp]),
    "spax_all_decode": (_i, [_vp, _vp, _vp, _vp, _d, _d, _d, _d, _vp, _vp, _vp]),
    "si_kv_create": (_i, [_vp, C.POINTER(_vp)]),
    "si_kv_destroy": (_i, [_vp]),
    "si_rope_create": (_i, [_i, C.POINTER(_d), C.POINTER(C.c_uint8), _i, _i, C.POINTER(_vp)]),
    "si_rope_destroy": (_i, [_vp]),
    "si_kv_append": (_i, [_vp, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "si_tree_attention": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, C.c_float, _vp, _vp, _vp]),
    "si_kv_accumulate": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, C.c_float, _vp, _vp]),
    "si_kv_evict": (_i, [_vp, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
}

SI_BF16, SI_FP16 = 0, 1


class KvDesc(C.Structure):
    """si_kv_desc of include/si.h."""
    _fields_ = [("dtype", _i), ("L", _i), ("B", _i), ("Hkv", _i), ("D", _i), ("cap", _i), ("n_slots", _ll),
                ("k", _vp), ("v", _vp), ("k_stride", _ll * 4), ("v_stride", _ll * 4),
                ("table", _vp), ("table_stride", _ll * 3), ("len", _vp), ("acc", _vp), ("acc_stride", _ll * 3)]

_lib = None


class SIError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("si error %d: %s" % (code, msg))
        self.code = code


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Loads libsi.so (building it first when absent or stale and nvcc exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise ImportError("libsi.so is not built; run __graft_entry__.build() first")
    L = C.CDLL(_build.LIB)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _check(rc):
    if rc != SI_OK:
        raise SIError(rc, _lib.si_last_error_string().decode())


# ------------------------------------------------------------------ helpers

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    torch = _torch()
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    return C.c_void_p(t.data_ptr())


_raw_stream = None


def _stream(stream=None):
    """The given stream's handle, or that of torch's current stream on the current device."""
    global _raw_stream
    if stream is not None:
        return C.c_void_p(stream.cuda_stream)
    if _raw_stream is None:
        cuda = _torch().cuda
        cuda.init()
        get, dev = (getattr(_torch()._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        # torch.cuda.current_stream() builds a stream object (4 us); the raw handle is all that is needed
        _raw_stream = (lambda: get(dev())) if get and dev else (lambda: cuda.current_stream().cuda_stream)
    return _raw_stream()


def _bf16(t, name):
    """bf16 tensors travel as their bit patterns: accept torch.bfloat16 or int16/uint16 views."""
    torch = _torch()
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise ValueError("%s must be bf16 (or its 16-bit pattern)" % name)
    return _ptr(t, None, name)


# ------------------------------------------------------------------ API


def si_count(ratio: float, n: int) -> int:
    return int(load().si_count(float(ratio), int(n)))


def si_counts(N, gamma, delta, phi):
    L = load()
    a, b, c, d = C.c_int(), C.c_int(), C.c_int(), C.c_int()
    _check(L.si_counts(int(N), float(gamma), float(delta), float(phi), C.byref(a), C.byref(b), C.byref(c),
                       C.byref(d)))
    return a.value, b.value, c.value, d.value


def si_packed_bytes(d, n_loaded) -> int:
    return int(load().si_packed_bytes(int(d), int(n_loaded)))


def si_device_error(clear: bool = True) -> int:
    L = load()
    v = C.c_uint32()
    _check(L.si_device_error(C.byref(v), 1 if clear else 0))
    return v.value


def si_sparse_layers(L: int, first: int = 5, last: int = -2):
    """Per-layer mask (numpy bool [L]) of the layers that run selection; the others stay dense."""
    import numpy as np
    out = np.zeros(max(int(L), 1), np.uint8)
    n = C.c_int(0)
    _check(load().si_sparse_layers(int(L), int(first), int(last), out.ctypes.data_as(C.c_void_p), C.byref(n)))
    return out[:int(L)].astype(bool)


def si_profile_scores(Wg, Wu, X, scores, stream=None):
    N, d = Wg.shape
    _check(load().si_profile_scores(_bf16(Wg, "Wg"), _bf16(Wu, "Wu"), d, N, _bf16(X, "X"), X.shape[0],
                                    _ptr(scores, _torch().float32, "scores"), _stream(stream)))
    return scores


def si_merge_scores(score_list, token_counts, out, stream=None):
    torch = _torch()
    ptrs = (C.c_void_p * len(score_list))(*[s.data_ptr() for s in score_list])
    for s in score_list:
        _ptr(s, torch.float32, "scores")
    toks = (C.c_longlong * len(score_list))(*[int(t) for t in token_counts])
    _check(load().si_merge_scores(ptrs, toks, len(score_list), out.shape[0], _ptr(out, torch.float32, "out"),
                                  _stream(stream)))
    return out


def si_scores_save(path, scores, token_count):
    """Writes a score file: `scores` (fp32 [N], on any device) and the token
    count they were summed over."""
    import numpy as np
    if hasattr(scores, "detach"):
        scores = scores.detach().to("cpu")
        scores = scores.numpy()
    h = np.ascontiguousarray(scores, dtype=np.float32).reshape(-1)
    _check(load().si_scores_save(os.fsencode(path), h.ctypes.data, int(h.size), int(token_count)))


def si_scores_load(path):
    """Reads a score file: (scores as a float32 numpy array [N], token count)."""
    import numpy as np
    n, t = C.c_int(), C.c_longlong()
    L = load()
    _check(L.si_scores_load(os.fsencode(path), None, 0, C.byref(n), C.byref(t)))
    out = np.empty(n.value, dtype=np.float32)
    _check(L.si_scores_load(os.fsencode(path), out.ctypes.data, int(out.size), C.byref(n), C.byref(t)))
    return out, t.value


class Layer:
    """A packed SelectInfer layer (owns the library handle)."""

    def __init__(self, handle):
        self._h = handle
        L = load()
        v = [C.c_int() for _ in range(5)]
        _check(L.si_layer_info(self._h, *[C.byref(x) for x in v]))
        self.d, self.N, self.n_loaded, self.n_static, self.n_pad = [x.value for x in v]

    @property
    def handle(self):
        return self._h

    def buffers(self):
        """(loaded_idx, is_static, packed) device pointers as ints."""
        a, b, c = C.c_void_p(), C.c_void_p(), C.c_void_p()
        _check(load().si_layer_buffers(self._h, C.byref(a), C.byref(b), C.byref(c)))
        return a.value, b.value, c.value

    def close(self):
        if self._h:
            load().si_layer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def si_pack_loaded(Wg, Wu, Wd, task_scores, model_scores, gamma, delta, stream=None) -> Layer:
    torch = _torch()
    N, d = Wg.shape
    h = C.c_void_p()
    _check(load().si_pack_loaded(_bf16(Wg, "Wg"), _bf16(Wu, "Wu"), _bf16(Wd, "Wd"), d, N,
                                 _ptr(task_scores, torch.float32, "task_scores"),
                                 _ptr(model_scores, torch.float32, "model_scores"), float(gamma), float(delta),
                                 C.byref(h), _stream(stream)))
    return Layer(h)


def si_select_dynamic(layer: Layer, X, T, B, alpha, phi, S, absact_out=None, stream=None):
    torch = _torch()
    _check(load().si_select_dynamic(layer.handle, _bf16(X, "X"), int(T), int(B), int(alpha), float(phi),
                                    _ptr(S, torch.int32, "S"), _ptr(absact_out, torch.float32, "absact_out"),
                                    _stream(stream)))
    return S


def si_layer_set_salience(layer: Layer, weight_aware: bool):
    """Prefill ranking key of this layer: |a| (False, default) or |a| * ||Wd[:, n]||_2 (True)."""
    _check(load().si_layer_set_salience(layer.handle, 1 if weight_aware else 0))


def si_layer_norms(layer: Layer) -> int:
    """Device pointer of the layer's fp32 [n_pad] down-column norms."""
    p = C.c_void_p()
    _check(load().si_layer_norms(layer.handle, C.byref(p)))
    return p.value


def si_set_gemm_tile(bnn: int):
    """Forces the activation GEMM's neuron-tile width (64, 80, 96, 112, 128) or, with 0, restores the per-launch choice."""
    _check(load().si_set_gemm_tile(int(bnn)))


def si_gemm_tile_for(M: int, N: int) -> int:
    """The neuron-tile width a GEMM launch over M token rows and N neurons would use now."""
    b = C.c_int(0)
    _check(load().si_gemm_tile_for(int(M), int(N), C.byref(b)))
    return b.value


def si_prefill_absact(layer: Layer, X, T, B, absact_out, stream=None):
    _check(load().si_prefill_absact(layer.handle, _bf16(X, "X"), int(T), int(B),
                                    _ptr(absact_out, _torch().float32, "absact_out"), _stream(stream)))
    return absact_out


def si_select_from_absact(layer: Layer, absA, T, B, alpha, phi, S, topmask=None, counts=None, stream=None):
    torch = _torch()
    u32 = torch.int32  # uint32 words travel in int32 tensors
    _check(load().si_select_from_absact(layer.handle, _ptr(absA, torch.float32, "absA"), absA.shape[1], int(T),
                                        int(B), int(alpha), float(phi), _ptr(S, torch.int32, "S"),
                                        _ptr(topmask, u32, "topmask"), _ptr(counts, u32, "counts"),
                                        _stream(stream)))
    return S


def si_expand_clusters(layer: Layer, S, n_sel, cluster, S_out, stream=None) -> int:
    """Whole clusters of `cluster` contiguous neurons around the selected positions S; returns len."""
    n = C.c_int(0)
    _check(load().si_expand_clusters(layer.handle, _ptr(S, _torch().int32, "S") if n_sel else None, int(n_sel),
                                     int(cluster), _ptr(S_out, _torch().int32, "S_out"), C.byref(n),
                                     _stream(stream)))
    return n.value


def si_decode_plan(layer: Layer, S, n_sel, B, stream=None):
    _check(load().si_decode_plan(layer.handle, _ptr(S, _torch().int32, "S"), int(n_sel), int(B), _stream(stream)))


def si_sparse_ffn_decode(layer: Layer, S, n_sel, B, x, y, stream=None):
    torch = _torch()
    _check(load().si_sparse_ffn_decode(layer.handle, _ptr(S, torch.int32, "S"), int(n_sel), int(B), _bf16(x, "x"),
                                       _ptr(y, torch.float32, "y"), _stream(stream)))
    return y


def si_sparse_ffn_decode_residual(layer: Layer, S, n_sel, B, x, y, stream=None):
    torch = _torch()
    _check(load().si_sparse_ffn_decode_residual(layer.handle, _ptr(S, torch.int32, "S"), int(n_sel), int(B),
                                                _bf16(x, "x"), _ptr(y, torch.float32, "y"), _stream(stream)))
    return y


def si_sparse_ffn_decode_noalloc(packed_ptr: int, n_records: int, d: int, S, n_sel, x, y, stream=None):
    """The no-allocation batch-1 decode; packed_ptr is a device address (int)."""
    torch = _torch()
    _check(load().si_sparse_ffn_decode_noalloc(C.c_void_p(packed_ptr), int(n_records), int(d),
                                               _ptr(S, torch.int32, "S"), int(n_sel), _bf16(x, "x"),
                                               _ptr(y, torch.float32, "y"), _stream(stream)))
    return y


class Stack:
    """A decode stack over packed layers (owns the library handle; the layers
    must outlive it, and it keeps references to them)."""

    def __init__(self, handle, layers):
        self._h = handle
        self.layers = list(layers)
        self.L = len(self.layers)
        self.d = self.layers[0].d

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load().si_stack_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def si_stack_create(layers) -> Stack:
    hs = (C.c_void_p * len(layers))(*[l.handle for l in layers])
    h = C.c_void_p()
    _check(load().si_stack_create(hs, len(layers), C.byref(h)))
    return Stack(h, layers)


def si_stack_plan(stack: Stack, S_list, n_sel_list, stream=None):
    """Copies each layer's computed set (device int32, ascending positions) into the stack."""
    torch = _torch()
    ptrs = []
    for S, n in zip(S_list, n_sel_list):
        ptrs.append(_ptr(S, torch.int32, "S").value if int(n) > 0 else None)
    arr = (C.c_void_p * stack.L)(*ptrs)
    ns = (C.c_int * stack.L)(*[int(n) for n in n_sel_list])
    _check(load().si_stack_plan(stack.handle, arr, ns, _stream(stream)))


def si_sparse_ffn_decode_stack(stack: Stack, h, x_out=None, stream=None):
    """One decode token through every layer of the stack: h (fp32 [d], read
    and written) is the residual stream; x_out (optional bf16 [L][d]) gets each
    layer's input."""
    torch = _torch()
    _check(load().si_sparse_ffn_decode_stack(stack.handle, _ptr(h, torch.float32, "h"),
                                             _bf16(x_out, "x_out") if x_out is not None else None,
                                             _stream(stream)))
    return h


class SpaxLayer:
    """An encoded SpAx down-projection (owns the library handle)."""

    def __init__(self, handle):
        self._h = handle
        v = [C.c_int() for _ in range(5)]
        _check(load().spax_layer_info(self._h, *[C.byref(x) for x in v]))
        self.d, self.N, self.bits, self.group, self.ngp = [x.value for x in v]

    @property
    def handle(self):
        return self._h

    def buffers(self):
        """(WdT, codes, params) device pointers as ints."""
        a, b, c = C.c_void_p(), C.c_void_p(), C.c_void_p()
        _check(load().spax_layer_buffers(self._h, C.byref(a), C.byref(b), C.byref(c)))
        return a.value, b.value, c.value

    def close(self):
        if self._h:
            load().spax_layer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def spax_encode(Wd, bits=4, group=128, stream=None) -> SpaxLayer:
    d, N = Wd.shape
    h = C.c_void_p()
    _check(load().spax_encode(_bf16(Wd, "Wd"), d, N, int(bits), int(group), C.byref(h), _stream(stream)))
    return SpaxLayer(h)


def spax_dense_act(Wg, Wu, x, a, stream=None):
    N, d = Wg.shape
    _check(load().spax_dense_act(_bf16(Wg, "Wg"), _bf16(Wu, "Wu"), d, N, _bf16(x, "x"),
                                 _ptr(a, _torch().float32, "a"), _stream(stream)))
    return a


def spax_tiered_down(layer: SpaxLayer, a, top_frac, mid_frac, y, top_idx=None, mid_idx=None, stream=None):
    torch = _torch()
    _check(load().spax_tiered_down(layer.handle, _ptr(a, torch.float32, "a"), float(top_frac), float(mid_frac),
                                   _ptr(y, torch.float32, "y"), _ptr(top_idx, torch.int32, "top_idx"),
                                   _ptr(mid_idx, torch.int32, "mid_idx"), _stream(stream)))
    return y


def spax_select_decode(layer: SpaxLayer, Wg, Wu, rows, x, top_frac, mid_frac, y, a_out=None, stream=None):
    """SpAx tiers inside a selected set: rows (device int32) are the neurons computed."""
    torch = _torch()
    n_rows = int(rows.numel()) if rows is not None else 0
    _check(load().spax_select_decode(layer.handle, _bf16(Wg, "Wg"), _bf16(Wu, "Wu"),
                                     _ptr(rows, torch.int32, "rows") if n_rows else None, n_rows, _bf16(x, "x"),
                                     float(top_frac), float(mid_frac), _ptr(y, torch.float32, "y"),
                                     _ptr(a_out, torch.float32, "a_out"), _stream(stream)))
    return y


def spax_ffn_decode(layer: SpaxLayer, Wg, Wu, x, top_frac, mid_frac, y, a_out=None, stream=None):
    torch = _torch()
    _check(load().spax_ffn_decode(layer.handle, _bf16(Wg, "Wg"), _bf16(Wu, "Wu"), _bf16(x, "x"), float(top_frac),
                                  float(mid_frac), _ptr(y, torch.float32, "y"),
                                  _ptr(a_out, torch.float32, "a_out"), _stream(stream)))
    return y


def spax_encode_rows(W, bits=4, group=128, stream=None) -> SpaxLayer:
    """Encodes a gate or up matrix W [N x d] for spax_gate_up: its columns
    (input channels) get the records, with groups along the N neurons."""
    N, d = W.shape
    h = C.c_void_p()
    _check(load().spax_encode(_bf16(W, "W"), N, d, int(bits), int(group), C.byref(h), _stream(stream)))
    return SpaxLayer(h)


def spax_gate_up(gate: SpaxLayer, up: SpaxLayer, x, top_frac, mid_frac, a, top_idx=None, mid_idx=None, stream=None):
    """a = silu(g) * u with g, u tiered over the input channels by |x|."""
    torch = _torch()
    _check(load().spax_gate_up(gate.handle, up.handle, _bf16(x, "x"), float(top_frac), float(mid_frac),
                               _ptr(a, torch.float32, "a"), _ptr(top_idx, torch.int32, "top_idx"),
                               _ptr(mid_idx, torch.int32, "mid_idx"), _stream(stream)))
    return a


def spax_all_decode(down: SpaxLayer, gate: SpaxLayer, up: SpaxLayer, x, in_top, in_mid, top_frac, mid_frac, y,
                    a_out=None, stream=None):
    """One SpAx-ALL FFN token: gate/up tiers by |x|, then the down tiers by |a|."""
    torch = _torch()
    _check(load().spax_all_decode(down.handle, gate.handle, up.handle, _bf16(x, "x"), float(in_top), float(in_mid),
                                  float(top_frac), float(mid_frac), _ptr(y, torch.float32, "y"),
                                  _ptr(a_out, torch.float32, "a_out"), _stream(stream)))
    return y


# ------------------------------------------------------------------ key/value cache


class Rope:
    """Rotary positions (owns the library handle): n_pairs pairs over n_axes axes."""

    def __init__(self, handle, n_pairs, n_axes):
        self._h, self.n_pairs, self.n_axes = handle, n_pairs, n_axes

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load().si_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def si_rope_create(D, base=10000.0, sections=None, interleaved=False, inv_freq=None, axis=None) -> Rope:
    """Rotary positions for heads of D elements.

    By default all D / 2 pairs turn, pair i by pos * base ** (-2 i / D).
    `sections` (pairs of each axis, in order; one section by default) says
    which axis of the positions a pair follows; `axis` (an axis index per
    pair) says it pair by pair. `inv_freq` (radians per position, one per
    pair) replaces the default frequencies, and fewer than D / 2 of them leave
    the elements past the pairs unrotated."""
    freq = [float(base) ** (-2.0 * i / D) for i in range(D // 2)] if inv_freq is None else [float(f) for f in inv_freq]
    n = len(freq)
    if axis is None:
        sections = [n] if sections is None else [int(c) for c in sections]
        if sum(sections) != n or min(sections) < 0:
            raise ValueError("sections must add up to the number of pairs (%d)" % n)
        axis, n_axes = [a for a, c in enumerate(sections) for _ in range(c)], len(sections)
    else:
        axis = [int(a) for a in axis]
        if len(axis) != n or min(axis) < 0 or max(axis) > 255:
            raise ValueError("axis needs an index for each of the %d pairs" % n)
        n_axes = max(axis) + 1
    if 2 * n > D:
        raise ValueError("%d pairs exceed D = %d" % (n, D))
    h = C.c_void_p()
    _check(load().si_rope_create(n, (C.c_double * n)(*freq), (C.c_uint8 * n)(*axis), n_axes, 1 if interleaved else 0,
                                 C.byref(h)))
    return Rope(h, n, n_axes)


class KV:
    """A key/value cache over the caller's tensors (owns the library handle
    and keeps references to the tensors)."""

    def __init__(self, handle, K, V, table, lens, acc):
        self._h = handle
        self.K, self.V, self.table, self.lens, self.acc = K, V, table, lens, acc
        self.L, self.B, self.Hkv, self.n_slots, self.D = K.shape
        self.cap = table.shape[3] if table is not None else self.n_slots
        self.dtype = K.dtype

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load().si_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _dev(t, dtype, name, shape=None, ndim=None):
    """A CUDA tensor of this type (and shape) whose last dimension is contiguous."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got %d" % (name, ndim, t.dim()))
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return t.data_ptr()


def _whole(t, dtype, name, shape):
    """The pointer of a contiguous CUDA tensor of this type and shape; None passes."""
    if t is None:
        return None
    # one look at what a decode step has right; _dev says what is wrong
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda):
        _dev(t, dtype, name, shape)
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


_stride_arrays = {}  # the C array of {sequence, token, head} strides, by a tensor's strides


def _strides(t, name):
    a = _stride_arrays.get(t.stride())
    if a is None:
        if t.stride(-1) != 1 and t.shape[-1] != 1:
            raise ValueError("the last dimension of %s must be contiguous" % name)
        if len(_stride_arrays) >= 1024:
            _stride_arrays.clear()
        a = _stride_arrays[t.stride()] = (_ll * 3)(*t.stride()[:3])
    return a


def _rows(t, kv, name, T):
    """(pointer, strides, heads) of a [B][T][heads][D] tensor of the cache's type."""
    if t.dim() != 4 or not (t.dtype is kv.dtype and t.is_cuda):
        _dev(t, kv.dtype, name, None, 4)
    b, n, heads, d = t.shape
    if b != kv.B or n != T or d != kv.D:
        raise ValueError("%s must have shape (%d, %d, heads, %d), got %s" % (name, kv.B, T, kv.D, tuple(t.shape)))
    return t.data_ptr(), _strides(t, name), heads


def si_kv_create(K, V, table, lens, acc=None) -> KV:
    """A cache over K, V [L][B][Hkv][n_slots][D] (bf16 or fp16), table int32
    [L][B][Hkv][cap] (None: entry i is slot i), lens int32 [L][B] and acc fp32
    [L][B][Hkv][n_slots] (None: no eviction)."""
    torch = _torch()
    if K.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("K must be bf16 or fp16")
    d = KvDesc()
    d.dtype = SI_FP16 if K.dtype == torch.float16 else SI_BF16
    d.k = _dev(K, K.dtype, "K", None, 5)
    d.v = _dev(V, K.dtype, "V", K.shape)
    d.L, d.B, d.Hkv, d.n_slots, d.D = K.shape
    d.k_stride[:], d.v_stride[:] = K.stride()[:4], V.stride()[:4]
    d.cap = min(d.n_slots, 2 ** 31 - 1)
    if table is not None:
        d.table = _dev(table, torch.int32, "table", None, 4)
        if table.shape[:3] != K.shape[:3]:
            raise ValueError("table must have shape (L, B, Hkv, cap), got %s" % (tuple(table.shape),))
        d.cap = table.shape[3]
        d.table_stride[:] = table.stride()[:3]
    d.len = _whole(lens, torch.int32, "lens", K.shape[:2])
    if acc is not None:
        d.acc = _dev(acc, torch.float32, "acc", K.shape[:4])
        d.acc_stride[:] = acc.stride()[:3]
    h = C.c_void_p()
    _check(load().si_kv_create(C.byref(d), C.byref(h)))
    return KV(h, K, V, table, lens, acc)


def si_kv_append(kv: KV, rope: Rope, q, k, v, pos, q_out, layer=0, stream=None):
    """Rotates q [B][T][Hq][D] into q_out and k [B][T][Hkv][D] into the
    cache, with v, at the first T free slots of every list. pos int32
    [B][T][n_axes]. q and q_out may be None."""
    torch = _torch()
    T = k.shape[1]
    kp, ks, hk = _rows(k, kv, "k", T)
    vp, vs, hv = _rows(v, kv, "v", T)
    if hk != kv.Hkv or hv != kv.Hkv:
        raise ValueError("k and v must have %d heads" % kv.Hkv)
    qp, qs, hq, op = None, None, 0, None
    if q is not None:
        qp, qs, hq = _rows(q, kv, "q", T)
        op = _whole(q_out, kv.dtype, "q_out", q.shape)
    rc = _lib.si_kv_append(kv._h, layer, rope._h, T, hq, qp, qs, kp, ks, vp, vs,
                           _whole(pos, torch.int32, "pos", (kv.B, T, rope.n_axes)), op, _stream(stream))
    if rc:
        _check(rc)
    return q_out


def si_tree_attention(kv: KV, q, out, mask=None, lse=None, scale=None, layer=0, stream=None):
    """Attention of the T new tokens q [B][T][Hq][D] over the cache and each
    other. mask int64 [B][T]: bit j of a node's word says that it sees node j
    (0: padding; None: a chain). out as q, contiguous; lse fp32 [B][T][Hq]
    (optional). scale defaults to D ** -0.5."""
    torch = _torch()
    B, T = kv.B, q.shape[1]
    qp, qs, hq = _rows(q, kv, "q", T)
    rc = _lib.si_tree_attention(kv._h, layer, T, hq, qp, qs, _whole(mask, torch.int64, "mask", (B, T)),
                                kv.D ** -0.5 if scale is None else scale, _whole(out, kv.dtype, "out", q.shape),
                                _whole(lse, torch.float32, "lse", (B, T, hq)), _stream(stream))
    if rc:
        _check(rc)
    return out


def si_kv_accumulate(kv: KV, q, lse, mask=None, rows=None, scale=None, acc_out=None, layer=0, stream=None):
    """Adds to every key's accumulated weight what it received from the
    counted nodes of q (rows int64 [B], bit t counts node t; None: all), with
    the lse of si_tree_attention. acc_out fp32 [B][Hkv][n_slots] with the
    cache's strides, or [1][B][Hkv][n_slots] (None: the cache's acc)."""
    torch = _torch()
    B, T = kv.B, q.shape[1]
    qp, qs, hq = _rows(q, kv, "q", T)
    ap = None
    if acc_out is not None:
        ap = _dev(acc_out, torch.float32, "acc_out")
        if kv.acc is None or acc_out.shape[-3:] != kv.acc.shape[1:] or acc_out.numel() != B * kv.Hkv * kv.n_slots \
                or any(n > 1 and x != y for n, x, y in zip(acc_out.shape[-3:], acc_out.stride()[-3:], kv.acc.stride()[1:])):
            raise ValueError("acc_out must have the shape and strides of one layer of the cache's acc")
    rc = _lib.si_kv_accumulate(kv._h, layer, T, hq, qp, qs, _whole(lse, torch.float32, "lse", (B, T, hq)),
                               _whole(mask, torch.int64, "mask", (B, T)), _whole(rows, torch.int64, "rows", (B,)),
                               kv.D ** -0.5 if scale is None else scale, ap, _stream(stream))
    if rc:
        _check(rc)


def si_kv_evict(kv: KV, T, budget, sinks=0, recent=0, path=None, n_path=None, table_out=None, len_out=None,
                layer=None, stream=None):
    """Takes the accepted ones of the T new nodes into the lists and drops the
    keys with the least accumulated weight beyond `budget` (0: none), but for
    the first `sinks` and the last `recent`. path int32 [B][T] and n_path int32
    [B] name the accepted nodes (path None: the first n_path; n_path None:
    all). All layers, or one. In place unless table_out and len_out are given."""
    torch = _torch()
    B = kv.B
    rc = _lib.si_kv_evict(kv._h, -1 if layer is None else layer, T, _whole(path, torch.int32, "path", (B, T)),
                          _whole(n_path, torch.int32, "n_path", (B,)), budget, sinks, recent,
                          _whole(table_out, torch.int32, "table_out", (kv.L, B, kv.Hkv, kv.cap)),
                          _whole(len_out, torch.int32, "len_out", (kv.L, B)), _stream(stream))
    if rc:
        _check(rc)
