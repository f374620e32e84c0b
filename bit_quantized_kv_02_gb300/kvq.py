"""Thin ctypes binding of libkvq (include/kvq.h): argument marshalling only.

Every step of the quantize / append / decode path runs in the CUDA kernels of
libkvq.so; PyTorch only provides device memory and the CUDA stream.  There is
no CPU fallback: if the library is missing the calls raise.

The functions keep the C names (``kvq_cache_bytes``, ``kvq_cache_create``,
``kvq_prefill_quantize``, ``kvq_append``, ``kvq_decode_attn``, ``kvq_export``,
...); ``KVQCache`` wraps a handle plus the torch buffer it lives in.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

PER_TOKEN, PER_CHANNEL = 0, 1
ASYM, SYM = 0, 1
F16, F32, BF16 = 0, 1, 2
WHOLE_VECTOR = -1
ROPE_PAIRS, ROPE_HALVES = 0, 1
ALL_LAYERS = -1

STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED", 3: "KVQ_ERR_CAPACITY",
          4: "KVQ_ERR_BUFFER_TOO_SMALL", 5: "KVQ_ERR_CUDA", 6: "KVQ_ERR_DEVICE_TIMEOUT",
          7: "KVQ_ERR_BAD_INDEX", 8: "KVQ_ERR_OUT_OF_PAGES"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")


class KVQError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))


class TensorCfg(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group", ctypes.c_int), ("axis", ctypes.c_int), ("mode", ctypes.c_int)]


class Config(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int), ("batch", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("k", TensorCfg), ("v", TensorCfg), ("meta_dtype", ctypes.c_int), ("max_splits", ctypes.c_int),
                ("recent_window", ctypes.c_int), ("rope_theta", ctypes.c_float)]


class Bytes(ctypes.Structure):
    _fields_ = [("tail", ctypes.c_double), ("packed", ctypes.c_double), ("metadata", ctypes.c_double),
                ("workspace", ctypes.c_double), ("total", ctypes.c_double), ("elements", ctypes.c_double),
                ("alloc", ctypes.c_size_t)]


class PagesConfig(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int), ("pages", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("k", TensorCfg), ("v", TensorCfg), ("dtype", ctypes.c_int)]


class _PagesBatch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("new_tokens", ctypes.c_int), ("max_new", ctypes.c_int),
                ("q_start", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("rows", ctypes.c_int), ("dim", ctypes.c_int), ("style", ctypes.c_int),
                ("positions", ctypes.c_void_p)]


class _Tree(ctypes.Structure):
    _fields_ = [("seen", ctypes.c_void_p), ("words", ctypes.c_int), ("positions", ctypes.c_void_p)]


class _ForkArgs(ctypes.Structure):
    _fields_ = [("rows_in", ctypes.c_int), ("rows_out", ctypes.c_int), ("parent", ctypes.c_void_p),
                ("table_in", ctypes.c_void_p), ("stride_in", ctypes.c_int64), ("lens_in", ctypes.c_void_p),
                ("refs_in", ctypes.c_void_p), ("table_out", ctypes.c_void_p), ("stride_out", ctypes.c_int64),
                ("lens_out", ctypes.c_void_p), ("refs_out", ctypes.c_void_p)]


class _GrowArgs(ctypes.Structure):
    _fields_ = [("sequences", ctypes.c_int), ("q_start", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("refs", ctypes.c_void_p),
                ("lens_out", ctypes.c_void_p)]


class _NormRopeArgs(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("k_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int)]


_lock = threading.Lock()
_lib = None

EXPORTED = ["kvq_cache_bytes", "kvq_cache_create", "kvq_cache_destroy", "kvq_prefill_quantize", "kvq_append",
            "kvq_decode_attn", "kvq_export", "kvq_cache_tcap", "kvq_get_lens", "kvq_decode_traffic",
            "kvq_device_status", "kvq_last_launches", "kvq_status_string", "kvq_last_error",
            "kvq_set_decode_plan", "kvq_refresh_lens", "kvq_decode_attn_static", "kvq_set_decode_kernel",
            "kvq_decode_kernel_specialized", "kvq_dequantize", "kvq_decode_attn_materialized",
            "kvq_append_decode_attn", "kvq_decode_cta_warps", "kvq_pages_bytes", "kvq_pages_create",
            "kvq_pages_destroy", "kvq_pages_append", "kvq_pages_attn", "kvq_pages_read", "kvq_pages_set_kernel",
            "kvq_pages_status", "kvq_pages_last_error", "kvq_qk_norm_rope", "kvq_pages_tree", "kvq_pages_tree_attn",
            "kvq_pages_cross_attn", "kvq_pages_keep", "kvq_pages_copy", "kvq_pages_fork", "kvq_pages_grow"]


def lib():
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkvq.so not built ({LIB_PATH}); run bit_quantized_kv_02_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
        L.kvq_cache_bytes.argtypes = [ctypes.POINTER(Config), P, ctypes.POINTER(Bytes)]
        L.kvq_cache_create.argtypes = [ctypes.POINTER(Config), P, ctypes.c_size_t, P, ctypes.POINTER(P)]
        L.kvq_cache_destroy.argtypes = [P]
        L.kvq_prefill_quantize.argtypes = [P, I, P, P, I, P, ctypes.c_int64, P]
        L.kvq_append.argtypes = [P, I, P, P, I, P]
        L.kvq_decode_attn.argtypes = [P, I, P, I, ctypes.c_float, P, P]
        L.kvq_append_decode_attn.argtypes = [P, I, P, P, I, P, I, ctypes.c_float, P, P]
        L.kvq_export.argtypes = [P, I, P, P, P, P, P, P, P, P]
        L.kvq_cache_tcap.argtypes = [P]
        L.kvq_cache_tcap.restype = I
        L.kvq_get_lens.argtypes = [P, I, P]
        L.kvq_decode_traffic.argtypes = [P, I, I, ctypes.POINTER(ctypes.c_double)]
        L.kvq_device_status.argtypes = [P, P]
        L.kvq_last_launches.argtypes = [P]
        L.kvq_last_launches.restype = I
        L.kvq_status_string.argtypes = [S]
        L.kvq_status_string.restype = ctypes.c_char_p
        L.kvq_decode_attn_static.argtypes = [P, I, P, I, ctypes.c_float, P, P]
        L.kvq_dequantize.argtypes = [P, I, P, P, P]
        L.kvq_decode_attn_materialized.argtypes = [P, I, P, P, P, I, ctypes.c_float, P, P]
        L.kvq_set_decode_plan.argtypes = [P, I]
        L.kvq_set_decode_kernel.argtypes = [P, I]
        L.kvq_decode_kernel_specialized.argtypes = [P]
        L.kvq_decode_kernel_specialized.restype = I
        L.kvq_decode_cta_warps.argtypes = [P, I]
        L.kvq_decode_cta_warps.restype = I
        L.kvq_refresh_lens.argtypes = [P, P]
        L.kvq_last_error.argtypes = [P]
        L.kvq_last_error.restype = ctypes.c_char_p
        PB, PR = ctypes.POINTER(_PagesBatch), ctypes.POINTER(_Rope)
        L.kvq_pages_bytes.argtypes = [ctypes.POINTER(PagesConfig), ctypes.POINTER(Bytes)]
        L.kvq_pages_create.argtypes = [ctypes.POINTER(PagesConfig), P, ctypes.c_size_t, P, ctypes.POINTER(P)]
        L.kvq_pages_destroy.argtypes = [P]
        L.kvq_pages_append.argtypes = [P, I, P, P, I, ctypes.c_int64, ctypes.c_int64, PB, PR, P]
        L.kvq_pages_attn.argtypes = [P, I, P, I, ctypes.c_int64, PB, ctypes.c_float, I, P, P]
        L.kvq_pages_read.argtypes = [P, I, PB, P, P, P]
        L.kvq_pages_tree.argtypes = [P, PB, P, I, P, P, P]
        L.kvq_pages_tree_attn.argtypes = [P, I, P, I, ctypes.c_int64, PB, ctypes.POINTER(_Tree), ctypes.c_float, I, P, P]
        L.kvq_pages_cross_attn.argtypes = [P, I, P, I, ctypes.c_int64, PB, ctypes.c_float, P, P]
        L.kvq_pages_keep.argtypes = [P, I, PB, P, P, P]
        L.kvq_pages_copy.argtypes = [P, I, P, P, I, P]
        L.kvq_pages_fork.argtypes = [P, ctypes.POINTER(_ForkArgs), P]
        L.kvq_pages_grow.argtypes = [P, ctypes.POINTER(_GrowArgs), P]
        L.kvq_pages_set_kernel.argtypes = [P, I]
        L.kvq_pages_status.argtypes = [P, P]
        L.kvq_pages_last_error.argtypes = [P]
        L.kvq_pages_last_error.restype = ctypes.c_char_p
        L.kvq_qk_norm_rope.argtypes = [ctypes.POINTER(_NormRopeArgs), PR, P]
        for name in ("kvq_pages_bytes", "kvq_pages_create", "kvq_pages_destroy", "kvq_pages_append", "kvq_pages_attn",
                     "kvq_pages_read", "kvq_pages_set_kernel", "kvq_pages_status", "kvq_qk_norm_rope"):
            getattr(L, name).restype = S
        for name in ("kvq_cache_bytes", "kvq_cache_create", "kvq_cache_destroy", "kvq_prefill_quantize",
                     "kvq_append", "kvq_decode_attn", "kvq_export", "kvq_get_lens", "kvq_decode_traffic",
                     "kvq_device_status", "kvq_set_decode_plan", "kvq_refresh_lens", "kvq_decode_attn_static",
                     "kvq_set_decode_kernel", "kvq_dequantize", "kvq_decode_attn_materialized"):
            getattr(L, name).restype = S
        _lib = L
        return L


def make_config(layers, batch, q_heads, kv_heads, head_dim, max_tokens, k, v, meta_dtype=F16, max_splits=0,
                recent_window=0, rope_theta=0.0):
    """k, v: (bits, group, axis, mode) tuples or dicts; recent_window: fp16 window
    of the newest tokens of both tensors (multiple of 16, 0 = none); rope_theta:
    base of the rotary embedding applied to the dequantized keys at decode (keys
    cached before RoPE; 0 = none)."""
    def tc(t):
        if isinstance(t, dict):
            return TensorCfg(t["bits"], t["group"], t["axis"], t.get("mode", ASYM))
        return TensorCfg(*t)
    return Config(layers, batch, q_heads, kv_heads, head_dim, max_tokens, tc(k), tc(v), meta_dtype, max_splits,
                  recent_window, float(rope_theta))


def _check(st: int, what: str, handle=None):
    if st != 0:
        detail = ""
        if handle is not None:
            detail = (lib().kvq_last_error(handle) or b"").decode()
        raise KVQError(st, what, detail)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (fp16 or fp32)")


# ------------------------------------------------------- C-named functions --

def kvq_cache_bytes(cfg: Config, lens=None) -> Bytes:
    out = Bytes()
    arr = None
    if lens is not None:
        arr = (ctypes.c_int32 * len(lens))(*[int(x) for x in lens])
    _check(lib().kvq_cache_bytes(ctypes.byref(cfg), arr, ctypes.byref(out)), "kvq_cache_bytes")
    return out


def kvq_status_string(status: int) -> str:
    return lib().kvq_status_string(status).decode()


class KVQCache:
    """A libkvq cache handle living in one torch uint8 device buffer."""

    def __init__(self, cfg: Config, device="cuda", stream=None):
        self.cfg = cfg
        self.bytes = kvq_cache_bytes(cfg)
        self.buffer = torch.empty(self.bytes.alloc, dtype=torch.uint8, device=device)
        h = ctypes.c_void_p()
        _check(lib().kvq_cache_create(ctypes.byref(cfg), _ptr(self.buffer), self.bytes.alloc, _stream(stream),
                                      ctypes.byref(h)), "kvq_cache_create")
        self.handle = h
        self.tcap = lib().kvq_cache_tcap(h)

    def close(self):
        if getattr(self, "handle", None):
            lib().kvq_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # C-named methods ---------------------------------------------------------
    def kvq_prefill_quantize(self, layer: int, k: torch.Tensor, v: torch.Tensor, lens, stream=None):
        """k, v: [batch][T][kv_heads][head_dim] contiguous fp16/fp32 on the device."""
        assert k.is_contiguous() and v.is_contiguous() and k.shape == v.shape and k.dtype == v.dtype
        arr = (ctypes.c_int32 * self.cfg.batch)(*[int(x) for x in lens])
        _check(lib().kvq_prefill_quantize(self.handle, layer, _ptr(k), _ptr(v), _dtype_code(k), arr, k.shape[1],
                                          _stream(stream)), "kvq_prefill_quantize", self.handle)

    def kvq_append(self, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        """k_new, v_new: [batch][kv_heads][head_dim] contiguous fp16/fp32 on the device."""
        assert k_new.is_contiguous() and v_new.is_contiguous() and k_new.dtype == v_new.dtype
        _check(lib().kvq_append(self.handle, layer, _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _stream(stream)),
               "kvq_append", self.handle)

    def kvq_decode_attn(self, layer: int, q: torch.Tensor, out: torch.Tensor | None = None, scale: float = 0.0,
                        stream=None) -> torch.Tensor:
        """q: [batch][q_heads][head_dim] fp16/fp32; returns fp32 [batch][q_heads][head_dim]."""
        assert q.is_contiguous()
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        _check(lib().kvq_decode_attn(self.handle, layer, _ptr(q), _dtype_code(q), float(scale), _ptr(out),
                                     _stream(stream)), "kvq_decode_attn", self.handle)
        return out

    def kvq_append_decode_attn(self, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                               out: torch.Tensor | None = None, scale: float = 0.0, stream=None) -> torch.Tensor:
        """kvq_append then kvq_decode_attn on `layer`, in one launch where the
        layout allows it: k_new, v_new [batch][kv_heads][head_dim]; q
        [batch][q_heads][head_dim]; returns fp32 [batch][q_heads][head_dim]."""
        assert k_new.is_contiguous() and v_new.is_contiguous() and k_new.dtype == v_new.dtype
        assert q.is_contiguous()
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        _check(lib().kvq_append_decode_attn(self.handle, layer, _ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                            _ptr(q), _dtype_code(q), float(scale), _ptr(out), _stream(stream)),
               "kvq_append_decode_attn", self.handle)
        return out

    def kvq_decode_attn_static(self, layer: int, q: torch.Tensor, out: torch.Tensor | None = None,
                               scale: float = 0.0, stream=None) -> torch.Tensor:
        """kvq_decode_attn with its scratch in the library's static device array
        (for callers that cannot provide device memory); same inputs and output."""
        assert q.is_contiguous()
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        _check(lib().kvq_decode_attn_static(self.handle, layer, _ptr(q), _dtype_code(q), float(scale), _ptr(out),
                                            _stream(stream)), "kvq_decode_attn_static", self.handle)
        return out

    def kvq_dequantize(self, layer: int, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                       stream=None):
        """Materialised baseline: fp16 K and V rows [batch][kv_heads][tcap][head_dim]
        of `layer` (rows past a sequence's length are left as they were)."""
        c = self.cfg
        shape = (c.batch, c.kv_heads, self.tcap, c.head_dim)
        if k_out is None:
            k_out = torch.zeros(shape, dtype=torch.float16, device=self.buffer.device)
        if v_out is None:
            v_out = torch.zeros(shape, dtype=torch.float16, device=self.buffer.device)
        assert k_out.shape == shape and v_out.shape == shape and k_out.dtype == torch.float16
        assert k_out.is_contiguous() and v_out.is_contiguous() and v_out.dtype == torch.float16
        _check(lib().kvq_dequantize(self.handle, layer, _ptr(k_out), _ptr(v_out), _stream(stream)), "kvq_dequantize",
               self.handle)
        return k_out, v_out

    def kvq_decode_attn_materialized(self, layer: int, k16: torch.Tensor, v16: torch.Tensor, q: torch.Tensor,
                                     out: torch.Tensor | None = None, scale: float = 0.0,
                                     stream=None) -> torch.Tensor:
        """Decode attention over rows from kvq_dequantize (the baseline the fused
        kvq_decode_attn is measured against); same query and output layout."""
        assert q.is_contiguous() and k16.is_contiguous() and v16.is_contiguous()
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        _check(lib().kvq_decode_attn_materialized(self.handle, layer, _ptr(k16), _ptr(v16), _ptr(q), _dtype_code(q),
                                                  float(scale), _ptr(out), _stream(stream)),
               "kvq_decode_attn_materialized", self.handle)
        return out

    def kvq_export(self, layer: int, stream=None) -> dict:
        c = self.cfg
        dev = self.buffer.device
        B, H, D, T = c.batch, c.kv_heads, c.head_dim, self.tcap

        def groups(t):
            if t.axis == PER_CHANNEL:
                return B * H * (T // t.group) * D
            if t.group == WHOLE_VECTOR:
                return B * T
            return B * H * T * (D // t.group)

        def rows(t):  # fp16 rows per (sequence, head): the unsealed tokens, row t - sealed
            if t.axis == PER_CHANNEL:
                return t.group + c.recent_window
            return c.recent_window + 16 if c.recent_window else 0

        out = {
            "codes_k": torch.zeros((B, H, T, D), dtype=torch.uint8, device=dev),
            "codes_v": torch.zeros((B, H, T, D), dtype=torch.uint8, device=dev),
            "meta_k": torch.zeros((groups(c.k), 2), dtype=torch.float32, device=dev),
            "meta_v": torch.zeros((groups(c.v), 2), dtype=torch.float32, device=dev),
            "tail_k": torch.zeros((B, H, rows(c.k), D), dtype=torch.int16, device=dev) if rows(c.k) else None,
            "tail_v": torch.zeros((B, H, rows(c.v), D), dtype=torch.int16, device=dev) if rows(c.v) else None,
            "lens": torch.zeros((B,), dtype=torch.int32, device=dev),
        }
        _check(lib().kvq_export(self.handle, layer, _ptr(out["codes_k"]), _ptr(out["codes_v"]), _ptr(out["meta_k"]),
                                _ptr(out["meta_v"]), _ptr(out["tail_k"]), _ptr(out["tail_v"]), _ptr(out["lens"]),
                                _stream(stream)), "kvq_export", self.handle)
        return out

    def kvq_get_lens(self, layer: int):
        arr = (ctypes.c_int32 * self.cfg.batch)()
        _check(lib().kvq_get_lens(self.handle, layer, arr), "kvq_get_lens", self.handle)
        return list(arr)

    def kvq_decode_traffic(self, layer: int, q_dtype: int = F16) -> float:
        v = ctypes.c_double()
        _check(lib().kvq_decode_traffic(self.handle, layer, q_dtype, ctypes.byref(v)), "kvq_decode_traffic")
        return v.value

    def kvq_device_status(self, stream=None) -> int:
        return lib().kvq_device_status(self.handle, _stream(stream))

    def kvq_set_decode_plan(self, plan_tokens: int):
        _check(lib().kvq_set_decode_plan(self.handle, int(plan_tokens)), "kvq_set_decode_plan")

    def kvq_set_decode_kernel(self, which: int):
        """0: compile-time specialisation when one matches (default); 1: generic kernel."""
        _check(lib().kvq_set_decode_kernel(self.handle, int(which)), "kvq_set_decode_kernel", self.handle)

    def kvq_decode_cta_warps(self, fused: bool = False) -> int:
        """Warps per CTA of the current decode (fused: decode-step) kernel; 0 if the step runs two kernels."""
        return int(lib().kvq_decode_cta_warps(self.handle, int(bool(fused))))

    def kvq_decode_kernel_specialized(self) -> bool:
        return bool(lib().kvq_decode_kernel_specialized(self.handle))

    def kvq_refresh_lens(self, stream=None):
        _check(lib().kvq_refresh_lens(self.handle, _stream(stream)), "kvq_refresh_lens", self.handle)

    def kvq_last_launches(self) -> int:
        return lib().kvq_last_launches(self.handle)


# -------------------------------------------------------------- paged cache --

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def make_pages_config(layers, pages, page_tokens, q_heads, kv_heads, head_dim, k=None, v=None,
                      dtype=F16) -> PagesConfig:
    """k, v: None for 16-bit values of `dtype` (F16 or BF16), or the (bits, group,
    axis, mode) of quantized pages: 8 or 4 bits, PER_TOKEN, ASYM."""
    def tc(t):
        return TensorCfg(16, 0, PER_TOKEN, ASYM) if t is None else TensorCfg(*t)
    return PagesConfig(layers, pages, page_tokens, q_heads, kv_heads, head_dim, tc(k), tc(v), dtype)


def kvq_pages_bytes(cfg: PagesConfig) -> Bytes:
    out = Bytes()
    _check(lib().kvq_pages_bytes(ctypes.byref(cfg), ctypes.byref(out)), "kvq_pages_bytes")
    return out


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(t, name, device=None):
    _need(isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.is_cuda, f"{name}: an int32 tensor on the GPU")
    _need(device is None or t.device == device, f"{name}: on another device")
    return t


def _row_stride(t, name, heads, head_dim, index):
    """Stride between tokens of [tokens][heads][head_dim] with heads and channels packed, on device `index`."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise ValueError(f"{name}: [tokens][{heads}][{head_dim}]")
    if t.get_device() != index:
        raise ValueError(f"{name}: on another device")
    if stride[2] != 1 or (stride[1] != head_dim and heads != 1):
        raise ValueError(f"{name}: heads and channels not contiguous")
    return stride[0] if shape[0] > 1 else heads * head_dim


# the current stream's handle without the stream object around it, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_device(index, stream, call, *args):
    """call(*args, stream handle) with device `index` current."""
    handle = stream.cuda_stream if stream is not None else _raw_stream(index)
    if _current_device() == index:
        return call(*args, handle)
    with torch.cuda.device(index):
        return call(*args, handle)


class PagesBatch:
    """The rows of paged-cache calls (kvq_pages_batch): q_start [batch + 1], lens
    [batch] and table [batch][pages] are int32 device tensors, read by the kernels
    when they run, so their contents may change between calls and graph replays.
    new_tokens: rows of k / v / q / out (at least q_start[batch]); max_new: the
    most new tokens of any sequence if known (speed only; a batch of one is taken
    to have as many)."""

    def __init__(self, q_start, lens, table, new_tokens: int, max_new: int = 0):
        _ints(q_start, "q_start")
        _ints(lens, "lens", q_start.device)
        _ints(table, "table", q_start.device)
        _need(lens.dim() == 1 and q_start.dim() == 1 and q_start.shape[0] == lens.shape[0] + 1,
              "q_start: one entry more than lens")
        _need(table.dim() == 2 and table.shape[0] == lens.shape[0] and table.shape[1] > 0, "table: [batch][pages]")
        _need(q_start.is_contiguous() and lens.is_contiguous() and table.is_contiguous(), "batch arrays are contiguous")
        self.q_start, self.lens, self.table = q_start, lens, table
        self.index = q_start.get_device()
        self.new_tokens = int(new_tokens)
        self.c = _PagesBatch(lens.shape[0], self.new_tokens, int(max_new), q_start.data_ptr(), lens.data_ptr(),
                             table.data_ptr(), table.shape[1])
        self.ref = ctypes.byref(self.c)


class PagesTree:
    """A step's trees of drafted tokens (kvq_tree): seen [new_tokens][words] int64, words 1
    to 4: bit j of word w says that the row sees new token 64 w + j of its sequence;
    positions [new_tokens] int32, or None (they are needed with a window only).  Device
    tensors, written by KVQPages.kvq_pages_tree or by the caller."""

    def __init__(self, seen, positions=None):
        _need(isinstance(seen, torch.Tensor) and seen.dtype == torch.int64 and seen.is_cuda and seen.dim() == 2 and
              seen.is_contiguous(), "seen: a contiguous int64 tensor [new_tokens][words] on the GPU")
        if positions is not None:
            _ints(positions, "positions", seen.device)
            _need(positions.dim() == 1 and positions.is_contiguous() and positions.shape[0] == seen.shape[0],
                  "positions: one a row of seen, contiguous")
        self.seen, self.positions = seen, positions
        self.index, self.rows = seen.get_device(), seen.shape[0]
        self.c = _Tree(seen.data_ptr(), seen.shape[1], positions.data_ptr() if positions is not None else None)
        self.ref = ctypes.byref(self.c)


class Rope:
    """Rotary embedding by a table of angles (kvq_rope): table [rows][dim / 2][2] fp32
    (cosine, sine); style ROPE_PAIRS (2i, 2i+1) or ROPE_HALVES (i, i + dim/2);
    positions: int32 [new_tokens] rows of the table, or None where the operator
    takes the position in the sequence."""

    def __init__(self, table, style: int = ROPE_PAIRS, positions=None):
        _need(isinstance(table, torch.Tensor) and table.is_cuda and table.dtype == torch.float32 and
              table.dim() == 3 and table.shape[2] == 2 and table.is_contiguous(), "table: fp32 [rows][dim / 2][2] on the GPU")
        if positions is not None:
            _ints(positions, "positions", table.device)
            _need(positions.dim() == 1 and positions.is_contiguous(), "positions: one a token, contiguous")
        self.table, self.positions = table, positions
        self.index = table.get_device()
        self.rows_given = positions.shape[0] if positions is not None else 0
        self.c = _Rope(table.data_ptr(), table.shape[0], 2 * table.shape[1], int(style),
                       positions.data_ptr() if positions is not None else None)
        self.ref = ctypes.byref(self.c)


def _new(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one), whose memory is that stream's."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _norm_side(x, out, w, name, tokens, head_dim, dtype, index, stream):
    """(out, heads, pointers, strides and weight) of one of kvq_qk_norm_rope's two sides."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens or x.dtype is not dtype:
        raise ValueError(f"{name}: queries and keys of the same tokens, type and head_dim")
    heads = shape[1]
    stride = _row_stride(x, name, heads, head_dim, index)
    if out is None:
        out = _new(shape, dtype, x.device, stream)
        out_stride = heads * head_dim
    else:
        out_stride = _row_stride(out, name + "_out", heads, head_dim, index)
        if out.shape[0] != tokens or out.dtype is not dtype:
            raise ValueError(f"{name}_out: of {name}'s shape and type")
    if w is None:
        return out, heads, x.data_ptr(), stride, out.data_ptr(), out_stride, None
    if w.dim() != 1 or w.numel() != head_dim or w.get_device() != index or w.stride(0) != 1:
        raise ValueError(f"{name}_weight: [{head_dim}], contiguous, on {name}'s device")
    if w.dtype is not dtype and w.dtype is not torch.float32:
        raise ValueError(f"{name}_weight: {dtype} or fp32")
    return out, heads, x.data_ptr(), stride, out.data_ptr(), out_stride, w.data_ptr()


def kvq_qk_norm_rope(q, k, q_weight=None, k_weight=None, eps: float = 1e-6, rope: Rope | None = None, q_out=None,
                     k_out=None, norm: bool = True, stream=None):
    """Norm of queries and keys per head and the rotary embedding, in one pass.

    q [tokens][q_heads][head_dim], k [tokens][kv_heads][head_dim] (either may be
    None): fp16, bf16 or fp32, slices of a joint projection included; weights
    [head_dim] of the same type or fp32, or None for ones; norm=False only
    rotates.  Returns (q_out, k_out), new tensors unless given (q and k themselves
    work)."""
    one = q if q is not None else k
    if not isinstance(one, torch.Tensor) or not one.is_cuda or one.dim() != 3:
        raise ValueError("q, k: [tokens][heads][head_dim] on the GPU")
    dtype = one.dtype
    code = weight_code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype} (fp16, bf16 or fp32)")
    tokens, _, d = one.shape
    index = one.get_device()
    qo = ko = qp = kp = qop = kop = qw = kw = ref = None
    qh = kh = qs = ks = qos = kos = 0
    if q is not None:
        qo, qh, qp, qs, qop, qos, qw = _norm_side(q, q_out, q_weight, "q", tokens, d, dtype, index, stream)
    if k is not None:
        ko, kh, kp, ks, kop, kos, kw = _norm_side(k, k_out, k_weight, "k", tokens, d, dtype, index, stream)
    if qw is not None:
        weight_code = _DTYPES[q_weight.dtype]
        if kw is not None and k_weight.dtype is not q_weight.dtype:
            raise ValueError("both weights have one type")
    elif kw is not None:
        weight_code = _DTYPES[k_weight.dtype]
    if rope is not None:
        ref = rope.ref
        if rope.index != index:
            raise ValueError("rope: on another device")
        if rope.positions is None or rope.rows_given < tokens:
            raise ValueError("rope: a position for every token")
    a = _NormRopeArgs(tokens, qh, kh, d, code, qp, kp, qs, ks, qop, kop, qos, kos, 1 if norm else 0, eps, qw, kw,
                      weight_code)
    st = _on_device(index, stream, (_lib or lib()).kvq_qk_norm_rope, ctypes.byref(a), ref)
    if st:
        raise KVQError(st, "kvq_qk_norm_rope")
    return qo, ko


class KVQPages:
    """A paged cache (kvq_pages_t) living in one torch uint8 device buffer."""

    def __init__(self, cfg: PagesConfig, device="cuda", stream=None):
        self.cfg = cfg
        self.bytes = kvq_pages_bytes(cfg)
        self.buffer = _new(self.bytes.alloc, torch.uint8, device, stream)  # (zero-filled on the same stream)
        self.device, self.index = self.buffer.device, self.buffer.get_device()
        self.dtype = torch.bfloat16 if cfg.dtype == BF16 else torch.float16
        self._kv, self._q = (cfg.kv_heads, cfg.head_dim), (cfg.q_heads, cfg.head_dim)
        self._lib = lib()
        h = ctypes.c_void_p()
        _check(_on_device(self.index, stream, lambda s: self._lib.kvq_pages_create(
            ctypes.byref(cfg), _ptr(self.buffer), self.bytes.alloc, s, ctypes.byref(h))), "kvq_pages_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            lib().kvq_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _fail(self, st, what):
        raise KVQError(st, what, (self._lib.kvq_pages_last_error(self.handle) or b"").decode())

    # C-named methods ---------------------------------------------------------
    def kvq_pages_append(self, layer: int, k: torch.Tensor, v: torch.Tensor, batch: PagesBatch,
                         rope: Rope | None = None, stream=None):
        """Store the new tokens of `batch`: k, v [new_tokens][kv_heads][head_dim]
        fp16, bf16 or fp32; the keys are turned by `rope` on the way."""
        index, n, dtype = self.index, batch.new_tokens, k.dtype
        ks = _row_stride(k, "k", *self._kv, index)
        vs = _row_stride(v, "v", *self._kv, index)
        code = _DTYPES.get(dtype)
        if code is None or v.dtype != dtype:
            raise ValueError("k, v: both fp16, bf16 or fp32")
        if k.shape[0] < n or v.shape[0] < n:
            raise ValueError("k, v: fewer rows than new tokens")
        if batch.index != index:
            raise ValueError("batch: on another device")
        ref = None
        if rope is not None:
            ref = rope.ref
            if rope.index != index:
                raise ValueError("rope: on another device")
            if rope.positions is not None and rope.rows_given < n:
                raise ValueError("rope: fewer positions than new tokens")
        r = _on_device(index, stream, self._lib.kvq_pages_append, self.handle, layer, k.data_ptr(), v.data_ptr(), code, ks,
                       vs, batch.ref, ref)
        if r:
            self._fail(r, "kvq_pages_append")

    def kvq_pages_attn(self, layer: int, q: torch.Tensor, batch: PagesBatch, out: torch.Tensor | None = None,
                       scale: float = 0.0, window: int = 0, stream=None) -> torch.Tensor:
        """Attention of the new tokens of `batch` over the pages: q [new_tokens][q_heads]
        [head_dim] fp16 or bf16; returns out of the same shape and type (rows behind
        the last sequence are left as they were; zeros in a new tensor).  A given out
        shares no memory with q."""
        return self._attend(self._lib.kvq_pages_attn, "kvq_pages_attn", layer, q, batch, out, stream, (scale, window))

    def kvq_pages_tree(self, parents: torch.Tensor, batch: PagesBatch, words: int = 1, tree: PagesTree | None = None,
                       stream=None) -> PagesTree:
        """The trees of a step's drafted tokens: parents [new_tokens] int32, each the index, among its
        sequence's new tokens, of the one that the token hangs on, or -1 for the past.  Returns the
        masks and positions (a given `tree` is written; new ones hold zeros in rows behind the last
        sequence).  A sequence has at most 64 * words new tokens.  One call serves all layers."""
        index, n = self.index, batch.new_tokens
        _ints(parents, "parents")
        _need(parents.dim() == 1 and parents.is_contiguous() and parents.shape[0] >= n, "parents: one a new token, contiguous")
        _need(parents.get_device() == index, "parents: on another device")
        _need(batch.index == index, "batch: on another device")
        if tree is None:
            shape = (parents.shape[0], int(words))
            with torch.cuda.stream(stream):  # (None: the current one)
                tree = PagesTree(torch.zeros(shape, dtype=torch.int64, device=self.device),
                                 torch.zeros(shape[:1], dtype=torch.int32, device=self.device))
        else:
            _need(tree.index == index, "tree: on another device")
            _need(tree.rows >= n, "tree: fewer rows than new tokens")
        c = tree.c
        r = _on_device(index, stream, self._lib.kvq_pages_tree, self.handle, batch.ref, parents.data_ptr(), c.words, c.seen,
                       c.positions)
        if r:
            self._fail(r, "kvq_pages_tree")
        return tree

    def kvq_pages_tree_attn(self, layer: int, q: torch.Tensor, batch: PagesBatch, tree: PagesTree,
                            out: torch.Tensor | None = None, scale: float = 0.0, window: int = 0, stream=None) -> torch.Tensor:
        """kvq_pages_attn where the new tokens form a tree: a row sees the past, and of the new tokens those
        that tree.seen names.  window: 0, or at least 64 * words."""
        if tree.index != self.index:
            raise ValueError("tree: on another device")
        if tree.rows < batch.new_tokens:
            raise ValueError("tree: fewer rows than new tokens")
        return self._attend(self._lib.kvq_pages_tree_attn, "kvq_pages_tree_attn", layer, q, batch, out, stream,
                            (tree.ref, scale, window))

    def kvq_pages_cross_attn(self, layer: int, q: torch.Tensor, batch: PagesBatch, out: torch.Tensor | None = None,
                             scale: float = 0.0, stream=None) -> torch.Tensor:
        """Attention of q's rows, as in kvq_pages_attn, over all tokens that the cache holds of their sequence:
        q_start deals out the queries, lens are those of the encoder's states, say, that were appended."""
        return self._attend(self._lib.kvq_pages_cross_attn, "kvq_pages_cross_attn", layer, q, batch, out, stream, (scale,))

    def kvq_pages_keep(self, keep: torch.Tensor, batch: PagesBatch, layer: int = ALL_LAYERS,
                       lens_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Keep the new tokens of `batch` that keep [new_tokens] (bool or uint8) marks, closing the gaps in
        the sequences' pages; returns the new lengths (int32 [batch])."""
        index = self.index
        _need(isinstance(keep, torch.Tensor) and keep.dtype in (torch.bool, torch.uint8) and keep.get_device() == index and
              keep.dim() == 1 and keep.is_contiguous(), "keep: bool or uint8 [new_tokens], contiguous, on the cache's device")
        _need(keep.shape[0] >= batch.new_tokens, "keep: fewer rows than new tokens")
        _need(batch.index == index, "batch: on another device")
        lens_out = self._ints_out(lens_out, "lens_out", batch.lens.shape, stream)
        r = _on_device(index, stream, self._lib.kvq_pages_keep, self.handle, layer, batch.ref, keep.data_ptr(),
                       lens_out.data_ptr())
        if r:
            self._fail(r, "kvq_pages_keep")
        return lens_out

    def kvq_pages_copy(self, src: torch.Tensor, dst: torch.Tensor, layer: int = ALL_LAYERS, stream=None):
        """Copy page src[i] to page dst[i] (int32 device tensors; negative entries skip the pair)."""
        index = self.index
        for t, name in ((src, "src"), (dst, "dst")):
            _ints(t, name)
            _need(t.dim() == 1 and t.is_contiguous() and t.get_device() == index, f"{name}: contiguous, on the cache's device")
        _need(src.shape == dst.shape, "src, dst: one page each a pair")
        r = _on_device(index, stream, self._lib.kvq_pages_copy, self.handle, layer, src.data_ptr(), dst.data_ptr(),
                       src.shape[0])
        if r:
            self._fail(r, "kvq_pages_copy")

    def _ints_out(self, t, name, shape, stream):
        """A given int32 output, checked, or a new one."""
        if t is None:
            return _new(shape, torch.int32, self.device, stream)
        _ints(t, name)
        _need(t.shape == shape and t.is_contiguous() and t.get_device() == self.index,
              f"{name}: contiguous, of {list(shape)}, on the cache's device")
        return t

    def _ints_in(self, t, name, shape):
        if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != self.index or not t.is_contiguous():
            raise ValueError(f"{name}: int32, contiguous, of {list(shape)}, on the cache's device")
        return t.data_ptr()

    def kvq_pages_fork(self, parent: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                       table_out: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
                       refs_out: torch.Tensor | None = None, stream=None):
        """A new table whose row b is row parent[b] (-1: empty) of `table` [rows][pages], sharing its pages, and
        the pages' reference counts with it: returns (table_out, lens_out, refs_out), new tensors unless given
        (refs itself works as refs_out).  All int32 device tensors; refs [pages]."""
        index, shape = self.index, table.shape
        if len(shape) != 2 or not shape[0] or not shape[1]:
            raise ValueError("table: [rows][pages]")
        if parent.dim() != 1 or not parent.shape[0]:
            raise ValueError("parent: one a new row")
        rows, n = shape[0], parent.shape[0]
        tp, pp = self._ints_in(table, "table", shape), self._ints_in(parent, "parent", (n,))
        lp, rp = self._ints_in(lens, "lens", (rows,)), self._ints_in(refs, "refs", (self.cfg.pages,))
        if table_out is not None:
            _need(table_out.dim() == 2 and table_out.shape[1] > 0, "table_out: [rows][pages]")
        width = table.shape[1] if table_out is None else table_out.shape[1]
        table_out = self._ints_out(table_out, "table_out", (n, width), stream)
        lens_out = self._ints_out(lens_out, "lens_out", (n,), stream)
        refs_out = self._ints_out(refs_out, "refs_out", (self.cfg.pages,), stream)
        a = _ForkArgs(rows, n, pp, tp, table.shape[1], lp, rp, table_out.data_ptr(), width, lens_out.data_ptr(),
                      refs_out.data_ptr())
        r = _on_device(index, stream, self._lib.kvq_pages_fork, self.handle, ctypes.byref(a))
        if r:
            self._fail(r, "kvq_pages_fork")
        return table_out, lens_out, refs_out

    def kvq_pages_grow(self, q_start: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                       lens_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Pages for q_start[b + 1] - q_start[b] new tokens behind the lens[b] of each row of `table`, dealt out
        where refs [pages] is zero, a shared last page copied; table and refs are changed in place.  Returns the
        lengths with the new tokens (lens itself works as lens_out); where pages ran out, -1 - lens[b]."""
        index, shape = self.index, table.shape
        if len(shape) != 2 or not shape[0] or not shape[1]:
            raise ValueError("table: [sequences][pages]")
        n = shape[0]
        tp, qp = self._ints_in(table, "table", shape), self._ints_in(q_start, "q_start", (n + 1,))
        lp, rp = self._ints_in(lens, "lens", (n,)), self._ints_in(refs, "refs", (self.cfg.pages,))
        lens_out = self._ints_out(lens_out, "lens_out", (n,), stream)
        a = _GrowArgs(n, qp, lp, tp, table.shape[1], rp, lens_out.data_ptr())
        r = _on_device(index, stream, self._lib.kvq_pages_grow, self.handle, ctypes.byref(a))
        if r:
            self._fail(r, "kvq_pages_grow")
        return lens_out

    def _attend(self, call, what, layer, q, batch, out, stream, tail):
        """call(handle, layer, q, type, stride, batch, *tail, out, stream) with the checks that attention calls share."""
        index, dtype = self.index, q.dtype
        qs = _row_stride(q, "q", *self._q, index)
        if dtype != torch.float16 and dtype != torch.bfloat16:
            raise ValueError("q: fp16 or bf16")
        if q.shape[0] < batch.new_tokens:
            raise ValueError("q: fewer rows than new tokens")
        if batch.index != index:
            raise ValueError("batch: on another device")
        if out is None:
            if stream is None:
                out = torch.zeros(q.shape, dtype=dtype, device=q.device)
            else:  # (as in _new; rows behind the last sequence are not written)
                with torch.cuda.stream(stream):
                    out = torch.zeros(q.shape, dtype=dtype, device=q.device)
        elif out.shape != q.shape or out.dtype != dtype or out.get_device() != index or not out.is_contiguous():
            raise ValueError("out: contiguous, of q's shape and type")
        r = _on_device(index, stream, call, self.handle, layer, q.data_ptr(), _DTYPES[dtype], qs, batch.ref, *tail,
                       out.data_ptr())
        if r:
            self._fail(r, what)
        return out

    def kvq_pages_read(self, layer: int, batch: PagesBatch, k_out: torch.Tensor | None = None,
                       v_out: torch.Tensor | None = None, stream=None):
        """What the pages hold for the new tokens of `batch`: (k, v), each [new_tokens]
        [kv_heads][head_dim] of the pages' type (fp16 for quantized pages); rows
        without a place are left as they were (new tensors are not cleared)."""
        index = self.index
        shape = (batch.new_tokens, *self._kv)
        if batch.index != index:
            raise ValueError("batch: on another device")
        if k_out is None:
            k_out = _new(shape, self.dtype, self.device, stream)
        elif k_out.shape != shape or k_out.dtype != self.dtype or k_out.get_device() != index or not k_out.is_contiguous():
            raise ValueError("k_out: contiguous [new_tokens][kv_heads][head_dim] of the pages' type")
        if v_out is None:
            v_out = _new(shape, self.dtype, self.device, stream)
        elif v_out.shape != shape or v_out.dtype != self.dtype or v_out.get_device() != index or not v_out.is_contiguous():
            raise ValueError("v_out: contiguous [new_tokens][kv_heads][head_dim] of the pages' type")
        r = _on_device(index, stream, self._lib.kvq_pages_read, self.handle, layer, batch.ref, k_out.data_ptr(),
                       v_out.data_ptr())
        if r:
            self._fail(r, "kvq_pages_read")
        return k_out, v_out

    def kvq_pages_set_kernel(self, which: int):
        """0: by the rows of each sequence (default); 1: the few-rows kernel; 2: the many-rows kernel."""
        _check(self._lib.kvq_pages_set_kernel(self.handle, int(which)), "kvq_pages_set_kernel")

    def kvq_pages_status(self, stream=None) -> int:
        """Synchronises and returns what kernels recorded since the last call (0: nothing): calls
        return before their kernels run, so a bad index or a wait that ran out shows only here.
        Of several the first in this order: 6 (a wait), 7 (an index), 8 (pages ran out), 7 for
        negative lengths alone; kvq_pages_last_error names all."""
        return _on_device(self.index, stream, self._lib.kvq_pages_status, self.handle)
