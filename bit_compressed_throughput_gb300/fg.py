"""ctypes binding of libfg (include/fg.h): argument marshalling only.

Every function here checks the status the C call returns and raises ``FgError`` on
failure.  Tensors are torch CUDA tensors (device memory and streams only); nothing is
computed in Python.  Importing this module loads ``libfg.so`` from this package and
raises ``ImportError`` if it has not been built -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional


class _LazyTorch:
    """Stands for torch until its first use, which imports it and puts it in this object's place:
    the library's host-side calls work where torch is not installed."""

    def __getattr__(self, name):
        import torch as module
        globals()["torch"] = module
        return getattr(module, name)


torch = _LazyTorch()

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfg.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libfg.so is not built ({LIB_PATH}); run "
                      "`python -c 'import __graft_entry__ as g; g.build()'` first")
lib = C.CDLL(LIB_PATH)

FG_OK, FG_ERR_ARG, FG_ERR_SHAPE, FG_ERR_WORKSPACE = 0, -1, -2, -3
FG_ERR_CUDA, FG_ERR_ARCH, FG_ERR_CAPACITY, FG_ERR_TIMEOUT = -4, -5, -6, -7
FG_EPI_NONE, FG_EPI_RELU, FG_EPI_RESIDUAL = 0, 1, 2
KINDS = ["q4g64_quantize", "q4g64_dequant", "q4_dequant_gemm_tc", "gemm_splitk_reduce",
         "q4kv_append", "q4kv_decode_attn", "decode_attn_combine", "prefill_attn", "layernorm",
         "q4_dequant_gemm_stream", "q4kv_decode_attn_topk", "q4_dequant_gemm_pair",
         "gemm_f16w_pair", "q4kv_read", "q4kv_decode_attn_window", "prefill_attn_window", "rope",
         "q4kv_attn_paged", "q4kv_attn_weights", "q4kv_evict"]
K_QUANT, K_DEQUANT, K_GEMM, K_GEMM_REDUCE, K_KV_APPEND, K_DECODE_ATTN, K_DECODE_COMBINE, \
    K_PREFILL_ATTN, K_LAYERNORM, K_GEMM_STREAM, K_DECODE_ATTN_TOPK, K_GEMM_PAIR, \
    K_GEMM_PAIR_F16W, K_KV_READ, K_DECODE_ATTN_WINDOW, K_PREFILL_ATTN_WINDOW, K_ROPE, \
    K_ATTN_PAGED, K_ATTN_WEIGHTS, K_KV_EVICT = range(20)


class fg_q4mat(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("ab", C.c_void_p), ("K", C.c_int64), ("N", C.c_int64)]


class fg_kvcache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_ab", C.c_void_p),
                ("v_ab", C.c_void_p), ("B", C.c_int32), ("cap", C.c_int32), ("h", C.c_int32),
                ("H", C.c_int32)]


class fg_kvpages(C.Structure):
    _fields_ = [("blocks", C.c_void_p), ("pages", C.c_int32), ("page", C.c_int32),
                ("h", C.c_int32), ("H", C.c_int32)]


class fg_rope_rows(C.Structure):
    _fields_ = [("angles", C.c_void_p), ("pos", C.c_void_p), ("positions", C.c_int32),
                ("rot", C.c_int32), ("interleaved", C.c_int32)]


class fg_dims(C.Structure):
    _fields_ = [("h", C.c_int32), ("H", C.c_int32), ("d", C.c_int32), ("f", C.c_int32),
                ("ln_eps", C.c_float)]


class fg_layer(C.Structure):
    _fields_ = [("wqkv", fg_q4mat), ("wo", fg_q4mat), ("w1", fg_q4mat), ("w2", fg_q4mat),
                ("bqkv", C.c_void_p), ("bo", C.c_void_p), ("b1", C.c_void_p), ("b2", C.c_void_p),
                ("ln1_g", C.c_void_p), ("ln1_b", C.c_void_p), ("ln2_g", C.c_void_p),
                ("ln2_b", C.c_void_p)]


_P, _I64, _I32, _F, _SZ = C.c_void_p, C.c_int64, C.c_int32, C.c_float, C.c_size_t
_SIGS = {
    "fg_quantize_g64": ([_P, _I64, _I64, _P, _P, _P], C.c_int),
    "fg_dequant_g64": ([_P, _P, _I64, _I64, _P, _P], C.c_int),
    "fg_dequant_gemm_q4": ([_P, _I64, C.POINTER(fg_q4mat), _P, C.c_int, _P, _P, _P, _SZ, _P],
                           C.c_int),
    "fg_gemm_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "fg_dequant_gemm_q4_kv": ([_P, _I64, C.POINTER(fg_q4mat), _P, _P, C.POINTER(fg_kvcache),
                               _I32, _I32, _P, _SZ, _P], C.c_int),
    "fg_dequant_gemm_q4_ln": ([_P, _I64, C.POINTER(fg_q4mat), _P, C.c_int, _P, _P, _P, _P, _F,
                               _P, _P, _SZ, _P], C.c_int),
    "fg_kv_append_q4": ([_P, _P, _I64, _I32, _I32, C.POINTER(fg_kvcache), _P], C.c_int),
    "fg_decode_attn_q4kv": ([_P, _I64, C.POINTER(fg_kvcache), _I32, _F, _P, _P, _SZ, _P],
                            C.c_int),
    "fg_decode_attn_workspace_bytes": ([C.POINTER(fg_kvcache), _I32], _SZ),
    "fg_decode_attn_q4kv_static": ([_P, _I64, C.POINTER(fg_kvcache), _I32, _F, _P, _P], C.c_int),
    "fg_decode_attn_q4kv_topk": ([_P, _I64, C.POINTER(fg_kvcache), _I32, _I32, _F, _P, _P, _P,
                                  _SZ, _P], C.c_int),
    "fg_decode_attn_topk_workspace_bytes": ([C.POINTER(fg_kvcache), _I32], _SZ),
    "fg_prefill_attn": ([_P, _I32, _I32, _I32, _I32, _F, _P, _P], C.c_int),
    "fg_kv_append_q4_ragged": ([_P, _P, _I64, _I32, _P, _P, C.POINTER(fg_kvcache), _P], C.c_int),
    "fg_kv_read_q4_ragged": ([C.POINTER(fg_kvcache), _P, _P, _I32, _P, _P, _I64, _P], C.c_int),
    "fg_decode_attn_q4kv_window": ([_P, _I64, _I32, C.POINTER(fg_kvcache), _P, _I32, _I32, _F, _P,
                                    _I64, _P, _SZ, _P], C.c_int),
    "fg_decode_attn_window_workspace_bytes": ([C.POINTER(fg_kvcache), _I32], _SZ),
    "fg_prefill_attn_window": ([_P, _I64, _I32, _P, _P, _P, _I64, _I32, _P, _I32, _I32, _I32, _I32,
                                _I32, _I32, _F, _P, _I64, _P], C.c_int),
    "fg_rope_table": ([_P, _I32, _I32, C.c_double, C.c_double, _I32, C.c_double, C.c_double,
                       C.c_double, _P], C.c_int),
    "fg_rope": ([_P, _I64, _I32, _I32, _I32, _P, _I32, C.POINTER(fg_rope_rows), _I32, _P, _I64, _P],
                C.c_int),
    "fg_kv_append_q4_paged": ([_P, _P, _I64, _I32, _P, _P, C.POINTER(fg_rope_rows),
                               C.POINTER(fg_kvpages), _P, _I64, _I32, _P], C.c_int),
    "fg_kv_read_q4_paged": ([C.POINTER(fg_kvpages), _P, _I64, _I32, _P, _P, _I32, _P, _P, _I64,
                             _P], C.c_int),
    "fg_attn_paged_workspace_bytes": ([C.POINTER(fg_kvpages), _I32, _I32], _SZ),
    "fg_attn_q4kv_paged": ([_P, _I64, _I32, _P, _I32, _I32, C.POINTER(fg_kvpages), _P, _I64, _P,
                            _I32, _I32, _I32, _F, _P, _I64, _P, _P, _SZ, _P], C.c_int),
    "fg_attn_weights_q4_paged": ([_P, _I64, _I32, _P, _I32, _I32, C.POINTER(fg_kvpages), _P, _I64,
                                  _P, _I32, _I32, _I32, _F, _P, _P, _P, _I64, _P], C.c_int),
    "fg_kv_evict_q4_paged": ([C.POINTER(fg_kvpages), _P, _I64, _I32, _P, _P, _I64, _I32, _I32, _P,
                              _I64, _P, _P, _P, _P], C.c_int),
    "fg_layernorm": ([_P, _I64, _I32, _P, _P, _F, _P, _P], C.c_int),
    "fg_layer_prefill": ([C.POINTER(fg_dims), C.POINTER(fg_layer), C.POINTER(fg_kvcache), _P, _P,
                          _I32, _I32, _I32, _P, _SZ, _P], C.c_int),
    "fg_layer_decode": ([C.POINTER(fg_dims), C.POINTER(fg_layer), C.POINTER(fg_kvcache), _P, _P,
                         _I32, _I32, _I32, _P, _SZ, _P], C.c_int),
    "fg_workspace_bytes": ([C.POINTER(fg_dims), _I32, _I32, _I32], _SZ),
    "fg_layer_workspace_bytes": ([C.POINTER(fg_dims), _I32, _I32, _I32], _SZ),
    "fg_status_string": ([C.c_int], C.c_char_p),
    "fg_last_error": ([], C.c_char_p),
    "fg_check_device_error": ([_P], C.c_int),
    "fg_prof_enable": ([C.c_int], C.c_int),
    "fg_prof_reset": ([], C.c_int),
    "fg_prof_query": ([C.c_int, C.POINTER(C.c_int64), C.POINTER(C.c_double),
                       C.POINTER(C.c_double)], C.c_int),
    "fg_kernel_name": ([C.c_int], C.c_char_p),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class FgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib.fg_status_string(status).decode()
        detail = lib.fg_last_error().decode()
        super().__init__(f"{fn}: {msg} ({status})" + (f": {detail}" if detail else ""))
        self.status = status


def _check(fn: str, status: int):
    if status != FG_OK:
        raise FgError(fn, status)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    # the handle of torch.cuda.current_stream(), without building a Stream object each call (0.3
    # instead of 2.9 us of a call's host time; torch 2.9 and 2.11 have it)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


# ----------------------------------------------------------------------------- containers


class Q4Weight:
    """A 4-bit weight W[K][N] on the device: ``codes`` uint8 [K][N/2], ``ab`` int32
    [K][N/64] (a in the low 16 bits, b in the high 16 bits)."""

    def __init__(self, codes, ab, K: int, N: int):
        self.codes, self.ab, self.K, self.N = codes, ab, int(K), int(N)

    @classmethod
    def from_fp16(cls, w, stream=None) -> "Q4Weight":
        K, N = w.shape
        codes = torch.empty((K, N // 2), dtype=torch.uint8, device=w.device)
        ab = torch.empty((K, N // 64), dtype=torch.int32, device=w.device)
        fg_quantize_g64(w, codes, ab, stream)
        return cls(codes, ab, K, N)

    def struct(self) -> fg_q4mat:
        return fg_q4mat(_ptr(self.codes), _ptr(self.ab), self.K, self.N)


class KVCacheQ4:
    """One layer's 4-bit KV cache: codes [B][H][cap][d/2] uint8, ab [B][H][cap][d/64]
    int32, for K and V.  ``cap`` is rounded up to a multiple of 16 positions."""

    def __init__(self, B: int, cap: int, h: int, H: int, device="cuda"):
        cap = (int(cap) + 15) // 16 * 16
        d = h // H
        self.B, self.cap, self.h, self.H, self.d = B, cap, h, H, d
        self.k_codes = torch.zeros((B, H, cap, d // 2), dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_ab = torch.zeros((B, H, cap, d // 64), dtype=torch.int32, device=device)
        self.v_ab = torch.zeros_like(self.k_ab)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_fits", False)

    def check(self):
        """ValueError unless the four tensors have the shapes that B, cap, h and H say, on one
        device.  Done once after an attribute was set; the ragged and windowed calls ask for it."""
        if self._fits:
            return
        if self.H <= 0 or self.h != self.H * self.d or self.d % 64:
            raise ValueError(f"cache: h = {self.h}, H = {self.H} and d = {self.d} do not fit")
        device = self.k_codes.device
        for name, dtype, width in (("k_codes", torch.uint8, self.d // 2),
                                   ("v_codes", torch.uint8, self.d // 2),
                                   ("k_ab", torch.int32, self.d // 64),
                                   ("v_ab", torch.int32, self.d // 64)):
            t, shape = getattr(self, name), (self.B, self.H, self.cap, width)
            if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
                raise ValueError(f"cache.{name}: contiguous {dtype} {shape} expected, got {t.dtype} "
                                 f"{tuple(t.shape)}")
            if t.device != device:
                raise ValueError(f"cache.{name} on {t.device}, cache.k_codes on {device}")
        object.__setattr__(self, "_fits", True)

    def struct(self) -> fg_kvcache:
        return fg_kvcache(_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_ab),
                          _ptr(self.v_ab), self.B, self.cap, self.h, self.H)


class KVPagesQ4:
    """One layer's 4-bit KV cache in pages of ``page`` positions (a power of two, 16 .. 1024):
    ``blocks`` uint8 [pages][H][page*9*d/8], per page and head K codes [page][d/2], K statistics
    [page][d/64] (int32), V codes, V statistics.  Which pages a sequence has is the caller's
    affair: calls take a page table, int32 [nseq][n] on the device.  ``blocks`` may be replaced (a
    grown or moved pool); the other attributes follow from it and ``d``."""

    def __init__(self, pages: int, page: int, h: int, H: int, device="cuda"):
        self._set(torch.zeros((pages, H, page * 9 * (h // H) // 8), dtype=torch.uint8,
                              device=device), h // H)
        if self.page != page or self.h != h:
            raise ValueError(f"pages of {page} positions with h = {h} and H = {H} do not fit")

    @classmethod
    def of(cls, blocks, d: int) -> "KVPagesQ4":
        """The cache that a tensor of blocks holds, heads of ``d`` channels."""
        self = cls.__new__(cls)
        self._set(blocks, d)
        return self

    def _set(self, blocks, d: int):
        if d not in (64, 128) or blocks.dim() != 3 or blocks.dtype is not torch.uint8 or \
                not blocks.is_contiguous() or blocks.shape[2] % (9 * d // 8):
            raise ValueError(f"blocks: contiguous uint8 [pages][H][page*9*d/8] expected, got "
                             f"{blocks.dtype} {tuple(blocks.shape)} for d = {d}")
        (pages, H), page = blocks.shape[:2], blocks.shape[2] * 8 // (9 * d)
        if page < 16 or page > 1024 or page & (page - 1):
            raise ValueError(f"pages of {page} positions: a power of two, 16 .. 1024, expected")
        self.__dict__.update(blocks=blocks, d=d, pages=pages, H=H, page=page, h=H * d,
                             _ptr=_ptr(blocks), _numel=blocks.numel(),
                             _struct=fg_kvpages(_ptr(blocks), pages, page, H * d, H))

    def __setattr__(self, name, value):
        if name in ("d", "H", "h", "page", "pages"):
            raise AttributeError(f"{name} follows from the blocks: set those")
        if name == "blocks":
            self._set(value, self.d)
        else:
            object.__setattr__(self, name, value)

    def parts(self):
        """Views of the blocks: K codes [pages][H][page][d/2] and statistics [..][page][d/64] (fp16
        pairs a, b in a last dimension), V codes and statistics."""
        nc, na = self.page * self.d // 2, self.page * self.d // 16
        out = []
        for at in (0, nc + na):
            out.append(self.blocks[..., at:at + nc].unflatten(-1, (self.page, self.d // 2)))
            out.append(self.blocks[..., at + nc:at + nc + na].view(torch.float16)
                       .unflatten(-1, (self.page, self.d // 64, 2)))
        return out

    def struct(self) -> fg_kvpages:
        t = self.blocks
        if t.data_ptr() != self._ptr or t.numel() != self._numel:    # resized in place
            self._set(t, self.d)
        return self._struct


class LayerQ4:
    """One decoder layer's device parameters (4-bit weights, fp16 vectors)."""

    def __init__(self, h: int, H: int, f: int, wqkv: Q4Weight, wo: Q4Weight,
                 w1: Optional[Q4Weight], w2: Optional[Q4Weight], vec: dict, ln_eps=1e-5):
        self.h, self.H, self.d, self.f, self.ln_eps = h, H, h // H, f, ln_eps
        self.wqkv, self.wo, self.w1, self.w2, self.vec = wqkv, wo, w1, w2, vec

    @classmethod
    def from_fp16(cls, params: dict, H: int, ln_eps=1e-5, device="cuda", stream=None):
        """Quantise fp16 parameters (numpy or torch, W[K][N] layout) on the device."""
        def dev(a):
            t = a if isinstance(a, torch.Tensor) else torch.from_numpy(a)
            return t.to(device=device, dtype=torch.float16).contiguous()

        h = params["wo"].shape[0]
        f = params["w1"].shape[1] if "w1" in params else 0
        wq = Q4Weight.from_fp16(dev(params["wqkv"]), stream)
        wo = Q4Weight.from_fp16(dev(params["wo"]), stream)
        w1 = Q4Weight.from_fp16(dev(params["w1"]), stream) if f else None
        w2 = Q4Weight.from_fp16(dev(params["w2"]), stream) if f else None
        vec = {k: dev(v) for k, v in params.items() if k not in ("wqkv", "wo", "w1", "w2")}
        return cls(h, H, f, wq, wo, w1, w2, vec, ln_eps)

    def dims(self) -> fg_dims:
        return fg_dims(self.h, self.H, self.d, self.f, self.ln_eps)

    def struct(self) -> fg_layer:
        z = fg_q4mat(None, None, 0, 0)
        v = self.vec
        return fg_layer(self.wqkv.struct(), self.wo.struct(),
                        self.w1.struct() if self.w1 else z, self.w2.struct() if self.w2 else z,
                        _ptr(v.get("bqkv")), _ptr(v.get("bo")), _ptr(v.get("b1")),
                        _ptr(v.get("b2")), _ptr(v["ln1_g"]), _ptr(v["ln1_b"]),
                        _ptr(v.get("ln2_g")), _ptr(v.get("ln2_b")))


# ----------------------------------------------------------------------------- calls


def fg_quantize_g64(x, codes, ab, stream=None):
    rows, cols = x.shape
    _check("fg_quantize_g64", lib.fg_quantize_g64(_ptr(x), rows, cols, _ptr(codes), _ptr(ab),
                                                  _stream(stream)))


def fg_dequant_g64(codes, ab, rows: int, cols: int, y, stream=None):
    _check("fg_dequant_g64", lib.fg_dequant_g64(_ptr(codes), _ptr(ab), rows, cols, _ptr(y),
                                                _stream(stream)))


def fg_gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib.fg_gemm_workspace_bytes(M, K, N))


def fg_dequant_gemm_q4(X, W: Q4Weight, bias, epilogue: int, residual, Y, ws=None, stream=None):
    M = X.shape[0]
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = W.struct()
    _check("fg_dequant_gemm_q4",
           lib.fg_dequant_gemm_q4(_ptr(X), M, C.byref(st), _ptr(bias), epilogue, _ptr(residual),
                                  _ptr(Y), _ptr(ws), wsb, _stream(stream)))


def fg_dequant_gemm_q4_kv(X, W: Q4Weight, bias, Y, cache: KVCacheQ4, T: int, pos: int, ws=None,
                          stream=None):
    M = X.shape[0]
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st, kst = W.struct(), cache.struct()
    _check("fg_dequant_gemm_q4_kv",
           lib.fg_dequant_gemm_q4_kv(_ptr(X), M, C.byref(st), _ptr(bias), _ptr(Y), C.byref(kst),
                                     T, pos, _ptr(ws), wsb, _stream(stream)))


def fg_dequant_gemm_q4_ln(X, W: Q4Weight, bias, epilogue: int, residual, Y, gamma, beta,
                          eps: float, Y_ln, ws=None, stream=None):
    M = X.shape[0]
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    st = W.struct()
    _check("fg_dequant_gemm_q4_ln",
           lib.fg_dequant_gemm_q4_ln(_ptr(X), M, C.byref(st), _ptr(bias), epilogue, _ptr(residual),
                                     _ptr(Y), _ptr(gamma), _ptr(beta), eps, _ptr(Y_ln), _ptr(ws),
                                     wsb, _stream(stream)))


def fg_kv_append_q4(k_new, v_new, row_stride: int, T: int, pos: int, cache: KVCacheQ4,
                    stream=None):
    st = cache.struct()
    _check("fg_kv_append_q4", lib.fg_kv_append_q4(_ptr(k_new), _ptr(v_new), row_stride, T, pos,
                                                  C.byref(st), _stream(stream)))


def fg_decode_attn_workspace_bytes(cache: KVCacheQ4, length: int) -> int:
    st = cache.struct()
    return int(lib.fg_decode_attn_workspace_bytes(C.byref(st), length))


def fg_decode_attn_q4kv(q, q_stride: int, cache: KVCacheQ4, length: int, scale: float, out,
                        ws=None, stream=None):
    st = cache.struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check("fg_decode_attn_q4kv",
           lib.fg_decode_attn_q4kv(_ptr(q), q_stride, C.byref(st), length, scale, _ptr(out),
                                   _ptr(ws), wsb, _stream(stream)))


def fg_decode_attn_topk_workspace_bytes(cache: KVCacheQ4, length: int) -> int:
    st = cache.struct()
    return int(lib.fg_decode_attn_topk_workspace_bytes(C.byref(st), length))


def fg_decode_attn_q4kv_topk(q, q_stride: int, cache: KVCacheQ4, length: int, k: int,
                             scale: float, out, ws, sel=None, stream=None):
    """Top-K sparse decode attention: softmax over all positions' scores, values of the k
    highest-scoring positions only; ``sel`` (optional int32 [B][H][k]) receives them."""
    st = cache.struct()
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check("fg_decode_attn_q4kv_topk",
           lib.fg_decode_attn_q4kv_topk(_ptr(q), q_stride, C.byref(st), length, k, scale,
                                        _ptr(out), _ptr(sel), _ptr(ws), wsb, _stream(stream)))


DECODE_ATTN_STATIC_SCRATCH_BYTES = 4 << 20


def fg_decode_attn_q4kv_static(q, q_stride: int, cache: KVCacheQ4, length: int, scale: float,
                               out, stream=None):
    """Decode attention for callers that cannot allocate: the split scratch is the
    library's own static device array (4 MiB), so no workspace is passed."""
    st = cache.struct()
    _check("fg_decode_attn_q4kv_static",
           lib.fg_decode_attn_q4kv_static(_ptr(q), q_stride, C.byref(st), length, scale,
                                          _ptr(out), _stream(stream)))


def fg_prefill_attn(qkv, nseq: int, s: int, H: int, d: int, scale: float, out, stream=None):
    _check("fg_prefill_attn", lib.fg_prefill_attn(_ptr(qkv), nseq, s, H, d, scale, _ptr(out),
                                                  _stream(stream)))


# The ragged calls take their row counts and strides from the tensors, and the kernels rely on
# them, so these are checked here (ValueError) before they become bare pointers.


def _rows(name: str, t, width: int):
    """(rows, row stride) of a 2-D fp16 tensor of rows of `width` contiguous values."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width or stride[1] != 1 or t.dtype is not torch.float16:
        raise ValueError(f"{name}: fp16 [rows][{width}] with contiguous rows expected, got "
                         f"{t.dtype} {tuple(shape)} with strides {stride}")
    # the stride of a dimension of one row (or none) is arbitrary and never used
    return shape[0], (stride[0] if shape[0] > 1 else (width + 7) // 8 * 8)


def _extents(name: str, t, n: int):
    if t.shape != (n,) or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 [{n}] expected, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _window(window: int, sinks: int):
    # what does not fit 32 bits would reach the library as another number
    if not (-1 << 31) <= window < 1 << 31 or not (-1 << 31) <= sinks < 1 << 31:
        raise ValueError(f"window and sinks are 32-bit integers, got {window} and {sinks}")


def _stream_for(stream, *tensors) -> int:
    """The handle to launch on, for tensors that are all on the device that the call launches on:
    the current one, and the stream's."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{here}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(here)
    if stream.device.index != here:
        raise ValueError(f"stream on {stream.device}, but the current device is cuda:{here}")
    return stream.cuda_stream


def fg_kv_append_q4_ragged(k_new, v_new, row_off, pos, cache: KVCacheQ4, stream=None):
    """Rows row_off[b] .. row_off[b+1]-1 of ``k_new`` and ``v_new`` (fp16 [rows][h], one row
    stride) quantised into positions pos[b] .. of sequence b; ``row_off`` int32 [B+1] and ``pos``
    int32 [B] on the device."""
    rows, stride = _rows("k_new", k_new, cache.h)
    if _rows("v_new", v_new, cache.h) != (rows, stride):
        raise ValueError("k_new and v_new differ in rows or row stride")
    _extents("row_off", row_off, cache.B + 1)
    _extents("pos", pos, cache.B)
    cache.check()
    handle = _stream_for(stream, k_new, v_new, row_off, pos, cache.k_codes)
    st = cache.struct()
    _check("fg_kv_append_q4_ragged",
           lib.fg_kv_append_q4_ragged(_ptr(k_new), _ptr(v_new), stride, rows, _ptr(row_off),
                                      _ptr(pos), C.byref(st), handle))


def fg_kv_read_q4_ragged(cache: KVCacheQ4, row_off, pos, k_out, v_out, stream=None):
    """Positions pos[b] .. of sequence b restored to fp16 rows row_off[b] .. row_off[b+1]-1 of
    ``k_out`` and ``v_out`` (fp16 [rows][h], one row stride; either may be None)."""
    outs = [_rows(n, t, cache.h) for n, t in (("k_out", k_out), ("v_out", v_out)) if t is not None]
    if not outs or outs[0] != outs[-1]:
        raise ValueError("k_out and v_out differ in rows or row stride, or both are None")
    rows, stride = outs[0]
    _extents("row_off", row_off, cache.B + 1)
    _extents("pos", pos, cache.B)
    cache.check()
    handle = _stream_for(stream, k_out, v_out, row_off, pos, cache.k_codes)
    st = cache.struct()
    _check("fg_kv_read_q4_ragged",
           lib.fg_kv_read_q4_ragged(C.byref(st), _ptr(row_off), _ptr(pos), rows, _ptr(k_out),
                                    _ptr(v_out), stride, handle))


def fg_decode_attn_window_workspace_bytes(cache: KVCacheQ4, Hq: int) -> int:
    st = cache.struct()
    return int(lib.fg_decode_attn_window_workspace_bytes(C.byref(st), Hq))


def fg_decode_attn_q4kv_window(q, Hq: int, cache: KVCacheQ4, lens, scale: float, out, ws=None,
                               window: int = 0, sinks: int = 0, stream=None):
    """Decode attention of the newest position of every sequence (``lens`` int32 [B] on the
    device) over its last ``window`` positions (0: all) and its first ``sinks``; ``q`` and ``out``
    fp16 [B][Hq*d], Hq a multiple of the cache's heads."""
    _window(window, sinks)
    nq, q_stride = _rows("q", q, Hq * cache.d)
    no, o_stride = _rows("out", out, Hq * cache.d)
    if nq != cache.B or no != cache.B:
        raise ValueError(f"q and out need {cache.B} rows, got {nq} and {no}")
    _extents("lens", lens, cache.B)
    cache.check()
    handle = _stream_for(stream, q, out, lens, ws, cache.k_codes)
    st = cache.struct()
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor expected")
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check("fg_decode_attn_q4kv_window",
           lib.fg_decode_attn_q4kv_window(_ptr(q), q_stride, Hq, C.byref(st), _ptr(lens), window,
                                          sinks, scale, _ptr(out), o_stride, _ptr(ws), wsb,
                                          handle))


def fg_prefill_attn_window(q, q_off, k, v, kv_off, Hq: int, Hkv: int, scale: float, out,
                           window: int = 0, sinks: int = 0, stream=None):
    """Attention of the newest positions of every sequence over its fp16 K/V rows: ``q`` and
    ``out`` [q_rows][Hq*d], ``k`` and ``v`` [kv_rows][Hkv*d] with one row stride, ``q_off`` and
    ``kv_off`` int32 [nseq+1] on the device; window and sinks as in
    ``fg_decode_attn_q4kv_window``."""
    _window(window, sinks)
    if Hq <= 0 or Hkv <= 0 or q.dim() != 2 or q.shape[1] % Hq:
        raise ValueError(f"q: [rows][Hq*d] expected, got {tuple(q.shape)} for {Hq} heads")
    d = q.shape[1] // Hq
    q_rows, q_stride = _rows("q", q, Hq * d)
    o_rows, o_stride = _rows("out", out, Hq * d)
    kv_rows, kv_stride = _rows("k", k, Hkv * d)
    if _rows("v", v, Hkv * d) != (kv_rows, kv_stride) or o_rows != q_rows:
        raise ValueError("k and v, or q and out, differ in rows, or k and v in row stride")
    nseq = q_off.shape[0] - 1
    _extents("q_off", q_off, nseq + 1)
    _extents("kv_off", kv_off, nseq + 1)
    handle = _stream_for(stream, q, out, k, v, q_off, kv_off)
    _check("fg_prefill_attn_window",
           lib.fg_prefill_attn_window(_ptr(q), q_stride, q_rows, _ptr(q_off), _ptr(k), _ptr(v),
                                      kv_stride, kv_rows, _ptr(kv_off), nseq, Hq, Hkv, d, window,
                                      sinks, scale, _ptr(out), o_stride, handle))


def _table(name: str, t):
    """(sequences, entries each) of a page table."""
    if t.dim() != 2 or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 [sequences][pages] expected, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.shape


def _angles(t):
    """(positions, rotated channels) of a table of angles."""
    if t.dim() != 3 or t.shape[2] != 2 or t.dtype is not torch.float32 or not t.is_contiguous():
        raise ValueError(f"angles: contiguous fp32 [positions][rot/2][2] expected, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.shape[0], 2 * t.shape[1]


def fg_rope_table(angles, base: float = 10000.0, factor: float = 1.0, original: int = 0,
                  low: float = 1.0, high: float = 4.0, gain: float = 1.0, stream=None):
    """Fills ``angles`` (fp32 [positions][rot/2][2]) with gain * (cos, sin) of every position's
    angles; ``factor`` stretches them for contexts longer than ``original`` positions (0: all of
    them, see include/fg.h)."""
    positions, rot = _angles(angles)
    _check("fg_rope_table",
           lib.fg_rope_table(_ptr(angles), positions, rot, base, factor, original, low, high, gain,
                             _stream_for(stream, angles)))


def fg_rope(x, d: int, row_off, pos, angles, y, interleaved: bool = False, transpose: bool = False,
            stream=None):
    """Rotary positions: rows row_off[b] .. row_off[b+1]-1 of ``x`` (fp16 [rows][heads*d]) turned as
    positions pos[b] .. into ``y`` (may be ``x``); ``transpose``: the gradient's (and, with a gain
    of 1, the inverse) turn."""
    if d <= 0 or x.dim() != 2 or x.shape[1] % d:
        raise ValueError(f"x: [rows][heads*{d}] expected, got {tuple(x.shape)}")
    rows, x_stride = _rows("x", x, x.shape[1])
    y_rows, y_stride = _rows("y", y, x.shape[1])
    if y_rows != rows:
        raise ValueError(f"x has {rows} rows, y {y_rows}")
    positions, rot = _angles(angles)
    nseq = pos.shape[0]
    _extents("row_off", row_off, nseq + 1)
    _extents("pos", pos, nseq)
    handle = _stream_for(stream, x, y, row_off, pos, angles)
    st = fg_rope_rows(_ptr(angles), _ptr(pos), positions, rot, int(interleaved))
    _check("fg_rope", lib.fg_rope(_ptr(x), x_stride, rows, x.shape[1] // d, d, _ptr(row_off), nseq,
                                  C.byref(st), int(transpose), _ptr(y), y_stride, handle))


def fg_kv_append_q4_paged(k_new, v_new, row_off, pos, pages: KVPagesQ4, table, angles=None,
                          rope_pos=None, interleaved: bool = False, stream=None):
    """Rows row_off[b] .. row_off[b+1]-1 of ``k_new`` and ``v_new`` (fp16 [rows][h], one row stride)
    quantised into positions pos[b] .. of sequence b's pages (``table`` int32 [nseq][n]).  With
    ``angles`` K is turned first, as positions rope_pos[b] .. (default: pos[b] ..)."""
    rows, stride = _rows("k_new", k_new, pages.h)
    if _rows("v_new", v_new, pages.h) != (rows, stride):
        raise ValueError("k_new and v_new differ in rows or row stride")
    nseq, n = _table("table", table)
    _extents("row_off", row_off, nseq + 1)
    _extents("pos", pos, nseq)
    rope = None
    if angles is not None:
        positions, rot = _angles(angles)
        if rope_pos is not None:
            _extents("rope_pos", rope_pos, nseq)
        rope = C.byref(fg_rope_rows(_ptr(angles), _ptr(rope_pos), positions, rot,
                                    int(interleaved)))
    elif rope_pos is not None:
        raise ValueError("rope_pos without angles")
    handle = _stream_for(stream, k_new, v_new, row_off, pos, table, angles, rope_pos, pages.blocks)
    _check("fg_kv_append_q4_paged",
           lib.fg_kv_append_q4_paged(_ptr(k_new), _ptr(v_new), stride, rows, _ptr(row_off),
                                     _ptr(pos), rope, C.byref(pages.struct()), _ptr(table), n, nseq,
                                     handle))


def fg_kv_read_q4_paged(pages: KVPagesQ4, table, row_off, pos, k_out, v_out, stream=None):
    """Positions pos[b] .. of sequence b's pages restored to fp16 rows row_off[b] .. row_off[b+1]-1
    of ``k_out`` and ``v_out`` (fp16 [rows][h], one row stride; either may be None)."""
    outs = [_rows(n, t, pages.h) for n, t in (("k_out", k_out), ("v_out", v_out)) if t is not None]
    if not outs or outs[0] != outs[-1]:
        raise ValueError("k_out and v_out differ in rows or row stride, or both are None")
    rows, stride = outs[0]
    nseq, n = _table("table", table)
    _extents("row_off", row_off, nseq + 1)
    _extents("pos", pos, nseq)
    handle = _stream_for(stream, k_out, v_out, row_off, pos, table, pages.blocks)
    _check("fg_kv_read_q4_paged",
           lib.fg_kv_read_q4_paged(C.byref(pages.struct()), _ptr(table), n, nseq, _ptr(row_off),
                                   _ptr(pos), rows, _ptr(k_out), _ptr(v_out), stride, handle))


def fg_attn_paged_workspace_bytes(pages: KVPagesQ4, Hq: int, max_q: int) -> int:
    return int(lib.fg_attn_paged_workspace_bytes(C.byref(pages.struct()), Hq, max_q))


def _paged_queries(q, q_off, Hq: int, pages: KVPagesQ4, table, lens, max_q, window, sinks):
    """What the two paged attention calls say of their queries: (rows, row stride, max_q, sequences,
    page table entries)."""
    _window(window, sinks)
    rows, stride = _rows("q", q, Hq * pages.d)
    nseq, n = _table("table", table)
    _extents("q_off", q_off, nseq + 1)
    _extents("lens", lens, nseq)
    return rows, stride, rows if max_q is None else max_q, nseq, n


def _scores(name: str, t, shape):
    if t.shape != shape or t.dtype is not torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous fp32 {tuple(shape)} expected, got {t.dtype} "
                         f"{tuple(t.shape)}")


def fg_attn_q4kv_paged(q, q_off, Hq: int, pages: KVPagesQ4, table, lens, scale: float, out, ws,
                       max_q: Optional[int] = None, window: int = 0, sinks: int = 0, lse=None,
                       stream=None):
    """Attention of the newest tokens of every sequence (rows q_off[b] .. q_off[b+1]-1 of ``q`` and
    ``out``, fp16 [rows][Hq*d]; at most ``max_q`` each, default all rows) over its ``lens[b]``
    cached positions; ``lse`` (optional fp32 [rows][Hq]) receives the scores' log-sum-exp; window
    and sinks as in ``fg_decode_attn_q4kv_window``."""
    rows, q_stride, max_q, nseq, n = _paged_queries(q, q_off, Hq, pages, table, lens, max_q, window,
                                                    sinks)
    o_rows, o_stride = _rows("out", out, Hq * pages.d)
    if o_rows != rows:
        raise ValueError(f"q has {rows} rows, out {o_rows}")
    if lse is not None:
        _scores("lse", lse, (rows, Hq))
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor expected")
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    handle = _stream_for(stream, q, out, q_off, table, lens, lse, ws, pages.blocks)
    _check("fg_attn_q4kv_paged",
           lib.fg_attn_q4kv_paged(_ptr(q), q_stride, rows, _ptr(q_off), max_q, Hq,
                                  C.byref(pages.struct()), _ptr(table), n, _ptr(lens), nseq, window,
                                  sinks, scale, _ptr(out), o_stride, _ptr(lse), _ptr(ws), wsb,
                                  handle))


def fg_attn_weights_q4_paged(q, q_off, Hq: int, pages: KVPagesQ4, table, lens, scale: float, lse,
                             acc, acc_out, max_q: Optional[int] = None, window: int = 0,
                             sinks: int = 0, stream=None):
    """The softmax weights that cached positions receive from the given queries, added to ``acc``
    (fp32 [nseq][H][n], or None for zeros) into ``acc_out`` (may be ``acc``); ``lse`` as
    ``fg_attn_q4kv_paged`` gives it."""
    rows, q_stride, max_q, nseq, n = _paged_queries(q, q_off, Hq, pages, table, lens, max_q, window,
                                                    sinks)
    _scores("lse", lse, (rows, Hq))
    if acc_out.dim() != 3:
        raise ValueError(f"acc_out: [nseq][H][positions] expected, got {tuple(acc_out.shape)}")
    shape = (nseq, pages.H, acc_out.shape[2])
    _scores("acc_out", acc_out, shape)
    if acc is not None:
        _scores("acc", acc, shape)
    handle = _stream_for(stream, q, q_off, table, lens, lse, acc, acc_out, pages.blocks)
    _check("fg_attn_weights_q4_paged",
           lib.fg_attn_weights_q4_paged(_ptr(q), q_stride, rows, _ptr(q_off), max_q, Hq,
                                        C.byref(pages.struct()), _ptr(table), n, _ptr(lens), nseq,
                                        window, sinks, scale, _ptr(lse), _ptr(acc), _ptr(acc_out),
                                        shape[2], handle))


def fg_kv_evict_q4_paged(pages: KVPagesQ4, table, lens, acc, recent: int, dst_table, kept, acc_out,
                         dst_lens, stream=None):
    """Every head of sequence b keeps its last ``recent`` positions and the heaviest others (``acc``
    fp32 [nseq][H][n]), as many as ``kept`` (int32 [nseq][H][keep]) has room for, moved into the
    pages of ``dst_table``; ``acc_out`` (fp32 as ``kept``) and ``dst_lens`` (int32 [nseq]) receive
    their weights and how many stayed."""
    nseq, n = _table("table", table)
    nd, m = _table("dst_table", dst_table)
    if nd != nseq or acc.dim() != 3 or kept.dim() != 3:
        raise ValueError("table and dst_table differ in sequences, or acc or kept is not "
                         "[nseq][H][..]")
    _scores("acc", acc, (nseq, pages.H, acc.shape[2]))
    keep = kept.shape[2]
    if kept.shape != (nseq, pages.H, keep) or kept.dtype is not torch.int32 or \
            not kept.is_contiguous():
        raise ValueError(f"kept: contiguous int32 {(nseq, pages.H, keep)} expected, got "
                         f"{kept.dtype} {tuple(kept.shape)}")
    _scores("acc_out", acc_out, (nseq, pages.H, keep))
    _extents("lens", lens, nseq)
    _extents("dst_lens", dst_lens, nseq)
    handle = _stream_for(stream, table, lens, acc, dst_table, kept, acc_out, dst_lens, pages.blocks)
    _check("fg_kv_evict_q4_paged",
           lib.fg_kv_evict_q4_paged(C.byref(pages.struct()), _ptr(table), n, nseq, _ptr(lens),
                                    _ptr(acc), acc.shape[2], keep, recent, _ptr(dst_table), m,
                                    _ptr(kept), _ptr(acc_out), _ptr(dst_lens), handle))


def fg_layernorm(x, gamma, beta, eps: float, y, stream=None):
    rows, h = x.shape
    _check("fg_layernorm", lib.fg_layernorm(_ptr(x), rows, h, _ptr(gamma), _ptr(beta), eps,
                                            _ptr(y), _stream(stream)))


def fg_workspace_bytes(layer: LayerQ4, g: int, m: int, s_max: int) -> int:
    """Scratch bytes of fg_layer_prefill / fg_layer_decode for this layer's dims."""
    dm = layer.dims()
    return int(lib.fg_workspace_bytes(C.byref(dm), g, m, s_max))


fg_layer_workspace_bytes = fg_workspace_bytes


def fg_layer_prefill(layer: LayerQ4, cache: KVCacheQ4, x, y, g: int, m: int, s: int, ws,
                     stream=None):
    dm, L, kv = layer.dims(), layer.struct(), cache.struct()
    _check("fg_layer_prefill",
           lib.fg_layer_prefill(C.byref(dm), C.byref(L), C.byref(kv), _ptr(x), _ptr(y), g, m, s,
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def fg_layer_decode(layer: LayerQ4, cache: KVCacheQ4, x, y, g: int, m: int, pos: int, ws,
                    stream=None):
    dm, L, kv = layer.dims(), layer.struct(), cache.struct()
    _check("fg_layer_decode",
           lib.fg_layer_decode(C.byref(dm), C.byref(L), C.byref(kv), _ptr(x), _ptr(y), g, m, pos,
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def fg_check_device_error(stream=None):
    _check("fg_check_device_error", lib.fg_check_device_error(_stream(stream)))


def fg_prof_enable(on: bool = True):
    lib.fg_prof_enable(1 if on else 0)


def fg_prof_reset():
    lib.fg_prof_reset()


def fg_prof_query(kind: int):
    n, ms, work = C.c_int64(), C.c_double(), C.c_double()
    _check("fg_prof_query", lib.fg_prof_query(kind, C.byref(n), C.byref(ms), C.byref(work)))
    return {"kernel": lib.fg_kernel_name(kind).decode(), "launches": n.value, "ms": ms.value,
            "work": work.value}


# ----------------------------------------------------------------------------- stack


class StackEngine:
    """A stack of layers over one block of B = g*m sequences: prefill over the prompt,
    then decode steps, each running every layer over the whole block before the next
    (the block schedule).  Orchestration only -- each layer step is one C call."""

    def __init__(self, layers, g: int, m: int, cap: int, s_max: int, device="cuda"):
        self.layers, self.g, self.m, self.cap = layers, g, m, cap
        L0 = layers[0]
        self.B = g * m
        self.caches = [KVCacheQ4(self.B, cap, L0.h, L0.H, device) for _ in layers]
        wsb = max(fg_workspace_bytes(L, g, m, max(s_max, cap)) for L in layers)
        self.ws = torch.empty((wsb + 255) // 256 * 256, dtype=torch.uint8, device=device)

    def prefill(self, x, y, s: int, stream=None):
        """x, y: [B][s][h] fp16 (may alias); runs every layer over the prompt."""
        cur = x
        for L, c in zip(self.layers, self.caches):
            fg_layer_prefill(L, c, cur, y, self.g, self.m, s, self.ws, stream)
            cur = y
        return y

    def decode(self, x, y, pos: int, stream=None):
        """One decode step: x, y [B][h]; appends at ``pos`` in every layer's cache."""
        cur = x
        for L, c in zip(self.layers, self.caches):
            fg_layer_decode(L, c, cur, y, self.g, self.m, pos, self.ws, stream)
            cur = y
        return y
