"""Python binding of libmla.so (the GB300 MLA sublayer).

Argument marshalling only: each function takes torch tensors for device
memory and the current torch stream, and calls the C entry point of the same
name (include/mla.h).  Every step of the computation runs in the library's
CUDA kernels; there is no fallback.  If the library has not been built the
import of ``lib()`` fails loudly.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

D, HEADS, Q_LORA, KV_LORA, QK_NOPE, QK_ROPE, QK, V = 7168, 64, 1536, 512, 128, 64, 192, 128
FFN_INTER = 18432
MODE_PREFILL, MODE_DECODE, MODE_DECODE_LATENT, MODE_FFN, MODE_CHUNK_LATENT, MODE_CHUNK_ABSORBED = 0, 1, 2, 3, 4, 5
MODE_FOLD = 6
MODE_PAGED_APPEND, MODE_PAGED_ATTN, MODE_WINDOW_ATTN, MODE_DECODE_PAGED, MODE_PREFILL_PAGED = 8, 9, 10, 11, 12
MODE_PAGES, MODE_DOCUMENTS = 13, 14
STAGES = ["input_norm", "a_proj", "latent", "q_b", "kv_b", "attn", "combine", "absorb_q", "absorb_o", "o_proj",
          "ffn_norm", "gate_up", "down"]
MAX_STAGES = len(STAGES)

STATUS = {0: "MLA_OK", -1: "MLA_ERR_INVALID_ARG", -2: "MLA_ERR_ALIGNMENT", -3: "MLA_ERR_WORKSPACE",
          -4: "MLA_ERR_UNSUPPORTED", -5: "MLA_ERR_CUDA", -6: "MLA_ERR_TIMEOUT", -7: "MLA_ERR_NO_PAGES"}

WEIGHT_NAMES = ["w_in_norm", "w_q_a", "w_q_a_norm", "w_q_b", "w_kv_a", "w_kv_a_norm", "w_kv_b", "w_o"]
WEIGHT_SHAPES = {
    "w_in_norm": (D,), "w_q_a": (Q_LORA, D), "w_q_a_norm": (Q_LORA,), "w_q_b": (HEADS * QK, Q_LORA),
    "w_kv_a": (KV_LORA + QK_ROPE, D), "w_kv_a_norm": (KV_LORA,), "w_kv_b": (HEADS * (QK_NOPE + V), KV_LORA),
    "w_o": (D, HEADS * V),
}
FFN_WEIGHT_NAMES = ["w_post_norm", "w_1", "w_3", "w_2"]
FFN_WEIGHT_SHAPES = {"w_post_norm": (D,), "w_1": (FFN_INTER, D), "w_3": (FFN_INTER, D), "w_2": (D, FFN_INTER)}


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class MlaWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_NAMES]


FP8_NAMES = ["w_q_a", "w_q_b", "w_kv_a", "w_kv_b", "w_o"]


class MlaWeightsFp8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ["w_in_norm", "w_q_a_norm", "w_kv_a_norm"] + FP8_NAMES] + \
               [("s_" + n[2:], ctypes.c_void_p) for n in FP8_NAMES]


class MlaFfnWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in FFN_WEIGHT_NAMES]


class MlaPagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_pe", "k_scales", "v_scales", "table")] + \
               [(n, ctypes.c_int) for n in ("n_pages", "max_pages", "page", "heads")]


class MlaPagePool(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "refs")] + \
               [(n, ctypes.c_int) for n in ("rows", "max_pages", "n_pages", "page")]


class MlaTiming(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p * MAX_STAGES), ("stop", ctypes.c_void_p * MAX_STAGES),
                ("n_launches", ctypes.c_int)]


class MlaParams(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("rope_base", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("delta_out", ctypes.c_void_p), ("timing", ctypes.POINTER(MlaTiming))]


_lib = None

_VP, _I, _SZ, _LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
_SIGS = {
    "mla_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "mla_prefill": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _VP, _VP, _VP, _VP,
                         _VP, _I, _VP, _SZ, _VP]),
    "mla_prefill_chunk": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _I, _VP, _VP,
                               _VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_prefill_chunk_latent": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _I, _VP,
                                      _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_prefill_chunk_absorbed": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _I,
                                        _VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_decode": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _VP, _VP, _I, _VP,
                        _VP, _SZ, _VP]),
    "mla_decode_latent": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _VP, _VP, _I,
                               _VP, _VP, _SZ, _VP]),
    "mla_fold_wuv_into_wo": (_I, [ctypes.POINTER(MlaWeights), _VP, _VP, _SZ, _VP]),
    "mla_decode_latent_folded": (_I, [ctypes.POINTER(MlaWeights), _VP, ctypes.POINTER(MlaParams), _VP, _I, _I, _VP,
                                      _VP, _I, _VP, _VP, _SZ, _VP]),
    "mla_decode_varlen": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _VP, _I, _VP, _VP,
                               _I, _VP, _VP, _SZ, _VP]),
    "mla_decode_latent_varlen": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _VP, _I, _VP,
                                      _VP, _I, _VP, _VP, _SZ, _VP]),
    "mla_decode_noalloc": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _VP, _VP, _I,
                                _VP, _VP]),
    "mla_ffn": (_I, [ctypes.POINTER(MlaFfnWeights), ctypes.POINTER(MlaParams), _VP, _I, _VP, _VP, _SZ, _VP]),
    "mla_quantize_fp8": (_I, [_VP, _I, _I, _VP, _VP, _VP]),
    "mla_decode_fp8": (_I, [ctypes.POINTER(MlaWeightsFp8), ctypes.POINTER(MlaParams), _VP, _I, _I, _VP, _VP, _I, _VP,
                            _VP, _SZ, _VP]),
    "mla_paged_append": (_I, [ctypes.POINTER(MlaPagedCache), ctypes.POINTER(MlaParams), _VP, _LL, _LL, _VP, _LL, _LL,
                              _VP, _LL, _VP, _VP, _I, _I, _I, _VP, _SZ, _VP]),
    "mla_paged_attention": (_I, [ctypes.POINTER(MlaPagedCache), ctypes.POINTER(MlaParams), _VP, _LL, _I, _I, _VP, _I,
                                 _I, _I, _VP, _LL, _VP, _SZ, _VP]),
    "mla_window_attention": (_I, [ctypes.POINTER(MlaParams), _VP, _I, _I, _I, _VP, _VP, _I, _I, _I, _VP, _VP, _SZ,
                                  _VP]),
    "mla_decode_paged": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _VP, _I,
                              ctypes.POINTER(MlaPagedCache), _I, _I, _VP, _VP, _SZ, _VP]),
    "mla_prefill_paged": (_I, [ctypes.POINTER(MlaWeights), ctypes.POINTER(MlaParams), _VP, _I, _I, _I,
                               ctypes.POINTER(MlaPagedCache), _I, _I, _VP, _VP, _SZ, _VP]),
    "mla_document_attention": (_I, [_VP, _VP, _LL, _I, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _VP, _LL, _VP, _SZ, _VP]),
    "mla_pages_free": (_I, [_VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_pages_reserve": (_I, [_VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_pages_fork": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_pages_compact": (_I, [_VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "mla_pages_copy": (_I, [_VP, _VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "mla_device_status": (_I, [_VP, _VP]),
    "mla_status_string": (ctypes.c_char_p, [_I]),
}


def lib():
    """The loaded libmla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: the CUDA library must be built "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != 0:
        raise MlaError(rc, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_weights(w: dict) -> MlaWeights:
    """Pack a dict of bf16 CUDA tensors (names of WEIGHT_NAMES) into the C struct."""
    import torch
    for n in WEIGHT_NAMES:
        t = w[n]
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != WEIGHT_SHAPES[n]:
            raise ValueError(f"weight {n}: need contiguous bf16 CUDA tensor of shape {WEIGHT_SHAPES[n]}")
    s = MlaWeights(*[w[n].data_ptr() for n in WEIGHT_NAMES])
    s._keep = dict(w)  # the struct holds raw pointers: keep the tensors alive with it
    return s


def make_ffn_weights(w: dict) -> MlaFfnWeights:
    """Pack a dict of bf16 CUDA tensors (names of FFN_WEIGHT_NAMES) into the C struct."""
    import torch
    for n in FFN_WEIGHT_NAMES:
        t = w[n]
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or \
                tuple(t.shape) != FFN_WEIGHT_SHAPES[n]:
            raise ValueError(f"weight {n}: need contiguous bf16 CUDA tensor of shape {FFN_WEIGHT_SHAPES[n]}")
    s = MlaFfnWeights(*[w[n].data_ptr() for n in FFN_WEIGHT_NAMES])
    s._keep = dict(w)
    return s


def make_params(eps=1e-6, rope_base=10000.0, softmax_scale=None, delta_out=None, timing=None) -> MlaParams:
    if softmax_scale is None:
        softmax_scale = 1.0 / (QK ** 0.5)
    return MlaParams(eps, rope_base, softmax_scale,
                     None if delta_out is None else delta_out.data_ptr(),
                     None if timing is None else ctypes.pointer(timing))


def workspace_size(mode: int, B: int, t_or_p: int, cap: int = 0) -> int:
    n = lib().mla_workspace_size(mode, B, t_or_p, cap)
    if n == 0:
        raise MlaError(-1, "mla_workspace_size")
    return n


def alloc_workspace(mode: int, B: int, t_or_p: int, device="cuda", cap: int = 0):
    import torch
    return torch.empty(workspace_size(mode, B, t_or_p, cap), dtype=torch.uint8, device=device)


def mla_prefill(weights: MlaWeights, x, out, workspace, k_cache=None, v_cache=None, ckv_cache=None,
                kpe_cache=None, cap=0, params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, T, 7168] (out None: fill the given caches only); caches as in include/mla.h."""
    B, T = x.shape[0], x.shape[1]
    rc = lib().mla_prefill(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x), B, T,
                           _ptr(out), _ptr(k_cache), _ptr(v_cache), _ptr(ckv_cache), _ptr(kpe_cache), cap,
                           _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_prefill")


def mla_prefill_chunk(weights: MlaWeights, x, P0: int, out, k_cache, v_cache, workspace, ckv_cache=None,
                      kpe_cache=None, params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, T, 7168], the chunk at positions P0..P0+T-1; k_cache [B, 64, cap, 192] and
    v_cache [B, 64, cap, 128] hold rows 0..P0-1 and receive rows P0..P0+T-1."""
    B, T = x.shape[0], x.shape[1]
    cap = k_cache.shape[2]
    rc = lib().mla_prefill_chunk(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x),
                                 B, T, P0, _ptr(out), _ptr(k_cache), _ptr(v_cache), _ptr(ckv_cache),
                                 _ptr(kpe_cache), cap, _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_prefill_chunk")


def mla_prefill_chunk_latent(weights: MlaWeights, x, P0: int, out, ckv_cache, kpe_cache, workspace,
                             params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, T, 7168] at positions P0..P0+T-1; ckv_cache [B, cap, 512] and kpe_cache
    [B, cap, 64] hold rows 0..P0-1 and receive rows P0..P0+T-1; workspace of MODE_CHUNK_LATENT
    sized with the same cap."""
    B, T = x.shape[0], x.shape[1]
    cap = ckv_cache.shape[1]
    rc = lib().mla_prefill_chunk_latent(ctypes.byref(weights), None if params is None else ctypes.byref(params),
                                        _ptr(x), B, T, P0, _ptr(out), _ptr(ckv_cache), _ptr(kpe_cache), cap,
                                        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_prefill_chunk_latent")


def mla_prefill_chunk_absorbed(weights: MlaWeights, x, P0: int, out, ckv_cache, kpe_cache, workspace,
                               params: MlaParams | None = None, stream=None):
    """The same chunk as mla_prefill_chunk_latent in the absorbed form (one latent decode row per new
    token); workspace of MODE_CHUNK_ABSORBED sized with the same B, T and cap."""
    B, T = x.shape[0], x.shape[1]
    cap = ckv_cache.shape[1]
    rc = lib().mla_prefill_chunk_absorbed(ctypes.byref(weights), None if params is None else ctypes.byref(params),
                                          _ptr(x), B, T, P0, _ptr(out), _ptr(ckv_cache), _ptr(kpe_cache), cap,
                                          _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_prefill_chunk_absorbed")


def mla_decode(weights: MlaWeights, x, P: int, k_cache, v_cache, out, workspace,
               params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, 7168]; k_cache [B, 64, cap, 192], v_cache [B, 64, cap, 128]."""
    B = x.shape[0]
    cap = k_cache.shape[2]
    rc = lib().mla_decode(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x), B, P,
                          _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _ptr(workspace), workspace.numel(),
                          _stream(stream))
    _check(rc, "mla_decode")


def mla_decode_latent(weights: MlaWeights, x, P: int, ckv_cache, kpe_cache, out, workspace,
                      params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, 7168]; ckv_cache [B, cap, 512], kpe_cache [B, cap, 64]."""
    B = x.shape[0]
    cap = ckv_cache.shape[1]
    rc = lib().mla_decode_latent(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x),
                                 B, P, _ptr(ckv_cache), _ptr(kpe_cache), cap, _ptr(out), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(rc, "mla_decode_latent")


def mla_fold_wuv_into_wo(weights: MlaWeights, w_fold, workspace, stream=None):
    """w_fold: bf16 [7168, 64 * 512] receives W_o's head blocks times W_UV per head; workspace of MODE_FOLD."""
    rc = lib().mla_fold_wuv_into_wo(ctypes.byref(weights), _ptr(w_fold), _ptr(workspace), workspace.numel(),
                                    _stream(stream))
    _check(rc, "mla_fold_wuv_into_wo")


def mla_decode_latent_folded(weights: MlaWeights, w_fold, x, P: int, ckv_cache, kpe_cache, out, workspace,
                             params: MlaParams | None = None, stream=None):
    """mla_decode_latent with W_UV folded into o_proj (w_fold from mla_fold_wuv_into_wo)."""
    B = x.shape[0]
    cap = ckv_cache.shape[1]
    rc = lib().mla_decode_latent_folded(ctypes.byref(weights), _ptr(w_fold),
                                        None if params is None else ctypes.byref(params), _ptr(x), B, P,
                                        _ptr(ckv_cache), _ptr(kpe_cache), cap, _ptr(out), _ptr(workspace),
                                        workspace.numel(), _stream(stream))
    _check(rc, "mla_decode_latent_folded")


def mla_decode_varlen(weights: MlaWeights, x, P, P_max: int, k_cache, v_cache, out, workspace,
                      params: MlaParams | None = None, stream=None):
    """Ragged decode: P is an int32 CUDA tensor [B] of per-sequence positions (<= P_max)."""
    B = x.shape[0]
    cap = k_cache.shape[2]
    rc = lib().mla_decode_varlen(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x), B,
                                 _ptr(P), P_max, _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(rc, "mla_decode_varlen")


def mla_decode_latent_varlen(weights: MlaWeights, x, P, P_max: int, ckv_cache, kpe_cache, out, workspace,
                             params: MlaParams | None = None, stream=None):
    """Ragged latent decode: P is an int32 CUDA tensor [B] of per-sequence positions (<= P_max)."""
    B = x.shape[0]
    cap = ckv_cache.shape[1]
    rc = lib().mla_decode_latent_varlen(ctypes.byref(weights), None if params is None else ctypes.byref(params),
                                        _ptr(x), B, _ptr(P), P_max, _ptr(ckv_cache), _ptr(kpe_cache), cap, _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_decode_latent_varlen")


def mla_decode_noalloc(weights: MlaWeights, x, P: int, k_cache, v_cache, out, params: MlaParams | None = None,
                       stream=None):
    """mla_decode with its scratch in the library's fixed static device array
    (for callers that cannot allocate device memory); no workspace argument."""
    B = x.shape[0]
    cap = k_cache.shape[2]
    rc = lib().mla_decode_noalloc(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x),
                                  B, P, _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _stream(stream))
    _check(rc, "mla_decode_noalloc")


def mla_ffn(weights: MlaFfnWeights, x, out, workspace, params: MlaParams | None = None, stream=None):
    """x, out: bf16 [..., 7168] (out = x + Delta_ffn, may be x itself)."""
    n_tok = x.numel() // D
    rc = lib().mla_ffn(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x), n_tok,
                       _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "mla_ffn")


def mla_quantize_fp8(w, codes, scales, stream=None):
    """w: bf16 CUDA [rows, cols] (cols % 128 == 0) -> codes uint8 block-major
    [ceil(rows/128), cols/128, 128, 128], scales float32 [ceil(rows/128), cols/128]."""
    rows, cols = w.shape
    _check(lib().mla_quantize_fp8(_ptr(w), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)),
           "mla_quantize_fp8")


def make_weights_fp8(w: dict, stream=None):
    """FP8 block-scaled copies of the five projection matrices of a bf16
    weight dict (quantized by the library) packed with the bf16 gains;
    returns (struct, dict of the tensors it points to)."""
    import torch
    t = {n: w[n] for n in ("w_in_norm", "w_q_a_norm", "w_kv_a_norm")}
    for n in FP8_NAMES:
        rows, cols = w[n].shape
        t[n] = torch.empty(((rows + 127) // 128, cols // 128, 128, 128), dtype=torch.uint8, device=w[n].device)
        t["s_" + n[2:]] = torch.empty(((rows + 127) // 128, (cols + 127) // 128), dtype=torch.float32,
                                     device=w[n].device)
        mla_quantize_fp8(w[n], t[n], t["s_" + n[2:]], stream)
    st = MlaWeightsFp8(*[t[f].data_ptr() for f, _ in MlaWeightsFp8._fields_])
    st._keep = t
    return st, t


def mla_decode_fp8(weights: MlaWeightsFp8, x, P: int, k_cache, v_cache, out, workspace,
                   params: MlaParams | None = None, stream=None):
    """mla_decode with FP8 block-scaled weights (make_weights_fp8)."""
    B = x.shape[0]
    cap = k_cache.shape[2]
    rc = lib().mla_decode_fp8(ctypes.byref(weights), None if params is None else ctypes.byref(params), _ptr(x), B, P,
                              _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _ptr(workspace), workspace.numel(),
                              _stream(stream))
    _check(rc, "mla_decode_fp8")


PAGED_TENSORS = ["k_codes", "v_codes", "k_pe", "k_scales", "v_scales"]


def alloc_paged_cache(n_pages: int, page: int = 64, heads: int = HEADS, device="cuda") -> dict:
    """The tensors of an empty paged 8-bit cache (codes uint8, E4M3; without a table)."""
    import torch
    t = {n: torch.zeros((n_pages, heads, page, 128), dtype=torch.uint8, device=device) for n in ("k_codes", "v_codes")}
    t["k_pe"] = torch.zeros((n_pages, page, QK_ROPE), dtype=torch.bfloat16, device=device)
    for n in ("k_scales", "v_scales"):
        t[n] = torch.ones((n_pages, heads), dtype=torch.float32, device=device)
    return t


def make_paged_cache(t: dict) -> MlaPagedCache:
    """Pack the tensors of a paged cache (PAGED_TENSORS) and its int32 table [B, max_pages] into the C struct.
    The struct points at the tensors: a table changed in place is seen by the next call."""
    import torch
    n_pages, heads, page, _ = t["k_codes"].shape
    shapes = {"k_codes": (n_pages, heads, page, 128), "v_codes": (n_pages, heads, page, 128),
              "k_pe": (n_pages, page, QK_ROPE), "k_scales": (n_pages, heads), "v_scales": (n_pages, heads)}
    dtypes = {"k_codes": torch.uint8, "v_codes": torch.uint8, "k_pe": torch.bfloat16, "k_scales": torch.float32,
              "v_scales": torch.float32, "table": torch.int32}
    for n in PAGED_TENSORS + ["table"]:
        x = t[n]
        if x.dtype != dtypes[n] or not x.is_cuda or not x.is_contiguous() or \
                (tuple(x.shape) != shapes[n] if n != "table" else x.dim() != 2) or x.device != t["k_codes"].device:
            raise ValueError(f"paged cache {n}: need a contiguous {dtypes[n]} CUDA tensor of shape "
                             f"{shapes.get(n, '[B, max_pages]')} on one device")
    if not t["table"].numel():
        raise ValueError("paged cache table: need at least one sequence and one page")
    s = MlaPagedCache(*[t[n].data_ptr() for n in PAGED_TENSORS], t["table"].data_ptr(), n_pages, t["table"].shape[1],
                      page, heads)
    s._keep = dict(t)
    # what every call of a decode loop looks up: read once here
    s._ref, s._device, s._batch = ctypes.byref(s), t["table"].get_device(), t["table"].shape[0]
    return s


# The paged calls take a few microseconds on the GPU at decode sizes, so that
# their argument checks are kept to one attribute each: get_device() is -1 for
# a tensor that is not on a GPU.
def _rows(x, what: str, cols: int, device: int) -> int:
    """Row stride of a bf16 tensor [rows, cols] on the device whose rows are contiguous."""
    shape, stride = x.shape, x.stride()
    if not (x.dtype is _torch.bfloat16 and x.get_device() == device and len(shape) == 2 and shape[1] == cols and
            stride[1] == 1):
        raise ValueError(f"{what}: need a bf16 tensor [rows, {cols}] with contiguous rows on the current device")
    return stride[0] if shape[0] > 1 else cols  # (the stride of a single row is arbitrary)


def _head_rows(x, what: str, heads: int, rows: int, device: int):
    """Token and head strides of a bf16 tensor [rows, heads, 128] on the device, its last dimension contiguous."""
    stride = x.stride()
    if not (x.dtype is _torch.bfloat16 and x.get_device() == device and x.shape == (rows, heads, 128) and
            stride[2] == 1):
        raise ValueError(f"{what}: need a bf16 tensor [{rows}, {heads}, 128] with a contiguous last dimension on the "
                         "current device")
    return stride[0] if rows > 1 else 0, stride[1]


def _ints(x, what: str, n: int, device: int) -> int:
    if not (x.dtype is _torch.int32 and x.get_device() == device and x.shape == (n,) and x.is_contiguous()):
        raise ValueError(f"{what}: need a contiguous int32 tensor of {n} elements on the current device")
    return x.data_ptr()


def _bytes(x, device: int) -> int:
    if x.get_device() != device or not x.is_contiguous():
        raise ValueError("workspace: need a contiguous tensor on the current device")
    return x.data_ptr()


def _stream_on(device: int, stream) -> int:
    """The stream's handle (the current one of the device if None); the device has to be the current one."""
    global _torch
    if _torch is None:
        import torch as _torch
    if device < 0 or _torch.cuda.current_device() != device:
        raise ValueError("the tensors are not on the current CUDA device")
    return stream.cuda_stream if stream is not None else _torch._C._cuda_getCurrentRawStream(device)


_torch = None


def mla_paged_append(cache: MlaPagedCache, k, v, k_pe, P, T: int, workspace, cu=None,
                     params: MlaParams | None = None, stream=None):
    """k, v: bf16 [N, heads, 128] (views of a kv_b product are fine); k_pe: bf16 [N, 64], unrotated; P: int32 [B],
    position of each sequence's first new token (-1: idle); T tokens each, or with cu (int32 [B + 1], row offsets)
    at most T; workspace of MODE_PAGED_APPEND."""
    dev, B = cache._device, cache._batch
    s = _stream_on(dev, stream)
    N = k.shape[0]
    k_token, k_head = _head_rows(k, "k", cache.heads, N, dev)
    v_token, v_head = _head_rows(v, "v", cache.heads, N, dev)
    pe_token = _rows(k_pe, "k_pe", QK_ROPE, dev)
    if k_pe.shape[0] != N:
        raise ValueError("k_pe: need as many rows as k and v")
    rc = lib().mla_paged_append(cache._ref, None if params is None else ctypes.byref(params), k.data_ptr(), k_token,
                                k_head, v.data_ptr(), v_token, v_head, k_pe.data_ptr(), pe_token,
                                _ints(P, "P", B, dev), None if cu is None else _ints(cu, "cu", B + 1, dev), B, T, N,
                                _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_paged_append")


def mla_paged_attention(cache: MlaPagedCache, q, P, P_max: int, out, workspace, window: int = 0, sinks: int = 0,
                        params: MlaParams | None = None, stream=None):
    """q: bf16 [B * T, heads * 192] (rotated); out: bf16 [B * T, heads * 128]; P: int32 [B], position of each
    sequence's first query (-1: idle, its rows become zeros), at most P_max; window 0 = every key, else the last
    `window` keys and the first `sinks`; workspace of MODE_PAGED_ATTN."""
    dev, B = cache._device, cache._batch
    s = _stream_on(dev, stream)
    q_row, out_row = _rows(q, "q", cache.heads * QK, dev), _rows(out, "out", cache.heads * V, dev)
    n = q.shape[0]
    if n % B or out.shape[0] != n:
        raise ValueError("q and out: need the same number of rows, T for each sequence of the table")
    rc = lib().mla_paged_attention(cache._ref, None if params is None else ctypes.byref(params), q.data_ptr(), q_row,
                                   B, n // B, _ints(P, "P", B, dev), P_max, window, sinks, out.data_ptr(), out_row,
                                   _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_paged_attention")


def mla_window_attention(q, P0: int, k_cache, v_cache, out, workspace, window: int, sinks: int = 0,
                         params: MlaParams | None = None, stream=None):
    """q: bf16 [B, T, 64 * 192] at positions P0..P0+T-1; k_cache [B, 64, cap, 192], v_cache [B, 64, cap, 128];
    out: bf16 [B, T, 64 * 128]; a query sees the last `window` keys up to its own and the first `sinks`;
    workspace of MODE_WINDOW_ATTN."""
    dev = q.get_device()
    s = _stream_on(dev, stream)
    B, T, cap = q.shape[0], q.shape[1], k_cache.shape[2]
    for x, what, shape in ((q, "q", (B, T, HEADS * QK)), (k_cache, "k_cache", (B, HEADS, cap, QK)),
                           (v_cache, "v_cache", (B, HEADS, cap, V)), (out, "out", (B, T, HEADS * V))):
        if not (x.dtype is _torch.bfloat16 and x.get_device() == dev and x.is_contiguous() and x.shape == shape):
            raise ValueError(f"{what}: need a contiguous bf16 tensor of shape {shape} on the current device")
    rc = lib().mla_window_attention(None if params is None else ctypes.byref(params), q.data_ptr(), B, T, P0,
                                    k_cache.data_ptr(), v_cache.data_ptr(), cap, window, sinks, out.data_ptr(),
                                    _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_window_attention")


def mla_document_attention(q, cu_q, k_cache, v_cache, out, workspace, cu_k=None, prefix=None, window: int = 0,
                           sinks: int = 0, params: MlaParams | None = None, stream=None):
    """q: bf16 [N, 64 * 192], out: bf16 [N, 64 * 128] (rows may be strided); k_cache [64, cap, 192], v_cache
    [64, cap, 128]; cu_q, cu_k: int32 [n + 1], the rows of q and of the caches where each document begins (cu_k None:
    cu_q); prefix: int32 [n], tokens that all queries of a document see; workspace of MODE_DOCUMENTS(n, N)."""
    dev, n = q.get_device(), cu_q.shape[0] - 1
    s = _stream_on(dev, stream)
    q_row, out_row = _rows(q, "q", HEADS * QK, dev), _rows(out, "out", HEADS * V, dev)
    N, cap = q.shape[0], k_cache.shape[1]
    if out.shape[0] != N:
        raise ValueError("q and out: need the same number of rows")
    for x, what, shape in ((k_cache, "k_cache", (HEADS, cap, QK)), (v_cache, "v_cache", (HEADS, cap, V))):
        if not (x.dtype is _torch.bfloat16 and x.get_device() == dev and x.is_contiguous() and x.shape == shape):
            raise ValueError(f"{what}: need a contiguous bf16 tensor of shape {shape} on the current device")
    rc = lib().mla_document_attention(None if params is None else ctypes.byref(params), q.data_ptr(), q_row, N,
                                      _ints(cu_q, "cu_q", n + 1, dev), k_cache.data_ptr(), v_cache.data_ptr(), cap,
                                      None if cu_k is None else _ints(cu_k, "cu_k", n + 1, dev),
                                      None if prefix is None else _ints(prefix, "prefix", n, dev), n, window, sinks,
                                      out.data_ptr(), out_row, _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_document_attention")


def make_page_pool(table, refs, page: int = 64) -> MlaPagePool:
    """Pack int32 CUDA tensors table [rows, max_pages] (-1: no page; the paged cache's table) and refs [n_pages]
    (holds on each page, 0: free) into the C struct, which points at them."""
    import torch
    for x, what, dims in ((table, "table", 2), (refs, "refs", 1)):
        if x.dtype is not torch.int32 or not x.is_cuda or not x.is_contiguous() or x.dim() != dims or \
                x.device != table.device or not x.numel():
            raise ValueError(f"page pool {what}: need a contiguous int32 CUDA tensor of {dims} dimension(s), not empty, "
                             "on the table's device")
    s = MlaPagePool(table.data_ptr(), refs.data_ptr(), table.shape[0], table.shape[1], refs.shape[0], page)
    s._keep = (table, refs)
    s._ref, s._device = ctypes.byref(s), table.get_device()
    return s


def mla_pages_free(pool: MlaPagePool, rows, P, workspace, stream=None):
    """Gives back the pages of each of the rows behind its first P positions; rows, P: int32 [n]; workspace of
    MODE_PAGES(n, n_pages, cap=rows of the table) here and below.  A row that then ends inside a page that others hold
    too (refs above 1) must not be appended to: fork its P positions into an empty row, which gets a page of its own."""
    dev, n = pool._device, rows.shape[0]
    s = _stream_on(dev, stream)
    rc = lib().mla_pages_free(pool._ref, _ints(rows, "rows", n, dev), _ints(P, "P", n, dev), n, _bytes(workspace, dev),
                              workspace.nbytes, s)
    _check(rc, "mla_pages_free")


def mla_pages_reserve(pool: MlaPagePool, rows, P, workspace, stream=None):
    """Takes free pages so that each of the rows holds its first P positions; rows, P: int32 [n]."""
    dev, n = pool._device, rows.shape[0]
    s = _stream_on(dev, stream)
    rc = lib().mla_pages_reserve(pool._ref, _ints(rows, "rows", n, dev), _ints(P, "P", n, dev), n,
                                 _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_pages_reserve")


def mla_pages_fork(cache: MlaPagedCache, pool: MlaPagePool, parents, children, P, workspace, stream=None):
    """Rows `children` get the first P positions of rows `parents`: whole pages shared, the rest of a page copied;
    int32 [n] each."""
    dev, n = pool._device, parents.shape[0]
    s = _stream_on(dev, stream)
    if cache._device != dev:
        raise ValueError("cache and pool: need the same device")
    rc = lib().mla_pages_fork(cache._ref, pool._ref, _ints(parents, "parents", n, dev),
                              _ints(children, "children", n, dev), _ints(P, "P", n, dev), n, _bytes(workspace, dev),
                              workspace.nbytes, s)
    _check(rc, "mla_pages_fork")


def mla_pages_compact(cache: MlaPagedCache, pool: MlaPagePool, moved, n_live, workspace, stream=None):
    """Moves the pages that are held to the lowest numbers; moved: int32 [n_pages] receives each page's new number
    (-1: free), n_live: int32 [1] the number of pages held; workspace of MODE_PAGES(1, n_pages, cap=rows)."""
    dev = pool._device
    s = _stream_on(dev, stream)
    if cache._device != dev:
        raise ValueError("cache and pool: need the same device")
    rc = lib().mla_pages_compact(cache._ref, pool._ref, _ints(moved, "moved", pool.n_pages, dev),
                                 _ints(n_live, "n_live", 1, dev), _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_pages_compact")


def mla_pages_copy(source: MlaPagedCache, target: MlaPagedCache, src, dst, workspace, stream=None):
    """Copies pages src of one cache to pages dst of another, or of the same one; int32 [n] each; workspace of
    MODE_PAGES(n, n_pages of the target)."""
    dev, n = target._device, src.shape[0]
    s = _stream_on(dev, stream)
    if source._device != dev:
        raise ValueError("source and target: need the same device")
    rc = lib().mla_pages_copy(source._ref, target._ref, _ints(src, "src", n, dev), _ints(dst, "dst", n, dev), n,
                              _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_pages_copy")


def mla_decode_paged(weights: MlaWeights, x, P, P_max: int, cache: MlaPagedCache, out, workspace, window: int = 0,
                     sinks: int = 0, params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, 7168]; P: int32 [B], positions of the new tokens (-1: idle), at most P_max; the cache has one
    table row per sequence; workspace of MODE_DECODE_PAGED sized with P_max."""
    dev, B = cache._device, cache._batch
    s = _stream_on(dev, stream)
    for t, what in ((x, "x"), (out, "out")):
        if _rows(t, what, D, dev) != D or t.shape[0] != B:
            raise ValueError(f"{what}: need a contiguous bf16 tensor [{B}, {D}], one row for each row of the table")
    rc = lib().mla_decode_paged(ctypes.byref(weights), None if params is None else ctypes.byref(params), x.data_ptr(), B,
                                _ints(P, "P", B, dev), P_max, cache._ref, window, sinks, out.data_ptr(),
                                _bytes(workspace, dev), workspace.nbytes, s)
    _check(rc, "mla_decode_paged")


def mla_prefill_paged(weights: MlaWeights, x, P0: int, cache: MlaPagedCache, out, workspace, window: int = 0,
                      sinks: int = 0, params: MlaParams | None = None, stream=None):
    """x, out: bf16 [B, T, 7168], tokens at positions P0..P0+T-1, appended to the pages; the cache has one table row
    per sequence; workspace of MODE_PREFILL_PAGED sized with T and cap = P0 + T."""
    dev, B, T = cache._device, cache._batch, x.shape[1]
    s = _stream_on(dev, stream)
    for t, what in ((x, "x"), (out, "out")):
        if t.dtype is not _torch.bfloat16 or t.get_device() != dev or not t.is_contiguous() or t.shape != (B, T, D):
            raise ValueError(f"{what}: need a contiguous bf16 tensor [{B}, {T}, {D}], a sequence for each row of the table")
    rc = lib().mla_prefill_paged(ctypes.byref(weights), None if params is None else ctypes.byref(params), x.data_ptr(),
                                 B, T, P0, cache._ref, window, sinks, out.data_ptr(), _bytes(workspace, dev),
                                 workspace.nbytes, s)
    _check(rc, "mla_prefill_paged")


def mla_device_status(workspace, stream=None) -> int:
    return lib().mla_device_status(_ptr(workspace), _stream(stream))


def mla_status_string(status: int) -> str:
    return lib().mla_status_string(status).decode()
