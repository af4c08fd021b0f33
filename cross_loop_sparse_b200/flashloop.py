"""Thin Python binding of libflashloop.so (the C ABI in include/flashloop.h).

Argument marshalling only: every step of the sublayer runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  If
the shared library is missing this module raises at import time; there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re
import warnings
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

MAX_LOOPS = 16
GROUP = 32
PAPER_GROUP = 64   # the pages' cache setting: groups of 64 and a 64-token bf16 tail
PAPER_TAIL = 64
_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libflashloop.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "flashloop.h")

STATUS = {0: "FLASHLOOP_OK", -1: "FLASHLOOP_ERR_INVALID_ARG", -2: "FLASHLOOP_ERR_UNSUPPORTED",
          -3: "FLASHLOOP_ERR_CUDA", -4: "FLASHLOOP_ERR_DEVICE", -5: "FLASHLOOP_ERR_ARCH"}


class FlashLoopError(RuntimeError):
    def __init__(self, fn, status, detail=""):
        self.status = status
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})" + (f": {detail}" if detail else ""))


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m cross_loop_sparse_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)


# ----------------------------------------------------------------------------- structs
class Params(ctypes.Structure):
    _fields_ = [("seq", c_int32), ("d_model", c_int32), ("n_heads", c_int32), ("head_dim", c_int32),
                ("n_loops", c_int32), ("batch", c_int32), ("tau", c_float), ("rope_theta", c_float),
                ("topk", c_int32 * MAX_LOOPS), ("bits", c_int32 * MAX_LOOPS),
                ("capacity", c_int32 * MAX_LOOPS), ("gate_topk", c_int32), ("fixed_mass", c_int32),
                ("attn_pairs", c_int32), ("kv_scheme", c_int32)]

    @classmethod
    def from_config(cls, cfg, capacity=None, topk=None, tau=None, seq=None, token_budgets=None,
                    fixed_mass=False, kv_scheme="spec"):
        """Params of a workload.Config; capacities default to S (no overflow possible).
        token_budgets (per loop) selects top-k token retention with those budgets;
        fixed_mass selects the fixed-mass form of the sparse update; attn_pairs
        (reserved) stays 0."""
        p = cls()
        p.kv_scheme = {"spec": 0, "paper": 1}[kv_scheme]
        p.fixed_mass = 1 if fixed_mass else 0
        p.attn_pairs = 0
        p.seq = cfg.seq if seq is None else seq
        p.d_model, p.n_heads, p.head_dim = cfg.d_model, cfg.n_heads, cfg.head_dim
        p.n_loops, p.batch = cfg.n_loops, (cfg.batch if cfg.decode else 1)
        p.tau = cfg.tau if tau is None else tau
        p.rope_theta = cfg.rope_theta
        ks = cfg.k_per_loop() if topk is None else list(topk)
        for r in range(cfg.n_loops):
            p.topk[r] = ks[r]
            p.bits[r] = cfg.bits[r]
            p.capacity[r] = p.seq if capacity is None else capacity[r]
        if token_budgets is not None:
            p.gate_topk = 1
            for r in range(1, cfg.n_loops):
                p.capacity[r] = token_budgets[r]
        return p


class KV(ctypes.Structure):
    _fields_ = [("base_codes", c_void_p), ("base_scales", c_void_p),
                ("res_codes", c_void_p * MAX_LOOPS), ("res_scales", c_void_p * MAX_LOOPS)]


class PaperKV(ctypes.Structure):
    _fields_ = [("codes", c_void_p * MAX_LOOPS), ("scale", c_void_p * MAX_LOOPS),
                ("minv", c_void_p * MAX_LOOPS), ("tail", c_void_p * MAX_LOOPS)]


class StateC(ctypes.Structure):
    _fields_ = [("k", KV), ("v", KV), ("active", c_void_p * MAX_LOOPS), ("slot", c_void_p * MAX_LOOPS),
                ("n_active", c_void_p), ("q", c_void_p * 3), ("m", c_void_p * 3), ("Z", c_void_p * 3),
                ("N", c_void_p * 3), ("colmass", c_void_p * 2), ("cols", c_void_p * MAX_LOOPS),
                ("O", c_void_p), ("Y", c_void_p), ("rope_cs", c_void_p), ("err_word", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("G", c_void_p * 3),
                ("paper_k", POINTER(PaperKV)), ("paper_v", POINTER(PaperKV))]


class DecodeStateC(ctypes.Structure):
    _fields_ = [("k", KV), ("v", KV), ("rope_cs", c_void_p), ("q", c_void_p * 3), ("m", c_void_p * 3),
                ("Z", c_void_p * 3), ("N", c_void_p * 3), ("probs", c_void_p), ("cols", c_void_p),
                ("O", c_void_p), ("Y", c_void_p), ("err_word", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t)]


class PagedParams(ctypes.Structure):
    """Shapes and host-known bounds of the many-request calls (flashloop_paged_params)."""
    _fields_ = [("batch", c_int32), ("max_tokens", c_int32), ("max_new", c_int32), ("n_heads", c_int32),
                ("n_kv_heads", c_int32), ("head_dim", c_int32), ("page_size", c_int32), ("n_pages", c_int32),
                ("max_blocks", c_int32), ("dtype", c_int32), ("scale", c_float)]

    @classmethod
    def make(cls, batch, max_tokens, max_new, n_heads, n_kv_heads, head_dim, page_size=64, n_pages=1, max_blocks=1,
             dtype=torch.bfloat16, scale=None):
        """batch requests with at most max_tokens rows in all and max_new rows each; the page
        fields matter to the calls that touch the paged cache; scale defaults to 1/sqrt(head_dim)."""
        if dtype not in PAGED_DTYPES or dtype == torch.float32:
            raise FlashLoopError("PagedParams.make", -2, f"dtype {dtype}: bfloat16 or float16")
        return cls(batch, max_tokens, max_new, n_heads, n_kv_heads, head_dim, page_size, n_pages, max_blocks,
                   PAGED_DTYPES[dtype], head_dim ** -0.5 if scale is None else scale)


PAGED_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class RowsC(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("stride_token", c_int64), ("stride_head", c_int64)]


class PagesC(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("stride_page", c_int64), ("stride_token", c_int64), ("stride_head", c_int64)]


# ----------------------------------------------------------------------------- prototypes
_P = POINTER(Params)
_S = POINTER(StateC)
_D = POINTER(DecodeStateC)
_V = c_void_p
_I = c_int32
_PP = POINTER(PagedParams)
_RW = POINTER(RowsC)
_PG = POINTER(PagesC)
_SIG = {
    "flashloop_workspace_bytes": (c_size_t, [_P]),
    "flashloop_cache_bytes": (c_size_t, [_P, _V]),
    "flashloop_rope_table": (_I, [_P, _I, _V, _V]),
    "flashloop_gate": (_I, [_P, _V, _V, _V, _V, _I, _V, _V, _V, _I, _V, _V, _V]),
    "flashloop_gate_noalloc": (_I, [_P, _V, _V, _V, _V, _I, _V, _V, _V, _I, _V, _V]),
    "flashloop_gate_topk": (_I, [_P, _V, _V, _V, _V, _I, _I, _V, _V, _V, _I, _V, _V, _V]),
    "flashloop_qkv_gathered": (_I, [_P, _V, _V, _V, _I, _V, _V, _V, _V, _V, _V]),
    "flashloop_kv_quant_residual": (_I, [_P, _I, _V, _V, _V, _V, _S, _V]),
    "flashloop_qkv_quant": (_I, [_P, _I, _V, _V, _V, _V, _S, _V, _V]),
    "flashloop_paper_kv_quant": (_I, [_P, _I, _V, _V, _V, _V, _S, _V]),
    "flashloop_topk_columns": (_I, [_P, _V, _V, _I, _I, _V, _V]),
    "flashloop_selcol_dequant": (_I, [_P, _I, _S, _V]),
    "flashloop_sparse_attn_update": (_I, [_P, _I, _S, _I, _V]),
    "flashloop_out_proj": (_I, [_P, _V, _V, _V, _I, _V, _V, _V]),
    "flashloop_loop_step": (_I, [_P, _I, _V, _V, _V, _V, _S, _V]),
    "flashloop_kv_step": (_I, [_P, _I, _V, _V, _V, _S, _V]),
    "flashloop_kv_workspace_bytes": (c_size_t, [_P]),
    "flashloop_decode_workspace_bytes": (c_size_t, [_P]),
    "flashloop_decode_attn": (_I, [_P, _I, _S, _D, _V]),
    "flashloop_decode_step": (_I, [_P, _I, _V, _V, _V, _S, _D, _V]),
    "flashloop_decode_qkv": (_I, [_P, _I, _V, _V, _D, _V]),
    "flashloop_decode_select": (_I, [_P, _D, _V]),
    "flashloop_decode_out": (_I, [_P, _V, _D, _V]),
    "flashloop_selection_loop": (_I, [_P, _I]),
    "flashloop_check_error_word": (_I, [_V, POINTER(c_int32), _V]),
    "flashloop_selftest_bounded_wait": (_I, [_I, _V, _V]),
    "flashloop_status_string": (ctypes.c_char_p, [_I]),
    "flashloop_paged_plan": (_I, [_PP, _V, _V, _V, _I, _V, _V, _V, _V, _V, _V, _V, _V, _V]),
    "flashloop_paged_kv_write": (_I, [_PP, _RW, _RW, _I, _V, _PG, _PG, _V, _V]),
    "flashloop_prompt_attn": (_I, [_PP, _RW, _RW, _RW, _V, _RW, _V, _V, _V]),
    "flashloop_paged_attn_workspace_bytes": (c_size_t, [_PP]),
    "flashloop_paged_attn": (_I, [_PP, _RW, _PG, _PG, _V, _V, _V, _RW, _V, _V, c_size_t, _V, _V]),
}
for _name, (_res, _args) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def header_functions():
    """Names of the functions include/flashloop.h declares."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(flashloop_[a-z_0-9]+)\s*\(",
                                 text, flags=re.M)))


def exported_symbols():
    return {n for n in header_functions() if hasattr(_lib, n)}


# ----------------------------------------------------------------------------- marshalling
def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(name, rc):
    if rc != 0:
        raise FlashLoopError(name, rc)
    return rc


def flashloop_workspace_bytes(params: Params) -> int:
    return int(_lib.flashloop_workspace_bytes(ctypes.byref(params)))


def flashloop_cache_bytes(params: Params, n_per_loop) -> int:
    arr = (c_int32 * MAX_LOOPS)(*list(n_per_loop))
    return int(_lib.flashloop_cache_bytes(ctypes.byref(params), ctypes.cast(arr, c_void_p)))


def flashloop_selection_loop(params: Params, loop: int) -> int:
    return int(_lib.flashloop_selection_loop(ctypes.byref(params), loop))


def flashloop_status_string(status: int) -> str:
    return _lib.flashloop_status_string(status).decode()


def flashloop_rope_table(params, n_pos, cs, stream=None):
    return _check("flashloop_rope_table",
                  _lib.flashloop_rope_table(ctypes.byref(params), n_pos, _ptr(cs), _stream(stream)))


def flashloop_gate(params, x_cur, x_prev, prev_active, n_prev, prev_capacity, active_out, slot_out,
                   n_active_out, out_capacity, workspace, err_word, stream=None):
    return _check("flashloop_gate", _lib.flashloop_gate(
        ctypes.byref(params), _ptr(x_cur), _ptr(x_prev), _ptr(prev_active), _ptr(n_prev),
        prev_capacity, _ptr(active_out), _ptr(slot_out), _ptr(n_active_out), out_capacity,
        _ptr(workspace), _ptr(err_word), _stream(stream)))


def flashloop_gate_topk(params, x_cur, x_prev, prev_active, n_prev, prev_capacity, budget, active_out,
                        slot_out, n_active_out, out_capacity, workspace, err_word, stream=None):
    return _check("flashloop_gate_topk", _lib.flashloop_gate_topk(
        ctypes.byref(params), _ptr(x_cur), _ptr(x_prev), _ptr(prev_active), _ptr(n_prev), prev_capacity,
        budget, _ptr(active_out), _ptr(slot_out), _ptr(n_active_out), out_capacity, _ptr(workspace),
        _ptr(err_word), _stream(stream)))


def flashloop_gate_noalloc(params, x_cur, x_prev, prev_active, n_prev, prev_capacity, active_out,
                           slot_out, n_active_out, out_capacity, err_word, stream=None):
    """flashloop_gate without a workspace: for callers that cannot allocate;
    its scratch is a fixed device array inside the library (see the header)."""
    return _check("flashloop_gate_noalloc", _lib.flashloop_gate_noalloc(
        ctypes.byref(params), _ptr(x_cur), _ptr(x_prev), _ptr(prev_active), _ptr(n_prev),
        prev_capacity, _ptr(active_out), _ptr(slot_out), _ptr(n_active_out), out_capacity,
        _ptr(err_word), _stream(stream)))


def flashloop_qkv_gathered(params, x, active, n_active, capacity, w_qkv, rope_cs, q_out, k_out,
                           v_out, stream=None):
    return _check("flashloop_qkv_gathered", _lib.flashloop_qkv_gathered(
        ctypes.byref(params), _ptr(x), _ptr(active), _ptr(n_active), capacity, _ptr(w_qkv),
        _ptr(rope_cs), _ptr(q_out), _ptr(k_out), _ptr(v_out), _stream(stream)))


def flashloop_kv_quant_residual(params, loop, k_new, v_new, active, n_active, state, stream=None):
    return _check("flashloop_kv_quant_residual", _lib.flashloop_kv_quant_residual(
        ctypes.byref(params), loop, _ptr(k_new), _ptr(v_new), _ptr(active), _ptr(n_active),
        ctypes.byref(state.c), _stream(stream)))


def flashloop_qkv_quant(params, loop, x, active, n_active, w_qkv, state, q_out, stream=None):
    return _check("flashloop_qkv_quant", _lib.flashloop_qkv_quant(
        ctypes.byref(params), loop, _ptr(x), _ptr(active), _ptr(n_active), _ptr(w_qkv),
        ctypes.byref(state.c), _ptr(q_out), _stream(stream)))


def flashloop_paper_kv_quant(params, loop, k_new, v_new, active, n_active, state, stream=None):
    return _check("flashloop_paper_kv_quant", _lib.flashloop_paper_kv_quant(
        ctypes.byref(params), loop, _ptr(k_new), _ptr(v_new), _ptr(active), _ptr(n_active),
        ctypes.byref(state.c), _stream(stream)))


def flashloop_topk_columns(params, mass, candidates, n_cand, k, out, stream=None):
    return _check("flashloop_topk_columns", _lib.flashloop_topk_columns(
        ctypes.byref(params), _ptr(mass), _ptr(candidates), n_cand, k, _ptr(out), _stream(stream)))


def flashloop_selcol_dequant(params, loop, state, stream=None):
    return _check("flashloop_selcol_dequant", _lib.flashloop_selcol_dequant(
        ctypes.byref(params), loop, ctypes.byref(state.c), _stream(stream)))


def flashloop_sparse_attn_update(params, loop, state, want_colmass=0, stream=None):
    return _check("flashloop_sparse_attn_update", _lib.flashloop_sparse_attn_update(
        ctypes.byref(params), loop, ctypes.byref(state.c), int(want_colmass), _stream(stream)))


def flashloop_out_proj(params, o, active, n_active, capacity, w_o, y, stream=None):
    return _check("flashloop_out_proj", _lib.flashloop_out_proj(
        ctypes.byref(params), _ptr(o), _ptr(active), _ptr(n_active), capacity, _ptr(w_o), _ptr(y),
        _stream(stream)))


def flashloop_loop_step(params, loop, x_cur, x_prev, w_qkv, w_o, state, stream=None):
    return _check("flashloop_loop_step", _lib.flashloop_loop_step(
        ctypes.byref(params), loop, _ptr(x_cur), _ptr(x_prev), _ptr(w_qkv), _ptr(w_o),
        ctypes.byref(state.c), _stream(stream)))


def flashloop_kv_step(params, loop, x_cur, x_prev, w_qkv, state, stream=None):
    return _check("flashloop_kv_step", _lib.flashloop_kv_step(
        ctypes.byref(params), loop, _ptr(x_cur), _ptr(x_prev), _ptr(w_qkv), ctypes.byref(state.c),
        _stream(stream)))


def flashloop_kv_workspace_bytes(params: Params) -> int:
    return int(_lib.flashloop_kv_workspace_bytes(ctypes.byref(params)))


def flashloop_decode_workspace_bytes(params: Params) -> int:
    return int(_lib.flashloop_decode_workspace_bytes(ctypes.byref(params)))


def flashloop_decode_attn(params, loop, ctx, dstate, stream=None):
    return _check("flashloop_decode_attn", _lib.flashloop_decode_attn(
        ctypes.byref(params), loop, ctypes.byref(ctx.c), ctypes.byref(dstate.c), _stream(stream)))


def flashloop_decode_qkv(params, loop, x_tok, w_qkv, dstate, stream=None):
    return _check("flashloop_decode_qkv", _lib.flashloop_decode_qkv(
        ctypes.byref(params), loop, _ptr(x_tok), _ptr(w_qkv), ctypes.byref(dstate.c), _stream(stream)))


def flashloop_decode_select(params, dstate, stream=None):
    return _check("flashloop_decode_select", _lib.flashloop_decode_select(
        ctypes.byref(params), ctypes.byref(dstate.c), _stream(stream)))


def flashloop_decode_out(params, w_o, dstate, stream=None):
    return _check("flashloop_decode_out", _lib.flashloop_decode_out(
        ctypes.byref(params), _ptr(w_o), ctypes.byref(dstate.c), _stream(stream)))


def flashloop_decode_step(params, loop, x_tok, w_qkv, w_o, ctx, dstate, stream=None):
    return _check("flashloop_decode_step", _lib.flashloop_decode_step(
        ctypes.byref(params), loop, _ptr(x_tok), _ptr(w_qkv), _ptr(w_o), ctypes.byref(ctx.c),
        ctypes.byref(dstate.c), _stream(stream)))


def flashloop_selftest_bounded_wait(kind, err_word, stream=None):
    return _check("flashloop_selftest_bounded_wait", _lib.flashloop_selftest_bounded_wait(
        int(kind), _ptr(err_word), _stream(stream)))


def flashloop_check_error_word(err_word, stream=None):
    """Returns the device error code (0 = none); synchronises the stream."""
    code = c_int32(0)
    rc = _lib.flashloop_check_error_word(_ptr(err_word), ctypes.byref(code), _stream(stream))
    if rc not in (0, -4):
        raise FlashLoopError("flashloop_check_error_word", rc)
    return int(code.value)


# ----------------------------------------------------------------------------- many requests
def _in_rows(shape, row):
    """Whether a contiguous tensor is rows of `row` elements: flat, or its last dimensions make up a row."""
    size = 1
    for d in reversed(shape):
        if size == row:
            return True
        size *= d
    return size == row or len(shape) < 2


def _vec(fn, name, t, n, dtype, dev, row=1):
    """Address of a contiguous vector of at least n elements, in rows of `row`, on CUDA device dev (an index)."""
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= n and t.is_contiguous() and (row == 1 or n == 0 or _in_rows(t.shape, row)):
        return t.data_ptr()
    raise FlashLoopError(fn, -1, f"{name}: a contiguous {dtype} tensor of at least {n} elements{f' in rows of {row}' if row > 1 else ''} "
                                 f"on cuda:{dev}, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(fn, name, t, shape, dtype, dev, written=False):
    """flashloop_rows of [tokens, heads, head_dim]."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise FlashLoopError(fn, -1, f"{name}: {dtype} {shape} on cuda:{dev}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    st, sh, se = t.stride()
    if se != 1:
        raise FlashLoopError(fn, -1, f"{name}: head_dim has to be contiguous")
    if written and (st == 0 and shape[0] > 1 or sh == 0 and shape[1] > 1):
        raise FlashLoopError(fn, -1, f"{name}: rows that overlap")
    # a dimension of one may have any stride
    return RowsC(t.data_ptr(), st if shape[0] > 1 else shape[2], sh if shape[1] > 1 else shape[2])


def _pages(fn, name, t, p, dtype, dev, written=False):
    """flashloop_pages of [n_pages, page_size, n_kv_heads, head_dim]."""
    shape = (p.n_pages, p.page_size, p.n_kv_heads, p.head_dim)
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise FlashLoopError(fn, -1, f"{name}: {dtype} {shape} on cuda:{dev}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    sp, st, sh, se = t.stride()
    if se != 1:
        raise FlashLoopError(fn, -1, f"{name}: head_dim has to be contiguous")
    if written and (sp == 0 and shape[0] > 1 or st == 0 or sh == 0 and shape[2] > 1):
        raise FlashLoopError(fn, -1, f"{name}: pages that overlap")
    return PagesC(t.data_ptr(), sp if shape[0] > 1 else shape[3], st, sh if shape[2] > 1 else shape[3])


def _paged_dtype(fn, p):
    if p.dtype not in (0, 1):
        raise FlashLoopError(fn, -2, f"dtype {p.dtype}")
    return torch.float16 if p.dtype else torch.bfloat16


# The same marshalling in C++ for the plain case, tensors on the current device; None where it leaves
# a call to the functions below.  It is built for one torch and interpreter; the functions below serve
# any, with 10 us of host time a call where it takes 4.
class _NoFastcall:
    plan = write = prompt = attn = staticmethod(lambda *args: None)
    bind = plan


from .build import fastcall_fits  # noqa: E402  (behind the library, without which there is nothing to build for)

try:
    if not fastcall_fits():
        raise ImportError("missing, or built for another torch or interpreter")
    from . import _fastcall
except ImportError as exc:
    _fastcall = _NoFastcall
    warnings.warn(f"{_PKG}/_fastcall.so: {exc}. The many-request calls take longer on the host; build it with "
                  "`python -m cross_loop_sparse_b200.build`", stacklevel=2)
_fastcall.bind(*(ctypes.cast(getattr(_lib, fn), c_void_p).value for fn in (
    "flashloop_paged_plan", "flashloop_paged_kv_write", "flashloop_prompt_attn", "flashloop_paged_attn")))


def _done(fn, rc):
    if rc:
        raise FlashLoopError(fn, rc)
    return rc


# The current stream's handle without a Stream object (a microsecond less a call) where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, dev, stream, *args):
    """Call into the library on the tensors' device, on its current stream by default."""
    if dev < 0:
        raise FlashLoopError(fn, -1, "tensors on a CUDA device")
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            rc = getattr(_lib, fn)(*args, _stream(stream))
    else:
        rc = getattr(_lib, fn)(*args, _raw_stream(dev) if stream is None and _raw_stream else _stream(stream))
    return _done(fn, rc)


def flashloop_paged_plan(params, kv_lens, new_lens, free_pages, n_free, block_table, cu, kv_lens_out, slot_map,
                         positions, n_free_out, err_word, stream=None):
    """Block tables, slot maps, positions and packed starts of the tokens that the requests
    append (see the header).  int32 tensors; block_table [batch, max_blocks] (or flat) and n_free_out,
    kv_lens_out, cu [batch + 1], slot_map and positions [max_tokens] are written."""
    rc = _fastcall.plan(params, kv_lens, new_lens, free_pages, n_free, block_table, cu, kv_lens_out, slot_map, positions,
                        n_free_out, err_word, stream)
    if rc is not None:
        return _done("flashloop_paged_plan", rc)
    fn, p, dev, i32 = "flashloop_paged_plan", params, kv_lens.get_device(), torch.int32
    B, T = max(p.batch, 0), max(p.max_tokens, 0)
    return _launch(fn, dev, stream, ctypes.byref(p), _vec(fn, "kv_lens", kv_lens, B, i32, dev),
                   _vec(fn, "new_lens", new_lens, B, i32, dev),
                   _vec(fn, "free_pages", free_pages, 0, i32, dev), min(free_pages.numel(), 2 ** 31 - 1), _vec(fn, "n_free", n_free, 1, i32, dev),
                   _vec(fn, "block_table", block_table, B * p.max_blocks, i32, dev, p.max_blocks),
                   _vec(fn, "cu", cu, B + 1, i32, dev), _vec(fn, "kv_lens_out", kv_lens_out, B, i32, dev),
                   _vec(fn, "slot_map", slot_map, T, i32, dev), _vec(fn, "positions", positions, T, i32, dev),
                   _vec(fn, "n_free_out", n_free_out, 1, i32, dev), _vec(fn, "err_word", err_word, 1, i32, dev))


def flashloop_paged_kv_write(params, k, v, slot_map, k_cache, v_cache, err_word, stream=None):
    """Write k and v [max_tokens, n_kv_heads, head_dim] (params.dtype or float32) into the pages
    [n_pages, page_size, n_kv_heads, head_dim] of their slots."""
    rc = _fastcall.write(params, k, v, slot_map, k_cache, v_cache, err_word, stream)
    if rc is not None:
        return _done("flashloop_paged_kv_write", rc)
    fn, p, dev = "flashloop_paged_kv_write", params, k_cache.get_device()
    dt = _paged_dtype(fn, p)
    shape = (p.max_tokens, p.n_kv_heads, p.head_dim)
    if k.dtype not in PAGED_DTYPES:
        raise FlashLoopError(fn, -2, f"k: {k.dtype}")
    kr, vr = _rows(fn, "k", k, shape, k.dtype, dev), _rows(fn, "v", v, shape, k.dtype, dev)
    kc, vc = _pages(fn, "k_cache", k_cache, p, dt, dev, True), _pages(fn, "v_cache", v_cache, p, dt, dev, True)
    return _launch(fn, dev, stream, ctypes.byref(p), ctypes.byref(kr), ctypes.byref(vr), PAGED_DTYPES[k.dtype],
                   _vec(fn, "slot_map", slot_map, p.max_tokens, torch.int32, dev), ctypes.byref(kc), ctypes.byref(vc),
                   _vec(fn, "err_word", err_word, 1, torch.int32, dev))


def flashloop_prompt_attn(params, q, k, v, cu, o, lse, err_word, stream=None):
    """Causal attention over packed prompts: q and o [max_tokens, n_heads, head_dim], k and v
    [max_tokens, n_kv_heads, head_dim], cu int32 [batch + 1], lse float32 [n_heads, max_tokens] or None."""
    rc = _fastcall.prompt(params, q, k, v, cu, o, lse, err_word, stream)
    if rc is not None:
        return _done("flashloop_prompt_attn", rc)
    fn, p, dev = "flashloop_prompt_attn", params, q.get_device()
    dt = _paged_dtype(fn, p)
    qs, ks = (p.max_tokens, p.n_heads, p.head_dim), (p.max_tokens, p.n_kv_heads, p.head_dim)
    qr, kr, vr = _rows(fn, "q", q, qs, dt, dev), _rows(fn, "k", k, ks, dt, dev), _rows(fn, "v", v, ks, dt, dev)
    orr = _rows(fn, "o", o, qs, dt, dev, True)
    return _launch(fn, dev, stream, ctypes.byref(p), ctypes.byref(qr), ctypes.byref(kr), ctypes.byref(vr),
                   _vec(fn, "cu", cu, p.batch + 1, torch.int32, dev), ctypes.byref(orr),
                   None if lse is None else _vec(fn, "lse", lse, p.n_heads * p.max_tokens, torch.float32, dev, p.max_tokens),
                   _vec(fn, "err_word", err_word, 1, torch.int32, dev))


def flashloop_paged_attn_workspace_bytes(params: PagedParams) -> int:
    return int(_lib.flashloop_paged_attn_workspace_bytes(ctypes.byref(params)))


def flashloop_paged_attn(params, q, k_cache, v_cache, block_table, kv_lens, cu, o, lse, workspace, err_word,
                         stream=None):
    """Attention of the requests' new rows q [max_tokens, n_heads, head_dim] over their pages
    (block_table int32 [batch, max_blocks], kv_lens int32 [batch] with the new tokens counted)."""
    rc = _fastcall.attn(params, q, k_cache, v_cache, block_table, kv_lens, cu, o, lse, workspace, err_word, stream)
    if rc is not None:
        return _done("flashloop_paged_attn", rc)
    fn, p, dev = "flashloop_paged_attn", params, q.get_device()
    dt = _paged_dtype(fn, p)
    qs = (p.max_tokens, p.n_heads, p.head_dim)
    qr, orr = _rows(fn, "q", q, qs, dt, dev), _rows(fn, "o", o, qs, dt, dev, True)
    kc, vc = _pages(fn, "k_cache", k_cache, p, dt, dev), _pages(fn, "v_cache", v_cache, p, dt, dev)
    i32 = torch.int32
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise FlashLoopError(fn, -1, "workspace: contiguous, on the tensors' device")
    return _launch(fn, dev, stream, ctypes.byref(p), ctypes.byref(qr), ctypes.byref(kc), ctypes.byref(vc),
                   _vec(fn, "block_table", block_table, p.batch * p.max_blocks, i32, dev, p.max_blocks),
                   _vec(fn, "kv_lens", kv_lens, p.batch, i32, dev), _vec(fn, "cu", cu, p.batch + 1, i32, dev),
                   ctypes.byref(orr),
                   None if lse is None else _vec(fn, "lse", lse, p.n_heads * p.max_tokens, torch.float32, dev, p.max_tokens),
                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                   _vec(fn, "err_word", err_word, 1, i32, dev))


# ----------------------------------------------------------------------------- state
class FlashLoopState:
    """Caller-owned device buffers of one sequence (torch tensors) and the
    C struct that points at them.  Allocation is the only work done here."""

    def __init__(self, params: Params, device="cuda", kv_only=False, rope_period=None):
        """kv_only: only what flashloop_kv_step touches (caches, active lists,
        slot maps, counts, the gate's scratch, RoPE table, error word).
        rope_period: positions restart every rope_period rows (sequences laid
        end to end, as a decode context is)."""
        self.params = params
        S, H, dh, d, R = params.seq, params.n_heads, params.head_dim, params.d_model, params.n_loops
        self.device = device
        dev = torch.device(device)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)  # noqa: E731
        self.t = {}
        c = StateC()
        self._paper = []
        if params.kv_scheme == 1:
            # the pages' cache setting: per loop INT4 codes, fp16 scales and minima, bf16 tail
            tail = min(PAPER_TAIL, S)
            body = S - tail
            for name in ("k", "v"):
                kv = PaperKV()
                for r in range(1, R + 1):
                    rows = max(body if r == 1 else params.capacity[r - 1], 1)
                    groups = (rows + PAPER_GROUP - 1) // PAPER_GROUP
                    gshape = (groups, H, dh) if name == "k" else (rows, H, dh // PAPER_GROUP)
                    self.t[f"p{name}_codes{r}"] = z((rows, H, dh // 2), torch.uint8)
                    self.t[f"p{name}_scale{r}"] = z(gshape, torch.float16)
                    self.t[f"p{name}_min{r}"] = z(gshape, torch.float16)
                    self.t[f"p{name}_tail{r}"] = z((max(tail, 1), H, dh), torch.bfloat16)
                    kv.codes[r - 1] = self.t[f"p{name}_codes{r}"].data_ptr()
                    kv.scale[r - 1] = self.t[f"p{name}_scale{r}"].data_ptr()
                    kv.minv[r - 1] = self.t[f"p{name}_min{r}"].data_ptr()
                    kv.tail[r - 1] = self.t[f"p{name}_tail{r}"].data_ptr()
                self._paper.append(kv)
            c.paper_k = ctypes.pointer(self._paper[0])
            c.paper_v = ctypes.pointer(self._paper[1])
        for name, kv in (("k", c.k), ("v", c.v)) if params.kv_scheme == 0 else ():
            base = z((S, H, dh), torch.int8)
            bs = z((S, H, dh // GROUP), torch.float16)
            self.t[f"{name}_base"], self.t[f"{name}_base_s"] = base, bs
            kv.base_codes, kv.base_scales = base.data_ptr(), bs.data_ptr()
            for r in range(2, R + 1):
                cap, b = params.capacity[r - 1], params.bits[r - 1]
                codes = z((cap, H, dh * b // 8), torch.uint8)
                sc = z((cap, H, dh // GROUP), torch.float16)
                self.t[f"{name}_res{r}"], self.t[f"{name}_res{r}_s"] = codes, sc
                kv.res_codes[r - 1], kv.res_scales[r - 1] = codes.data_ptr(), sc.data_ptr()
        for r in range(2, R + 1):
            act = z((params.capacity[r - 1],), torch.int32)
            slot = torch.full((S,), -1, dtype=torch.int32, device=dev)
            self.t[f"active{r}"], self.t[f"slot{r}"] = act, slot
            c.active[r - 1], c.slot[r - 1] = act.data_ptr(), slot.data_ptr()
        self.t["n_active"] = z((MAX_LOOPS,), torch.int32)
        c.n_active = self.t["n_active"].data_ptr()
        self.t["rope_cs"] = z((S, dh // 2, 2), torch.float32)
        self.t["err"] = z((1,), torch.int32)
        c.rope_cs, c.err_word = self.t["rope_cs"].data_ptr(), self.t["err"].data_ptr()
        self.c = c
        if rope_period is None:
            flashloop_rope_table(params, S, self.t["rope_cs"])
        else:
            assert S % rope_period == 0
            one = z((rope_period, dh // 2, 2), torch.float32)
            flashloop_rope_table(params, rope_period, one)
            self.t["rope_cs"].copy_(one.repeat(S // rope_period, 1, 1))
        if kv_only:
            ws = flashloop_kv_workspace_bytes(params)
            self.t["workspace"] = z((max(ws, 256),), torch.uint8)
            c.workspace, c.workspace_bytes = self.t["workspace"].data_ptr(), ws
            return
        for i in range(3):
            self.t[f"q{i}"] = z((S, d), torch.bfloat16)
            self.t[f"m{i}"] = z((H, S), torch.float32)
            self.t[f"Z{i}"] = z((H, S), torch.float32)
            self.t[f"N{i}"] = z((H, S, dh), torch.float32)
            c.q[i], c.m[i] = self.t[f"q{i}"].data_ptr(), self.t[f"m{i}"].data_ptr()
            c.Z[i], c.N[i] = self.t[f"Z{i}"].data_ptr(), self.t[f"N{i}"].data_ptr()
            if params.fixed_mass:
                self.t[f"G{i}"] = z((H, S), torch.float32)
                c.G[i] = self.t[f"G{i}"].data_ptr()
        for i in range(2):
            self.t[f"colmass{i}"] = z((H, S), torch.float32)
            c.colmass[i] = self.t[f"colmass{i}"].data_ptr()
        for r in range(2, R + 1):
            if flashloop_selection_loop(params, r) == r:
                self.t[f"cols{r}"] = z((H, params.topk[r - 1]), torch.int32)
                c.cols[r - 1] = self.t[f"cols{r}"].data_ptr()
        self.t["O"] = z((S, d), torch.bfloat16)
        self.t["Y"] = z((S, d), torch.bfloat16)
        ws = flashloop_workspace_bytes(params)
        self.t["workspace"] = z((max(ws, 256),), torch.uint8)
        c.O, c.Y = self.t["O"].data_ptr(), self.t["Y"].data_ptr()
        c.workspace, c.workspace_bytes = self.t["workspace"].data_ptr(), ws

    def __getitem__(self, key):
        return self.t[key]

    def cols_for_loop(self, r):
        return self.t[f"cols{flashloop_selection_loop(self.params, r)}"]

    def q_slot(self, r):
        return 0 if r == 1 else 1 + (r % 2)

    def error_code(self, stream=None):
        return flashloop_check_error_word(self.t["err"], stream)


# ----------------------------------------------------------------------------- decode
def decode_context_params(params: Params, capacity=None) -> Params:
    """Params of the B contexts of a decode laid end to end (seq = B*S), the
    layout flashloop_decode_attn reads; capacities default to B*S."""
    p = Params()
    ctypes.pointer(p)[0] = params
    p.seq = params.batch * params.seq
    p.batch = 1
    for r in range(params.n_loops):
        p.capacity[r] = p.seq if capacity is None else capacity[r]
    return p


class DecodeContext(FlashLoopState):
    """Caches of the B contexts of a decode (kv-only state of B*S rows, RoPE
    positions restarting at every sequence)."""

    def __init__(self, params: Params, device="cuda", capacity=None):
        self.dec_params = params
        super().__init__(decode_context_params(params, capacity), device, kv_only=True,
                         rope_period=params.seq)

    def prepare(self, xs, w_qkv, stream=None):
        """KV path of loops 1..R: xs[r-1] is bf16 [B*S, d] (the contexts of loop r)."""
        p = self.params
        for r in range(1, p.n_loops + 1):
            flashloop_kv_step(p, r, xs[r - 1], xs[r - 2] if r > 1 else None, w_qkv, self, stream)


class DecodeState:
    """Caller-owned device buffers of a decode step (B sequences, one token
    each at position S) and the C struct that points at them."""

    def __init__(self, params: Params, device="cuda"):
        self.params = params
        S, H, dh, d, R, B = (params.seq, params.n_heads, params.head_dim, params.d_model, params.n_loops,
                             params.batch)
        dev = torch.device(device)
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)  # noqa: E731
        self.t = {}
        c = DecodeStateC()
        for name, kv in (("k", c.k), ("v", c.v)):
            base = z((B, H, dh), torch.int8)
            bs = z((B, H, dh // GROUP), torch.float16)
            self.t[f"{name}_base"], self.t[f"{name}_base_s"] = base, bs
            kv.base_codes, kv.base_scales = base.data_ptr(), bs.data_ptr()
            for r in range(2, R + 1):
                b = params.bits[r - 1]
                codes = z((B, H, dh * b // 8), torch.uint8)
                sc = z((B, H, dh // GROUP), torch.float16)
                self.t[f"{name}_res{r}"], self.t[f"{name}_res{r}_s"] = codes, sc
                kv.res_codes[r - 1], kv.res_scales[r - 1] = codes.data_ptr(), sc.data_ptr()
        for i in range(3):
            self.t[f"q{i}"] = z((B, d), torch.bfloat16)
            self.t[f"m{i}"] = z((B, H), torch.float32)
            self.t[f"Z{i}"] = z((B, H), torch.float32)
            self.t[f"N{i}"] = z((B, H, dh), torch.float32)
            c.q[i], c.m[i] = self.t[f"q{i}"].data_ptr(), self.t[f"m{i}"].data_ptr()
            c.Z[i], c.N[i] = self.t[f"Z{i}"].data_ptr(), self.t[f"N{i}"].data_ptr()
        self.t["probs"] = z((B, H, S + 1), torch.float32)
        k = params.topk[1] if R >= 2 else 1
        self.t["cols"] = z((B, H, k), torch.int32)
        self.t["O"] = z((B, d), torch.bfloat16)
        self.t["Y"] = z((B, d), torch.bfloat16)
        self.t["err"] = z((1,), torch.int32)
        table = z((S + 1, dh // 2, 2), torch.float32)
        flashloop_rope_table(params, S + 1, table)
        self.t["rope_cs"] = table[S].clone()
        ws = flashloop_decode_workspace_bytes(params)
        if ws == 0:
            raise FlashLoopError("flashloop_decode_workspace_bytes", -2)
        self.t["workspace"] = z((ws,), torch.uint8)
        c.rope_cs, c.probs, c.cols = (self.t["rope_cs"].data_ptr(), self.t["probs"].data_ptr(),
                                      self.t["cols"].data_ptr())
        c.O, c.Y, c.err_word = self.t["O"].data_ptr(), self.t["Y"].data_ptr(), self.t["err"].data_ptr()
        c.workspace, c.workspace_bytes = self.t["workspace"].data_ptr(), ws
        self.c = c

    def __getitem__(self, key):
        return self.t[key]

    def q_slot(self, r):
        return 0 if r == 1 else 1 + (r % 2)

    def error_code(self, stream=None):
        return flashloop_check_error_word(self.t["err"], stream)
