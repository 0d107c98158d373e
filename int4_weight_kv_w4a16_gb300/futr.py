"""Thin ctypes binding of libfutr.so (C ABI in include/futr.h).

Every function here only marshals arguments: device buffers are torch CUDA
tensors (passed by ``data_ptr()``), streams are torch streams (or None for the
current stream), descriptors are the ctypes mirrors of the C structs.  All
arithmetic runs in the library's kernels; if the library is missing, ``lib()``
raises and nothing falls back to another implementation.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfutr.so")
LIB_DEBUG_PATH = os.path.join(PKG, "libfutr_debug.so")

FUTR_OK = 0
FUTR_ERR_INVALID_ARG = 1
FUTR_ERR_UNSUPPORTED = 2
FUTR_ERR_CUDA = 3
FUTR_ERR_OUT_OF_RANGE = 4
FUTR_ERR_TIMEOUT = 5
FUTR_ERR_BAD_BLOB = 6
FUTR_ERR_NOT_PD = 7
FUTR_ERR_CORRUPT = 8
FUTR_ERR_BOUNDS = 9
FUTR_ERR_NOT_FINITE = 10

FUTR_ERR_NO_PAGES = 11
FUTR_ERR_NOT_HELD = 12
FUTR_ERR_SHARED = 13

FUTR_DTYPE_BF16, FUTR_DTYPE_F16, FUTR_DTYPE_F32 = range(3)

FUTR_PROJ_QKV, FUTR_PROJ_O, FUTR_PROJ_GATE, FUTR_PROJ_UP, FUTR_PROJ_DOWN = range(5)


class futr_shape(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_q_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("inter", C.c_int32), ("group", C.c_int32),
                ("had_block", C.c_int32), ("rms_eps", C.c_float), ("rope_theta", C.c_float)]


class futr_kv(C.Structure):
    _fields_ = [("shape", futr_shape), ("n_layers", C.c_int32), ("max_batch", C.c_int32),
                ("capacity", C.c_int32), ("_pad", C.c_int32), ("base", C.c_void_p),
                ("bytes", C.c_uint64), ("stream_bytes", C.c_uint64), ("rope_offset", C.c_uint64),
                ("err_offset", C.c_uint64), ("magic", C.c_uint64)]


class futr_ws(C.Structure):
    _fields_ = [("shape", futr_shape), ("max_batch", C.c_int32), ("capacity", C.c_int32),
                ("n_sm", C.c_int32), ("_pad", C.c_int32), ("base", C.c_void_p), ("bytes", C.c_uint64),
                ("off_err", C.c_uint64), ("off_qrot", C.c_uint64), ("off_o", C.c_uint64),
                ("off_h", C.c_uint64), ("off_a", C.c_uint64), ("off_xin", C.c_uint64),
                ("off_yout", C.c_uint64), ("off_pos", C.c_uint64), ("off_part", C.c_uint64),
                ("part_bytes", C.c_uint64), ("off_apart", C.c_uint64), ("apart_bytes", C.c_uint64),
                ("off_cnt", C.c_uint64), ("cnt_words", C.c_uint64), ("magic", C.c_uint64)]


class futr_paged(C.Structure):
    _fields_ = [("shape", futr_shape), ("n_layers", C.c_int32), ("n_pages", C.c_int32), ("page", C.c_int32),
                ("max_pos", C.c_int32), ("rope", C.c_int32), ("base", C.c_void_p), ("bytes", C.c_uint64),
                ("scale_offset", C.c_uint64), ("rope_offset", C.c_uint64), ("err_offset", C.c_uint64),
                ("copy_map", C.c_uint64 * 16), ("magic", C.c_uint64)]


class futr_paged_ws(C.Structure):
    _fields_ = [("head_dim", C.c_int32), ("ctas", C.c_int32), ("base", C.c_void_p), ("bytes", C.c_uint64),
                ("err_offset", C.c_uint64), ("rec_offset", C.c_uint64), ("magic", C.c_uint64)]


class futr_moe_shape(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("inter", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("group", C.c_int32), ("renorm", C.c_int32), ("rms_eps", C.c_float)]


class futr_moe_ws(C.Structure):
    _fields_ = [("shape", futr_moe_shape), ("max_batch", C.c_int32), ("ctas", C.c_int32), ("_pad", C.c_int32),
                ("base", C.c_void_p), ("bytes", C.c_uint64), ("off_cnt", C.c_uint64), ("off_rms", C.c_uint64),
                ("off_logits", C.c_uint64), ("off_x", C.c_uint64), ("off_act", C.c_uint64), ("off_rec", C.c_uint64), ("blob_bytes", C.c_uint64),
                ("magic", C.c_uint64)]


class futr_beam_ws(C.Structure):
    _fields_ = [("rows", C.c_int32), ("keep", C.c_int32), ("ctas", C.c_int32), ("_pad", C.c_int32),
                ("base", C.c_void_p), ("bytes", C.c_uint64), ("err_offset", C.c_uint64), ("cnt_offset", C.c_uint64),
                ("row_offset", C.c_uint64), ("rec_offset", C.c_uint64), ("magic", C.c_uint64)]


class futr_pages(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("max_seqs", C.c_int32), ("base", C.c_void_p), ("bytes", C.c_uint64),
                ("refs_offset", C.c_uint64), ("free_offset", C.c_uint64), ("plan_offset", C.c_uint64),
                ("err_offset", C.c_uint64), ("magic", C.c_uint64)]


class FutrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.futr_status_string(status).decode() if _lib else status}")


_lib: Optional[C.CDLL] = None
P = C.c_void_p
I32 = C.c_int32
_SIGS = {
    "futr_status_string": (C.c_char_p, [I32]),
    "futr_version": (I32, []),
    "futr_weights_size": (I32, [C.POINTER(futr_shape), C.POINTER(C.c_size_t)]),
    "futr_pack_weights": (I32, [C.POINTER(futr_shape)] + [P] * 10 + [C.c_size_t, P]),
    "futr_gptq_scratch_size": (I32, [C.POINTER(futr_shape), C.POINTER(C.c_size_t)]),
    "futr_pack_weights_gptq": (I32, [C.POINTER(futr_shape)] + [P] * 13 + [C.c_double, P, C.c_size_t, P,
                                                                          C.c_size_t, P]),
    "futr_unpack_weights": (I32, [C.POINTER(futr_shape), P, I32, P, P, P]),
    "futr_kv_size": (I32, [C.POINTER(futr_shape), I32, I32, I32, C.POINTER(C.c_size_t)]),
    "futr_kv_init": (I32, [C.POINTER(futr_shape), I32, I32, I32, P, C.c_size_t, C.POINTER(futr_kv), P]),
    "futr_kv_append": (I32, [C.POINTER(futr_kv), I32, I32, I32, P, I32, P, P, P]),
    "futr_kv_read": (I32, [C.POINTER(futr_kv), I32, I32, I32, P, P, P, P, P]),
    "futr_workspace_size": (I32, [C.POINTER(futr_shape), I32, I32, C.POINTER(C.c_size_t)]),
    "futr_workspace_init": (I32, [C.POINTER(futr_shape), I32, I32, P, C.c_size_t, C.POINTER(futr_ws), P]),
    "futr_decode_block": (I32, [P, P, C.POINTER(futr_kv), I32, I32, P, P, C.POINTER(futr_ws), P]),
    "futr_decode_block_timed": (I32, [P, P, C.POINTER(futr_kv), I32, I32, P, P, C.POINTER(futr_ws), P,
                                      C.POINTER(C.c_float)]),
    "futr_decode_block_host": (I32, [P, P, C.POINTER(futr_kv), I32, I32, P, P, C.POINTER(futr_ws), P]),
    "futr_check": (I32, [C.POINTER(futr_ws), C.POINTER(futr_kv), P]),
    "futr_decode_block_noalloc": (I32, [P, P, C.POINTER(futr_kv), I32, I32, P, P, P]),
    "futr_paged_size": (I32, [C.POINTER(futr_shape), I32, I32, I32, I32, C.POINTER(C.c_size_t)]),
    "futr_paged_init": (I32, [C.POINTER(futr_shape), I32, I32, I32, I32, I32, P, C.c_size_t,
                              C.POINTER(futr_paged), P]),
    "futr_paged_append": (I32, [P, I32, I32, P, P, I32, P, I32, P, C.c_int64, P, C.c_int64, I32, P]),
    "futr_paged_workspace_size": (I32, [C.POINTER(futr_shape), C.POINTER(C.c_size_t)]),
    "futr_paged_workspace_init": (I32, [C.POINTER(futr_shape), P, C.c_size_t, C.POINTER(futr_paged_ws), P]),
    "futr_paged_attention": (I32, [P, I32, I32, P, P, I32, P, I32, P, C.c_int64, P, C.c_int64, I32, C.c_float, I32,
                                   P, P]),
    "futr_paged_attention_sinks": (I32, [P, I32, I32, P, P, I32, P, I32, P, C.c_int64, P, C.c_int64, I32, C.c_float,
                                         I32, I32, P, P]),
    "futr_paged_check": (I32, [P, P, P]),
    "futr_beam_workspace_size": (I32, [I32, I32, C.POINTER(C.c_size_t)]),
    "futr_beam_workspace_init": (I32, [I32, I32, P, C.c_size_t, C.POINTER(futr_beam_ws), P]),
    "futr_beam_select": (I32, [P, C.c_int64, I32, I32, I32, I32, P, P, I32, I32, I32, P, P, P, P, P, P]),
    "futr_beam_check": (I32, [P, P]),
    "futr_kv_reorder": (I32, [P, I32, P, P, P]),
    "futr_pages_size": (I32, [I32, I32, C.POINTER(C.c_size_t)]),
    "futr_pages_init": (I32, [I32, I32, P, C.c_size_t, C.POINTER(futr_pages), P]),
    "futr_pages_hold": (I32, [P, P, I32, P, I32, P]),
    "futr_pages_grow": (I32, [P, P, I32, P, P, P, I32, P]),
    "futr_pages_free": (I32, [P, P, I32, P, P, I32, I32, I32, P]),
    "futr_pages_fork": (I32, [P, P, I32, P, P, P, I32, P]),
    "futr_pages_compact": (I32, [P, P, I32, P, I32, I32, I32, P]),
    "futr_pages_check": (I32, [P, C.POINTER(I32), P]),
    "futr_moe_weights_size": (I32, [C.POINTER(futr_moe_shape), C.POINTER(C.c_size_t)]),
    "futr_moe_pack": (I32, [C.POINTER(futr_moe_shape), I32, P, P, P, P, P, C.c_size_t, P]),
    "futr_moe_unpack": (I32, [C.POINTER(futr_moe_shape), P, I32, I32, P, P, P]),
    "futr_moe_workspace_size": (I32, [C.POINTER(futr_moe_shape), I32, C.POINTER(C.c_size_t)]),
    "futr_moe_workspace_init": (I32, [C.POINTER(futr_moe_shape), I32, P, C.c_size_t, C.POINTER(futr_moe_ws), P]),
    "futr_moe_layer": (I32, [P, P, P, P, I32, P, P, P, P, P, P]),
    "futr_moe_check": (I32, [P, P]),
    "futr_decode_step": (I32, [P, P, I32, C.POINTER(C.c_void_p), I32, C.POINTER(futr_kv), I32, P, P, P, P,
                               C.POINTER(futr_ws), P]),
}


def lib() -> C.CDLL:
    """Load libfutr.so (built by ``build.py``), or its debug variant
    libfutr_debug.so (``build.py --debug``: device bounds checks) when the
    environment has FUTR_DEBUG=1; raises if that library is missing."""
    global _lib
    if _lib is None:
        path = LIB_DEBUG_PATH if os.environ.get("FUTR_DEBUG") == "1" else LIB_PATH
        if not os.path.exists(path):
            flag = " --debug" if path == LIB_DEBUG_PATH else ""
            raise RuntimeError(f"{path} is not built; run int4_weight_kv_w4a16_gb300/build.py{flag}")
        h = C.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def _ok(status: int, where: str) -> None:
    if status != FUTR_OK:
        raise FutrError(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if hasattr(t, "ctypes"):  # numpy (host buffers)
        return t.ctypes.data
    raise TypeError(f"cannot pass {type(t)} as a buffer")


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(s) -> futr_shape:
    """futr_shape from any object with the BlockShape attributes."""
    return futr_shape(s.hidden, s.n_q_heads, s.n_kv_heads, s.head_dim, s.inter, s.group, s.had_block,
                      s.rms_eps, s.rope_theta)


def futr_status_string(status: int) -> str:
    return lib().futr_status_string(status).decode()


def futr_version() -> int:
    return lib().futr_version()


def futr_weights_size(shape: futr_shape) -> int:
    n = C.c_size_t()
    _ok(lib().futr_weights_size(C.byref(shape), C.byref(n)), "futr_weights_size")
    return n.value


def futr_pack_weights(shape, wq, wk, wv, wo, wgate, wup, wdown, g_attn, g_mlp, blob, stream=None):
    _ok(lib().futr_pack_weights(C.byref(shape), *[_ptr(t) for t in (wq, wk, wv, wo, wgate, wup, wdown,
                                                                    g_attn, g_mlp, blob)],
                                blob.numel() * blob.element_size(), _stream(stream)), "futr_pack_weights")


def futr_gptq_scratch_size(shape) -> int:
    n = C.c_size_t()
    _ok(lib().futr_gptq_scratch_size(C.byref(shape), C.byref(n)), "futr_gptq_scratch_size")
    return n.value


def futr_pack_weights_gptq(shape, wq, wk, wv, wo, wgate, wup, wdown, g_attn, g_mlp, h_attn, h_o, h_mlp, h_down,
                           damp, scratch, blob, stream=None):
    _ok(lib().futr_pack_weights_gptq(C.byref(shape), *[_ptr(t) for t in (wq, wk, wv, wo, wgate, wup, wdown,
                                                                         g_attn, g_mlp, h_attn, h_o, h_mlp,
                                                                         h_down)],
                                     float(damp), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                     _ptr(blob), blob.numel() * blob.element_size(), _stream(stream)),
        "futr_pack_weights_gptq")


def futr_unpack_weights(shape, blob, which, codes, scales, stream=None):
    _ok(lib().futr_unpack_weights(C.byref(shape), _ptr(blob), which, _ptr(codes), _ptr(scales),
                                  _stream(stream)), "futr_unpack_weights")


def futr_kv_size(shape, n_layers, max_batch, capacity) -> int:
    n = C.c_size_t()
    _ok(lib().futr_kv_size(C.byref(shape), n_layers, max_batch, capacity, C.byref(n)), "futr_kv_size")
    return n.value


def futr_kv_init(shape, n_layers, max_batch, capacity, kv_mem, stream=None) -> futr_kv:
    kv = futr_kv()
    _ok(lib().futr_kv_init(C.byref(shape), n_layers, max_batch, capacity, _ptr(kv_mem),
                           kv_mem.numel() * kv_mem.element_size(), C.byref(kv), _stream(stream)), "futr_kv_init")
    kv._mem = kv_mem  # keep the device buffer alive with the descriptor
    return kv


def futr_kv_append(kv, layer, seq0, batch, pos, n_tok, k, v, stream=None):
    _ok(lib().futr_kv_append(C.byref(kv), layer, seq0, batch, _ptr(pos), n_tok, _ptr(k), _ptr(v),
                             _stream(stream)), "futr_kv_append")


def futr_kv_read(kv, layer, seq, n_pos, k_codes, k_scales, v_codes, v_scales, stream=None):
    _ok(lib().futr_kv_read(C.byref(kv), layer, seq, n_pos, _ptr(k_codes), _ptr(k_scales), _ptr(v_codes),
                           _ptr(v_scales), _stream(stream)), "futr_kv_read")


def futr_workspace_size(shape, max_batch, capacity) -> int:
    n = C.c_size_t()
    _ok(lib().futr_workspace_size(C.byref(shape), max_batch, capacity, C.byref(n)), "futr_workspace_size")
    return n.value


def futr_workspace_init(shape, max_batch, capacity, ws_mem, stream=None) -> futr_ws:
    ws = futr_ws()
    _ok(lib().futr_workspace_init(C.byref(shape), max_batch, capacity, _ptr(ws_mem),
                                  ws_mem.numel() * ws_mem.element_size(), C.byref(ws), _stream(stream)),
        "futr_workspace_init")
    ws._mem = ws_mem
    return ws


def futr_decode_block(x, blob, kv, layer, batch, pos, y, ws, stream=None):
    _ok(lib().futr_decode_block(_ptr(x), _ptr(blob), C.byref(kv), layer, batch, _ptr(pos), _ptr(y),
                                C.byref(ws), _stream(stream)), "futr_decode_block")


def futr_decode_block_timed(x, blob, kv, layer, batch, pos, y, ws, stream=None) -> Sequence[float]:
    out = (C.c_float * 5)()
    _ok(lib().futr_decode_block_timed(_ptr(x), _ptr(blob), C.byref(kv), layer, batch, _ptr(pos), _ptr(y),
                                      C.byref(ws), _stream(stream), out), "futr_decode_block_timed")
    return list(out)


def futr_decode_block_host(x_host, blob, kv, layer, batch, pos_host, y_host, ws, stream=None):
    _ok(lib().futr_decode_block_host(_ptr(x_host), _ptr(blob), C.byref(kv), layer, batch, _ptr(pos_host),
                                     _ptr(y_host), C.byref(ws), _stream(stream)), "futr_decode_block_host")


def futr_decode_step(tokens, embedding, vocab, blobs, kv, batch, pos, g_final, lm_head, logits, ws, stream=None):
    """One complete decode step (embedding, every block in ``blobs``, final
    norm, bf16 LM head) -> fp32 logits [batch, vocab]."""
    arr = (C.c_void_p * len(blobs))(*[_ptr(b) for b in blobs])
    _ok(lib().futr_decode_step(_ptr(tokens), _ptr(embedding), vocab, arr, len(blobs), C.byref(kv), batch,
                               _ptr(pos), _ptr(g_final), _ptr(lm_head), _ptr(logits), C.byref(ws),
                               _stream(stream)), "futr_decode_step")


def futr_decode_block_noalloc(x, blob, kv, layer, batch, pos, y, stream=None):
    """futr_decode_block with the library's fixed scratch array instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _ok(lib().futr_decode_block_noalloc(_ptr(x), _ptr(blob), C.byref(kv), layer, batch, _ptr(pos), _ptr(y),
                                        _stream(stream)), "futr_decode_block_noalloc")


def futr_check(ws=None, kv=None, stream=None) -> int:
    """Synchronize and return the device status (0 = ok); does not raise."""
    return lib().futr_check(C.byref(ws) if ws is not None else None, C.byref(kv) if kv is not None else None,
                            _stream(stream))


# ----------------------------------------------------------------------------
# paged 8-bit cache.  Row tensors, positions and tables are torch CUDA tensors;
# their types, shapes and strides are checked here, the C side cannot see them.
# ----------------------------------------------------------------------------

# Decoding calls these once per layer and token, so the checks cost as few
# Python steps as they can: types and devices are bound once.
_T = None


class _Torch:
    """What the checks need of torch (imported on first use)."""

    def __init__(self):
        import torch
        self.int32, self.float32, self.bfloat16 = torch.int32, torch.float32, torch.bfloat16
        self.rows = {torch.bfloat16: FUTR_DTYPE_BF16, torch.float16: FUTR_DTYPE_F16}
        self.logits = dict(self.rows) | {torch.float32: FUTR_DTYPE_F32}
        # (torch.cuda's own functions ask first whether CUDA is set up: tensors on it are at hand here)
        self.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)


def _torch() -> _Torch:
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _bad_tensor(t, name, want, device):
    where = "" if t.get_device() == device else f" on CUDA device {device}, the current one"
    raise ValueError(f"{name} must be {want}{where}, not {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _elsewhere(descriptor, name, device):
    raise ValueError(f"{name} is on {descriptor._mem.device}, not on CUDA device {device}, the current one")


def _row_dtype(T, a, b, names) -> int:
    dtype = a.dtype
    if b.dtype is not dtype or dtype not in T.rows:
        raise TypeError(f"{names} must both be bfloat16 or both float16, not {dtype} and {b.dtype}")
    return T.rows[dtype]


def _row_stride(t, name, device, shape) -> int:
    """Elements from one row to the next of a row tensor (rows, heads, head_dim)."""
    ld, sh, sd = t.stride()
    n, heads, d = shape
    if t.shape != shape or sd != 1 or (sh != d and heads != 1) or t.get_device() != device:
        _bad_tensor(t, name, f"rows {shape}, the heads of a row contiguous,", device)
    return ld if n > 1 else -(-heads * d // 8) * 8


def _paged_rows(T, batch, pos, start, table, n_rows, device):
    """The arguments pos, start, n_rows, table, table_ld of a paged call."""
    int32 = T.int32
    if pos.dtype is not int32 or pos.shape != (batch,) or not pos.is_contiguous() or pos.get_device() != device:
        _bad_tensor(pos, "pos", f"a contiguous int32 tensor ({batch},)", device)
    if start is not None and (start.dtype is not int32 or start.shape != (batch + 1,) or not start.is_contiguous() or
                              start.get_device() != device):
        _bad_tensor(start, "start", f"a contiguous int32 tensor ({batch + 1},)", device)
    shape = table.shape
    if (table.dtype is not int32 or len(shape) != 2 or shape[0] != batch or not table.is_contiguous() or
            table.get_device() != device):
        _bad_tensor(table, "table", f"a contiguous int32 tensor ({batch}, pages)", device)
    return pos.data_ptr(), None if start is None else start.data_ptr(), n_rows, table.data_ptr(), shape[1]


def futr_paged_size(shape, n_layers, n_pages, page, max_pos) -> int:
    n = C.c_size_t()
    _ok(lib().futr_paged_size(C.byref(shape), n_layers, n_pages, page, max_pos, C.byref(n)), "futr_paged_size")
    return n.value


def futr_paged_init(shape, n_layers, n_pages, page, max_pos, rope, mem, stream=None) -> futr_paged:
    cache = futr_paged()
    _ok(lib().futr_paged_init(C.byref(shape), n_layers, n_pages, page, max_pos, int(rope), _ptr(mem),
                              mem.numel() * mem.element_size(), C.byref(cache), _stream(stream)), "futr_paged_init")
    cache._mem = mem
    return cache


def paged_views(cache):
    """The cache's codes (float8_e4m3fn [layers, pages, kv-heads, 2, page, head_dim])
    and scales (float32 [layers, pages, kv-heads, 2]) as tensors on its memory:
    index 0 keys, 1 values; a value is code * scale."""
    import torch
    s = cache.shape
    lead = (cache.n_layers, cache.n_pages, s.n_kv_heads, 2)
    n = cache.n_layers * cache.n_pages * s.n_kv_heads * 2
    codes = cache._mem[:n * cache.page * s.head_dim].view(torch.float8_e4m3fn)
    scales = cache._mem[cache.scale_offset:cache.scale_offset + 4 * n].view(torch.float32)
    return codes.view(*lead, cache.page, s.head_dim), scales.view(*lead)


def futr_paged_append(cache, layer, batch, pos, start, table, k, v, stream=None):
    """Append the rows k, v [n_rows, kv-heads, head_dim]; start None: one row per sequence."""
    T = _T or _torch()
    device = T.device()
    n = k.shape[0]
    rows = (n, cache.shape.n_kv_heads, cache.shape.head_dim)
    dtype = _row_dtype(T, k, v, "k and v")
    if cache._mem.get_device() != device:
        _elsewhere(cache, "the cache", device)
    ld_k, ld_v = _row_stride(k, "k", device, rows), _row_stride(v, "v", device, rows)
    p, s, n, t, ld = _paged_rows(T, batch, pos, start, table, n, device)
    _ok(lib().futr_paged_append(C.addressof(cache), layer, batch, p, s, n, t, ld, k.data_ptr(), ld_k, v.data_ptr(),
                                ld_v, dtype, T.stream(device) if stream is None else _stream(stream)),
        "futr_paged_append")


def futr_paged_workspace_size(shape) -> int:
    n = C.c_size_t()
    _ok(lib().futr_paged_workspace_size(C.byref(shape), C.byref(n)), "futr_paged_workspace_size")
    return n.value


def futr_paged_workspace_init(shape, mem, stream=None) -> futr_paged_ws:
    ws = futr_paged_ws()
    _ok(lib().futr_paged_workspace_init(C.byref(shape), _ptr(mem), mem.numel() * mem.element_size(), C.byref(ws),
                                        _stream(stream)), "futr_paged_workspace_init")
    ws._mem = mem
    return ws


def futr_paged_attention(cache, layer, batch, pos, start, table, q, out, ws, scale=0.0, window=0, stream=None, sinks=0):
    """Attention of the rows q [n_rows, heads, head_dim] over the cache into out
    (same shape and type); scale 0 is 1/sqrt(head_dim), window 0 is none, the first
    `sinks` positions of a sequence are visible through any window."""
    T = _T or _torch()
    device = T.device()
    n = q.shape[0]
    rows = (n, cache.shape.n_q_heads, cache.shape.head_dim)
    dtype = _row_dtype(T, q, out, "q and out")
    if cache._mem.get_device() != device:
        _elsewhere(cache, "the cache", device)
    if ws._mem.get_device() != device:
        _elsewhere(ws, "the workspace", device)
    ld_q, ld_out = _row_stride(q, "q", device, rows), _row_stride(out, "out", device, rows)
    p, s, n, t, ld = _paged_rows(T, batch, pos, start, table, n, device)
    _ok(lib().futr_paged_attention_sinks(C.addressof(cache), layer, batch, p, s, n, t, ld, q.data_ptr(), ld_q,
                                         out.data_ptr(), ld_out, dtype, scale, window, sinks, C.addressof(ws),
                                         T.stream(device) if stream is None else _stream(stream)),
        "futr_paged_attention")


def futr_paged_attention_sinks(cache, layer, batch, pos, start, table, q, out, ws, window, sinks, scale=0.0, stream=None):
    """futr_paged_attention with a window and the first `sinks` positions, which every row sees."""
    futr_paged_attention(cache, layer, batch, pos, start, table, q, out, ws, scale, window, stream, sinks)


def futr_paged_check(cache, ws=None, stream=None) -> int:
    """Synchronize and return the device status (0 = ok); does not raise."""
    return lib().futr_paged_check(C.byref(cache), C.byref(ws) if ws is not None else None, _stream(stream))


# ----------------------------------------------------------------------------
# mixture of experts
# ----------------------------------------------------------------------------

def make_moe_shape(hidden, inter, n_experts, top_k, renorm=True, rms_eps=1e-5, group=128) -> futr_moe_shape:
    return futr_moe_shape(hidden, inter, n_experts, top_k, group, int(renorm), rms_eps)


def futr_moe_weights_size(shape) -> int:
    n = C.c_size_t()
    _ok(lib().futr_moe_weights_size(C.byref(shape), C.byref(n)), "futr_moe_weights_size")
    return n.value


def _dense(t, name: str, dtype, shape, device: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _bad_tensor(t, name, f"a contiguous {dtype} tensor {shape}", device)
    return t.data_ptr()


def _moe_blob(blob, nbytes, device):
    if blob.nbytes < nbytes or not blob.is_contiguous() or blob.get_device() != device:
        raise ValueError(f"blob must hold the layer's packed experts, {nbytes} contiguous bytes on CUDA device "
                         f"{device}, the current one")
    return blob.data_ptr()


def futr_moe_pack(shape, expert, wgate, wup, wdown, gain, blob, stream=None):
    T = _T or _torch()
    device = T.device()
    H, I, f32 = shape.hidden, shape.inter, T.float32
    _moe_blob(blob, futr_moe_weights_size(shape), device)
    _ok(lib().futr_moe_pack(C.byref(shape), expert, _dense(wgate, "wgate", f32, (I, H), device),
                            _dense(wup, "wup", f32, (I, H), device), _dense(wdown, "wdown", f32, (H, I), device),
                            _dense(gain, "gain", f32, (H,), device), _ptr(blob), blob.numel() * blob.element_size(),
                            _stream(stream)), "futr_moe_pack")


def futr_moe_unpack(shape, blob, expert, which, codes, scales, stream=None):
    import torch
    device = torch.cuda.current_device() if _T is None else _T.device()
    r, c = (shape.hidden, shape.inter) if which == FUTR_PROJ_DOWN else (shape.inter, shape.hidden)
    _ok(lib().futr_moe_unpack(C.byref(shape), _moe_blob(blob, futr_moe_weights_size(shape), device), expert, which,
                              _dense(codes, "codes", torch.int8, (r, c), device),
                              _dense(scales, "scales", torch.float16, (r, c // 128), device), _stream(stream)),
        "futr_moe_unpack")


def futr_moe_workspace_size(shape, max_batch) -> int:
    n = C.c_size_t()
    _ok(lib().futr_moe_workspace_size(C.byref(shape), max_batch, C.byref(n)), "futr_moe_workspace_size")
    return n.value


def futr_moe_workspace_init(shape, max_batch, mem, stream=None) -> futr_moe_ws:
    ws = futr_moe_ws()
    _ok(lib().futr_moe_workspace_init(C.byref(shape), max_batch, _ptr(mem), mem.numel() * mem.element_size(),
                                      C.byref(ws), _stream(stream)), "futr_moe_workspace_init")
    ws._mem = mem
    return ws


def futr_moe_layer(x, gain, router, blob, resid, y, ws, ids=None, weights=None, stream=None):
    """The layer of x [batch, hidden] (bf16) into y; resid, gain, ids and weights may be None."""
    T = _T or _torch()
    device = T.device()
    s = ws.shape
    H, K, bf, n = s.hidden, s.top_k, T.bfloat16, x.shape[0]
    rows = (n, H)
    _moe_blob(blob, ws.blob_bytes, device)
    if ws._mem.get_device() != device:
        _elsewhere(ws, "the workspace", device)
    _ok(lib().futr_moe_layer(_dense(x, "x", bf, rows, device), _dense(gain, "gain", T.float32, (H,), device),
                             _dense(router, "router", bf, (s.n_experts, H), device), blob.data_ptr(), n,
                             _dense(resid, "resid", bf, rows, device), _dense(y, "y", bf, rows, device),
                             _dense(ids, "ids", T.int32, (n, K), device),
                             _dense(weights, "weights", T.float32, (n, K), device), C.addressof(ws),
                             T.stream(device) if stream is None else _stream(stream)), "futr_moe_layer")


def futr_moe_check(ws, stream=None) -> int:
    """Synchronize and return the device status (0 = ok); does not raise."""
    return lib().futr_moe_check(C.byref(ws), _stream(stream))


# ----------------------------------------------------------------------------
# beams
# ----------------------------------------------------------------------------

def futr_beam_workspace_size(rows, keep) -> int:
    n = C.c_size_t()
    _ok(lib().futr_beam_workspace_size(rows, keep, C.byref(n)), "futr_beam_workspace_size")
    return n.value


def futr_beam_workspace_init(rows, keep, mem, stream=None) -> futr_beam_ws:
    ws = futr_beam_ws()
    _ok(lib().futr_beam_workspace_init(rows, keep, _ptr(mem), mem.numel() * mem.element_size(), C.byref(ws),
                                       _stream(stream)), "futr_beam_workspace_init")
    ws._mem = mem
    return ws


def futr_beam_select(logits, scores, score_out, parent, token, ws, done=None, done_out=None, end=-1, stay=False,
                     stream=None):
    """The best continuations of the beams scores [batch, beams] by the logits
    [batch * beams, vocab] into score_out, parent, token and done_out [batch, keep]."""
    T = _T or _torch()
    device = T.device()
    f32, i32 = T.float32, T.int32
    shape, kept, rows = scores.shape, score_out.shape, logits.shape
    if len(shape) != 2 or len(kept) != 2 or kept[0] != shape[0]:
        raise ValueError(f"scores and score_out must be [batch, beams] and [batch, keep], not {tuple(shape)} and "
                         f"{tuple(kept)}")
    batch, beams = shape
    dtype = T.logits.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, not {logits.dtype}")
    n = batch * beams
    if len(rows) != 2 or rows[0] != n or logits.get_device() != device:
        _bad_tensor(logits, "logits", f"rows ({n}, vocab), a row contiguous,", device)
    vocab, (ld, step) = rows[1], logits.stride()
    if step != 1 and vocab > 1:
        _bad_tensor(logits, "logits", f"rows ({n}, vocab), a row contiguous,", device)
    if ws._mem.get_device() != device:
        _elsewhere(ws, "the workspace", device)
    _ok(lib().futr_beam_select(logits.data_ptr(), ld if n > 1 else vocab, dtype, batch, beams, vocab,
                               _dense(scores, "scores", f32, shape, device),
                               None if done is None else _dense(done, "done", i32, shape, device), end, kept[1],
                               1 if stay else 0, _dense(score_out, "score_out", f32, kept, device),
                               _dense(parent, "parent", i32, kept, device), _dense(token, "token", i32, kept, device),
                               None if done_out is None else _dense(done_out, "done_out", i32, kept, device),
                               C.addressof(ws), T.stream(device) if stream is None else _stream(stream)),
        "futr_beam_select")


def futr_beam_check(ws, stream=None) -> int:
    """Synchronize and return the device status (0 = ok); does not raise."""
    return lib().futr_beam_check(C.byref(ws), _stream(stream))


def futr_kv_reorder(kv, parent, pos, stream=None):
    """Slot i of the INT4 cache continues slot parent[i] (int32 [batch]); pos [batch] follows."""
    T = _T or _torch()
    device = T.device()
    shape = (parent.shape[0],) if parent.dim() == 1 else (parent.numel(),)
    if kv._mem.get_device() != device:
        _elsewhere(kv, "the cache", device)
    _ok(lib().futr_kv_reorder(C.addressof(kv), shape[0], _dense(parent, "parent", T.int32, shape, device),
                              _dense(pos, "pos", T.int32, shape, device),
                              T.stream(device) if stream is None else _stream(stream)), "futr_kv_reorder")


# ----------------------------------------------------------------------------
# pages of a paged cache.  Tables are contiguous int32 tensors [batch, pages] and
# are changed in place.
# ----------------------------------------------------------------------------

def futr_pages_size(n_pages, max_seqs) -> int:
    n = C.c_size_t()
    _ok(lib().futr_pages_size(n_pages, max_seqs, C.byref(n)), "futr_pages_size")
    return n.value


def futr_pages_init(n_pages, max_seqs, mem, stream=None) -> futr_pages:
    pool = futr_pages()
    _ok(lib().futr_pages_init(n_pages, max_seqs, _ptr(mem), mem.numel() * mem.element_size(), C.byref(pool),
                              _stream(stream)), "futr_pages_init")
    pool._mem = mem
    return pool


def pages_refs(pool):
    """How many places of the page tables name each page (int32 [n_pages], a view of the pool)."""
    import torch
    return pool._mem[pool.refs_offset:pool.refs_offset + 4 * pool.n_pages].view(torch.int32)


def _pages(T, cache, pool, table, device):
    """The table's rows and places, after the checks that every call on a table shares."""
    if table.dtype is not T.int32 or table.dim() != 2 or not table.is_contiguous() or table.get_device() != device:
        _bad_tensor(table, "table", "a contiguous int32 tensor (batch, pages)", device)
    if cache._mem.get_device() != device:
        _elsewhere(cache, "the cache", device)
    if pool._mem.get_device() != device:
        _elsewhere(pool, "the pool", device)
    return table.shape


def futr_pages_hold(cache, pool, table, stream=None):
    """Count the pages that a table made by hand names."""
    T = _T or _torch()
    device = T.device()
    batch, ld = _pages(T, cache, pool, table, device)
    _ok(lib().futr_pages_hold(C.addressof(cache), C.addressof(pool), batch, table.data_ptr(), ld,
                              T.stream(device) if stream is None else _stream(stream)), "futr_pages_hold")


def futr_pages_grow(cache, pool, pos, start, table, stream=None):
    """Take pages for the new rows of a call (start None: one row per sequence)."""
    T = _T or _torch()
    device = T.device()
    batch, ld = _pages(T, cache, pool, table, device)
    _ok(lib().futr_pages_grow(C.addressof(cache), C.addressof(pool), batch,
                              _dense(pos, "pos", T.int32, (batch,), device),
                              _dense(start, "start", T.int32, (batch + 1,), device), table.data_ptr(), ld,
                              T.stream(device) if stream is None else _stream(stream)), "futr_pages_grow")


def futr_pages_free(cache, pool, pos, table, window=0, sinks=0, stream=None):
    """Give back the pages that no row at pos or later sees, and those behind pos."""
    T = _T or _torch()
    device = T.device()
    batch, ld = _pages(T, cache, pool, table, device)
    _ok(lib().futr_pages_free(C.addressof(cache), C.addressof(pool), batch,
                              _dense(pos, "pos", T.int32, (batch,), device), table.data_ptr(), ld, window, sinks,
                              T.stream(device) if stream is None else _stream(stream)), "futr_pages_free")


def futr_pages_fork(cache, pool, parent, pos, table, stream=None):
    """Row i of the table continues row parent[i] (-1: empty); pos follows.  Every page that the table names is held."""
    T = _T or _torch()
    device = T.device()
    batch, ld = _pages(T, cache, pool, table, device)
    _ok(lib().futr_pages_fork(C.addressof(cache), C.addressof(pool), batch,
                              _dense(parent, "parent", T.int32, (batch,), device),
                              _dense(pos, "pos", T.int32, (batch,), device), table.data_ptr(), ld,
                              T.stream(device) if stream is None else _stream(stream)), "futr_pages_fork")


def futr_pages_compact(cache, pool, table, lo, hi=None, stream=None):
    """Move the pages in use of [lo, hi) (hi None: the end) to the lowest free pages outside of it.  Every page that
    the table names is held."""
    T = _T or _torch()
    device = T.device()
    batch, ld = _pages(T, cache, pool, table, device)
    _ok(lib().futr_pages_compact(C.addressof(cache), C.addressof(pool), batch, table.data_ptr(), ld, lo,
                                 pool.n_pages if hi is None else hi,
                                 T.stream(device) if stream is None else _stream(stream)), "futr_pages_compact")


def futr_pages_check(pool, stream=None):
    """Synchronize and return (device status, number of free pages); does not raise."""
    n = I32()
    return lib().futr_pages_check(C.byref(pool), C.byref(n), _stream(stream)), n.value


# ----------------------------------------------------------------------------
# allocation helpers (torch provides the device memory)
# ----------------------------------------------------------------------------

def alloc_bytes(n: int, device="cuda"):
    import torch
    # 256-byte aligned: the caching allocator aligns blocks to at least 512 bytes
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


def ws_view(ws: futr_ws, name: str, shape, dtype):
    """A tensor view of one workspace region (e.g. 'h', 'a', 'o', 'qrot')."""
    import torch
    off = getattr(ws, "off_" + name)
    n = 1
    for s in shape:
        n *= s
    esize = torch.empty((), dtype=dtype).element_size()
    return ws._mem[off:off + n * esize].view(dtype).view(*shape)
