"""Thin ctypes binding of the C ABI in ``include/csa.h`` (``libcsa.so``).

Argument marshalling only: tensors are torch CUDA tensors, passed by device
pointer; every step of the path runs in the library's CUDA kernels. The
functions keep the C names. A non-OK status raises ``CsaError``.

The library is loaded from the package directory (built in-tree by
``long_context_sparse_07_b200.build``). There is no fallback: if it is missing
or fails to load, import of this module's functions raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcsa.so")

CSA_F32, CSA_BF16, CSA_E4M3, CSA_E2M1 = 0, 1, 2, 3
STATUS = {0: "CSA_OK", -1: "CSA_ERR_INVALID_ARG", -2: "CSA_ERR_UNSUPPORTED",
          -3: "CSA_ERR_CUDA", -4: "CSA_ERR_TIMEOUT", -5: "CSA_ERR_BOUNDS"}

# every symbol that include/csa.h declares
EXPORTS = ("csa_abi_version", "csa_status_string", "csa_last_message", "csa_compress_kv",
           "csa_indexer_scores", "csa_topk", "csa_topk_workspace_size", "csa_indexer_topk",
           "csa_indexer_topk_workspace_size", "csa_indexer_topk_launches", "csa_sparse_mqa",
           "hca_dense_mqa", "csa_mqa_workspace_size", "csa_sparse_mqa_noalloc",
           "csa_noalloc_scratch_bytes", "csa_norm_rope", "csa_grouped_out_proj",
           "csa_add_norm_quant", "csa_quantize_weight", "csa_fp8_proj",
           "csa_debug_fp8_proj_form", "csa_debug_wait_probe", "csa_get_error")


class CsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


class _Entries(ctypes.Structure):
    _fields_ = [("body", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("c", ctypes.c_int), ("rope_dims", ctypes.c_int),
                ("scale_group", ctypes.c_int), ("dt", ctypes.c_int)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_S = ctypes.c_size_t
_lib = None


def load(path: str = LIB_PATH):
    """Load ``libcsa.so`` and declare its signatures (raises if missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libcsa.so not built: run `python -m long_context_sparse_07_b200.build`")
    L = ctypes.CDLL(path)
    L.csa_abi_version.restype = _I
    L.csa_status_string.restype = ctypes.c_char_p
    L.csa_status_string.argtypes = [_I]
    L.csa_last_message.restype = ctypes.c_char_p
    L.csa_compress_kv.restype = _I
    L.csa_compress_kv.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _Entries, _P]
    L.csa_indexer_scores.restype = _I
    L.csa_indexer_scores.argtypes = [_P, _P, _P, _Entries, _P, _I, _I64, _I64, _I, _I, _I, _I,
                                     _P, _I64, _P]
    L.csa_topk.restype = _I
    L.csa_topk.argtypes = [_P, _I64, _I64, _I64, _P, _I, _I, _P, _P, _S, _P]
    L.csa_topk_workspace_size.restype = _S
    L.csa_topk_workspace_size.argtypes = [_I64, _I64, _I]
    L.csa_indexer_topk.restype = _I
    L.csa_indexer_topk.argtypes = [_P, _P, _P, _Entries, _P, _I, _I64, _I64, _I, _I, _I, _I, _I,
                                   _P, _P, _S, _P]
    L.csa_indexer_topk_workspace_size.restype = _S
    L.csa_indexer_topk_workspace_size.argtypes = [_I, _I64, _I64, _I, _I, _I, _I]
    L.csa_indexer_topk_launches.restype = _I
    L.csa_indexer_topk_launches.argtypes = [_I, _I64, _I64, _I, _I, _I, _I]
    L.csa_sparse_mqa.restype = _I
    L.csa_sparse_mqa.argtypes = [_P, _I, _Entries, _I64, _I, _P, _I, _P, _I64, _P, _I, _P, _P,
                                 _I, _I64, _I, _F, _P, _P, _P, _S, _P]
    L.hca_dense_mqa.restype = _I
    L.hca_dense_mqa.argtypes = [_P, _I, _Entries, _I64, _I, _P, _I64, _P, _I, _P, _P, _I, _I64,
                                _I, _F, _P, _P, _P, _S, _P]
    L.csa_mqa_workspace_size.restype = _S
    L.csa_mqa_workspace_size.argtypes = [_I, _I64, _I, _I, _I64]
    L.csa_sparse_mqa_noalloc.restype = _I
    L.csa_sparse_mqa_noalloc.argtypes = [_P, _I, _Entries, _I64, _I, _P, _I, _P, _I64, _P, _I, _P,
                                         _P, _I, _I64, _I, _F, _P, _P, _P]
    L.csa_noalloc_scratch_bytes.restype = _S
    L.csa_noalloc_scratch_bytes.argtypes = []
    L.csa_norm_rope.restype = _I
    L.csa_norm_rope.argtypes = [_P, _I, _P, _I64, _I, _I, _I, _P, _I64, _I64, _I, _F, _F, _P]
    L.csa_grouped_out_proj.restype = _I
    L.csa_grouped_out_proj.argtypes = [_P, _P, _P, _I64, _I, _I, _I, _I, _I, _P, _P, _P]
    L.csa_add_norm_quant.restype = _I
    L.csa_add_norm_quant.argtypes = [_P, _P, _P, _I, _I64, _I, _I, _F, _P, _P, _P, _P, _P]
    L.csa_quantize_weight.restype = _I
    L.csa_quantize_weight.argtypes = [_P, _I, _I64, _I, _P, _P, _P]
    L.csa_fp8_proj.restype = _I
    L.csa_fp8_proj.argtypes = [_P, _P, _P, _P, _I64, _I, _I, _I, _I, _P, _P, _P]
    L.csa_debug_fp8_proj_form.restype = _I
    L.csa_debug_fp8_proj_form.argtypes = [_I64, _I, _I, _I, _I]
    L.csa_debug_wait_probe.restype = _I
    L.csa_debug_wait_probe.argtypes = [ctypes.c_uint64, _P]
    L.csa_get_error.restype = _I
    L.csa_get_error.argtypes = [ctypes.c_char_p, _S]
    _lib = L
    return L


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return CSA_F32
    if t.dtype == torch.bfloat16:
        return CSA_BF16
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        return CSA_E4M3
    raise TypeError("unsupported dtype %s" % t.dtype)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _check(st: int):
    if st != 0:
        msg = load().csa_last_message().decode()
        raise CsaError(st, msg)


@dataclasses.dataclass
class Entries:
    """A table of KV entries (``csa_entries``): plain [rows, c] f32/bf16, or
    the fp8 layout (e4m3 body [rows, c - rope_dims] with per-group float32
    scales, optional bf16 rope part [rows, rope_dims]), or the fp4 layout of
    indexer keys (fp4=True: uint8 body [rows, c / 2] of packed e2m1 codes,
    uint8 block exponents [rows, c / 32] in ``scale``, scale_group 32)."""
    body: torch.Tensor
    c: int
    scale: Optional[torch.Tensor] = None
    rope: Optional[torch.Tensor] = None
    rope_dims: int = 0
    scale_group: int = 0
    fp4: bool = False

    def struct(self) -> _Entries:
        dt = CSA_E2M1 if self.fp4 else dtype_code(self.body)
        return _Entries(_ptr(self.body), _ptr(self.scale), _ptr(self.rope), self.c,
                        self.rope_dims, self.scale_group, dt)


def csa_abi_version() -> int:
    return load().csa_abi_version()


def csa_compress_kv(Ca, Cb, Za, Zb, Ba, Bb, m: int, overlap: bool, out: Entries, stream=None):
    n, c = Ca.shape[0], Ca.shape[-1]
    _check(load().csa_compress_kv(_ptr(Ca), _ptr(Cb), _ptr(Za), _ptr(Zb), _ptr(Ba), _ptr(Bb),
                                  n, c, m, int(bool(overlap)), dtype_code(Ca), out.struct(),
                                  _stream(stream)))


def csa_indexer_scores(qI, qI_scale, wI, kI: Entries, q_pos, m: int, scores, E: int,
                       stream=None):
    B, n_q, hI, cI = qI.shape
    _check(load().csa_indexer_scores(_ptr(qI), _ptr(qI_scale), _ptr(wI), kI.struct(),
                                     _ptr(q_pos), B, n_q, E, hI, cI, m, dtype_code(qI),
                                     _ptr(scores), scores.shape[-1], _stream(stream)))


def csa_topk_workspace_size(rows: int, E: int, k: int) -> int:
    return int(load().csa_topk_workspace_size(rows, E, k))


def csa_topk(scores, q_pos, m: int, k: int, idx, E: Optional[int] = None, workspace=None,
             stream=None):
    ld = scores.shape[-1]
    rows = scores.numel() // ld if ld else 0
    E = ld if E is None else E
    ws = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().csa_topk(_ptr(scores), rows, E, ld, _ptr(q_pos), m, k, _ptr(idx),
                           _ptr(workspace), ws, _stream(stream)))


def csa_indexer_topk_workspace_size(B: int, n_q: int, E: int, hI: int, cI: int, k: int,
                                    dt) -> int:
    code = dt if isinstance(dt, int) else dtype_code(dt)
    return int(load().csa_indexer_topk_workspace_size(B, n_q, E, hI, cI, k, code))


def csa_indexer_topk_launches(B: int, n_q: int, E: int, hI: int, cI: int, k: int, dt) -> int:
    """Kernel launches of csa_indexer_topk for these shapes (6: candidate path)."""
    code = dt if isinstance(dt, int) else dtype_code(dt)
    return int(load().csa_indexer_topk_launches(B, n_q, E, hI, cI, k, code))


def csa_indexer_topk(qI, qI_scale, wI, kI: Entries, q_pos, m: int, k: int, idx, E: int,
                     workspace=None, stream=None):
    """Indexer scores and top-k in one call: idx [B * n_q, k] as
    csa_indexer_scores followed by csa_topk would give."""
    B, n_q, hI, cI = qI.shape
    ws = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().csa_indexer_topk(_ptr(qI), _ptr(qI_scale), _ptr(wI), kI.struct(), _ptr(q_pos),
                                   B, n_q, E, hI, cI, m, dtype_code(qI), k, _ptr(idx),
                                   _ptr(workspace), ws, _stream(stream)))


def csa_mqa_workspace_size(B: int, n_q: int, h: int, c: int, max_keys: int) -> int:
    return int(load().csa_mqa_workspace_size(B, n_q, h, c, max_keys))


def csa_sparse_mqa(q, kv: Entries, E: int, m: int, idx, k: int, kwin, win_pos0, n_win: int,
                   q_pos, sink, scale: float, out, lse=None, workspace=None, stream=None):
    B, n_q, h, c = q.shape
    win_rows = kwin.shape[-2] if kwin is not None else 0
    ws = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().csa_sparse_mqa(_ptr(q), dtype_code(q), kv.struct(), E, m, _ptr(idx), k,
                                 _ptr(kwin), win_rows, _ptr(win_pos0), n_win, _ptr(q_pos),
                                 _ptr(sink), B, n_q, h, scale, _ptr(out), _ptr(lse),
                                 _ptr(workspace), ws, _stream(stream)))


def csa_sparse_mqa_noalloc(q, kv: Entries, E: int, m: int, idx, k: int, kwin, win_pos0,
                           n_win: int, q_pos, sink, scale: float, out, lse=None, stream=None):
    """csa_sparse_mqa with the library's fixed device scratch instead of a
    workspace: for callers that cannot allocate device memory."""
    B, n_q, h, c = q.shape
    win_rows = kwin.shape[-2] if kwin is not None else 0
    _check(load().csa_sparse_mqa_noalloc(_ptr(q), dtype_code(q), kv.struct(), E, m, _ptr(idx), k,
                                         _ptr(kwin), win_rows, _ptr(win_pos0), n_win,
                                         _ptr(q_pos), _ptr(sink), B, n_q, h, scale, _ptr(out),
                                         _ptr(lse), _stream(stream)))


def csa_noalloc_scratch_bytes() -> int:
    return int(load().csa_noalloc_scratch_bytes())


def hca_dense_mqa(q, kv: Entries, E: int, m: int, kwin, win_pos0, n_win: int, q_pos, sink,
                  scale: float, out, lse=None, workspace=None, stream=None):
    B, n_q, h, c = q.shape
    win_rows = kwin.shape[-2] if kwin is not None else 0
    ws = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().hca_dense_mqa(_ptr(q), dtype_code(q), kv.struct(), E, m, _ptr(kwin),
                                win_rows, _ptr(win_pos0), n_win, _ptr(q_pos), _ptr(sink), B,
                                n_q, h, scale, _ptr(out), _ptr(lse), _ptr(workspace), ws,
                                _stream(stream)))


def csa_norm_rope(x, rope_dims: int, pos=None, pos_mul: int = 1, pos_add: int = 0, gamma=None,
                  normalise: bool = True, eps: float = 1e-6, base: float = 10000.0, stream=None):
    """In-place RMSNorm and partial RoPE of x [rows, heads, c] or [rows, c]."""
    c = x.shape[-1]
    rows = x.shape[0]
    heads = x.numel() // (rows * c) if rows else 1
    _check(load().csa_norm_rope(_ptr(x), dtype_code(x), _ptr(gamma), rows, heads, c, rope_dims,
                                _ptr(pos), pos_mul, pos_add, int(bool(normalise)), eps, base,
                                _stream(stream)))


def csa_grouped_out_proj(o, Wg, Wo, g: int, u, out, stream=None):
    """Grouped output projection: o [n, h, c] -> u [n, g dg] -> out [n, d]."""
    n, h, c = o.shape
    dg = Wg.shape[0] // g
    d = Wo.shape[0]
    _check(load().csa_grouped_out_proj(_ptr(o), _ptr(Wg), _ptr(Wo), n, h, c, g, dg, d, _ptr(u),
                                       _ptr(out), _stream(stream)))


_PLAIN = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)
_CODES = (torch.float8_e4m3fn, torch.uint8)
_DTYPE_CODE = {torch.float32: CSA_F32, torch.bfloat16: CSA_BF16, torch.float8_e4m3fn: CSA_E4M3,
               torch.uint8: CSA_E4M3}


def _operand(t, dtypes, shape, dev, has=None):
    """Device pointer of an operand that is as a call needs it, else 0: a dense
    tensor of a listed dtype and of this shape, on CUDA device `dev`. `has` is
    its shape where the caller has read it."""
    if (t.dtype in dtypes and (has or t.shape) == shape and t.is_contiguous()
            and t.get_device() == dev >= 0):
        return t.data_ptr() or _EMPTY
    return 0


_EMPTY = 16          # stands for the null address of a tensor without elements


def _refuse(what: str, dev: int, **operands):
    """Raises what is wrong with the first of name = (tensor, dtypes, shape)."""
    for name, (t, dtypes, shape) in operands.items():
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError("%s: %s is %s" % (what, name, t.dtype))
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s: %s is %s, expected %s" % (what, name, tuple(t.shape),
                                                            tuple(shape)))
        if not t.is_contiguous():
            raise ValueError("%s: %s must be contiguous" % (what, name))
    raise ValueError("%s: operands must be on one CUDA device" % what)


def _call_on(dev: int, fn, stream, *args):
    """Calls fn(*args, stream) with `dev` current, on its current stream when
    none is given."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call_on(dev, fn, stream, *args)
    st = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else
            getattr(stream, "cuda_stream", stream))
    if st:
        _check(st)


def csa_add_norm_quant(x, residual=None, gamma=None, normalise: bool = True, eps: float = 1e-6,
                       total=None, y=None, codes=None, scale=None, stream=None):
    """total <- x + residual, its RMSNorm (times gamma) to y and, in e4m3 with
    a scale per 128 channels, to codes and scale; x [..., d]. Outputs that are
    None are not written."""
    shape = x.shape
    d = shape[-1]
    same, dev = (x.dtype,), x.get_device()
    blocks = shape[:-1] + ((d + 127) >> 7,)
    px = _operand(x, _PLAIN, shape, dev, shape)
    pr = None if residual is None else _operand(residual, same, shape, dev)
    pg = None if gamma is None else _operand(gamma, _F32, (d,), dev)
    pt = None if total is None else _operand(total, same, shape, dev)
    py = None if y is None else _operand(y, same, shape, dev)
    pc = None if codes is None else _operand(codes, _CODES, shape, dev)
    ps = None if scale is None else _operand(scale, _F32, blocks, dev)
    if 0 in (px, pr, pg, pt, py, pc, ps):
        _refuse("csa_add_norm_quant", dev, x=(x, _PLAIN, shape), residual=(residual, same, shape),
                gamma=(gamma, _F32, (d,)), total=(total, same, shape), y=(y, same, shape),
                codes=(codes, _CODES, shape), scale=(scale, _F32, blocks))
    _call_on(dev, (_lib or load()).csa_add_norm_quant, stream, px, pr, pg, _DTYPE_CODE[x.dtype],
             x.numel() // d if d else 0, d, 1 if normalise else 0, eps, pt, py, pc, ps)


def csa_quantize_weight(W, codes, scale, stream=None):
    """W [N, K] to e4m3 codes [N, K] with a scale per 128 x 128 block,
    [ceil(N / 128), ceil(K / 128)]."""
    N, K = W.shape
    dev = W.get_device()
    blocks = ((N + 127) >> 7, (K + 127) >> 7)
    pw = _operand(W, _PLAIN, (N, K), dev, (N, K))
    pc = _operand(codes, _CODES, (N, K), dev)
    ps = _operand(scale, _F32, blocks, dev)
    if not (pw and pc and ps):
        _refuse("csa_quantize_weight", dev, W=(W, _PLAIN, (N, K)), codes=(codes, _CODES, (N, K)),
                scale=(scale, _F32, blocks))
    _call_on(dev, (_lib or load()).csa_quantize_weight, stream, pw, _DTYPE_CODE[W.dtype], N, K, pc, ps)


def csa_fp8_proj(A, A_scale, W, W_scale, out, out_scale=None, groups: int = 1, stream=None):
    """out [M, groups N] = A [M, groups K] times W [groups N, K] (group by
    group), e4m3 operands with block scales; out bf16, f32, or e4m3 codes with
    out_scale [M, ceil(groups N / 128)]."""
    a, (GN, K) = A.shape, W.shape
    M = a[0]
    if groups < 1 or GN % groups:
        raise ValueError("csa_fp8_proj: groups must divide the rows of W")
    dev = A.get_device()
    nb, nbo = (K + 127) >> 7, (GN + 127) >> 7
    pa = _operand(A, _CODES, (M, groups * K), dev, a)
    pas = _operand(A_scale, _F32, (M, groups * nb), dev)
    pw = _operand(W, _CODES, (GN, K), dev, (GN, K))
    pws = _operand(W_scale, _F32, (nbo, nb), dev)
    po = _operand(out, _DTYPE_CODE, (M, GN), dev)
    pos = None if out_scale is None else _operand(out_scale, _F32, (M, nbo), dev)
    if not (pa and pas and pw and pws and po) or pos == 0:
        _refuse("csa_fp8_proj", dev, A=(A, _CODES, (M, groups * K)),
                A_scale=(A_scale, _F32, (M, groups * nb)), W=(W, _CODES, (GN, K)),
                W_scale=(W_scale, _F32, (nbo, nb)), out=(out, _DTYPE_CODE, (M, GN)),
                out_scale=(out_scale, _F32, (M, nbo)))
    _call_on(dev, (_lib or load()).csa_fp8_proj, stream, pa, pas, pw, pws, M, GN // groups, K, groups,
             _DTYPE_CODE[out.dtype], po, pos)


FP8_PROJ_FORMS = ("few", "cluster16", "cluster32", "cluster64", "tiles", "pairs")


def csa_debug_fp8_proj_form(M: int, N: int, K: int, groups: int, dtype) -> str:
    """The kernel (one of FP8_PROJ_FORMS) that csa_fp8_proj takes for M tokens,
    N features and K inputs a group, and results of this dtype."""
    st = load().csa_debug_fp8_proj_form(M, N, K, groups, _DTYPE_CODE[dtype])
    if st < 0:
        _check(st)
    return FP8_PROJ_FORMS[st]


def csa_debug_wait_probe(limit_ns: int, stream=None):
    """Launch bounded device waits that run out (a thread's after `limit_ns`,
    then a warp's of which one lane gives up); the next csa_get_error() reports
    CSA_ERR_TIMEOUT."""
    _check(load().csa_debug_wait_probe(int(limit_ns), _stream(stream)))


def csa_get_error() -> int:
    """Synchronise, read and clear the device error word; raises on error."""
    buf = ctypes.create_string_buffer(256)
    st = load().csa_get_error(buf, 256)
    if st != 0:
        raise CsaError(st, buf.value.decode())
    return st
