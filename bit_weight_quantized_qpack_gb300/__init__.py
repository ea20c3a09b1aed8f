"""qpack for GB300: fused dequantization + matrix-vector / small-batch / prefill products over group-quantized
low-bit weights (INT4 group-32 and the 2/3/5/6-bit 256-weight super-block formats).

This module is a thin ctypes binding over the C ABI of ``libqpack.so`` (declared in ``include/qpack.h``). It
only marshals arguments: every computation runs in the library's CUDA kernels. PyTorch supplies device memory
and streams. There is no CPU fallback: importing works anywhere, but every compute call raises ``QpackError``
when the CUDA library is not built or no GPU is present.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

Q4G32, Q2S, Q3S, Q5S, Q6S, Q4G32H, Q4G16, Q4G32A = 0, 1, 2, 3, 4, 5, 6, 7
FORMATS = {"Q4G32": Q4G32, "Q2S": Q2S, "Q3S": Q3S, "Q5S": Q5S, "Q6S": Q6S, "Q4G32H": Q4G32H, "Q4G16": Q4G16,
           "Q4G32A": Q4G32A}
F32, F16, BF16 = 0, 1, 2
FLAG_RANGE = 1
FAULT_NONFINITE_X = 16
FAULT_PAGE, FAULT_NO_PAGES = 32, 64
KV_ATTEND_ZEROED = 1 << 20
KV_I8, KV_F16, KV_BF16 = 0, 1, 2
# (sub-blocks per super-block, asymmetric) for the super-block formats
_SB = {Q2S: (16, True), Q3S: (16, False), Q5S: (8, True), Q6S: (16, False)}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqpack.so")
_lock = threading.Lock()
_lib = None


class QpackError(RuntimeError):
    pass


class Layout(ctypes.Structure):
    _fields_ = [("row_stride", ctypes.c_int64), ("packed_bytes", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("scale_bytes", ctypes.c_int64),
                ("block_bytes", ctypes.c_int64), ("nsub", ctypes.c_int64),
                ("weight_bytes", ctypes.c_int64)]


class _Pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("scale_layer_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("layers", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("dim", ctypes.c_int32), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _Tables(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("stride", ctypes.c_int64), ("pages", ctypes.c_int64), ("seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


def lib():
    """Load libqpack.so (raises QpackError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise QpackError(f"libqpack.so not built ({LIB_PATH}); run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            sigs = {
                "qpack_layout": ([I, I64, I64, ctypes.POINTER(Layout)], I),
                "qpack_quantize": ([I, P, I, I64, I64, P, P, P, P, P, P, P, P], I),
                "qpack_pack": ([I, I64, I64, P, P, P, P, P, P, P, P, P], I),
                "qpack_quantize_pack": ([I, P, I, I64, I64, P, P, P, P], I),
                "qpack_unpack": ([I, I64, I64, P, P, P, P, P, P, P, P, P], I),
                "qpack_dequant": ([I, I64, I64, P, P, P, P], I),
                "qgemv": ([I, P, P, I64, I64, P, P, P], I),
                "qgemm_small": ([I, P, P, I64, I64, I, P, I64, P, I64, P], I),
                "qgemm_prefill": ([I, P, P, I64, I64, I64, P, I64, P, I64, P], I),
                "qpack_kv_quantize": ([P, I64, P, P, P], I),
                "qpack_kv_dequant": ([P, P, I64, P, P], I),
                "qpack_kv_append": ([P, I, P, P, P, I64, P, P, I, I64, I64, P, I64, P], I),
                "qpack_kv_read": ([P, I, P, P, P, I64, P, P, I, I64, I64, P], I),
                "qpack_kv_attend": ([P, I, P, P, I, P, I, I64, I, ctypes.c_float, I64, P, I64, P, I, I64, P, P, I64, P],
                                    I),
                "qpack_kv_attend_workspace": ([P, I, I, ctypes.POINTER(I64)], I),
                "qpack_kv_reserve": ([P, P, P, P, I64, P], I),
                "qpack_kv_fork": ([P, P, P, P, I64, P, I64, P], I),
                "qpack_kv_free": ([P, P, I64, P], I),
                "qpack_kv_compact": ([P, P, P, P, P, P, I64, P], I),
                "qpack_kv_copy_pages": ([P, P, P, I64, P], I),
                "qpack_kv_page_workspace": ([P, P, ctypes.POINTER(I64)], I),
                "qpack_status_string": ([I], ctypes.c_char_p),
                "qpack_fetch_fault_flags": ([ctypes.POINTER(ctypes.c_int32)], I),
                "qpack_version": ([], I),
                "qpack_set_option": ([I, I], I),
            }
            for name, (args, res) in sigs.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = lib().qpack_status_string(rc).decode()
        raise QpackError(f"{what}: {msg} (status {rc})")


def _need(t, dtype, what, numel=None, rows=None, cols=None):
    """Argument checks the C ABI cannot make (it sees only pointers): element type, size and, for matrices, a row-major
    layout with unit column stride. Raises QpackError before anything is launched."""
    if t.dtype != dtype:
        raise QpackError(f"{what}: expected {dtype}, got {t.dtype}")
    if rows is not None:
        if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or (t.shape[1] > 1 and t.stride(1) != 1):
            raise QpackError(f"{what}: expected a row-major matrix of at least {rows} x {cols}, got {tuple(t.shape)} "
                             f"with strides {tuple(t.stride())}")
    elif numel is not None:
        if not t.is_contiguous() or t.numel() < numel:
            raise QpackError(f"{what}: expected a contiguous tensor of at least {numel} elements, got "
                             f"{tuple(t.shape)}")


def _need_packed(fmt, N, K, packed, group_scales):
    L = layout(fmt, N, K)
    _need(packed, torch.uint8, "packed", numel=L["packed_bytes"])
    if L["scale_bytes"]:
        if group_scales is None:
            raise QpackError("group_scales: required by this format")
        gdt = torch.float16 if int(fmt) == Q4G32H else torch.float32
        if group_scales.dtype == torch.int16 and gdt == torch.float16:
            gdt = torch.int16                                   # fp16 bit patterns held as int16
        _need(group_scales, gdt, "group_scales", numel=L["scale_bytes"] // group_scales.element_size())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise QpackError("qpack kernels take CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t):
    d = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}.get(t.dtype)
    if d is None:
        raise QpackError(f"W: expected float32, float16 or bfloat16, got {t.dtype}")
    if t.dim() != 2 or not t.is_contiguous():
        raise QpackError(f"W: expected a contiguous [N, K] matrix, got {tuple(t.shape)}")
    return d


def layout(fmt: int, N: int, K: int) -> dict:
    out = Layout()
    _check(lib().qpack_layout(int(fmt), int(N), int(K), ctypes.byref(out)), "qpack_layout")
    return {f: getattr(out, f) for f, _ in Layout._fields_}


def alloc_packed(fmt, N, K, device="cuda"):
    """Caller-owned packed buffers of the right sizes: (packed uint8 [N, row_stride], scales or None)."""
    L = layout(fmt, N, K)
    packed = torch.empty((N, L["row_stride"]), dtype=torch.uint8, device=device)
    gs = None
    if fmt in (Q4G32, Q4G32H, Q4G16, Q4G32A):   # fp32 or fp16 group scales (Q4G32A: fp32 (s, z) pairs)
        gs = torch.empty((N, L["scale_stride"]), dtype=torch.float16 if fmt == Q4G32H else torch.float32, device=device)
    return packed, gs


def alloc_parts(fmt, N, K, device="cuda"):
    parts = dict(q=torch.empty((N, K), dtype=torch.int8, device=device), gscale=None, sub_scale=None,
                 sub_min=None, d=None, dmin=None)
    if fmt in (Q4G32, Q4G16, Q4G32A):
        parts["gscale"] = torch.empty((N, K // (32 if fmt == Q4G32 else 16)), dtype=torch.float32, device=device)
    elif fmt == Q4G32H:
        parts["d"] = torch.empty((N, K // 32), dtype=torch.int16, device=device)   # fp16 group-scale bits
    else:
        nsub, asym = _SB[fmt]
        nb = K // 256
        parts["sub_scale"] = torch.empty((N, nb * nsub), dtype=torch.uint8, device=device)
        parts["d"] = torch.empty((N, nb), dtype=torch.int16, device=device)
        if asym:
            parts["sub_min"] = torch.empty((N, nb * nsub), dtype=torch.uint8, device=device)
            parts["dmin"] = torch.empty((N, nb), dtype=torch.int16, device=device)
    return parts


def qpack_quantize(fmt, W, parts=None, status=None, stream=None):
    wdt = _dt(W)
    N, K = W.shape
    parts = alloc_parts(fmt, N, K, W.device) if parts is None else parts
    rc = lib().qpack_quantize(int(fmt), _ptr(W), wdt, N, K, _ptr(parts["q"]), _ptr(parts["gscale"]),
                              _ptr(parts["sub_scale"]), _ptr(parts["sub_min"]), _ptr(parts["d"]),
                              _ptr(parts["dmin"]), _ptr(status), _stream(stream))
    _check(rc, "qpack_quantize")
    return parts


def qpack_pack(fmt, N, K, parts, packed=None, group_scales=None, stream=None):
    if packed is None:
        packed, group_scales = alloc_packed(fmt, N, K, parts["q"].device)
    rc = lib().qpack_pack(int(fmt), N, K, _ptr(parts["q"]), _ptr(parts["gscale"]), _ptr(parts["sub_scale"]),
                          _ptr(parts["sub_min"]), _ptr(parts["d"]), _ptr(parts["dmin"]), _ptr(packed),
                          _ptr(group_scales), _stream(stream))
    _check(rc, "qpack_pack")
    return packed, group_scales


def qpack_quantize_pack(fmt, W, packed=None, group_scales=None, status=None, stream=None):
    wdt = _dt(W)
    N, K = W.shape
    if packed is None:
        packed, group_scales = alloc_packed(fmt, N, K, W.device)
    rc = lib().qpack_quantize_pack(int(fmt), _ptr(W), wdt, N, K, _ptr(packed), _ptr(group_scales),
                                   _ptr(status), _stream(stream))
    _check(rc, "qpack_quantize_pack")
    return packed, group_scales


def qpack_unpack(fmt, N, K, packed, group_scales=None, parts=None, stream=None):
    parts = alloc_parts(fmt, N, K, packed.device) if parts is None else parts
    rc = lib().qpack_unpack(int(fmt), N, K, _ptr(packed), _ptr(group_scales), _ptr(parts["q"]),
                            _ptr(parts["gscale"]), _ptr(parts["sub_scale"]), _ptr(parts["sub_min"]),
                            _ptr(parts["d"]), _ptr(parts["dmin"]), _stream(stream))
    _check(rc, "qpack_unpack")
    return parts


def qpack_dequant(fmt, N, K, packed, group_scales=None, out=None, stream=None):
    out = torch.empty((N, K), dtype=torch.float32, device=packed.device) if out is None else out
    rc = lib().qpack_dequant(int(fmt), N, K, _ptr(packed), _ptr(group_scales), _ptr(out), _stream(stream))
    _check(rc, "qpack_dequant")
    return out


def qgemv(fmt, packed, group_scales, N, K, x, y=None, stream=None):
    _need_packed(fmt, N, K, packed, group_scales)
    _need(x, torch.float16, "x", numel=K)
    y = torch.empty(N, dtype=torch.float32, device=x.device) if y is None else y
    _need(y, torch.float32, "y", numel=N)
    rc = lib().qgemv(int(fmt), _ptr(packed), _ptr(group_scales), N, K, _ptr(x), _ptr(y), _stream(stream))
    _check(rc, "qgemv")
    return y


def qgemm_small(fmt, packed, group_scales, N, K, X, Y=None, stream=None):
    _need_packed(fmt, N, K, packed, group_scales)
    M = X.shape[0]
    _need(X, torch.float16, "X", rows=M, cols=K)
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if Y is None else Y
    _need(Y, torch.float32, "Y", rows=M, cols=N)
    rc = lib().qgemm_small(int(fmt), _ptr(packed), _ptr(group_scales), N, K, M, _ptr(X), X.stride(0), _ptr(Y),
                           Y.stride(0), _stream(stream))
    _check(rc, "qgemm_small")
    return Y


def qgemm_prefill(fmt, packed, group_scales, N, K, X, Y=None, stream=None):
    _need_packed(fmt, N, K, packed, group_scales)
    M = X.shape[0]
    _need(X, torch.bfloat16, "X", rows=M, cols=K)
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device) if Y is None else Y
    _need(Y, torch.bfloat16, "Y", rows=M, cols=N)
    rc = lib().qgemm_prefill(int(fmt), _ptr(packed), _ptr(group_scales), N, K, M, _ptr(X), X.stride(0),
                             _ptr(Y), Y.stride(0), _stream(stream))
    _check(rc, "qgemm_prefill")
    return Y


def qpack_kv_quantize(v, codes=None, scales=None, stream=None):
    """fp16 KV tensor (any shape, contiguous, numel a multiple of 32) -> (int8 codes of its shape, fp16 scales
    [numel / 32]): one fp16 scale per 32 consecutive elements."""
    n = v.numel()
    _need(v, torch.float16, "v", numel=n)
    codes = torch.empty(v.shape, dtype=torch.int8, device=v.device) if codes is None else codes
    scales = torch.empty(n // 32, dtype=torch.float16, device=v.device) if scales is None else scales
    _need(codes, torch.int8, "codes", numel=n)
    _need(scales, torch.float16, "scales", numel=n // 32)
    _check(lib().qpack_kv_quantize(_ptr(v), n, _ptr(codes), _ptr(scales), _stream(stream)), "qpack_kv_quantize")
    return codes, scales


def qpack_kv_dequant(codes, scales, out=None, stream=None):
    """int8 codes + fp16 scales -> fp16 tensor of the codes' shape."""
    _need(codes, torch.int8, "codes", numel=codes.numel())
    _need(scales, torch.float16, "scales", numel=codes.numel() // 32)
    out = torch.empty(codes.shape, dtype=torch.float16, device=codes.device) if out is None else out
    _need(out, torch.float16, "out", numel=codes.numel())
    _check(lib().qpack_kv_dequant(_ptr(codes), _ptr(scales), codes.numel(), _ptr(out), _stream(stream)),
           "qpack_kv_dequant")
    return out


# A decode step makes these calls for every layer, a few microseconds of kernel each, so their marshalling is kept
# short: pointers and streams as plain integers.
def _addr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise QpackError("qpack kernels take CUDA tensors")
    return t.data_ptr()


# of a torch without CUDA neither exists, and no call gets as far as asking for its stream
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream):
    return _current_stream(_current_device()) if stream is None else stream.cuda_stream


_HERE = contextlib.nullcontext()


def _on(stream):
    """Where a call allocates what the caller did not give: in the order of the stream that it runs on, so that zeroing comes
    before the kernels, and memory that is given back is not handed out again before they end. `stream` is a torch stream, or
    anything with a `cuda_stream` handle, as for the launch."""
    if stream is None:
        return _HERE
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream))


def _out(stream, shape, dtype, device):
    """An output of a call on `stream`, to be read on the current stream too."""
    with _on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream())
    return t


class KVPool:
    """A paged KV cache: keys and values [layers, pages, heads, page_tokens, dim], int8 codes with fp16 scales
    [layers, pages, heads, page_tokens, dim / 32], or fp16 / bf16 without scales. The layer and page strides are free (a
    slice of a larger buffer will do), everything inside a page is contiguous. Holds its tensors; it can be kept for as
    long as they live."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        kind = {torch.int8: KV_I8, torch.float16: KV_F16, torch.bfloat16: KV_BF16}.get(k.dtype)
        if kind is None:
            raise QpackError(f"k: expected int8, float16 or bfloat16, got {k.dtype}")
        if (kind == KV_I8) != (k_scales is not None) or (kind == KV_I8) != (v_scales is not None):
            raise QpackError("k_scales, v_scales: given for int8 pools and for no other")
        sets = [("k", k, k.dtype, 0), ("v", v, k.dtype, 0)]
        if kind == KV_I8:
            sets += [("k_scales", k_scales, torch.float16, 1), ("v_scales", v_scales, torch.float16, 1)]
        for name, t, dtype, scales in sets:
            if t.dtype != dtype:
                raise QpackError(f"{name}: expected {dtype}, got {t.dtype}")
            shape = tuple(k.shape[:-1]) + ((k.shape[-1] // 32,) if scales else (k.shape[-1],))
            if t.dim() != 5 or tuple(t.shape) != shape:
                raise QpackError(f"{name}: expected [layers, pages, heads, page_tokens, dim{' / 32' if scales else ''}] "
                                 f"of {shape}, got {tuple(t.shape)}")
            inner = (t.shape[3] * t.shape[4], t.shape[4], 1)
            if any(n > 1 and st != want for n, st, want in zip(t.shape[2:], t.stride()[2:], inner)):
                raise QpackError(f"{name}: pages are not contiguous, strides {tuple(t.stride())}")
            same = (k if not scales else k_scales).stride()
            if any(n > 1 and a != b for n, a, b in zip(t.shape[:2], t.stride()[:2], same)):
                raise QpackError(f"{name}: layer and page strides differ from {'k_scales' if scales else 'k'}'s")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        layers, pages, heads, page_tokens, dim = k.shape
        self.layers, self.pages, self.heads, self.page_tokens, self.dim = layers, pages, heads, page_tokens, dim

        def strides(t):                                         # of an extent of one they mean nothing
            st = t.stride()
            return (st[0] if layers > 1 else 0), (st[1] if pages > 1 else heads * page_tokens * t.shape[4])

        ls, ps = strides(k)
        sls, sps = strides(k_scales) if kind == KV_I8 else (0, 0)
        self._c = _Pool(_addr(k), _addr(v), _addr(k_scales), _addr(v_scales), ls, ps, sls, sps, pages, layers, heads,
                        page_tokens, dim, kind, 0)
        self._ref = ctypes.addressof(self._c)


def alloc_kv_pool(kind, layers, pages, heads, page_tokens, dim, device="cuda") -> KVPool:
    """An empty pool of the kind KV_I8, KV_F16 or KV_BF16."""
    dt = {KV_I8: torch.int8, KV_F16: torch.float16, KV_BF16: torch.bfloat16}.get(kind)
    if dt is None:
        raise QpackError(f"kind: expected KV_I8, KV_F16 or KV_BF16, got {kind!r}")
    shape = (layers, pages, heads, page_tokens, dim)
    k, v = (torch.zeros(shape, dtype=dt, device=device) for _ in range(2))
    if kind != KV_I8:
        return KVPool(k, v)
    ks, vs = (torch.zeros(shape[:-1] + (dim // 32,), dtype=torch.float16, device=device) for _ in range(2))
    return KVPool(k, v, ks, vs)


class KVTables:
    """The sequences of a pool: page table int32 [seqs, max_pages] (-1: no page), lengths int32 [seqs] and reference
    counts int32 [pages] (not needed by append, read and attend). Holds its tensors."""

    def __init__(self, tables, lens, refs=None):
        if tables.dtype != torch.int32 or tables.dim() != 2 or (tables.shape[1] > 1 and tables.stride(1) != 1):
            raise QpackError(f"tables: expected a row-major int32 matrix, got {tables.dtype} {tuple(tables.shape)} with "
                             f"strides {tuple(tables.stride())}")
        _need(lens, torch.int32, "lens", numel=tables.shape[0])
        if refs is not None:
            _need(refs, torch.int32, "refs", numel=0)
        self.tables, self.lens, self.refs = tables, lens, refs
        stride = tables.stride(0) if tables.shape[0] > 1 else tables.shape[1]
        self._c = _Tables(_addr(tables), _addr(lens), _addr(refs), stride, 0 if refs is None else refs.numel(),
                          tables.shape[0], tables.shape[1])
        self._ref = ctypes.addressof(self._c)


def alloc_kv_tables(seqs, max_pages, pages, device="cuda") -> KVTables:
    """Empty sequences over a pool of `pages` free pages."""
    return KVTables(torch.full((seqs, max_pages), -1, dtype=torch.int32, device=device),
                    torch.zeros(seqs, dtype=torch.int32, device=device),
                    torch.zeros(pages, dtype=torch.int32, device=device))


_DTYPE_CODE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


def _need_rows(t, what, heads, dim):
    """Token rows: [n, heads * dim] or [n, heads, dim], a row contiguous. Returns (dtype code, row stride, n)."""
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise QpackError(f"{what}: expected float32, float16 or bfloat16, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        n, h, d = shape
        ok = h == heads and d == dim and st[2] == 1 and (st[1] == dim or heads == 1)
    else:
        ok = len(shape) == 2 and shape[1] == heads * dim and st[1] == 1
        n = shape[0] if ok else 0
    if not ok:
        raise QpackError(f"{what}: expected rows of {heads} x {dim}, got {tuple(shape)} with strides {tuple(st)}")
    return code, (st[0] if n > 1 else heads * dim), n


def _need_i32(t, what, n):
    if t is not None and (t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous()):
        _need(t, torch.int32, what, numel=n)


def _need_rope(rope, dim):
    """Rows of the rotation table."""
    if rope is None:
        return 0
    shape = rope.shape
    if rope.dtype is not torch.float32 or len(shape) != 2 or shape[1] != dim or not rope.is_contiguous():
        raise QpackError(f"rope: expected a contiguous float32 [positions, {dim}] table, got {rope.dtype} {tuple(shape)}")
    return shape[0]


def qpack_kv_append(pool, layer, tables, k, v, seqs=None, pos=None, rope=None, stream=None):
    """Write new tokens' keys and values (rows [n, heads, dim], float32, float16 or bfloat16) into a layer of the cache:
    token i at position pos[i] of sequence seqs[i] (default: the last token of sequence i). Keys are rotated first
    where `rope` (float32 [positions, dim]: cos | sin) is given; int8 pools quantize by qpack_kv_quantize's rule."""
    dt, ldk, n = _need_rows(k, "k", pool.heads, pool.dim)
    dtv, ldv, nv = _need_rows(v, "v", pool.heads, pool.dim)
    if dtv != dt or nv != n:
        raise QpackError("k, v: expected the same type and number of rows")
    _need_i32(seqs, "seqs", n)
    _need_i32(pos, "pos", n)
    rows = _need_rope(rope, pool.dim)
    rc = (_lib or lib()).qpack_kv_append(pool._ref, layer, tables._ref, _addr(seqs), _addr(pos), n, _addr(k), _addr(v),
                                         dt, ldk, ldv, _addr(rope), rows, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_append")


def qpack_kv_read(pool, layer, tables, seqs=None, pos=None, k_out=None, v_out=None, n=None, stream=None):
    """Rows of the cache: token i from position pos[i] of sequence seqs[i] (as in qpack_kv_append). Returns (k, v),
    [n, heads, dim], float16 (bfloat16 for a bfloat16 pool) unless given."""
    if n is None:
        given = seqs if seqs is not None else pos if pos is not None else k_out if k_out is not None else v_out
        if given is None:
            raise QpackError("n: needed where neither seqs, pos nor an output is given")
        n = given.shape[0]
    if k_out is None and v_out is None:
        dt = torch.bfloat16 if pool.k.dtype == torch.bfloat16 else torch.float16
        k_out, v_out = (_out(stream, (n, pool.heads, pool.dim), dt, pool.k.device) for _ in range(2))
    dk = dv = None
    ldk = ldv = 0
    if k_out is not None:
        dk, ldk, rows = _need_rows(k_out, "k_out", pool.heads, pool.dim)
        if rows < n:
            raise QpackError(f"k_out: expected at least {n} rows, got {rows}")
    if v_out is not None:
        dv, ldv, rows = _need_rows(v_out, "v_out", pool.heads, pool.dim)
        if rows < n:
            raise QpackError(f"v_out: expected at least {n} rows, got {rows}")
        if dk is not None and dk != dv:
            raise QpackError("k_out, v_out: expected the same type")
    _need_i32(seqs, "seqs", n)
    _need_i32(pos, "pos", n)
    rc = (_lib or lib()).qpack_kv_read(pool._ref, layer, tables._ref, _addr(seqs), _addr(pos), n, _addr(k_out),
                                       _addr(v_out), dv if dk is None else dk, ldk, ldv, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_read")
    return k_out, v_out


class KVWorkspace:
    """Scratch memory of a call, laid out once, its first `zeroed` bytes zeroed: attention counts in them, and every
    call leaves them as it found them. Calls that may run at the same time need a workspace each. It is allocated and zeroed
    on the current stream: a call on another one has to be ordered behind that, and the workspace has to outlive the call
    there (as with any tensor that torch allocates)."""

    def __init__(self, bytes, device, zeroed=0):
        self.buffer = torch.empty(bytes, dtype=torch.uint8, device=device)
        if zeroed:
            self.buffer[:zeroed].zero_()
        self._p = _addr(self.buffer)
        self.bytes = bytes


def alloc_kv_workspace(pool, batch, q_heads) -> KVWorkspace:
    """For qpack_kv_attend with up to `batch` rows."""
    n = ctypes.c_int64(0)
    rc = (_lib or lib()).qpack_kv_attend_workspace(pool._ref, batch, q_heads, ctypes.byref(n))
    if rc:
        _check(rc, "qpack_kv_attend_workspace")
    return KVWorkspace(n.value, pool.k.device, KV_ATTEND_ZEROED)


def alloc_kv_page_workspace(pool, tables) -> KVWorkspace:
    """For qpack_kv_fork and qpack_kv_compact."""
    n = ctypes.c_int64(0)
    rc = (_lib or lib()).qpack_kv_page_workspace(pool._ref, tables._ref, ctypes.byref(n))
    if rc:
        _check(rc, "qpack_kv_page_workspace")
    return KVWorkspace(n.value, pool.k.device)


def qpack_kv_attend(pool, layer, tables, q, seqs=None, scale=None, window=0, rope=None, out=None, lse=None,
                    workspace=None, stream=None):
    """Attention of one new token a row: q [B, q_heads, dim] or [B, q_heads * dim] (float32, float16 or bfloat16) over
    the cache of sequence seqs[b] (default b), its last `window` tokens where that is not 0. scale defaults to dim ** -0.5.
    Returns out, of q's shape, float16 unless given (float32 and bfloat16 too); lse, a float32 [B, q_heads] tensor if
    wanted, gets the log-sum-exp. A kept workspace (alloc_kv_workspace) saves its allocation."""
    D, shape = pool.dim, q.shape
    q_heads = shape[1] if len(shape) == 3 else shape[-1] // D
    qdt, ldq, B = _need_rows(q, "q", q_heads, D)
    if out is None:
        out = _out(stream, shape, torch.float16, q.device)
    odt, ldo, rows = _need_rows(out, "out", q_heads, D)
    if rows < B:
        raise QpackError(f"out: expected at least {B} rows, got {rows}")
    _need_i32(seqs, "seqs", B)
    if seqs is None and tables.tables.shape[0] < B:
        raise QpackError(f"q: {B} rows, but the table has {tables.tables.shape[0]} sequences")
    if lse is not None:
        _need(lse, torch.float32, "lse", numel=B * q_heads)
    if workspace is None:
        with _on(stream):
            workspace = alloc_kv_workspace(pool, B, q_heads)
    rows = _need_rope(rope, D)
    rc = (_lib or lib()).qpack_kv_attend(pool._ref, layer, tables._ref, _addr(seqs), B, _addr(q), qdt, ldq, q_heads,
                                         D ** -0.5 if scale is None else scale, window, _addr(rope), rows, _addr(out),
                                         odt, ldo, _addr(lse), workspace._p, workspace.bytes, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_attend")
    return out


def _need_refs(tables):
    if tables.refs is None:
        raise QpackError("tables: this call needs the reference counts")


def qpack_kv_reserve(pool, tables, seqs, add, stream=None):
    """Extend sequence seqs[i] by add[i] tokens, taking the lowest-numbered free pages in the order of the requests. A
    request without enough pages is left as it was and sets FAULT_NO_PAGES."""
    _need_refs(tables)
    n = seqs.numel()
    _need_i32(seqs, "seqs", n)
    _need_i32(add, "add", n)
    rc = (_lib or lib()).qpack_kv_reserve(pool._ref, tables._ref, _addr(seqs), _addr(add), n, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_reserve")


def qpack_kv_fork(pool, tables, src, dst, workspace=None, stream=None):
    """Make the empty sequences dst[i] copies of src[i]: full pages are shared, a part-filled last page is copied."""
    _need_refs(tables)
    n = src.numel()
    _need_i32(src, "src", n)
    _need_i32(dst, "dst", n)
    if workspace is None:
        with _on(stream):
            workspace = alloc_kv_page_workspace(pool, tables)
    rc = (_lib or lib()).qpack_kv_fork(pool._ref, tables._ref, _addr(src), _addr(dst), n, workspace._p,
                                       workspace.bytes, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_fork")


def qpack_kv_free(tables, seqs, stream=None):
    """Release the pages of sequences seqs[i]; they become empty."""
    _need_refs(tables)
    n = seqs.numel()
    _need_i32(seqs, "seqs", n)
    rc = (_lib or lib()).qpack_kv_free(tables._ref, _addr(seqs), n, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_free")


def qpack_kv_compact(pool, tables, tables_out=None, refs_out=None, moved=None, workspace=None, stream=None):
    """Move the live pages to the lowest numbers and renumber the tables and reference counts (in place unless outputs
    of the same layout are given). moved, an int32 tensor if wanted, gets the number of pages moved."""
    _need_refs(tables)
    tables_out = tables.tables if tables_out is None else tables_out
    refs_out = tables.refs if refs_out is None else refs_out
    if tables_out.dtype != torch.int32 or tables_out.shape != tables.tables.shape or \
            tables_out.stride() != tables.tables.stride():
        raise QpackError("tables_out: expected the tables' type, shape and strides")
    _need(refs_out, torch.int32, "refs_out", numel=tables.refs.numel())
    _need_i32(moved, "moved", 1)
    if workspace is None:
        with _on(stream):
            workspace = alloc_kv_page_workspace(pool, tables)
    rc = (_lib or lib()).qpack_kv_compact(pool._ref, tables._ref, _addr(tables_out), _addr(refs_out), _addr(moved),
                                          workspace._p, workspace.bytes, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_compact")
    return tables_out, refs_out


def qpack_kv_copy_pages(pool, src, dst, stream=None):
    """Copy page src[i] to page dst[i] over all layers."""
    n = src.numel()
    _need_i32(src, "src", n)
    _need_i32(dst, "dst", n)
    rc = (_lib or lib()).qpack_kv_copy_pages(pool._ref, _addr(src), _addr(dst), n, _raw_stream(stream))
    if rc:
        _check(rc, "qpack_kv_copy_pages")


def qpack_fetch_fault_flags() -> int:
    v = ctypes.c_int32(0)
    _check(lib().qpack_fetch_fault_flags(ctypes.byref(v)), "qpack_fetch_fault_flags")
    return int(v.value)


def qpack_status_string(status: int) -> str:
    return lib().qpack_status_string(int(status)).decode()


OPT_WEIGHT_PREFETCH = 1
OPT_PREFILL_TILE_ROWS = 2


def qpack_set_option(option: int, value: int) -> None:
    _check(lib().qpack_set_option(int(option), int(value)), "qpack_set_option")


def qpack_version() -> int:
    return int(lib().qpack_version())
