"""ctypes binding of include/magicpig.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmagicpig_b200.so")

MP_OK = 0
MP_ERR_ARG = -1
MP_ERR_SHAPE = -2
MP_ERR_ALIGN = -3
MP_ERR_CAPACITY = -4
MP_ERR_WORKSPACE = -5
MP_ERR_CUDA = -6
MP_ERR_TOO_LARGE = -7
MP_CODES_AUTO = 0
MP_CODES_BYTES = 1
MP_CODES_PLANES = 2
MP_PATH_AUTO = 0
MP_PATH_SPLIT = 1
MP_PATH_FUSED = 2
MP_PATH_TC = 3


class MagicPIGError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class _CShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "n_q_heads", "n_kv_heads", "head_dim", "capacity", "k_bits", "n_tables",
                 "sink", "window", "code_layout")]


class _CDebug(ctypes.Structure):
    _fields_ = [("qcodes_in", ctypes.c_void_p), ("qcodes_out", ctypes.c_void_p),
                ("member_out", ctypes.c_void_p), ("path", ctypes.c_int32), ("skip_scan", ctypes.c_int32)]


class _CPromptShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "n_q_heads", "n_kv_heads", "head_dim", "total", "q_stride", "k_stride", "v_stride")]


class _CPagesShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "n_q_heads", "n_kv_heads", "head_dim", "n_pages", "page_size", "max_pages")]


MP_CODES_AUTO_PLANES_MIN = 1 << 21  # include/magicpig.h


def auto_planes(batch: int, n_kv_heads: int, capacity: int, k_bits: int) -> bool:
    """MP_CODES_AUTO: bit planes, except byte codes for K = 8 problems with
    fewer than MP_CODES_AUTO_PLANES_MIN (token, kv head) slots."""
    return k_bits != 8 or batch * n_kv_heads * capacity >= MP_CODES_AUTO_PLANES_MIN


@dataclasses.dataclass(frozen=True)
class Shape:
    """Problem shape (see mp_shape in include/magicpig.h)."""
    batch: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    capacity: int
    k_bits: int
    n_tables: int
    sink: int
    window: int
    code_layout: int = 0  # MP_CODES_AUTO

    @property
    def planes(self) -> bool:
        """Whether the key codes are bit planes (the library's rule for MP_CODES_AUTO)."""
        if self.code_layout == MP_CODES_AUTO:
            return auto_planes(self.batch, self.n_kv_heads, self.capacity, self.k_bits)
        return self.code_layout == MP_CODES_PLANES

    def c(self) -> _CShape:
        return _CShape(*dataclasses.astuple(self))


_lib = None


def library() -> ctypes.CDLL:
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise MagicPIGError(MP_ERR_CUDA, f"{library_path} not built (run __graft_entry__.build())")
        lib = ctypes.CDLL(library_path)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        SP = ctypes.POINTER(_CShape)
        lib.mp_codes_bytes.argtypes = [SP, ctypes.POINTER(SZ)]
        lib.mp_hash_keys.argtypes = [SP, P, P, P, I32, P, P, P]
        lib.mp_hash_keys_range.argtypes = [SP, P, P, I32, I32, P, P, P]
        lib.mp_hash_queries.argtypes = [SP, P, P, P, P]
        lib.mp_append_token.argtypes = [SP, P, P, P, P, P, P, P, P, P]
        lib.mp_decode_workspace_bytes.argtypes = [SP, I32, ctypes.POINTER(SZ)]
        lib.mp_decode_attend.argtypes = [SP, P, P, P, P, P, P, I32, P, P, P, P, SZ,
                                         ctypes.POINTER(_CDebug), P]
        lib.mp_decode_attend_noalloc.argtypes = [SP, P, P, P, P, P, P, I32, P, P, P, P, P]
        lib.mp_quantize_keys.argtypes = [SP, P, P, I32, I32, P, P]
        lib.mp_append_token_q8.argtypes = [SP, P, P, P, P, P, P, P, P, P, P]
        lib.mp_decode_attend_q8.argtypes = [SP, P, P, P, P, P, P, I32, P, P, P, P, SZ,
                                            ctypes.POINTER(_CDebug), P]
        PP, GP = ctypes.POINTER(_CPromptShape), ctypes.POINTER(_CPagesShape)
        lib.mp_prompt_attend.argtypes = [PP, P, P, P, P, P, P, P, P]
        lib.mp_paged_workspace_bytes.argtypes = [GP, I32, ctypes.POINTER(SZ)]
        lib.mp_paged_attend.argtypes = [GP, P, P, P, P, P, I32, P, P, P, SZ, P, P]
        lib.mp_paged_append.argtypes = [GP, P, P, I32, I32, P, I32, I32, P, P, P, P, P, P]
        lib.mp_pages_reserve.argtypes = [GP, P, P, P, P, P, P]
        lib.mp_pages_fork.argtypes = [GP, P, P, I32, P, P, P, P, P, P]
        lib.mp_pages_free.argtypes = [GP, P, I32, P, P, P, P, P]
        lib.mp_pages_compact.argtypes = [GP, P, P, P, P, P]
        lib.mp_pages_copy.argtypes = [GP, P, I32, P, P, P, P]
        lib.mp_read_status.argtypes = [P, ctypes.POINTER(I32), P]
        lib.mp_status_string.argtypes = [ctypes.c_int]
        lib.mp_status_string.restype = ctypes.c_char_p
        for f in ("mp_codes_bytes", "mp_hash_keys", "mp_hash_keys_range", "mp_hash_queries", "mp_append_token",
                  "mp_decode_workspace_bytes", "mp_decode_attend", "mp_decode_attend_noalloc",
                  "mp_quantize_keys", "mp_append_token_q8", "mp_decode_attend_q8", "mp_read_status",
                  "mp_prompt_attend", "mp_paged_workspace_bytes", "mp_paged_attend", "mp_paged_append",
                  "mp_pages_reserve", "mp_pages_fork", "mp_pages_free", "mp_pages_compact", "mp_pages_copy"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


def status_string(code: int) -> str:
    try:
        return library().mp_status_string(int(code)).decode()
    except MagicPIGError:
        return f"status {code}"


def _check(code: int, where: str):
    if code != MP_OK:
        raise MagicPIGError(code, where)


def _ptr(t) -> Optional[int]:
    """Device pointer of a torch tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:  # torch.cuda.current_stream() without building its Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def codes_bytes(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check(library().mp_codes_bytes(ctypes.byref(shape.c()), ctypes.byref(n)), "mp_codes_bytes")
    return n.value


def codes_shape(shape: Shape):
    """(dtype name, tensor shape) of the key codes: uint8 [B,Hkv,L,Ncap] for
    byte codes, int32 bit planes [B,Hkv,L,Ncap/32,K] for plane codes."""
    B, Hkv, L, K, N = shape.batch, shape.n_kv_heads, shape.n_tables, shape.k_bits, shape.capacity
    if not shape.planes:
        return "uint8", (B, Hkv, L, N)
    return "int32", (B, Hkv, L, N // 32, K)


def decode_workspace_bytes(shape: Shape, max_len: int) -> int:
    n = ctypes.c_size_t()
    _check(library().mp_decode_workspace_bytes(ctypes.byref(shape.c()), int(max_len), ctypes.byref(n)),
           "mp_decode_workspace_bytes")
    return n.value


def hash_keys(shape: Shape, keys, W, n_tokens: int, codes, seq_lens=None, status=None, stream=None):
    _check(library().mp_hash_keys(ctypes.byref(shape.c()), _ptr(keys), _ptr(W), _ptr(seq_lens), int(n_tokens),
                                  _ptr(codes), _ptr(status), _stream(stream)), "mp_hash_keys")


def hash_keys_range(shape: Shape, keys, W, first_token: int, n_tokens: int, codes, status=None, stream=None):
    """Hashes tokens [first_token, first_token + n_tokens) of every unit (a
    streamed prefill block; first_token a multiple of 128)."""
    _check(library().mp_hash_keys_range(ctypes.byref(shape.c()), _ptr(keys), _ptr(W), int(first_token),
                                        int(n_tokens), _ptr(codes), _ptr(status), _stream(stream)),
           "mp_hash_keys_range")


def hash_queries(shape: Shape, q, W, qcodes, stream=None):
    _check(library().mp_hash_queries(ctypes.byref(shape.c()), _ptr(q), _ptr(W), _ptr(qcodes), _stream(stream)),
           "mp_hash_queries")


def append_token(shape: Shape, k_new, v_new, W, k_cache, v_cache, codes, seq_lens, status=None, stream=None):
    _check(library().mp_append_token(ctypes.byref(shape.c()), _ptr(k_new), _ptr(v_new), _ptr(W),
                                     _ptr(k_cache), _ptr(v_cache), _ptr(codes), _ptr(seq_lens), _ptr(status),
                                     _stream(stream)), "mp_append_token")


def decode_attend(shape: Shape, q, W, codes, k_cache, v_cache, seq_lens, max_len: int, out, lse, n_sampled,
                  workspace, qcodes_in=None, qcodes_out=None, member_out=None, path: int = 0, skip_scan: bool = False,
                  stream=None):
    dbg = None
    if qcodes_in is not None or qcodes_out is not None or member_out is not None or path or skip_scan:
        dbg = ctypes.byref(_CDebug(_ptr(qcodes_in), _ptr(qcodes_out), _ptr(member_out), int(path),
                                   int(bool(skip_scan))))
    nbytes = workspace.numel() * workspace.element_size()
    _check(library().mp_decode_attend(ctypes.byref(shape.c()), _ptr(q), _ptr(W), _ptr(codes), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(seq_lens), int(max_len), _ptr(out), _ptr(lse),
                                      _ptr(n_sampled), _ptr(workspace), nbytes, dbg, _stream(stream)),
           "mp_decode_attend")


def decode_attend_noalloc(shape: Shape, q, W, codes, k_cache, v_cache, seq_lens, max_len: int, out, lse,
                          n_sampled, status=None, stream=None):
    """mp_decode_attend with the library's fixed scratch array instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _check(library().mp_decode_attend_noalloc(ctypes.byref(shape.c()), _ptr(q), _ptr(W), _ptr(codes),
                                              _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), int(max_len),
                                              _ptr(out), _ptr(lse), _ptr(n_sampled), _ptr(status),
                                              _stream(stream)), "mp_decode_attend_noalloc")


Q8_ROW_BYTES = 144  # MP_Q8_ROW_BYTES


def quantize_keys(shape: Shape, k_cache, k8, first_token: int = 0, n_tokens: Optional[int] = None,
                  seq_lens=None, stream=None):
    """Writes the int8 rows of key rows [first_token, first_token + n_tokens)
    (default: the whole capacity) into k8, int8 [B,Hkv,Ncap,144]: 128 int8
    values, then the fp32 record {power-of-two scale, squared norm of the
    int8 row times the scale, 0, 0}."""
    n = shape.capacity - int(first_token) if n_tokens is None else int(n_tokens)
    _check(library().mp_quantize_keys(ctypes.byref(shape.c()), _ptr(k_cache), _ptr(seq_lens), int(first_token), n,
                                      _ptr(k8), _stream(stream)), "mp_quantize_keys")


def append_token_q8(shape: Shape, k_new, v_new, W, k_cache, v_cache, codes, seq_lens, k8, status=None,
                    stream=None):
    _check(library().mp_append_token_q8(ctypes.byref(shape.c()), _ptr(k_new), _ptr(v_new), _ptr(W),
                                        _ptr(k_cache), _ptr(v_cache), _ptr(codes), _ptr(seq_lens), _ptr(k8),
                                        _ptr(status), _stream(stream)), "mp_append_token_q8")


def decode_attend_q8(shape: Shape, q, W, codes, k8, v_cache, seq_lens, max_len: int, out, lse, n_sampled,
                     workspace, qcodes_in=None, qcodes_out=None, member_out=None, path: int = 0, stream=None):
    """decode_attend with the K rows gathered from the int8 copy."""
    dbg = None
    if qcodes_in is not None or qcodes_out is not None or member_out is not None or path:
        dbg = ctypes.byref(_CDebug(_ptr(qcodes_in), _ptr(qcodes_out), _ptr(member_out), int(path)))
    nbytes = workspace.numel() * workspace.element_size()
    _check(library().mp_decode_attend_q8(ctypes.byref(shape.c()), _ptr(q), _ptr(W), _ptr(codes), _ptr(k8),
                                         _ptr(v_cache), _ptr(seq_lens), int(max_len), _ptr(out),
                                         _ptr(lse), _ptr(n_sampled), _ptr(workspace), nbytes, dbg,
                                         _stream(stream)), "mp_decode_attend_q8")


# ---- exact attention: prompts and the paged cache (include/magicpig.h) ----

def _i32(n: int, what: str) -> int:
    """n, refused where the library's 32-bit argument does not hold it (ctypes keeps the low bits without a word)."""
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError(f"{what}: {n} does not fit 32 bits")
    return n


def _fields32(shape):
    """A shape's fields, in order, each checked by _i32."""
    return [_i32(getattr(shape, f.name), f.name) for f in dataclasses.fields(shape)]

@dataclasses.dataclass(frozen=True)
class PromptShape:
    """Shape of packed prompts (see mp_prompt_shape; the strides come from the tensors)."""
    batch: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    total: int

    def __post_init__(self):
        _fields32(self)


@dataclasses.dataclass(frozen=True)
class PagesShape:
    """Shape of a paged key-value cache (see mp_pages_shape)."""
    batch: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    n_pages: int
    page_size: int
    max_pages: int

    def __post_init__(self):
        # frozen, so the C struct and the tensors' shapes are made once
        def put(name, value):
            object.__setattr__(self, name, value)
        put("_c", _CPagesShape(*_fields32(self)))
        put("_ref", ctypes.byref(self._c))
        put("_pool", (self.n_pages, self.n_kv_heads, self.page_size, self.head_dim))
        put("_table", (self.batch, self.max_pages))
        put("_q", (self.batch, self.n_q_heads, self.head_dim))

    def __reduce__(self):  # the C struct is made anew where a copy or a pickle arrives
        return PagesShape, dataclasses.astuple(self)

    def c(self) -> _CPagesShape:
        return self._c


def _refuse(t, what: str, dtype, shape, device: int):
    raise ValueError(f"{what}: expected {tuple(shape)} of {dtype} on cuda:{device} (the current device), got "
                     f"{tuple(t.shape)}, strides {tuple(t.stride())}, of {t.dtype} on {t.device}")


def _arg(t, what: str, dtype, shape, device: int) -> int:
    """Device pointer of a contiguous tensor of this type and shape on the current device."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(t, what, dtype, shape, device)
    return t.data_ptr()


def _rows_arg(t, what: str, dtype, shape, device: int):
    """(device pointer, token stride in elements) of [tokens, heads, head_dim] rows whose heads lie side by side."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, what, dtype, shape, device)
    rows, heads, d = shape
    s0, s1, s2 = t.stride()
    if rows and (s2 != 1 or (heads > 1 and s1 != d)) or rows > 1 and s0 < heads * d:
        _refuse(t, what, dtype, shape, device)
    return t.data_ptr(), _i32(s0, f"{what}: token stride") if rows > 1 else 0  # (0 is "side by side" to the library)


def _opt(t, what: str, dtype, shape, device: int) -> Optional[int]:
    return None if t is None else _arg(t, what, dtype, shape, device)


def prompt_attend(shape: PromptShape, q, k, v, cu_lens, out, lse=None, status=None, stream=None):
    """Causal attention over packed prompts: q bf16 [T,Hq,d], k / v bf16 [T,Hkv,d] (token rows may be strided:
    parts of a fused projection), cu_lens int32 [B+1], out bf16 [T,Hq,d], lse fp32 [T,Hq] or None."""
    import torch
    dev, bf16 = torch.cuda.current_device(), torch.bfloat16
    T, Hq, Hkv, d = shape.total, shape.n_q_heads, shape.n_kv_heads, shape.head_dim
    qp, qs = _rows_arg(q, "q", bf16, (T, Hq, d), dev)
    kp, ks = _rows_arg(k, "k", bf16, (T, Hkv, d), dev)
    vp, vs = _rows_arg(v, "v", bf16, (T, Hkv, d), dev)
    cs = _CPromptShape(shape.batch, Hq, Hkv, d, T, qs, ks, vs)
    _check(library().mp_prompt_attend(ctypes.byref(cs), qp, kp, vp,
                                      _arg(cu_lens, "cu_lens", torch.int32, (shape.batch + 1,), dev),
                                      _arg(out, "out", bf16, (T, Hq, d), dev), _opt(lse, "lse", torch.float32, (T, Hq), dev),
                                      _opt(status, "status", torch.int32, (1,), dev), _stream(stream)),
           "mp_prompt_attend")


def paged_workspace_bytes(shape: PagesShape, max_len: int) -> int:
    n = ctypes.c_size_t()
    _check(library().mp_paged_workspace_bytes(shape._ref, _i32(int(max_len), "max_len"), ctypes.byref(n)),
           "mp_paged_workspace_bytes")
    return n.value


def paged_attend(shape: PagesShape, q, k_pages, v_pages, page_table, seq_lens, max_len: int, out, lse, workspace,
                 status=None, stream=None):
    """One exact decode step over a paged cache: q bf16 [B,Hq,d], pools bf16 [P,Hkv,S,d], page_table int32 [B,M],
    seq_lens int32 [B], out fp32 [B,Hq,d], lse fp32 [B,Hq], workspace of paged_workspace_bytes(shape, max_len)
    bytes or more."""
    import torch
    dev, bf16, i32, f32 = torch.cuda.current_device(), torch.bfloat16, torch.int32, torch.float32
    _check(library().mp_paged_attend(shape._ref, _arg(q, "q", bf16, shape._q, dev),
                                     _arg(k_pages, "k_pages", bf16, shape._pool, dev),
                                     _arg(v_pages, "v_pages", bf16, shape._pool, dev),
                                     _arg(page_table, "page_table", i32, shape._table, dev),
                                     _arg(seq_lens, "seq_lens", i32, (shape.batch,), dev), _i32(int(max_len), "max_len"),
                                     _arg(out, "out", f32, shape._q, dev), _arg(lse, "lse", f32, shape._q[:2], dev),
                                     _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev),
                                     workspace.numel() * workspace.element_size(),
                                     _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_paged_attend")


def paged_append(shape: PagesShape, k_new, v_new, page_table, seq_lens, k_pages, v_pages, cu_new=None,
                 advance: bool = True, status=None, stream=None):
    """Writes new rows k_new / v_new bf16 [n,Hkv,d] behind the sequences' tokens: one for each sequence (n == B),
    or rows [cu_new[b], cu_new[b+1]) for sequence b (cu_new int32 [B+1]).  advance: seq_lens grow."""
    import torch
    dev, bf16, i32 = torch.cuda.current_device(), torch.bfloat16, torch.int32
    rows = (_i32(k_new.shape[0], "rows of k_new"), shape.n_kv_heads, shape.head_dim)
    knp, ks = _rows_arg(k_new, "k_new", bf16, rows, dev)
    vnp, vs = _rows_arg(v_new, "v_new", bf16, rows, dev)
    _check(library().mp_paged_append(shape._ref, knp, vnp, ks, vs, _opt(cu_new, "cu_new", i32, (shape.batch + 1,), dev),
                                     rows[0], 1 if advance else 0, _arg(page_table, "page_table", i32, shape._table, dev),
                                     _arg(seq_lens, "seq_lens", i32, (shape.batch,), dev),
                                     _arg(k_pages, "k_pages", bf16, shape._pool, dev),
                                     _arg(v_pages, "v_pages", bf16, shape._pool, dev),
                                     _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_paged_append")


def pages_reserve(shape: PagesShape, n_new, page_table, seq_lens, refs, status=None, stream=None):
    """Takes the lowest free pages so that sequence b can hold n_new[b] tokens more (n_new int32 [B])."""
    import torch
    dev, i32 = torch.cuda.current_device(), torch.int32
    _check(library().mp_pages_reserve(shape._ref, _arg(n_new, "n_new", i32, (shape.batch,), dev),
                                      _arg(page_table, "page_table", i32, shape._table, dev),
                                      _arg(seq_lens, "seq_lens", i32, (shape.batch,), dev),
                                      _arg(refs, "refs", i32, (shape.n_pages,), dev),
                                      _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_pages_reserve")


def pages_fork(shape: PagesShape, src, dst, page_table, seq_lens, refs, copies, status=None, stream=None):
    """Makes sequence dst[i] a copy of src[i] (int32 [n] both); copies int32 [1+n,4] receives the page copies that
    pages_copy has to make in every layer's pools."""
    import torch
    dev, i32, n = torch.cuda.current_device(), torch.int32, _i32(src.numel(), "entries of src")
    _check(library().mp_pages_fork(shape._ref, _arg(src, "src", i32, (n,), dev), _arg(dst, "dst", i32, (n,), dev), n,
                                   _arg(page_table, "page_table", i32, shape._table, dev),
                                   _arg(seq_lens, "seq_lens", i32, (shape.batch,), dev),
                                   _arg(refs, "refs", i32, (shape.n_pages,), dev),
                                   _arg(copies, "copies", i32, (1 + n, 4), dev),
                                   _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_pages_fork")


def pages_free(shape: PagesShape, seqs, page_table, seq_lens, refs, status=None, stream=None):
    """Ends the sequences seqs (int32 [n]): their pages lose a count, their rows become -1, their lengths 0."""
    import torch
    dev, i32, n = torch.cuda.current_device(), torch.int32, _i32(seqs.numel(), "entries of seqs")
    _check(library().mp_pages_free(shape._ref, _arg(seqs, "seqs", i32, (n,), dev), n,
                                   _arg(page_table, "page_table", i32, shape._table, dev),
                                   _arg(seq_lens, "seq_lens", i32, (shape.batch,), dev),
                                   _arg(refs, "refs", i32, (shape.n_pages,), dev),
                                   _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_pages_free")


def pages_compact(shape: PagesShape, page_table, refs, copies, status=None, stream=None):
    """Brings the pages in use to the front of the pools; copies int32 [1+P//2,4] receives the page copies that
    pages_copy has to make in every layer's pools."""
    import torch
    dev, i32 = torch.cuda.current_device(), torch.int32
    _check(library().mp_pages_compact(shape._ref, _arg(page_table, "page_table", i32, shape._table, dev),
                                      _arg(refs, "refs", i32, (shape.n_pages,), dev),
                                      _arg(copies, "copies", i32, (1 + shape.n_pages // 2, 4), dev),
                                      _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_pages_compact")


def pages_copy(shape: PagesShape, copies, k_pages, v_pages, status=None, stream=None):
    """Copies pages within one layer's pools: copies int32 [1+n,4], entry 0 {count,0,0,0}, then {src, dst, rows, 0}."""
    import torch
    dev, bf16, i32 = torch.cuda.current_device(), torch.bfloat16, torch.int32
    n = _i32(copies.shape[0], "entries of copies")
    _check(library().mp_pages_copy(shape._ref, _arg(copies, "copies", i32, (n, 4), dev), n - 1,
                                   _arg(k_pages, "k_pages", bf16, shape._pool, dev),
                                   _arg(v_pages, "v_pages", bf16, shape._pool, dev),
                                   _opt(status, "status", i32, (1,), dev), _stream(stream)), "mp_pages_copy")


def read_status(workspace, stream=None) -> int:
    v = ctypes.c_int32()
    _check(library().mp_read_status(_ptr(workspace), ctypes.byref(v), _stream(stream)), "mp_read_status")
    return v.value
