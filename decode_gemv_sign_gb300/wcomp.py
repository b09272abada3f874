"""Python binding of the C-ABI library (argument marshalling only).

Every operation runs in the CUDA kernels of libwcomp.so; this module passes
device pointers, sizes and the current CUDA stream through ctypes and turns
status codes into exceptions.  PyTorch is used for device memory and streams.
There is no fallback: if the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libwcomp.so")

BYTESPLIT = 0
K15 = 1
SCHEMES = {"bytesplit": BYTESPLIT, "byte-split": BYTESPLIT, "k15": K15, BYTESPLIT: BYTESPLIT, K15: K15}

SCORING = {"softmax": 0, "sigmoid": 1}

OK, EINVAL, ENOMEM, ECORRUPT, ECUDA, EUNSUPPORTED, ETIMEOUT, EINTERNAL, EBOUNDS = 0, -1, -2, -3, -4, -5, -6, -7, -8


class WcompError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_strerror(status)} ({status})")


class CorruptContainer(WcompError):
    pass


class Info(ctypes.Structure):
    _fields_ = [
        ("scheme", ctypes.c_int32), ("version", ctypes.c_int32),
        ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("n", ctypes.c_int64),
        ("n_escapes", ctypes.c_uint64), ("tile_elems", ctypes.c_uint32), ("n_tiles", ctypes.c_uint32),
        ("table", ctypes.c_uint16 * 15), ("pad_", ctypes.c_uint16),
        ("bytes_codes", ctypes.c_uint64), ("bytes_raw", ctypes.c_uint64), ("bytes_index", ctypes.c_uint64),
        ("bytes_escapes", ctypes.c_uint64), ("serialized_bytes", ctypes.c_uint64),
        ("entropy_bpw", ctypes.c_double), ("physical_bpw", ctypes.c_double),
        ("serialized_compact_bytes", ctypes.c_uint64), ("physical_compact_bpw", ctypes.c_double),
    ]

    def as_dict(self) -> dict:
        d = {k: getattr(self, k) for k, _ in self._fields_ if k not in ("table", "pad_")}
        d["table"] = list(self.table)
        return d


class Q4Info(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("group", ctypes.c_int32),
                ("pad_", ctypes.c_int32), ("bytes", ctypes.c_uint64)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "pad_"}


class Kv4Info(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("bytes", ctypes.c_uint64)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_}


class Kv4Seqs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_table", "d_lengths", "d_starts")] + [
        ("B", ctypes.c_int32), ("width", ctypes.c_int32)]


class Kv4AttendArgs(ctypes.Structure):
    _fields_ = [("s", Kv4Seqs), ("d_q", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("d_out", ctypes.c_void_p), ("d_lse", ctypes.c_void_p), ("d_mass", ctypes.c_void_p),
                ("T", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class Kv4EvictArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_table", "d_lengths", "d_mass", "d_table_out", "d_lengths_out",
                                               "d_mass_out", "d_kept")] + [
        (n, ctypes.c_int32) for n in ("B", "width", "width_out", "keep", "recent")]


class LogprobsArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_logits", "d_ids", "d_logprob", "d_entropy", "d_lse",
                                               "d_top_logprobs", "d_top_ids")] + [
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("row", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_x", "d_router", "d_bias", "d_gate", "d_up", "d_down", "q4_gate",
                                               "q4_up", "q4_down", "d_y", "d_ids", "d_weights")] + [
        ("H", ctypes.c_int64), ("F", ctypes.c_int64), ("T", ctypes.c_int32), ("E", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("scoring", ctypes.c_int32), ("renormalize", ctypes.c_int32),
        ("factor", ctypes.c_float)]


_lib = None
P = ctypes.c_void_p


def lib():
    """Load libwcomp.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
    L = ctypes.CDLL(LIB_PATH)
    L.wcomp_encode.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P, ctypes.POINTER(P)]
    L.wcomp_encode_batched.argtypes = [ctypes.POINTER(P), ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                       P, ctypes.POINTER(P)]
    L.wcomp_encode_hist_grid.argtypes = [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_uint32)]
    L.wcomp_decode.argtypes = [P, P, P]
    L.wcomp_gemv.argtypes = [P, P, ctypes.c_int, P, P]
    L.wcomp_gemv_noalloc.argtypes = [P, P, ctypes.c_int, P, P]
    L.wcomp_gemv_bf16.argtypes = [P, ctypes.c_int64, ctypes.c_int64, P, ctypes.c_int, P, P]
    L.wcomp_gemv_bf16_batched.argtypes = [ctypes.POINTER(P), ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(P), ctypes.c_int,
                                          ctypes.POINTER(P), ctypes.c_int, P]
    L.wcomp_decode_batched.argtypes = [ctypes.POINTER(P), ctypes.POINTER(P), ctypes.c_int, P]
    L.wcomp_gemv_batched.argtypes = [ctypes.POINTER(P), ctypes.POINTER(P), ctypes.c_int, ctypes.POINTER(P),
                                     ctypes.c_int, P]
    L.wcomp_info.argtypes = [P, ctypes.POINTER(Info)]
    L.wcomp_serialize.argtypes = [P, P, ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64), P]
    L.wcomp_serialize_compact.argtypes = [P, P, ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64), P]
    L.wcomp_deserialize.argtypes = [P, ctypes.c_uint64, P, ctypes.POINTER(P)]
    L.wcomp_free.argtypes = [P, P]
    L.wcomp_free.restype = None
    L.wcomp_strerror.argtypes = [ctypes.c_int]
    L.wcomp_strerror.restype = ctypes.c_char_p
    L.wcomp_version.argtypes = []
    L.wcomp_device_check.argtypes = [P]
    L.wcomp_device_check.restype = ctypes.c_int
    L.wcomp_debug_skip_first_copy.argtypes = [ctypes.c_int]
    L.wcomp_debug_skip_first_copy.restype = ctypes.c_int
    L.wcomp_q4_encode.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P,
                                  ctypes.POINTER(P)]
    L.wcomp_q4_pack.argtypes = [P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P,
                                ctypes.POINTER(P)]
    L.wcomp_q4_unpack.argtypes = [P, P, P, P]
    L.wcomp_q4_decode.argtypes = [P, P, P]
    L.wcomp_q4_gemv.argtypes = [P, P, ctypes.c_int, P, P]
    L.wcomp_q4_info.argtypes = [P, ctypes.POINTER(Q4Info)]
    L.wcomp_q4_free.argtypes = [P, P]
    L.wcomp_q4_free.restype = None
    L.wcomp_moe.argtypes = [ctypes.POINTER(MoeArgs), P]
    L.wcomp_kv4_create.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, P, ctypes.POINTER(P)]
    L.wcomp_kv4_append.argtypes = [P, ctypes.POINTER(Kv4Seqs), P, ctypes.c_int64, ctypes.c_int64, P, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int64, P]
    L.wcomp_kv4_read.argtypes = [P, ctypes.POINTER(Kv4Seqs), P, P, ctypes.c_int64, P]
    L.wcomp_kv4_attend.argtypes = [P, ctypes.POINTER(Kv4AttendArgs), P]
    L.wcomp_kv4_evict.argtypes = [P, ctypes.POINTER(Kv4EvictArgs), P]
    L.wcomp_kv4_info.argtypes = [P, ctypes.POINTER(Kv4Info)]
    L.wcomp_kv4_free.argtypes = [P, P]
    L.wcomp_kv4_free.restype = None
    L.wcomp_logprobs.argtypes = [ctypes.POINTER(LogprobsArgs), P]
    L.wcomp_launch_count.argtypes = []
    L.wcomp_launch_count.restype = ctypes.c_uint64
    for name in ("wcomp_encode", "wcomp_encode_batched", "wcomp_encode_hist_grid", "wcomp_decode", "wcomp_gemv", "wcomp_gemv_noalloc",
                 "wcomp_gemv_bf16", "wcomp_gemv_bf16_batched",
                 "wcomp_decode_batched",
                 "wcomp_gemv_batched", "wcomp_info", "wcomp_serialize", "wcomp_serialize_compact",
                 "wcomp_deserialize", "wcomp_version", "wcomp_debug_skip_first_copy", "wcomp_q4_encode",
                 "wcomp_q4_pack", "wcomp_q4_unpack", "wcomp_q4_decode", "wcomp_q4_gemv", "wcomp_q4_info",
                 "wcomp_moe", "wcomp_kv4_create", "wcomp_kv4_append", "wcomp_kv4_read", "wcomp_kv4_attend",
                 "wcomp_kv4_evict", "wcomp_kv4_info", "wcomp_logprobs"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _strerror(s: int) -> str:
    try:
        return lib().wcomp_strerror(s).decode()
    except Exception:  # pragma: no cover
        return "error"


def _check(status: int, what: str):
    if status == ECORRUPT:
        raise CorruptContainer(status, what)
    if status != OK:
        raise WcompError(status, what)


# The current stream's handle alone: making torch's stream object takes longer
# than a small launch.  Not part of torch's documented interface, so it may be gone.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> int:
    if stream is None:
        if _raw_stream is None:
            return int(torch.cuda.current_stream().cuda_stream)
        return _raw_stream(torch.cuda.current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _bits16(t: torch.Tensor, what: str) -> torch.Tensor:
    """A contiguous CUDA tensor of 16-bit BF16 bit patterns (bf16, int16 or uint16)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{what} must hold BF16 bits (bfloat16, int16 or uint16), got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


class Container:
    """An encoded tensor living on the GPU (owned by the library)."""

    def __init__(self, handle: int, shape=None):
        self._h = handle
        self._info = None
        self._shape = tuple(shape) if shape is not None else None  # (N, K) when the caller knows it

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("container was freed")
        return self._h

    def info(self) -> dict:
        if self._info is None:
            inf = Info()
            _check(lib().wcomp_info(P(self.handle), ctypes.byref(inf)), "wcomp_info")
            self._info = inf.as_dict()
        return self._info

    @property
    def shape(self) -> tuple:
        """(N, K), without a description call when the shape is known from the encode."""
        if self._shape is None:
            inf = self.info()
            self._shape = (inf["N"], inf["K"])
        return self._shape

    @property
    def N(self) -> int:
        return self.shape[0]

    @property
    def K(self) -> int:
        return self.shape[1]

    @property
    def scheme(self) -> int:
        return self.info()["scheme"]

    def free(self, stream=None):
        if self._h:
            lib().wcomp_free(P(self._h), P(_stream(stream)))
            self._h = 0

    def __del__(self):
        try:
            if self._h and torch.cuda.is_available():
                self.free()
        except Exception:
            pass


def encode(w: torch.Tensor, scheme, stream=None) -> Container:
    """Encode BF16 weights W[N, K] (a 1-D tensor is one row)."""
    w = _bits16(w, "w")
    N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, w.numel())
    if w.dim() not in (1, 2):
        raise ValueError("w must be 1-D or 2-D")
    h = P()
    _check(lib().wcomp_encode(P(w.data_ptr()), N, K, SCHEMES[scheme], P(_stream(stream)), ctypes.byref(h)),
           "wcomp_encode")
    return Container(h.value, (N, K))


def encode_batched(ws: Sequence[torch.Tensor], schemes, stream=None) -> List[Container]:
    """Encode several tensors in one batched pass (one host synchronization).

    ``schemes`` is one scheme for all tensors or a sequence with one per tensor.
    """
    n = len(ws)
    if isinstance(schemes, (str, int)):
        schemes = [schemes] * n
    Ns, Ks = [], []
    for w in ws:
        _bits16(w, "w")
        if w.dim() not in (1, 2):
            raise ValueError("w must be 1-D or 2-D")
        Ns.append(w.shape[0] if w.dim() == 2 else 1)
        Ks.append(w.shape[1] if w.dim() == 2 else w.numel())
    outs = (P * n)()
    _check(lib().wcomp_encode_batched(_ptr_array([w.data_ptr() for w in ws]), (ctypes.c_int64 * n)(*Ns),
                                      (ctypes.c_int64 * n)(*Ks), (ctypes.c_int * n)(*[SCHEMES[x] for x in schemes]),
                                      n, P(_stream(stream)), outs), "wcomp_encode_batched")
    return [Container(outs[i], (Ns[i], Ks[i])) for i in range(n)]


def decode(c: Container, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Exact BF16 bits of W[N, K] as an int16 tensor (``out`` if given)."""
    inf = c.info()
    if out is None:
        out = torch.empty((inf["N"], inf["K"]), dtype=torch.int16, device="cuda")
    out = _bits16(out, "out")
    if out.numel() != inf["n"]:
        raise ValueError("out has the wrong size")
    _check(lib().wcomp_decode(P(c.handle), P(out.data_ptr()), P(_stream(stream))), "wcomp_decode")
    return out


def gemv(c: Container, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[B, N] (fp32) = x[B, K] @ W.T with W decoded in registers."""
    x = _bits16(x, "x")
    N, K = c.shape
    B = x.shape[0] if x.dim() == 2 else 1
    if x.numel() != B * K:
        raise ValueError("x has the wrong size")
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device="cuda")
    if y.dtype != torch.float32 or not y.is_contiguous() or y.numel() != B * N:
        raise ValueError("y must be a contiguous float32 tensor of B*N elements")
    _check(lib().wcomp_gemv(P(c.handle), P(x.data_ptr()), B, P(y.data_ptr()), P(_stream(stream))), "wcomp_gemv")
    return y


def gemv_noalloc(c: Container, x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """wcomp_gemv without any device allocation by the library.

    For callers that cannot let a library allocate device memory (a fixed
    memory budget, or no implicit synchronisation from cudaMalloc / cudaFree).
    ``y`` must be supplied by the caller.  Calls share one small static device
    array: do not let two of them run at the same time on different streams.
    """
    x = _bits16(x, "x")
    N, K = c.shape
    B = x.shape[0] if x.dim() == 2 else 1
    if x.numel() != B * K:
        raise ValueError("x has the wrong size")
    if y.dtype != torch.float32 or not y.is_contiguous() or y.numel() != B * N:
        raise ValueError("y must be a contiguous float32 tensor of B*N elements")
    _check(lib().wcomp_gemv_noalloc(P(c.handle), P(x.data_ptr()), B, P(y.data_ptr()), P(_stream(stream))),
           "wcomp_gemv_noalloc")
    return y


def gemv_bf16(w: torch.Tensor, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Plain BF16 GEMV (the comparison kernel)."""
    w = _bits16(w, "w")
    x = _bits16(x, "x")
    N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, w.numel())
    B = x.shape[0] if x.dim() == 2 else 1
    if x.numel() != B * K:
        raise ValueError("x has the wrong size")
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device="cuda")
    _check(lib().wcomp_gemv_bf16(P(w.data_ptr()), N, K, P(x.data_ptr()), B, P(y.data_ptr()), P(_stream(stream))),
           "wcomp_gemv_bf16")
    return y


def gemv_bf16_batched(ws: Sequence[torch.Tensor], xs: Sequence[torch.Tensor],
                      ys: Optional[List[torch.Tensor]] = None, stream=None):
    """Plain BF16 GEMV over several weight tensors in one launch."""
    B = xs[0].shape[0] if xs[0].dim() == 2 else 1
    Ns, Ks = [], []
    for w, x in zip(ws, xs):
        _bits16(w, "w")
        _bits16(x, "x")
        N, K = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, w.numel())
        if x.numel() != B * K:
            raise ValueError("x has the wrong size")
        Ns.append(N)
        Ks.append(K)
    if ys is None:
        ys = [torch.empty((B, N), dtype=torch.float32, device="cuda") for N in Ns]
    n_arr = (ctypes.c_int64 * len(ws))(*Ns)
    k_arr = (ctypes.c_int64 * len(ws))(*Ks)
    _check(lib().wcomp_gemv_bf16_batched(_ptr_array([w.data_ptr() for w in ws]), n_arr, k_arr,
                                         _ptr_array([x.data_ptr() for x in xs]), B,
                                         _ptr_array([y.data_ptr() for y in ys]), len(ws), P(_stream(stream))),
           "wcomp_gemv_bf16_batched")
    return ys


def _ptr_array(ptrs: Sequence[int]):
    arr = (P * len(ptrs))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


def decode_batched(cs: Sequence[Container], outs: Optional[List[torch.Tensor]] = None, stream=None):
    if outs is None:
        outs = [torch.empty((c.N, c.K), dtype=torch.int16, device="cuda") for c in cs]
    for c, o in zip(cs, outs):
        _bits16(o, "out")
        N, K = c.shape
        if o.numel() != N * K:
            raise ValueError("output has the wrong size")
    _check(lib().wcomp_decode_batched(_ptr_array([c.handle for c in cs]), _ptr_array([o.data_ptr() for o in outs]),
                                      len(cs), P(_stream(stream))), "wcomp_decode_batched")
    return outs


def gemv_batched(cs: Sequence[Container], xs: Sequence[torch.Tensor], ys: Optional[List[torch.Tensor]] = None,
                 stream=None):
    B = xs[0].shape[0] if xs[0].dim() == 2 else 1
    for c, x in zip(cs, xs):
        _bits16(x, "x")
        if x.numel() != B * c.K:
            raise ValueError("x has the wrong size")
    if ys is None:
        ys = [torch.empty((B, c.N), dtype=torch.float32, device="cuda") for c in cs]
    _check(lib().wcomp_gemv_batched(_ptr_array([c.handle for c in cs]), _ptr_array([x.data_ptr() for x in xs]), B,
                                    _ptr_array([y.data_ptr() for y in ys]), len(cs), P(_stream(stream))),
           "wcomp_gemv_batched")
    return ys


def serialize(c: Container, stream=None, compact: bool = False) -> bytes:
    """Container bytes: format version 1, or version 2 (compact) with compact=True."""
    fn = lib().wcomp_serialize_compact if compact else lib().wcomp_serialize
    name = "wcomp_serialize_compact" if compact else "wcomp_serialize"
    n = ctypes.c_uint64()
    _check(fn(P(c.handle), None, 0, ctypes.byref(n), P(_stream(stream))), name)
    buf = ctypes.create_string_buffer(n.value)
    _check(fn(P(c.handle), buf, n.value, ctypes.byref(n), P(_stream(stream))), name)
    return buf.raw[: n.value]


def deserialize(data: bytes, stream=None) -> Container:
    h = P()
    buf = ctypes.create_string_buffer(bytes(data), len(data))
    _check(lib().wcomp_deserialize(buf, len(data), P(_stream(stream)), ctypes.byref(h)), "wcomp_deserialize")
    return Container(h.value)


class Q4:
    """A weight in 4 bits with group scales, living on the GPU (owned by the library).

    ``shape`` is (N, K), or (M, N, K) for M matrices held together.  ``free``, and
    dropping the last reference, return its memory in the order of the (current)
    stream: have that wait for other streams whose calls still use the weight.
    """

    def __init__(self, handle: int, shape, group: int):
        self._h = handle
        self.shape = tuple(shape)
        self.group = group

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("weight was freed")
        return self._h

    def info(self) -> dict:
        inf = Q4Info()
        _check(lib().wcomp_q4_info(self.handle, ctypes.byref(inf)), "wcomp_q4_info")
        return inf.as_dict()

    def free(self, stream=None):
        if self._h:
            lib().wcomp_q4_free(self._h, _stream(stream))
            self._h = 0

    def __del__(self):
        try:
            if self._h and torch.cuda.is_available():
                self.free()
        except Exception:
            pass


def _matrices(shape, what: str) -> tuple:
    if len(shape) not in (2, 3):
        raise ValueError(f"{what} must be 2-D [N, K] or 3-D [M, N, K]")
    return tuple(shape) if len(shape) == 3 else (1, *shape)


def _output(t: torch.Tensor, what: str, dtype: torch.dtype, shape: tuple) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or not t.is_contiguous() \
            or t.shape != shape:
        raise ValueError(f"{what} must be a contiguous {dtype} CUDA tensor of shape {list(shape)}")
    return t.data_ptr()


def q4_encode(w: torch.Tensor, group: int = 128, stream=None) -> Q4:
    """Quantise BF16 weights W[N, K] or [M, N, K]: 4-bit codes, one BF16 scale per ``group`` columns."""
    w = _bits16(w, "w")
    M, N, K = _matrices(w.shape, "w")
    h = P()
    _check(lib().wcomp_q4_encode(w.data_ptr(), M, N, K, group, _stream(stream), ctypes.byref(h)), "wcomp_q4_encode")
    return Q4(h.value, w.shape, group)


def q4_pack(codes: torch.Tensor, scales: torch.Tensor, K: int, group: int = 128, stream=None) -> Q4:
    """Take weights quantised elsewhere: a code c stands for (c - 8) * scale.

    ``codes`` uint8 [(M,) N, ceil(K / 2)], the even column in the low nibble;
    ``scales`` BF16 [(M,) N, ceil(K / group)].
    """
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dtype != torch.uint8:
        raise TypeError("codes must be a CUDA uint8 tensor")
    scales = _bits16(scales, "scales")
    M, N, kb = _matrices(codes.shape, "codes")
    if not codes.is_contiguous():
        raise ValueError("codes must be contiguous")
    if group not in (32, 64, 128) or K < 1 or kb != (K + 1) // 2:
        raise ValueError("codes must have ceil(K / 2) bytes a row, and group be 32, 64 or 128")
    if scales.shape != (*codes.shape[:-1], -(-K // group)):
        raise ValueError("scales must be [..., N, ceil(K / group)] like codes")
    if scales.device != codes.device:
        raise ValueError("codes and scales must be on one device")
    h = P()
    _check(lib().wcomp_q4_pack(codes.data_ptr(), scales.data_ptr(), M, N, K, group, _stream(stream), ctypes.byref(h)),
           "wcomp_q4_pack")
    return Q4(h.value, (*codes.shape[:-1], K), group)


def q4_unpack(c: Q4, stream=None) -> tuple:
    """(codes, scales) in the layout that q4_pack takes."""
    K = c.shape[-1]
    codes = torch.empty((*c.shape[:-1], (K + 1) // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*c.shape[:-1], -(-K // c.group)), dtype=torch.bfloat16, device="cuda")
    _check(lib().wcomp_q4_unpack(c.handle, codes.data_ptr(), scales.data_ptr(), _stream(stream)), "wcomp_q4_unpack")
    return codes, scales


def q4_decode(c: Q4, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The weights' values rounded once to BF16, as an int16 tensor of their bits (``out`` if given)."""
    if out is None:
        out = torch.empty(c.shape, dtype=torch.int16, device="cuda")
    else:
        out = _bits16(out, "out")
        if out.shape != c.shape:
            raise ValueError("out has the wrong shape")
    _check(lib().wcomp_q4_decode(c.handle, out.data_ptr(), _stream(stream)), "wcomp_q4_decode")
    return out


def q4_gemv(c: Q4, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[B, N] (fp32) = x[B, K] @ W.T with the 4-bit weights expanded in registers, 1 <= B <= 16."""
    x = _bits16(x, "x")
    M, N, K = _matrices(c.shape, "c")
    if M != 1:
        raise ValueError("c must hold one matrix")
    B = x.shape[0] if x.dim() == 2 else 1
    if x.numel() != B * K:
        raise ValueError("x has the wrong size")
    if y is None:
        y = torch.empty((B, N), dtype=torch.float32, device=x.device)
    elif not y.is_cuda or y.dtype != torch.float32 or not y.is_contiguous() or y.numel() != B * N:
        raise ValueError("y must be a contiguous float32 CUDA tensor of B*N elements")
    _check(lib().wcomp_q4_gemv(c.handle, x.data_ptr(), B, y.data_ptr(), _stream(stream)), "wcomp_q4_gemv")
    return y


def moe(x: torch.Tensor, router: torch.Tensor, gate, up, down, top_k: int, *, scoring: str = "softmax",
        bias: Optional[torch.Tensor] = None, renormalize: bool = True, factor: float = 1.0,
        y: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
        weights: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One mixture-of-experts layer for x[T, H], 1 <= T <= 16: y[T, H] in x's type.

    ``router`` [E, H] gives the logits; the ``top_k`` experts of largest score
    (softmax or sigmoid) plus ``bias`` [E] are weighted by their scores,
    divided by the chosen scores' sum with ``renormalize``, times ``factor``.
    ``gate``, ``up`` [E, F, H] and ``down`` [E, H, F] are BF16 tensors or Q4
    weights.  ``ids`` (int32) and ``weights`` (float32) [T, top_k] receive the
    choice if given.
    """
    x = _bits16(x, "x")
    router = _bits16(router, "router")
    if x.dim() != 2 or router.dim() != 2 or router.shape[1] != x.shape[1]:
        raise ValueError("x must be [T, H] and router [E, H]")
    (T, H), E = x.shape, router.shape[0]
    if scoring not in SCORING:
        raise ValueError("scoring must be 'softmax' or 'sigmoid'")
    q4 = isinstance(gate, Q4)
    if isinstance(up, Q4) != q4 or isinstance(down, Q4) != q4:
        raise TypeError("gate, up and down must be all BF16 tensors or all Q4 weights")
    F = gate.shape[1] if len(gate.shape) == 3 else 0
    if gate.shape != (E, F, H) or up.shape != (E, F, H) or down.shape != (E, H, F):
        raise ValueError(f"gate and up must be [{E}, F, {H}] and down [{E}, {H}, F], got {list(gate.shape)}, "
                         f"{list(up.shape)}, {list(down.shape)}")
    if q4:
        ws = (None, None, None, gate.handle, up.handle, down.handle)
    else:
        ws = (_bits16(gate, "gate").data_ptr(), _bits16(up, "up").data_ptr(), _bits16(down, "down").data_ptr(),
              None, None, None)
    if y is None:
        y = torch.empty_like(x)
    else:
        _output(_bits16(y, "y"), "y", y.dtype, (T, H))
    a = MoeArgs(x.data_ptr(), router.data_ptr(), None if bias is None else _output(bias, "bias", torch.float32, (E,)),
                *ws, y.data_ptr(), None if ids is None else _output(ids, "ids", torch.int32, (T, top_k)),
                None if weights is None else _output(weights, "weights", torch.float32, (T, top_k)),
                H, F, T, E, top_k, SCORING[scoring], renormalize, factor)
    _check(lib().wcomp_moe(ctypes.byref(a), _stream(stream)), "wcomp_moe")
    return y


class KV4:
    """A cache of keys and values in 4 bits, living on the GPU (owned by the library).

    ``pages`` pages of 64 tokens with ``heads`` rows of ``dim`` columns of keys and of values each, one BF16
    scale per 32 columns.  ``free``, and dropping the last reference, return its memory in the order of the
    (current) stream: have that wait for other streams whose calls still use the cache.

    The calls on it take ``table`` (int32 [B, width]: the pages of each sequence; position p is place p % 64 of
    page table[b, p // 64]), ``lengths`` (int32 [B]: the tokens that each sequence holds, the call's own rows
    among them) and ``starts`` (int32 [B + 1]: rows starts[b] to starts[b + 1] - 1 are the newest tokens of
    sequence b; None: one row a sequence).  All three are on the device; a page or length out of range is
    skipped there, starts that descend or leave the call's rows reach no others, and ``device_check`` reports them.
    """

    def __init__(self, handle: int, pages: int, heads: int, dim: int, device: torch.device):
        self._h = handle
        self.pages, self.heads, self.dim, self.device = pages, heads, dim, device

    @property
    def handle(self) -> int:
        if not self._h:
            raise ValueError("cache was freed")
        return self._h

    def info(self) -> dict:
        inf = Kv4Info()
        _check(lib().wcomp_kv4_info(self.handle, ctypes.byref(inf)), "wcomp_kv4_info")
        return inf.as_dict()

    def free(self, stream=None):
        if self._h:
            lib().wcomp_kv4_free(self._h, _stream(stream))
            self._h = 0

    def __del__(self):
        try:
            if self._h and torch.cuda.is_available():
                self.free()
        except Exception:
            pass


def kv4_create(pages: int, heads: int, dim: int, stream=None) -> KV4:
    """A new cache on the current device; ``dim`` is 64, 128 or 256.  Its rows read as zeros."""
    if not (-2 ** 63 <= pages < 2 ** 63 and -2 ** 31 <= heads < 2 ** 31 and -2 ** 31 <= dim < 2 ** 31):
        raise ValueError("heads and dim must be within 32 bits, pages within 64")  # ctypes would cut them off
    h = P()
    _check(lib().wcomp_kv4_create(pages, heads, dim, _stream(stream), ctypes.byref(h)), "wcomp_kv4_create")
    return KV4(h.value, pages, heads, dim, torch.device("cuda", torch.cuda.current_device()))


def _stream_of(stream, device: torch.device) -> int:
    """``stream``, or the current one of that device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream(stream)


def _array(t: torch.Tensor, what: str, dtype: torch.dtype, shape: tuple, device: torch.device) -> int:
    """The address of a contiguous tensor of that type and shape on that device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device \
            and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")


def _kv4_seqs(c: KV4, table: torch.Tensor, lengths: torch.Tensor, starts: Optional[torch.Tensor]) -> Kv4Seqs:
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [B, width]")
    B, width = table.shape
    return Kv4Seqs(_array(table, "table", torch.int32, (B, width), c.device),
                   _array(lengths, "lengths", torch.int32, (B,), c.device),
                   None if starts is None else _array(starts, "starts", torch.int32, (B + 1,), c.device), B, width)


def _kv4_rows(c: KV4, t: torch.Tensor, what: str, heads: Optional[int] = None) -> tuple:
    """Address and strides of BF16 rows [T, heads, dim] whose columns are contiguous."""
    if not isinstance(t, torch.Tensor) or t.device != c.device:
        raise TypeError(f"{what} must be a CUDA tensor on {c.device}")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{what} must hold BF16 bits (bfloat16, int16 or uint16), got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != c.dim or t.stride(2) != 1 or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what} must be [T, {'heads' if heads is None else heads}, {c.dim}] with contiguous columns")
    return t.data_ptr(), t.stride(0), t.stride(1)


def kv4_append(c: KV4, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
               starts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise rows k, v [T, heads, dim] (BF16, any strides between rows and heads) into the cache."""
    s = _kv4_seqs(c, table, lengths, starts)
    kp, vp = _kv4_rows(c, k, "k", c.heads), _kv4_rows(c, v, "v", c.heads)
    T = k.shape[0]
    if v.shape[0] != T or (starts is None and T != s.B):
        raise ValueError("k and v must have the same rows, one a sequence without starts")
    _check(lib().wcomp_kv4_append(c.handle, ctypes.byref(s), *kp, *vp, T, _stream_of(stream, c.device)), "wcomp_kv4_append")


def kv4_read(c: KV4, table: torch.Tensor, lengths: torch.Tensor, starts: Optional[torch.Tensor] = None, *,
             rows: Optional[int] = None, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
             stream=None) -> tuple:
    """(k, v): the newest tokens of each sequence as BF16 rows [rows, heads, dim].

    ``rows`` is starts[B] (the number of sequences without starts).  Rows without a position read as zeros; rows
    of ``k`` and ``v``, where they are given, that belong to no sequence are left as they were.
    """
    s = _kv4_seqs(c, table, lengths, starts)
    if rows is None:
        given = k if k is not None else v
        if given is None and starts is not None:
            raise ValueError("rows must be given with starts")
        rows = s.B if given is None else given.shape[0]
    if starts is None and rows != s.B:
        raise ValueError("without starts there is one row a sequence")
    shape = (rows, c.heads, c.dim)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=c.device) if t is None else t for t in (k, v))
    _check(lib().wcomp_kv4_read(c.handle, ctypes.byref(s), _array(_bits16(k, "k"), "k", k.dtype, shape, c.device),
                                _array(_bits16(v, "v"), "v", v.dtype, shape, c.device), rows, _stream_of(stream, c.device)),
           "wcomp_kv4_read")
    return k, v


def kv4_attend(c: KV4, q: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
               starts: Optional[torch.Tensor] = None, *, scale: Optional[float] = None, window: int = 0,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               mass: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of query rows q [T, q_heads, dim] over the cache: BF16 rows of the same shape.

    Each row sees the tokens of its sequence up to its own position (append its keys and values first), the last
    ``window`` of them if that is not 0.  ``scale`` is dim ** -0.5 by default.  ``lse`` (float32 [T, q_heads])
    receives the log of the sum of exponentials, and ``mass`` (float32 [B, heads, width * 64]) is added the
    attention weight of each cached token, as ``kv4_evict`` takes it.  A row that sees nothing gets zeros.
    """
    s = _kv4_seqs(c, table, lengths, starts)
    qp = _kv4_rows(c, q, "q")
    T, Hq = q.shape[:2]
    if Hq < 1 or Hq % c.heads or (starts is None and T != s.B):
        raise ValueError("q must have a multiple of the cache's heads, and one row a sequence without starts")
    if not 0 <= window < 2 ** 31:
        raise ValueError("window must be within 0..2^31 - 1")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=c.device)
    a = Kv4AttendArgs(s, *qp, _array(_bits16(out, "out"), "out", out.dtype, (T, Hq, c.dim), c.device),
                      None if lse is None else _array(lse, "lse", torch.float32, (T, Hq), c.device),
                      None if mass is None else _array(mass, "mass", torch.float32, (s.B, c.heads, s.width * 64),
                                                       c.device),
                      T, Hq, window, c.dim ** -0.5 if scale is None else scale)
    _check(lib().wcomp_kv4_attend(c.handle, ctypes.byref(a), _stream_of(stream, c.device)), "wcomp_kv4_attend")
    return out


def kv4_evict(c: KV4, table: torch.Tensor, lengths: torch.Tensor, mass: torch.Tensor, keep: int, recent: int,
              table_out: torch.Tensor, *, lengths_out: Optional[torch.Tensor] = None,
              mass_out: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Bring sequences down to ``keep`` tokens a head: the last ``recent`` and those of largest ``mass``.

    They are copied in their order to the pages of ``table_out`` (int32 [B, width_out], none of them in
    ``table``).  Returns (lengths, mass) of the sequences there, as the other calls take them.  ``kept``
    (int32 [B, heads, keep]) receives the positions that were kept, then -1.
    """
    s = _kv4_seqs(c, table, lengths, None)
    if not isinstance(table_out, torch.Tensor) or table_out.dim() != 2:
        raise ValueError("table_out must be [B, width_out]")
    wide = table_out.shape[1]
    if keep < 1 or not 0 <= recent <= keep or wide * 64 < keep:
        raise ValueError("keep must be above 0, recent within 0..keep, and table_out have pages for keep tokens")
    if lengths_out is None:
        lengths_out = torch.empty_like(lengths)
    if mass_out is None:
        mass_out = torch.empty((s.B, c.heads, wide * 64), dtype=torch.float32, device=c.device)
    a = Kv4EvictArgs(s.d_table, s.d_lengths,
                     _array(mass, "mass", torch.float32, (s.B, c.heads, s.width * 64), c.device),
                     _array(table_out, "table_out", torch.int32, (s.B, wide), c.device),
                     _array(lengths_out, "lengths_out", torch.int32, (s.B,), c.device),
                     _array(mass_out, "mass_out", torch.float32, (s.B, c.heads, wide * 64), c.device),
                     None if kept is None else _array(kept, "kept", torch.int32, (s.B, c.heads, keep), c.device),
                     s.B, s.width, wide, keep, recent)
    _check(lib().wcomp_kv4_evict(c.handle, ctypes.byref(a), _stream_of(stream, c.device)), "wcomp_kv4_evict")
    return lengths_out, mass_out


def logprobs(logits: torch.Tensor, ids: Optional[torch.Tensor] = None, top_k: int = 0, *, scale: float = 1.0,
             lse: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """(logprob [T], entropy [T], top_logprobs [T, top_k], top_ids [T, top_k]) of logits [T, V] times ``scale``.

    ``logits`` are float32 (what ``gemv`` gives) or bfloat16, a row's columns contiguous; ``scale`` is above 0 and at
    most 2^127; ``ids`` (int64 [T]) are
    the given tokens: a negative one gets logprob 0, one beyond the vocabulary NaN.  logprob is None without
    ids.  ``top_k`` (at most 64) alternatives, the largest first, ties by the lowest index; ids are int32; both are
    None for 0.  ``lse`` (float32 [T]) receives the log of the sum of exponentials.
    """
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise TypeError("logits must be a CUDA tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T, V] with contiguous columns")
    if top_k < 0 or top_k > logits.shape[1]:
        raise ValueError("top_k must be within 0..V")
    (T, V), dev = logits.shape, logits.device
    if dev.index != torch.cuda.current_device():
        raise ValueError("logits must be on the current device")
    row = logits.stride(0) if T > 1 else V
    entropy = torch.empty(T, dtype=torch.float32, device=dev)
    logprob = None if ids is None else torch.empty(T, dtype=torch.float32, device=dev)
    top = top_ids = None
    if top_k:
        top = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        top_ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    a = LogprobsArgs(logits.data_ptr(), None if ids is None else _array(ids, "ids", torch.int64, (T,), dev),
                     None if ids is None else logprob.data_ptr(), entropy.data_ptr(),
                     None if lse is None else _array(lse, "lse", torch.float32, (T,), dev),
                     top.data_ptr() if top_k else None, top_ids.data_ptr() if top_k else None, T, V, row,
                     0 if logits.dtype == torch.float32 else 1, top_k, scale)
    _check(lib().wcomp_logprobs(ctypes.byref(a), _stream_of(stream, dev)), "wcomp_logprobs")
    return logprob, entropy, top, top_ids


def version() -> int:
    return lib().wcomp_version()


def device_check(stream=None) -> None:
    """Raise if a kernel on this device reported a timed-out wait or an index out of range (clears the report)."""
    _check(lib().wcomp_device_check(P(_stream(stream))), "wcomp_device_check")


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().wcomp_launch_count())
