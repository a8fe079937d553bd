"""Python binding of libtb (include/tb.h): argument marshalling only.

Every operation runs in the CUDA library; this module converts tensors,
integers and streams into the plain pointers and sizes the C ABI takes, and
turns error codes into ``TBError``.  PyTorch is optional here: anything with
``data_ptr()`` (a tensor) or a plain integer address is accepted as a
pointer, and anything with ``cuda_stream`` (a ``torch.cuda.Stream``) or an
integer handle as a stream.

Importing this module loads ``lib/libtb.so`` and fails loudly when it has not
been built: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as ct
import os
import sys
from dataclasses import dataclass

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libtb.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libtb.so is not built ({LIB_PATH} missing): run "
        "`python -c 'import __graft_entry__ as g; g.build()'` first")

lib = ct.CDLL(LIB_PATH)

TB_OK = 0
TB_EINVAL = -1
TB_ENOMEM = -2
TB_ECUDA = -3
TB_EVALIDATE = -4
TB_ETIMEOUT = -5
TB_ENOTSUP = -6
TB_MAX_SRCS = 16

TB_PATTERN_DEFAULT = 0
TB_PATTERN_COMPRESS = 1
TB_PATTERN_REPEAT = 2

_u64, _i64, _i32, _u32, _vp = ct.c_uint64, ct.c_int64, ct.c_int32, ct.c_uint32, ct.c_void_p


class Options(ct.Structure):
    """tb_options: see include/tb.h for every field's meaning and default."""
    _fields_ = [
        ("rotate_bytes", _u64),
        ("byte_offset", _u64),
        ("warmup", _i32),
        ("always_validate", _i32),
        ("memset_byte", _u32),
        ("ctas_per_subexec", _i32),
        ("block_threads", _i32),
        ("small_max_bytes", _u64),
        ("slot_items", _u32),
        ("num_slots", _u32),
        ("wait_timeout_ns", _u64),
        ("use_gate", _i32),
        ("vec_bytes", _i32),
        ("unroll", _i32),
        ("time_kernels", _i32),
        ("reduce_engine", _i32),
        ("ce_min_bytes", _u64),
        ("use_graph", _i32),
        ("use_pdl", _i32),
        ("kernel_wait_ns", _u64),
        ("validate_direct", _i32),
        ("validate_source", _i32),
        ("check_overlap", _i32),
        ("batch_min_copies", _i32),
        ("batch_short_shape", _i32),
        ("batch_max_ctas", _i32),
        ("early_reads", _i32),
    ]


class Pattern(ct.Structure):
    _fields_ = [
        ("kind", _i32),
        ("compress_pct", _u32 * 5),
        ("seed", _u64),
        ("repeat", ct.POINTER(ct.c_float)),
        ("repeat_len", _u32),
    ]


class Result(ct.Structure):
    _fields_ = [
        ("K", _u64),
        ("slice_stride", _u64),
        ("alloc_bytes", _u64),
        ("prep_h2d_bytes", _u64),
        ("iters", _i32),
        ("num_subexec", _i32),
        ("ctas", _i32),
        ("block_threads", _i32),
        ("gated", _i32),
        ("graphed", _i32),
        ("engine", _i32),
        ("validated", _i32),
        ("total_ms", ct.c_double),
        ("mean_ms", ct.c_double),
        ("median_ms", ct.c_double),
        ("min_ms", ct.c_double),
        ("max_ms", ct.c_double),
        ("gbps", ct.c_double),
        ("iter_ms", ct.POINTER(ct.c_float)),
        ("mismatch_index", _i64),
        ("mismatch_expected", _u32),
        ("mismatch_actual", _u32),
        ("executor", _i32),
    ]


class LaunchInfo(ct.Structure):
    _fields_ = [
        ("engine", _i32),
        ("vec_bytes", _i32),
        ("unroll", _i32),
        ("block_threads", _i32),
        ("grid", _i32),
        ("num_subexec", _i32),
        ("head_elems", _u64),
        ("body_vectors", _u64),
        ("tail_elems", _u64),
        ("smem_bytes", _u64),
        ("stages", _i32),
        ("tile_bytes", _i32),
    ]


class Transfer(ct.Structure):
    _fields_ = [
        ("srcs", ct.POINTER(_vp)),
        ("n_src", _i32),
        ("dst", _vp),
        ("num_bytes", _u64),
        ("num_subexec", _i32),
        ("iters", _i32),
        ("rotate_bytes", _u64),
        ("expected", _vp),
        ("expected_device", _vp),
        ("executor", _i32),
    ]


class CopyDesc(ct.Structure):
    _fields_ = [("src", _u64), ("dst", _u64), ("len", _u64)]


class BatchStats(ct.Structure):
    _fields_ = [
        ("descs", _u64),
        ("warp_items", _u64),
        ("cta_items", _u64),
        ("launches", _u64),
        ("bytes", _u64),
        ("upload_bytes", _u64),
        ("ce_copies", _u64),
        ("direct_launches", _u64),
    ]


class KvCacheStruct(ct.Structure):
    """tb_kv_cache: see include/tb.h."""
    _fields_ = [
        ("k", _vp),
        ("v", _vp),
        ("table", _vp),
        ("held", _vp),
        ("lens", _vp),
        ("refs", _vp),
        ("dtype", _i32),
        ("layers", _i32),
        ("pages", _i32),
        ("page_tokens", _i32),
        ("kv_heads", _i32),
        ("head_dim", _i32),
        ("slots", _i32),
        ("table_width", _i32),
        ("layer_stride", _i64),
        ("page_stride", _i64),
        ("token_stride", _i64),
        ("head_stride", _i64),
    ]


class Tree(ct.Structure):
    """tb_tree: see include/tb.h."""
    _fields_ = [
        ("cache", ct.POINTER(KvCacheStruct)),
        ("layer", _i32),
        ("seqs", _i32),
        ("seq_slots", _vp),
        ("q_start", _vp),
        ("rows", _i32),
        ("q_heads", _i32),
        ("scale", ct.c_float),
        ("q", _vp),
        ("out", _vp),
        ("q_row_stride", _i64),
        ("q_head_stride", _i64),
        ("out_row_stride", _i64),
        ("out_head_stride", _i64),
        ("lse", _vp),
        ("mask", _vp),
        ("mask_words", _i32),
        ("workspace", _vp),
        ("workspace_bytes", _u64),
    ]


class Mismatch(ct.Structure):
    _fields_ = [("index", _i64), ("expected", _u32), ("actual", _u32)]


def _sig(name, restype, *argtypes):
    fn = getattr(lib, name)
    fn.restype = restype
    fn.argtypes = list(argtypes)
    return fn


_P = ct.POINTER
_sig("tb_strerror", ct.c_char_p, ct.c_int)
_sig("tb_last_error", ct.c_char_p, _vp)
_sig("tb_options_default", None, _P(Options))
_sig("tb_options_from_env", ct.c_int, _P(Options))
_sig("tb_parse_bytes", ct.c_int, ct.c_char_p, _P(_u64))
_sig("tb_create", ct.c_int, _P(_vp), ct.c_int, _P(Options))
_sig("tb_destroy", None, _vp)
_sig("tb_get_options", ct.c_int, _vp, _P(Options))
_sig("tb_rotation_plan", ct.c_int, _u64, _u64, _u64, _P(_u64), _P(_u64), _P(_u64))
_sig("tb_slice_for_iteration", _u64, _i64, _u64)
_sig("tb_fill_source", ct.c_int, _vp, _vp, _u64, _P(Pattern), ct.c_int, _vp)
_sig("tb_upload_sources", ct.c_int, _vp, _P(_vp), _P(_vp), ct.c_int, _u64)
_sig("tb_prepare_sources", ct.c_int, _vp, _P(_vp), ct.c_int, _u64, _u64)
_sig("tb_prep_h2d_bytes", _u64, _vp)
_sig("tb_reduce_copy", ct.c_int, _vp, _P(_vp), ct.c_int, _vp, _u64, ct.c_int, _vp)
_sig("tb_reduce_plan", ct.c_int, _vp, _P(_vp), ct.c_int, _vp, _u64, ct.c_int, _P(LaunchInfo))
_sig("tb_run_transfer_ex", ct.c_int, _vp, _P(Transfer), _P(Result))
_sig("tb_run_transfer", ct.c_int, _vp, _P(_vp), ct.c_int, _vp, _u64, ct.c_int, ct.c_int, _u64,
     _P(Result))
_sig("tb_reduce_copy_host", ct.c_int, _vp, _P(_vp), ct.c_int, _vp, _u64, _P(_vp), _vp, ct.c_int,
     _vp)
_sig("tb_batch_copy", ct.c_int, _vp, _vp, ct.c_size_t, _vp)  # desc: a CopyDesc array's address
_sig("tb_last_batch_stats", ct.c_int, _vp, _P(BatchStats))
_sig("tb_last_batch_kernel_ms", ct.c_int, _vp, _P(ct.c_double))
_sig("tb_copy_each", ct.c_int, _vp, _vp, ct.c_size_t, _vp)  # desc: a CopyDesc array's address
_sig("tb_validate", ct.c_int, _vp, _vp, _vp, _u64, _u32, _P(Mismatch))
_sig("tb_validate_device", ct.c_int, _vp, _vp, _vp, _u64, _u32, _P(Mismatch))
_sig("tb_batch_copy_noalloc", ct.c_int, _vp, ct.c_size_t, _vp)  # desc: as tb_batch_copy
_KV = _P(KvCacheStruct)
_sig("tb_kv_copy_pages", ct.c_int, _vp, _KV, _vp, _vp, _vp, _i32, _vp)
_sig("tb_kv_resize", ct.c_int, _vp, _KV, _vp, _vp, _vp)
_sig("tb_kv_fork", ct.c_int, _vp, _KV, _vp, _vp, _vp, _vp, _vp, _vp)
_sig("tb_kv_compact", ct.c_int, _vp, _KV, _vp, _vp, _i32, _vp, _vp, _vp)
_sig("tb_tree_attention", ct.c_int, _vp, _P(Tree), _vp)
_sig("tb_tree_attention_workspace", ct.c_int, _vp, _KV, _i32, _P(_u64))

TB_NOALLOC_MAX_ITEMS = 65536
TB_EXEC_GPU = 0
TB_EXEC_DMA = 1


class TBError(RuntimeError):
    """A libtb call returned a negative code."""

    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code


def strerror(code: int) -> str:
    return lib.tb_strerror(code).decode()


def _check(code: int, ctx_handle=None, what: str = "") -> int:
    if code != TB_OK:
        detail = lib.tb_last_error(ctx_handle).decode() if ctx_handle else ""
        raise TBError(code, f"{what}: {strerror(code)}" + (f" ({detail})" if detail else ""))
    return code


def addr(x) -> int:
    """Device or host address of a tensor / array / integer."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    if hasattr(x, "ctypes"):  # numpy array
        return int(x.ctypes.data)
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def stream_handle(s) -> int:
    if s is None:
        return 0
    if isinstance(s, int):
        return s
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    raise TypeError(f"not a stream: {type(s).__name__}")


def _ptr_array(xs):
    arr = (_vp * max(1, len(xs)))(*[addr(x) for x in xs])
    return arr


def options(**overrides) -> Options:
    """Default options (no environment), with keyword overrides."""
    o = Options()
    lib.tb_options_default(ct.byref(o))
    for k, v in overrides.items():
        if not hasattr(o, k):
            raise AttributeError(f"tb_options has no field {k}")
        setattr(o, k, v)
    return o


def options_from_env(base: Options | None = None) -> Options:
    o = base if base is not None else options()
    _check(lib.tb_options_from_env(ct.byref(o)), None, "tb_options_from_env")
    return o


def parse_bytes(text: str) -> int:
    out = _u64()
    _check(lib.tb_parse_bytes(text.encode(), ct.byref(out)), None, f"tb_parse_bytes({text!r})")
    return out.value


@dataclass
class RotationPlan:
    K: int
    slice_stride: int
    alloc_bytes: int


def rotation_plan(num_bytes: int, rotate_bytes: int, byte_offset: int = 0) -> RotationPlan:
    k, s, a = _u64(), _u64(), _u64()
    _check(lib.tb_rotation_plan(num_bytes, rotate_bytes, byte_offset, ct.byref(k), ct.byref(s),
                                ct.byref(a)), None, "tb_rotation_plan")
    return RotationPlan(k.value, s.value, a.value)


def slice_for_iteration(iteration: int, K: int) -> int:
    return int(lib.tb_slice_for_iteration(iteration, K))


def default_pattern() -> Pattern:
    return Pattern(kind=TB_PATTERN_DEFAULT)


def compress_pattern(pct, seed: int) -> Pattern:
    p = Pattern(kind=TB_PATTERN_COMPRESS, seed=seed & (2**64 - 1))
    for i, v in enumerate(pct):
        p.compress_pct[i] = v
    return p


def repeat_pattern(values) -> tuple[Pattern, object]:
    buf = (ct.c_float * len(values))(*values)
    p = Pattern(kind=TB_PATTERN_REPEAT, repeat=ct.cast(buf, ct.POINTER(ct.c_float)),
                repeat_len=len(values))
    return p, buf  # keep buf alive for the call


# ---------------------------------------------------------------------------
# Paged key/value cache
# ---------------------------------------------------------------------------
TB_DTYPE_F16 = 0
TB_DTYPE_BF16 = 1
TB_DTYPE_F32 = 2
TB_DTYPE_BYTE = 3
TB_KV_MAX_SLOTS = 8192
TB_TREE_MAX_SEQS = 4096


def _dtype_name(t) -> str:
    return str(t.dtype).replace("torch.", "")


def _kv_dtype(t) -> int:
    name = _dtype_name(t)
    known = {"float16": TB_DTYPE_F16, "bfloat16": TB_DTYPE_BF16, "float32": TB_DTYPE_F32}
    if name in known:
        return known[name]
    if t.element_size() == 1:
        return TB_DTYPE_BYTE
    raise TypeError(f"no cache of {name}")


_INT32 = set()  # the tensor library's int32, once seen: comparing it is cheaper than its name


def _int32(t, what: str, shape: tuple) -> int:
    """Address of a dense int32 device tensor of this shape (None: any size)."""
    if t is not None and t.dtype in _INT32 and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t is None or _dtype_name(t) != "int32" or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{what} must be a contiguous int32 CUDA tensor")
    if len(t.shape) != len(shape) or any(n is not None and m != n for m, n in zip(t.shape, shape)):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {shape}")
    _INT32.add(t.dtype)
    return t.data_ptr()


class KvCache:
    """A tb_kv_cache with the tensors it points into (see kv_cache)."""

    def __init__(self, struct: KvCacheStruct, tensors: tuple):
        self.struct = struct
        self.ref = ct.byref(struct)
        self.ptr = ct.pointer(struct)
        self.tensors = tensors
        self.dtype = tensors[0].dtype if tensors[0] is not None else None
        # What the calls check their lists against, as plain values.
        self.per_slot = (struct.slots,)
        self.table_shape = (struct.slots, struct.table_width)
        self.head_dim = struct.head_dim


def kv_cache(k=None, v=None, table=None, held=None, lens=None, refs=None, layout: str = "NHD",
             page_tokens: int | None = None) -> KvCache:
    """Describes a paged key/value cache held in CUDA tensors (tb_kv_cache).

    k, v: [layers, pages, page_tokens, heads, dim] for layout "NHD" or
    [layers, pages, heads, page_tokens, dim] for "HND", of any strides with
    dense dim.  table: int32 [slots, width]; held, lens: int32 [slots]; refs:
    int32 [pages].  A cache described without k and v (page_tokens given
    instead) serves kv_resize, one without the table kv_copy_pages.  The
    description holds addresses: describe the cache again when a tensor is
    replaced.
    """
    if layout not in ("NHD", "HND"):
        raise ValueError(f"layout {layout!r} is neither NHD nor HND")
    s = KvCacheStruct(dtype=TB_DTYPE_BYTE)
    if (k is None) != (v is None):
        raise ValueError("k and v come together")
    if k is not None:
        if not k.is_cuda or not v.is_cuda or k.dim() != 5 or k.shape != v.shape \
                or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 5-d CUDA tensors of one shape, type and strides")
        if k.shape[4] > 1 and k.stride(4) != 1:
            raise ValueError("the last dimension of k and v must be dense")
        e, tokens, heads = k.element_size(), *((2, 3) if layout == "NHD" else (3, 2))
        if page_tokens is not None and page_tokens != k.shape[tokens]:
            raise ValueError(f"page_tokens is {page_tokens}, the pools have {k.shape[tokens]}")
        s.k, s.v, s.dtype = k.data_ptr(), v.data_ptr(), _kv_dtype(k)
        s.layers, s.pages, s.head_dim = k.shape[0], k.shape[1], k.shape[4]
        s.page_tokens, s.kv_heads = k.shape[tokens], k.shape[heads]
        s.layer_stride, s.page_stride = k.stride(0) * e, k.stride(1) * e
        s.token_stride, s.head_stride = k.stride(tokens) * e, k.stride(heads) * e
    else:
        s.page_tokens = page_tokens or 0
    if table is not None:
        s.table = _int32(table, "table", (None, None))
        s.slots, s.table_width = table.shape
        s.held, s.lens = _int32(held, "held", (s.slots,)), _int32(lens, "lens", (s.slots,))
        s.refs = _int32(refs, "refs", (s.pages if k is not None else None,))
        s.pages = refs.shape[0]
    return KvCache(s, (k, v, table, held, lens, refs))


def tree_mask(parents) -> list[list[int]]:
    """Mask rows of one draft tree for tree_attention: for each drafted token
    the words whose bits name the token itself and its ancestors.  parents[i]
    is the index of token i's parent, smaller than i, or negative for a child
    of the last committed token.  Words are signed, as int32 tensors hold them."""
    words = (len(parents) + 31) // 32
    seen: list[int] = []
    for i, parent in enumerate(parents):
        if parent >= i:
            raise ValueError(f"token {i} comes before its parent {parent}")
        seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
    rows = [[bits >> 32 * w & 0xFFFFFFFF for w in range(words)] for bits in seen]
    return [[w - (1 << 32) if w >> 31 else w for w in row] for row in rows]


class Context:
    """A libtb context on one CUDA device (tb_create / tb_destroy)."""

    def __init__(self, device: int = 0, opts: Options | None = None, env: bool = False):
        self._h = _vp()
        if opts is None and env:
            popt = None
        else:
            popt = ct.byref(opts if opts is not None else options())
        code = lib.tb_create(ct.byref(self._h), device, popt)
        if code != TB_OK:
            raise TBError(code, f"tb_create(device={device}): {strerror(code)}")
        self.device = device

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            lib.tb_destroy(self._h)
            self._h = _vp()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _ok(self, code, what):
        return _check(code, self._h, what)

    def get_options(self) -> Options:
        o = Options()
        self._ok(lib.tb_get_options(self._h, ct.byref(o)), "tb_get_options")
        return o

    # -- source preparation ------------------------------------------------
    def fill_source(self, dst, num_bytes: int, pattern: Pattern, buffer_idx: int, stream=None):
        self._ok(lib.tb_fill_source(self._h, addr(dst), num_bytes, ct.byref(pattern), buffer_idx,
                                    stream_handle(stream)), "tb_fill_source")

    def upload_sources(self, srcs, host_srcs, num_bytes: int):
        self._ok(lib.tb_upload_sources(self._h, _ptr_array(srcs), _ptr_array(host_srcs), len(srcs),
                                       num_bytes), "tb_upload_sources")

    def prepare_sources(self, srcs, num_bytes: int, rotate_bytes: int):
        self._ok(lib.tb_prepare_sources(self._h, _ptr_array(srcs), len(srcs), num_bytes,
                                        rotate_bytes), "tb_prepare_sources")

    @property
    def prep_h2d_bytes(self) -> int:
        return int(lib.tb_prep_h2d_bytes(self._h))

    # -- reduce-copy -------------------------------------------------------
    def reduce_copy(self, srcs, dst, num_bytes: int, num_subexec: int = 0, stream=None):
        self._ok(lib.tb_reduce_copy(self._h, _ptr_array(srcs), len(srcs), addr(dst), num_bytes,
                                    num_subexec, stream_handle(stream)), "tb_reduce_copy")

    def reduce_plan(self, srcs, dst, num_bytes: int, num_subexec: int = 0) -> dict:
        """The launch tb_reduce_copy would make (tb_reduce_plan), as a dict."""
        info = LaunchInfo()
        self._ok(lib.tb_reduce_plan(self._h, _ptr_array(srcs), len(srcs), addr(dst), num_bytes,
                                    num_subexec, ct.byref(info)), "tb_reduce_plan")
        return {name: getattr(info, name) for name, _ in LaunchInfo._fields_}

    def run_transfer(self, srcs, dst, num_bytes: int, num_subexec: int = 0, iters: int = 1,
                     rotate_bytes: int | None = None, expected=None,
                     expected_device=None, executor: int = 0) -> dict:
        """tb_run_transfer_ex; returns the tb_result fields as a dict.

        ``expected`` (host bytes, e.g. a numpy array) turns on validation; a
        mismatch raises TBError with code TB_EVALIDATE after filling the
        result, which is attached to the exception as ``.result``.
        ``executor``: TB_EXEC_GPU (the reduce-copy kernel) or TB_EXEC_DMA (one
        copy-engine copy per iteration, one source).
        """
        if rotate_bytes is None:
            rotate_bytes = self.get_options().rotate_bytes
        arr = _ptr_array(srcs)
        t = Transfer(srcs=ct.cast(arr, ct.POINTER(_vp)), n_src=len(srcs), dst=addr(dst),
                     num_bytes=num_bytes, num_subexec=num_subexec, iters=iters,
                     rotate_bytes=rotate_bytes, expected=addr(expected) if expected is not None else 0,
                     expected_device=addr(expected_device), executor=executor)
        r = Result()
        code = lib.tb_run_transfer_ex(self._h, ct.byref(t), ct.byref(r))
        res = {name: getattr(r, name) for name, _ in Result._fields_ if name != "iter_ms"}
        res["iter_ms"] = [r.iter_ms[i] for i in range(r.iters)] if r.iters > 0 and r.iter_ms else []
        if code != TB_OK:
            err = TBError(code, f"tb_run_transfer_ex: {strerror(code)} "
                                f"({lib.tb_last_error(self._h).decode()})")
            err.result = res
            raise err
        return res

    def reduce_copy_host(self, host_srcs, host_dst, num_bytes: int, dev_srcs, dev_dst,
                         num_subexec: int = 0, stream=None):
        self._ok(lib.tb_reduce_copy_host(self._h, _ptr_array(host_srcs), len(host_srcs),
                                         addr(host_dst), num_bytes, _ptr_array(dev_srcs),
                                         addr(dev_dst), num_subexec, stream_handle(stream)),
                 "tb_reduce_copy_host")

    # -- batched copy ------------------------------------------------------
    @staticmethod
    def descriptor_array(descs):
        """(address, count, keep-alive) for a ctypes CopyDesc array or an
        (n, 3) uint64 array of (src, dst, len) rows.  The address is taken
        without a ctypes pointer object, which would cost more than the rest
        of a small call's host work."""
        if isinstance(descs, ct.Array):
            return ct.addressof(descs), len(descs), descs
        import numpy as np
        a = np.ascontiguousarray(descs, dtype=np.uint64)
        if a.ndim != 2 or a.shape[1] != 3:
            raise ValueError("descriptors must be an (n, 3) array of (src, dst, len)")
        n = a.shape[0]
        if n == 0:
            return None, 0, a
        try:
            ptr = ct.addressof(ct.c_uint64.from_buffer(a))
        except (TypeError, ValueError):  # a read-only array
            ptr = a.ctypes.data
        return ptr, n, a

    def batch_copy(self, descs, stream=None):
        """tb_batch_copy of (src, dst, len) descriptors (see descriptor_array)."""
        ptr, n, keep = self.descriptor_array(descs)
        self._ok(lib.tb_batch_copy(self._h, ptr, n, stream_handle(stream)), "tb_batch_copy")
        del keep

    def copy_each(self, descs, stream=None):
        """tb_copy_each: one cudaMemcpyAsync per descriptor (the baseline)."""
        ptr, n, keep = self.descriptor_array(descs)
        self._ok(lib.tb_copy_each(self._h, ptr, n, stream_handle(stream)), "tb_copy_each")
        del keep

    def last_batch_kernel_ms(self) -> float:
        ms = ct.c_double()
        self._ok(lib.tb_last_batch_kernel_ms(self._h, ct.byref(ms)), "tb_last_batch_kernel_ms")
        return ms.value

    def last_batch_stats(self) -> dict:
        s = BatchStats()
        self._ok(lib.tb_last_batch_stats(self._h, ct.byref(s)), "tb_last_batch_stats")
        return {name: getattr(s, name) for name, _ in BatchStats._fields_}

    # -- paged key/value cache ---------------------------------------------
    # Their lists are tensors, often ones made a line before: without a stream
    # the calls run on PyTorch's current one, behind what made the tensors, and
    # memory that a dropped tensor gives back is written only after they have read it.
    def _stream(self, stream) -> int:
        if stream is None and "torch" in sys.modules:
            return sys.modules["torch"].cuda.current_stream(self.device).cuda_stream
        return stream_handle(stream)

    def kv_copy_pages(self, cache: KvCache, src, dst, n: int | None = None, tokens=None,
                      stream=None):
        """tb_kv_copy_pages: page src[i] to page dst[i] in every layer, keys
        and values, for the first n entries of the lists (default: all)."""
        s, d, m = _int32(src, "src", src.shape[:1]), _int32(dst, "dst", dst.shape[:1]), 0
        most = min(src.shape[0], dst.shape[0])
        if tokens is not None:
            m = _int32(tokens, "tokens", tokens.shape[:1])
            most = min(most, tokens.shape[0])
        if n is None:
            n = most
        elif n > most:
            raise ValueError(f"n is {n}, the shortest list has {most} entries")
        self._ok(lib.tb_kv_copy_pages(self._h, cache.ref, s, d, m, n, self._stream(stream)),
                 "tb_kv_copy_pages")

    def kv_resize(self, cache: KvCache, capacity, status, stream=None):
        """tb_kv_resize: each slot gets exactly the pages of capacity[s] tokens;
        status: 0, pages missing, or -1 (past the table's width, or a cut inside
        a page that other slots share)."""
        self._ok(lib.tb_kv_resize(self._h, cache.ref, _int32(capacity, "capacity", cache.per_slot),
                                  _int32(status, "status", (1,)), self._stream(stream)),
                 "tb_kv_resize")

    def kv_fork(self, cache: KvCache, parents, table_out, held_out, lens_out, status, stream=None):
        """tb_kv_fork: slot s becomes the sequence of slot parents[s]."""
        slots = cache.per_slot
        self._ok(lib.tb_kv_fork(self._h, cache.ref, _int32(parents, "parents", slots),
                                _int32(table_out, "table_out", cache.table_shape),
                                _int32(held_out, "held_out", slots),
                                _int32(lens_out, "lens_out", slots),
                                _int32(status, "status", (1,)), self._stream(stream)),
                 "tb_kv_fork")

    def kv_compact(self, cache: KvCache, start, keep, count, status, stream=None):
        """tb_kv_compact: token start[s] + keep[s, i] moves to start[s] + i;
        status per slot: 0, 1 (pages shared with other slots), 2 (a bad list)."""
        slots, width = cache.per_slot, keep.shape[-1]
        self._ok(lib.tb_kv_compact(self._h, cache.ref, _int32(start, "start", slots),
                                   _int32(keep, "keep", slots + (width,)), width,
                                   _int32(count, "count", slots), _int32(status, "status", slots),
                                   self._stream(stream)), "tb_kv_compact")

    def tree_attention_workspace(self, cache: KvCache, q_heads: int) -> int:
        """Bytes of workspace tree_attention needs (tb_tree_attention_workspace)."""
        n = _u64()
        self._ok(lib.tb_tree_attention_workspace(self._h, cache.ref, q_heads, ct.byref(n)),
                 "tb_tree_attention_workspace")
        return n.value

    def tree_attention(self, cache: KvCache, layer: int, q, q_start, mask, out, workspace,
                       scale: float | None = None, lse=None, seq_slots=None, stream=None):
        """tb_tree_attention: q and out [rows, q_heads, dim] of the cache's
        type, q_start int32 [seqs + 1], mask int32 [rows, words] (bits, see
        tree_mask), workspace uint8 of tree_attention_workspace bytes; lse
        float32 [rows, q_heads] when wanted; scale defaults to dim ** -0.5."""
        rows, heads, dim = q.shape
        if q.dtype != cache.dtype or out.dtype != cache.dtype or not q.is_cuda or not out.is_cuda \
                or out.shape != q.shape or dim != cache.head_dim:
            raise ValueError(f"q and out must be [rows, heads, {cache.head_dim}] CUDA tensors of the "
                             "cache's type")
        (q_row, q_head, q_dim), (o_row, o_head, o_dim) = q.stride(), out.stride()
        if dim > 1 and (q_dim != 1 or o_dim != 1):
            raise ValueError("the last dimension of q and out must be dense")
        starts = _int32(q_start, "q_start", q_start.shape[:1])
        seqs, words = q_start.shape[0] - 1, mask.shape[-1]
        bits = _int32(mask, "mask", (rows, words))
        slots = 0 if seq_slots is None else _int32(seq_slots, "seq_slots", (seqs,))
        if lse is not None and (_dtype_name(lse) != "float32" or not lse.is_cuda
                                or not lse.is_contiguous() or lse.shape != (rows, heads)):
            raise ValueError("lse must be a contiguous float32 [rows, q_heads] CUDA tensor")
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        e = q.element_size()
        t = Tree(cache.ptr, layer, seqs, slots, starts, rows, heads,
                 dim ** -0.5 if scale is None else scale, q.data_ptr(), out.data_ptr(),
                 q_row * e, q_head * e, o_row * e, o_head * e,
                 0 if lse is None else lse.data_ptr(), bits, words, workspace.data_ptr(),
                 workspace.numel() * workspace.element_size())
        self._ok(lib.tb_tree_attention(self._h, ct.byref(t), self._stream(stream)),
                 "tb_tree_attention")

    # -- validation --------------------------------------------------------
    def validate_device(self, dst_device, expected_device, num_bytes: int, elem_size: int = 4):
        """tb_validate_device: None when equal, else (index, expected_bits, actual_bits)."""
        m = Mismatch()
        code = lib.tb_validate_device(self._h, addr(dst_device), addr(expected_device), num_bytes,
                                      elem_size, ct.byref(m))
        if code == TB_EVALIDATE:
            return (m.index, m.expected, m.actual)
        self._ok(code, "tb_validate_device")
        return None

    def validate(self, dst_device, expected_host, num_bytes: int, elem_size: int = 4):
        """Returns None when equal, else (index, expected_bits, actual_bits)."""
        m = Mismatch()
        code = lib.tb_validate(self._h, addr(dst_device), addr(expected_host), num_bytes,
                               elem_size, ct.byref(m))
        if code == TB_EVALIDATE:
            return (m.index, m.expected, m.actual)
        self._ok(code, "tb_validate")
        return None


def batch_copy_noalloc(descs, stream=None) -> None:
    """tb_batch_copy_noalloc on the current CUDA device: the batched copy for
    callers that cannot allocate device memory (its work items live in a
    fixed array inside the library).  Raises TBError on a nonzero code."""
    ptr, n, keep = Context.descriptor_array(descs)
    code = lib.tb_batch_copy_noalloc(ptr, n, stream_handle(stream))
    del keep
    _check(code, None, "tb_batch_copy_noalloc")
