"""Python binding of libmrr, the MI355X N-rank allreduce reduction library.

Argument marshalling only: every function forwards to the C entry point of the
same name in ``libmrr.so`` (declared in ``include/mrr.h``) and returns its
``mrr_status`` as an int.  Buffers may be torch tensors (their ``data_ptr()``
is passed) or raw device addresses (ints).  ``stream=None`` means torch's
current HIP stream on the current device.

The library must have been built (``__graft_entry__.build()`` or
``python allreduce_reduction_nranks_amd/build.py``); without it every call
raises -- there is no fallback path.
"""
from __future__ import annotations

import builtins
import ctypes
import operator
import os
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmrr.so")

# mrr_status
MRR_OK, MRR_EINVAL, MRR_EUNSUPPORTED, MRR_EALIGN, MRR_EOVERLAP, MRR_ESCRATCH, \
    MRR_ETIMEDOUT, MRR_EHIP = range(8)
STATUS_NAMES = ["MRR_OK", "MRR_EINVAL", "MRR_EUNSUPPORTED", "MRR_EALIGN", "MRR_EOVERLAP",
                "MRR_ESCRATCH", "MRR_ETIMEDOUT", "MRR_EHIP"]
# mrr_dtype
MRR_AUTO, MRR_F32, MRR_F16, MRR_BF16, MRR_FP8_E4M3B15, MRR_FP8_E4M3FN = range(6)
DTYPES = {"auto": MRR_AUTO, "f32": MRR_F32, "f16": MRR_F16, "bf16": MRR_BF16,
          "fp8": MRR_FP8_E4M3B15, "fp8_e4m3b15": MRR_FP8_E4M3B15,
          "fp8fn": MRR_FP8_E4M3FN, "fp8_e4m3fn": MRR_FP8_E4M3FN}
MAX_RANKS = 32
PKT_FLAG_SLOTS = 1024
MRR_NOALLOC_SCRATCH_BYTES = 32 << 20  # packet scratch of mrr_allreduce_packet_noalloc


class MrrError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__("%s%s" % (name, (": " + what) if what else ""))


_lock = threading.Lock()
_lib = None


def load_library() -> ctypes.CDLL:
    """Loads libmrr.so (once).  Raises if it has not been built."""
    global _lib
    lib = _lib
    if lib is not None:  # loaded: no lock on the per-call path
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmrr.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32
        f32, i64 = ctypes.c_float, ctypes.c_int64
        pp = ctypes.POINTER(vp)
        sigs = {
            "mrr_allreduce_rsag": ([pp, pp, sz, i, i, vp], i),
            "mrr_allreduce_rsag_ex": ([pp, pp, sz, i, i, i, i, i, vp], i),
            "mrr_allreduce_rsag_dual": ([pp, pp, pp, sz, i, i, i, i, vp], i),
            "mrr_packet_scratch_bytes": ([sz, i, i], sz),
            "mrr_packet_flag_bytes": ([i], sz),
            "mrr_allreduce_packet": ([pp, pp, vp, sz, vp, sz, i, i, i, u32, vp, vp], i),
            "mrr_allreduce_packet_ex": ([pp, pp, vp, sz, vp, sz, i, i, i, u32, vp, i, i, vp], i),
            "mrr_allreduce_packet_noalloc": ([pp, pp, sz, i, i, i, u32, vp, vp], i),
            "mrr_packet_reduce": ([pp, vp, sz, i, i, i, u32, u32, u32, vp, vp], i),
            "mrr_allreduce": ([pp, pp, sz, i, i, i, vp, sz, vp, sz, u32, vp, vp], i),
            "mrr_packet_rsag_scratch_bytes": ([sz, i, i], sz),
            "mrr_allreduce_packet_rsag": ([pp, pp, vp, sz, vp, sz, i, i, i, u32, vp, i, i, vp], i),
            "mrr_fullmesh_scratch_bytes": ([sz, i, i], sz),
            "mrr_allreduce_fullmesh": ([pp, pp, vp, sz, vp, sz, i, i, i, u32, vp, i, i, vp], i),
            "mrr_pack": ([vp, vp, sz, u32, vp], i),
            "mrr_unpack": ([vp, vp, sz, vp], i),
            "mrr_fp8b15_to_f16": ([vp, vp, sz, vp], i),
            "mrr_fp8b15_to_f32": ([vp, vp, sz, vp], i),
            "mrr_f16_to_fp8b15": ([vp, vp, sz, vp], i),
            "mrr_f32_to_fp8b15": ([vp, vp, sz, vp], i),
            "mrr_layernorm_fwd": ([vp, i, vp, vp, vp, vp, vp, vp, vp, sz, sz, sz, sz, f32, i, i, vp], i),
            "mrr_layernorm_bwd_workspace_bytes": ([sz, sz], sz),
            "mrr_layernorm_bwd": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, sz, sz, sz, i, i, vp, sz, vp], i),
            "mrr_linear_xent_workspace_bytes": ([sz, sz, vp, i, i, i], sz),
            "mrr_linear_xent_workspace_bytes_in_place": ([sz, sz, vp, i, i, i], sz),
            "mrr_linear_xent_fwd": ([vp, vp, vp, i, vp, i64, vp, vp, sz, sz, sz, sz, i, vp, sz, vp], i),
            "mrr_linear_xent_bwd": ([vp, vp, vp, i, vp, i64, vp, vp, sz, vp, vp, sz, sz, sz, sz, i, vp, sz, vp], i),
            "mrr_qknorm_rope_fwd": ([vp, i, vp, vp, vp, sz, vp, vp, vp, sz, vp, sz, sz, i, sz, vp, vp, f32, i, i, vp], i),
            "mrr_qknorm_rope_bwd_workspace_bytes": ([sz, vp, sz], sz),
            "mrr_qknorm_rope_bwd": ([vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, sz, vp, sz, sz, i, sz, vp, vp, f32, i, i, vp,
                                     sz, vp], i),
            "mrr_orthogonalize_workspace_bytes": ([sz, sz, sz, i, i], sz),
            "mrr_orthogonalize": ([vp, vp, sz, sz, sz, sz, sz, sz, sz, i, vp, f32, i, i, vp, sz, vp], i),
            "mrr_muon_workspace_bytes": ([sz, sz, sz, i, i, i], sz),
            "mrr_muon_step": ([vp, i, f32, vp, vp, f32, i, vp, vp, f32, f32, sz, sz, sz, sz, sz, sz, sz, i, vp, f32, i, i,
                               i, vp, sz, vp], i),
            "mrr_stream_copy": ([vp, vp, sz, vp], i),
            "mrr_rank_buffer_pitch": ([sz, i], sz),
            "mrr_status_string": ([i], ctypes.c_char_p),
            "mrr_version": ([], i),
            "mrr_reload_env": ([], None),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return _lib


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _ptrs(xs):
    if xs is None:
        return None  # the C ABI refuses a null array with MRR_EINVAL
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _dt(d) -> int:
    v = DTYPES.get(d) if type(d) is str else None
    if v is not None:
        return v
    if isinstance(d, int):
        return d
    if isinstance(d, str):
        raise KeyError("unknown type name %r" % d)
    import torch
    return {torch.float32: MRR_F32, torch.float16: MRR_F16, torch.bfloat16: MRR_BF16,
            torch.uint8: MRR_FP8_E4M3B15}[d]


_ESIZE = {MRR_F32: 4, MRR_F16: 2, MRR_BF16: 2, MRR_FP8_E4M3B15: 1, MRR_FP8_E4M3FN: 1}


def _nbytes(count, dtype) -> int:
    """Bytes of `count` elements of dtype (0 for AUTO or an unknown id, which
    the C ABI refuses on its own)."""
    return (count if count > 0 else 0) * _ESIZE.get(_dt(dtype), 0)


def _room(x, nbytes: int, what: str) -> None:
    """A tensor argument must hold at least nbytes bytes.  Raw addresses
    (ints) and None pass unchecked: the C ABI validates what it can see."""
    if x is None or isinstance(x, int):
        return
    if x.nbytes < nbytes:
        raise ValueError("%s holds %d bytes, the call needs %d" % (what, x.nbytes, nbytes))


def _rank_ptrs(xs, nranks: int, nbytes: int, what: str):
    """Host array of device pointers for a per-rank argument.  The C ABI reads
    `nranks` entries, so a shorter list is refused here rather than letting it
    read past the array; tensor entries must hold nbytes bytes each."""
    if xs is None:
        return None
    if nranks > 0 and len(xs) < nranks:
        raise ValueError("%s has %d entries, nranks is %d" % (what, len(xs), nranks))
    ptrs = []
    for x in xs:
        if x is None or type(x) is int:
            ptrs.append(x or 0)
        else:
            if x.nbytes < nbytes and len(ptrs) < nranks:
                _room(x, nbytes, "%s[%d]" % (what, len(ptrs)))
            ptrs.append(x.data_ptr())
    return (_VP * len(ptrs))(*ptrs)


_VP = ctypes.c_void_p


_raw_stream = None


def _stream(stream) -> int:
    """HIP stream handle: torch's current stream on the current device when
    stream is None.  torch's raw-handle getter is used when it exists: it
    returns the same handle as torch.cuda.current_stream().cuda_stream without
    building a Stream object (measured on MI355X: 0.07 us against 2.96 us,
    a third of an eager call's host cost)."""
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            getter = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
            _raw_stream = (lambda: getter(device())) if getter else \
                (lambda: int(torch.cuda.current_stream().cuda_stream))
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def check(status: int, what: str = "") -> None:
    """Raises MrrError for a non-OK status."""
    if status != MRR_OK:
        raise MrrError(status, what)


def mrr_status_string(status: int) -> str:
    return load_library().mrr_status_string(status).decode()


def mrr_version() -> int:
    return load_library().mrr_version()


def mrr_reload_env() -> None:
    """Makes the library read its MRR_* environment overrides again."""
    load_library().mrr_reload_env()


def mrr_rank_buffer_pitch(bytes_per_rank: int, nranks: int) -> int:
    return load_library().mrr_rank_buffer_pitch(bytes_per_rank, nranks)


def alloc_rank_buffers(nranks: int, count: int, dtype, device=None):
    """N rank buffers of `count` elements carved from one device allocation
    at mrr_rank_buffer_pitch() spacing.  Returns (pool, [views])."""
    import torch
    tdt = dtype if isinstance(dtype, torch.dtype) else \
        {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
         "fp8": torch.uint8, "fp8_e4m3b15": torch.uint8, "fp8fn": torch.uint8,
         "fp8_e4m3fn": torch.uint8}[dtype]
    esize = torch.empty((), dtype=tdt).element_size()
    nbytes = count * esize
    pitch = mrr_rank_buffer_pitch(nbytes, nranks)
    pool = torch.empty(max(1, nranks * pitch), dtype=torch.uint8,
                       device=device if device is not None else "cuda")
    views = [pool[r * pitch: r * pitch + nbytes].view(tdt) for r in range(nranks)]
    return pool, views


def mrr_allreduce_rsag(inputs, outputs, count, dtype, nranks, stream=None) -> int:
    nb = _nbytes(count, dtype)
    return load_library().mrr_allreduce_rsag(_rank_ptrs(inputs, nranks, nb, "inputs"),
                                             _rank_ptrs(outputs, nranks, nb, "outputs"), count,
                                             _dt(dtype), nranks, _stream(stream))


def mrr_allreduce_rsag_ex(inputs, outputs, count, dtype_in, accum, dtype_out, nranks, rank=-1,
                          stream=None) -> int:
    tout = dtype_in if _dt(dtype_out) == MRR_AUTO else dtype_out
    return load_library().mrr_allreduce_rsag_ex(
        _rank_ptrs(inputs, nranks, _nbytes(count, dtype_in), "inputs"),
        _rank_ptrs(outputs, nranks, _nbytes(count, tout), "outputs"), count, _dt(dtype_in),
        _dt(accum), _dt(dtype_out), nranks, rank, _stream(stream))


def mrr_allreduce_rsag_dual(inputs, outputs, outputs2, count, dtype_in, accum, nranks, rank=-1,
                            stream=None) -> int:
    nb = _nbytes(count, dtype_in)
    return load_library().mrr_allreduce_rsag_dual(
        _rank_ptrs(inputs, nranks, nb, "inputs"),
        _rank_ptrs(outputs, nranks, _nbytes(count, MRR_F16), "outputs"),
        _rank_ptrs(outputs2, nranks, nb, "outputs2"), count, _dt(dtype_in), _dt(accum), nranks,
        rank, _stream(stream))


def mrr_packet_scratch_bytes(count, dtype, nranks) -> int:
    return load_library().mrr_packet_scratch_bytes(count, _dt(dtype), nranks)


def mrr_packet_flag_bytes(nranks) -> int:
    return load_library().mrr_packet_flag_bytes(nranks)


def mrr_allreduce_packet(inputs, outputs, scratch, scratch_bytes, flags, count, dtype, accum,
                         nranks, max_spins, dev_err=None, stream=None) -> int:
    nb = _nbytes(count, dtype)
    _room(scratch, scratch_bytes, "scratch")
    _room(flags, 4 * PKT_FLAG_SLOTS * max(0, nranks), "flags")
    return load_library().mrr_allreduce_packet(
        _rank_ptrs(inputs, nranks, nb, "inputs"), _rank_ptrs(outputs, nranks, nb, "outputs"),
        _ptr(scratch), scratch_bytes, _ptr(flags), count, _dt(dtype), _dt(accum), nranks,
        max_spins, _ptr(dev_err), _stream(stream))


def mrr_allreduce_packet_ex(inputs, outputs, scratch, scratch_bytes, flags, count, dtype, accum,
                            nranks, max_spins, dev_err=None, blocks_per_rank=0, threads=0,
                            stream=None) -> int:
    nb = _nbytes(count, dtype)
    _room(scratch, scratch_bytes, "scratch")
    _room(flags, 4 * PKT_FLAG_SLOTS * max(0, nranks), "flags")
    return load_library().mrr_allreduce_packet_ex(
        _rank_ptrs(inputs, nranks, nb, "inputs"), _rank_ptrs(outputs, nranks, nb, "outputs"),
        _ptr(scratch), scratch_bytes, _ptr(flags), count, _dt(dtype), _dt(accum), nranks,
        max_spins, _ptr(dev_err), blocks_per_rank, threads, _stream(stream))


def mrr_allreduce_packet_noalloc(inputs, outputs, count, dtype, accum, nranks, max_spins,
                                 dev_err=None, stream=None) -> int:
    nb = _nbytes(count, dtype)
    return load_library().mrr_allreduce_packet_noalloc(
        _rank_ptrs(inputs, nranks, nb, "inputs"), _rank_ptrs(outputs, nranks, nb, "outputs"),
        count, _dt(dtype), _dt(accum), nranks, max_spins, _ptr(dev_err), _stream(stream))


def mrr_packet_rsag_scratch_bytes(count, dtype, nranks) -> int:
    return load_library().mrr_packet_rsag_scratch_bytes(count, _dt(dtype), nranks)


def mrr_allreduce_packet_rsag(inputs, outputs, scratch, scratch_bytes, flags, count, dtype, accum,
                              nranks, max_spins, dev_err=None, blocks_per_rank=0, threads=0,
                              stream=None) -> int:
    nb = _nbytes(count, dtype)
    _room(scratch, scratch_bytes, "scratch")
    _room(flags, 4 * PKT_FLAG_SLOTS * max(0, nranks), "flags")
    return load_library().mrr_allreduce_packet_rsag(
        _rank_ptrs(inputs, nranks, nb, "inputs"), _rank_ptrs(outputs, nranks, nb, "outputs"),
        _ptr(scratch), scratch_bytes, _ptr(flags), count, _dt(dtype), _dt(accum), nranks,
        max_spins, _ptr(dev_err), blocks_per_rank, threads, _stream(stream))


def mrr_fullmesh_scratch_bytes(count, dtype, nranks) -> int:
    return load_library().mrr_fullmesh_scratch_bytes(count, _dt(dtype), nranks)


def mrr_allreduce_fullmesh(inputs, outputs, scratch, scratch_bytes, flags, count, dtype, accum,
                           nranks, max_spins, dev_err=None, blocks_per_rank=0, threads=0,
                           stream=None) -> int:
    nb = _nbytes(count, dtype)
    _room(scratch, scratch_bytes, "scratch")
    _room(flags, 4 * PKT_FLAG_SLOTS * max(0, nranks), "flags")
    return load_library().mrr_allreduce_fullmesh(
        _rank_ptrs(inputs, nranks, nb, "inputs"), _rank_ptrs(outputs, nranks, nb, "outputs"),
        _ptr(scratch), scratch_bytes, _ptr(flags), count, _dt(dtype), _dt(accum), nranks,
        max_spins, _ptr(dev_err), blocks_per_rank, threads, _stream(stream))


def mrr_allreduce(inputs, outputs, count, dtype, accum, nranks, scratch=None, scratch_bytes=0,
                  flags=None, packet_max_bytes=0, max_spins=0, dev_err=None, stream=None) -> int:
    nb = _nbytes(count, dtype)
    _room(scratch, scratch_bytes, "scratch")
    _room(flags, 4 * PKT_FLAG_SLOTS * max(0, nranks), "flags")
    return load_library().mrr_allreduce(_rank_ptrs(inputs, nranks, nb, "inputs"),
                                        _rank_ptrs(outputs, nranks, nb, "outputs"), count,
                                        _dt(dtype), _dt(accum), nranks, _ptr(scratch),
                                        scratch_bytes, _ptr(flags), packet_max_bytes, max_spins,
                                        _ptr(dev_err), _stream(stream))


def mrr_packet_reduce(in_pkts, out_pkts, npkts, dtype, accum, nranks, flag_in, flag_out,
                      max_spins, dev_err=None, stream=None) -> int:
    _room(out_pkts, 8 * max(0, int(npkts)), "out_pkts")
    return load_library().mrr_packet_reduce(_rank_ptrs(in_pkts, nranks, 8 * max(0, int(npkts)),
                                                       "in_pkts"), _ptr(out_pkts), npkts,
                                            _dt(dtype), _dt(accum), nranks, flag_in, flag_out,
                                            max_spins, _ptr(dev_err), _stream(stream))


def mrr_pack(src, pkts, nbytes, flag, stream=None) -> int:
    _room(src, nbytes, "src")
    _room(pkts, (max(0, int(nbytes)) + 3) // 4 * 8, "pkts")
    return load_library().mrr_pack(_ptr(src), _ptr(pkts), nbytes, flag, _stream(stream))


def mrr_unpack(pkts, dst, nbytes, stream=None) -> int:
    _room(pkts, (max(0, int(nbytes)) + 3) // 4 * 8, "pkts")
    _room(dst, nbytes, "dst")
    return load_library().mrr_unpack(_ptr(pkts), _ptr(dst), nbytes, _stream(stream))


def _codec_room(src, ein, dst, eout, n):
    _room(src, max(0, int(n)) * ein, "src")
    _room(dst, max(0, int(n)) * eout, "dst")


def mrr_fp8b15_to_f16(src, dst, n, stream=None) -> int:
    _codec_room(src, 1, dst, 2, n)
    return load_library().mrr_fp8b15_to_f16(_ptr(src), _ptr(dst), n, _stream(stream))


def mrr_fp8b15_to_f32(src, dst, n, stream=None) -> int:
    _codec_room(src, 1, dst, 4, n)
    return load_library().mrr_fp8b15_to_f32(_ptr(src), _ptr(dst), n, _stream(stream))


def mrr_f16_to_fp8b15(src, dst, n, stream=None) -> int:
    _codec_room(src, 2, dst, 1, n)
    return load_library().mrr_f16_to_fp8b15(_ptr(src), _ptr(dst), n, _stream(stream))


def mrr_f32_to_fp8b15(src, dst, n, stream=None) -> int:
    _codec_room(src, 4, dst, 1, n)
    return load_library().mrr_f32_to_fp8b15(_ptr(src), _ptr(dst), n, _stream(stream))


def _matrix_bytes(rows, cols, ld, esize) -> int:
    """Bytes from the first element to the last of rows x cols elements, rows ld apart."""
    return ((rows - 1) * ld + cols) * esize if rows > 0 and cols > 0 else 0


def _span(x) -> int:
    """Bytes from a tensor's first element to its last, strides counted."""
    if x.is_contiguous():
        return x.nbytes
    if x.numel() == 0:
        return 0
    return (1 + builtins.sum((n - 1) * s for n, s in zip(x.shape, x.stride()))) * x.element_size()


_bytes_of = operator.attrgetter("nbytes")
_is_whole = operator.methodcaller("is_contiguous")
_address = operator.methodcaller("data_ptr")


def _rows_arg(x, nbytes: int, what: str) -> int:
    """Address of an argument whose rows may lie apart: a tensor must hold nbytes
    bytes, a view of a wider one counting with its strides, and the elements of a row
    must lie side by side.  (Checks and address in one step, and below lists taken
    whole: marshalling is half of an eager call's host cost, which is what a small
    call takes.)"""
    if x is None:
        return 0
    try:
        if x.nbytes >= nbytes and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        return x
    if x.dim() and x.size(-1) > 1 and x.stride(-1) != 1:
        raise ValueError("%s has its rows' elements %d apart" % (what, x.stride(-1)))
    if _span(x) < nbytes:
        raise ValueError("%s spans %d bytes, the call needs %d" % (what, _span(x), nbytes))
    return x.data_ptr()


def _spaced_arg(x, nbytes: int, what: str) -> int:
    """_rows_arg() for single values that a call takes at a stride of its own.  The span alone
    counts: an expanded tensor (what autograd hands to a sum's gradient) has fewer bytes than
    elements."""
    if x is None or isinstance(x, int):
        return x or 0
    if _span(x) < nbytes:
        raise ValueError("%s spans %d bytes, the call needs %d" % (what, _span(x), nbytes))
    return x.data_ptr()


def _flat_arg(x, nbytes: int, what: str) -> int:
    """_rows_arg() for an argument without a row stride: its elements lie side by side."""
    if x is None:
        return 0
    try:
        if x.nbytes >= nbytes and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        return x
    if x.nbytes < nbytes:
        raise ValueError("%s holds %d bytes, the call needs %d" % (what, x.nbytes, nbytes))
    raise ValueError("%s is not contiguous" % what)


_words: dict = {}


def _pack(values) -> bytes:
    """Host array of 64-bit words for the C ABI (it lives as long as the call's arguments)."""
    n = len(values)
    p = _words.get(n)
    if p is None:
        p = _words[n] = struct.Struct("%dQ" % n).pack
    return p(*values)


def _rows_args(xs, n: int, nbytes, what: str):
    """Packed addresses of per-rank matrices; nbytes[r] is what entry r has to span
    (one number: all of them)."""
    if xs is None:
        return None
    if len(xs) < n:
        raise ValueError("%s has %d entries, nranks is %d" % (what, len(xs), n))
    one = type(nbytes) is int
    if 0 < n == len(xs):
        try:
            fits = builtins.min(map(_bytes_of, xs)) >= nbytes if one else all(map(operator.ge, map(_bytes_of, xs), nbytes))
            if fits and all(map(_is_whole, xs)):
                return _pack(list(map(_address, xs)))
        except AttributeError:
            pass  # addresses among them, or no shard
    ptrs = []
    for r, x in enumerate(xs):
        need = 0 if r >= n else nbytes if one else nbytes[r]
        ptrs.append(_rows_arg(x, need, "%s[%d]" % (what, r)))
    return _pack(ptrs)


def _wtype(t: int, wdtype) -> int:
    return _dt(wdtype) or t  # MRR_AUTO is 0


def mrr_layernorm_fwd(inputs, nranks, residual, weight, bias, sum, out, mean, rstd, rows, cols,
                      ld_in, ld_out, eps, dtype, wdtype="auto", stream=None) -> int:
    t = _dt(dtype)
    tw = _wtype(t, wdtype)
    e, wb, rb = _ESIZE.get(t, 0), cols * _ESIZE.get(tw, 0), 4 * rows
    nin = nout = _matrix_bytes(rows, cols, ld_in, e)
    if ld_out != ld_in:
        nout = _matrix_bytes(rows, cols, ld_out, e)
    return load_library().mrr_layernorm_fwd(
        _rows_args(inputs, nranks, nin, "inputs"), nranks, _rows_arg(residual, nin, "residual"),
        _flat_arg(weight, wb, "weight"), _flat_arg(bias, wb, "bias"), _rows_arg(sum, nout, "sum"),
        _rows_arg(out, nout, "out"), _flat_arg(mean, rb, "mean"), _flat_arg(rstd, rb, "rstd"),
        rows, cols, ld_in, ld_out, eps, t, tw, _stream(stream))


def mrr_layernorm_bwd_workspace_bytes(rows, cols) -> int:
    return load_library().mrr_layernorm_bwd_workspace_bytes(rows, cols)


def mrr_layernorm_bwd(dout, sum, weight, mean, rstd, dresidual, dsum, dweight, dbias, rows, cols,
                      ld_in, ld_out, dtype, wdtype="auto", workspace=None, workspace_bytes=0,
                      stream=None) -> int:
    t = _dt(dtype)
    tw = _wtype(t, wdtype)
    e, wb, rb = _ESIZE.get(t, 0), cols * _ESIZE.get(tw, 0), 4 * rows
    nin = nout = _matrix_bytes(rows, cols, ld_in, e)
    if ld_out != ld_in:
        nout = _matrix_bytes(rows, cols, ld_out, e)
    return load_library().mrr_layernorm_bwd(
        _rows_arg(dout, nin, "dout"), _rows_arg(sum, nin, "sum"), _flat_arg(weight, wb, "weight"),
        _flat_arg(mean, rb, "mean"), _flat_arg(rstd, rb, "rstd"),
        _rows_arg(dresidual, nin, "dresidual"), _rows_arg(dsum, nout, "dsum"), _flat_arg(dweight, wb, "dweight"),
        _flat_arg(dbias, wb, "dbias"), rows, cols, ld_in, ld_out, t, tw,
        _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def _shard_bytes(rows, n: int, cols, ld, esize):
    """_matrix_bytes() of each shard."""
    if rows is None:
        return []
    pitch, last = ld * esize, (cols - ld) * esize
    return [r * pitch + last if r > 0 and cols > 0 else 0 for r in rows[:n if n > 0 else 0]]


def _sizes(rows, n: int):
    if rows is None:
        return None
    if len(rows) < n:
        raise ValueError("rows has %d entries, nranks is %d" % (len(rows), n))
    return _pack(rows) if len(rows) else _pack((0,))


def mrr_linear_xent_workspace_bytes(tokens, cols, rows, nranks, dtype, backward) -> int:
    return load_library().mrr_linear_xent_workspace_bytes(tokens, cols, _sizes(rows, nranks), nranks, _dt(dtype),
                                                          1 if backward else 0)


def mrr_linear_xent_workspace_bytes_in_place(tokens, cols, rows, nranks, dtype, backward) -> int:
    return load_library().mrr_linear_xent_workspace_bytes_in_place(tokens, cols, _sizes(rows, nranks), nranks, _dt(dtype),
                                                                   1 if backward else 0)


def mrr_linear_xent_fwd(hidden, weights, rows, nranks, targets, ignore_index, loss, lse, tokens, cols,
                        ld_hidden, ld_weight, dtype, workspace=None, workspace_bytes=0, stream=None) -> int:
    t = _dt(dtype)
    e = _ESIZE.get(t, 0)
    sizes = _sizes(rows, nranks)
    need = _shard_bytes(rows, nranks, cols, ld_weight, e)
    return load_library().mrr_linear_xent_fwd(
        _rows_arg(hidden, _matrix_bytes(tokens, cols, ld_hidden, e), "hidden"),
        _rows_args(weights, len(need), need, "weights"), sizes, nranks, _flat_arg(targets, 8 * tokens, "targets"),
        ignore_index, _flat_arg(loss, 4 * tokens, "loss"), _flat_arg(lse, 4 * tokens, "lse"), tokens, cols, ld_hidden,
        ld_weight, t, _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def mrr_linear_xent_bwd(hidden, weights, rows, nranks, targets, ignore_index, lse, dloss, dloss_stride, dhidden,
                        dweights, tokens, cols, ld_hidden, ld_weight, dtype, workspace=None, workspace_bytes=0,
                        stream=None) -> int:
    t = _dt(dtype)
    e = _ESIZE.get(t, 0)
    sizes = _sizes(rows, nranks)
    nh = _matrix_bytes(tokens, cols, ld_hidden, e)
    need = _shard_bytes(rows, nranks, cols, ld_weight, e)
    return load_library().mrr_linear_xent_bwd(
        _rows_arg(hidden, nh, "hidden"), _rows_args(weights, len(need), need, "weights"), sizes, nranks,
        _flat_arg(targets, 8 * tokens, "targets"), ignore_index, _flat_arg(lse, 4 * tokens, "lse"),
        _spaced_arg(dloss, 4 * ((tokens - 1) * dloss_stride + 1) if tokens > 0 else 0, "dloss"), dloss_stride,
        _rows_arg(dhidden, nh, "dhidden"), _rows_args(dweights, len(need), need, "dweights"), tokens, cols, ld_hidden,
        ld_weight, t, _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def _three(xs, what: str):
    """Packed host array of three sizes: of the queries, keys and values."""
    if xs is None:
        return None
    if len(xs) != 3:
        raise ValueError("%s has %d entries, not 3" % (what, len(xs)))
    return _pack(xs)


def _head_args(xs, tokens, heads, dim, lds, strides, esize, what: str):
    """Packed addresses of the queries', keys' and values' tensors, each to span what its strides reach."""
    if xs is None or heads is None or lds is None or strides is None:
        return None
    if len(xs) != 3:
        raise ValueError("%s has %d entries, not 3" % (what, len(xs)))
    ptrs = [0, 0, 0]
    for k, x in enumerate(xs):
        n = heads[k]
        if x is None or not n:
            continue
        need = ((tokens - 1) * lds[k] + (n - 1) * strides[k] + dim) * esize if tokens > 0 and dim > 0 else 0
        ptrs[k] = _rows_arg(x, need, "%s[%d]" % (what, k) if type(x) is int else what)
    return _pack(ptrs)


def mrr_qknorm_rope_fwd(inputs, nranks, q_weight, k_weight, table, table_rows, positions, sum, outs, tokens, heads, head_dim,
                        rot_dim, pairs, ld_in, ld_outs, head_strides, eps, dtype, wdtype="auto", stream=None) -> int:
    t = _dt(dtype)
    tw = _wtype(t, wdtype)
    e, wb = _ESIZE.get(t, 0), head_dim * _ESIZE.get(tw, 0)
    counts, lds, strides = _three(heads, "heads"), _three(ld_outs, "ld_outs"), _three(head_strides, "head_strides")
    need = _matrix_bytes(tokens, (heads[0] + heads[1] + heads[2]) * head_dim, ld_in, e) if heads is not None else 0
    return load_library().mrr_qknorm_rope_fwd(
        _rows_args(inputs, nranks, need, "inputs"), nranks, _flat_arg(q_weight, wb, "q_weight"),
        _flat_arg(k_weight, wb, "k_weight"), _flat_arg(table, 4 * table_rows * rot_dim, "table"), table_rows,
        _flat_arg(positions, 8 * tokens, "positions"), _rows_arg(sum, need, "sum"),
        _head_args(outs, tokens, heads, head_dim, ld_outs, head_strides, e, "outs"), tokens, counts, head_dim, rot_dim,
        1 if pairs else 0, ld_in, lds, strides, eps, t, tw, _stream(stream))


def mrr_qknorm_rope_bwd_workspace_bytes(tokens, heads, head_dim) -> int:
    return load_library().mrr_qknorm_rope_bwd_workspace_bytes(tokens, _three(heads, "heads"), head_dim)


def mrr_qknorm_rope_bwd(douts, sum, q_weight, k_weight, table, table_rows, positions, dsum, dq_weight, dk_weight, tokens, heads,
                        head_dim, rot_dim, pairs, ld_in, ld_douts, head_strides, eps, dtype, wdtype="auto", workspace=None,
                        workspace_bytes=0, stream=None) -> int:
    t = _dt(dtype)
    tw = _wtype(t, wdtype)
    e, wb = _ESIZE.get(t, 0), head_dim * _ESIZE.get(tw, 0)
    counts, lds, strides = _three(heads, "heads"), _three(ld_douts, "ld_douts"), _three(head_strides, "head_strides")
    need = _matrix_bytes(tokens, (heads[0] + heads[1] + heads[2]) * head_dim, ld_in, e) if heads is not None else 0
    return load_library().mrr_qknorm_rope_bwd(
        _head_args(douts, tokens, heads, head_dim, ld_douts, head_strides, e, "douts"), _rows_arg(sum, need, "sum"),
        _flat_arg(q_weight, wb, "q_weight"), _flat_arg(k_weight, wb, "k_weight"),
        _flat_arg(table, 4 * table_rows * rot_dim, "table"), table_rows, _flat_arg(positions, 8 * tokens, "positions"),
        _rows_arg(dsum, need, "dsum"), _flat_arg(dq_weight, wb, "dq_weight"), _flat_arg(dk_weight, wb, "dk_weight"), tokens,
        counts, head_dim, rot_dim, 1 if pairs else 0, ld_in, lds, strides, eps, t, tw,
        _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def _batch_bytes(rows, cols, ld, batch, stride, esize) -> int:
    """Bytes from the first element to the last of `batch` matrices, `stride` elements apart."""
    return (batch - 1) * stride * esize + _matrix_bytes(rows, cols, ld, esize) if batch > 0 and rows > 0 and cols > 0 else 0


def _coefficients(xs, steps):
    """Host array of three floats a step."""
    if xs is None:
        return None
    if len(xs) < 3 * steps:
        raise ValueError("coefficients has %d entries, the call needs %d" % (len(xs), 3 * steps))
    return struct.pack("%df" % len(xs), *xs)


def mrr_orthogonalize_workspace_bytes(rows, cols, batch, dtype, products="auto") -> int:
    return load_library().mrr_orthogonalize_workspace_bytes(rows, cols, batch, _dt(dtype), _dt(products))


def mrr_orthogonalize(x, out, rows, cols, ld_in, ld_out, batch, stride_in, stride_out, steps, coefficients, eps, dtype,
                      products="auto", workspace=None, workspace_bytes=0, stream=None) -> int:
    t = _dt(dtype)
    e = _ESIZE.get(t, 0)
    return load_library().mrr_orthogonalize(
        _rows_arg(x, _batch_bytes(rows, cols, ld_in, batch, stride_in, e), "x"),
        _rows_arg(out, _batch_bytes(rows, cols, ld_out, batch, stride_out, e), "out"), rows, cols, ld_in, ld_out, batch, stride_in,
        stride_out, steps, _coefficients(coefficients, steps), eps, t, _dt(products),
        _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def mrr_muon_workspace_bytes(rows, cols, batch, wdtype, products="auto", nesterov=True) -> int:
    return load_library().mrr_muon_workspace_bytes(rows, cols, batch, 1 if nesterov else 0, _dt(wdtype), _dt(products))


def mrr_muon_step(grads, nranks, grad_scale, momentum, momentum_out, mu, nesterov, weight, weights_out, rate, decay, rows, cols,
                  ld_grad, ld_weight, batch, stride_grad, stride_weight, steps, coefficients, eps, gdtype, wdtype="auto",
                  products="auto", workspace=None, workspace_bytes=0, stream=None) -> int:
    tg = _dt(gdtype)
    tw = _wtype(tg, wdtype)
    ng = _batch_bytes(rows, cols, ld_grad, batch, stride_grad, _ESIZE.get(tg, 0))
    nm = _batch_bytes(rows, cols, ld_weight, batch, stride_weight, 4)
    nw = nm // 4 * _ESIZE.get(tw, 0)
    return load_library().mrr_muon_step(
        _rows_args(grads, nranks, ng, "grads"), nranks, grad_scale, _rows_arg(momentum, nm, "momentum"),
        _rows_arg(momentum_out, nm, "momentum_out"), mu, 1 if nesterov else 0, _rows_arg(weight, nw, "weight"),
        _rows_args(weights_out, nranks, nw, "weights_out"), rate, decay, rows, cols, ld_grad, ld_weight, batch, stride_grad,
        stride_weight, steps, _coefficients(coefficients, steps), eps, tg, tw, _dt(products),
        _flat_arg(workspace, workspace_bytes, "workspace"), workspace_bytes, _stream(stream))


def mrr_stream_copy(src, dst, nbytes, stream=None) -> int:
    _room(src, nbytes, "src")
    _room(dst, nbytes, "dst")
    return load_library().mrr_stream_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream))
