"""Thin Python binding of liblw (the C ABI in include/lw.h).

Argument marshalling and checks only: every step of the path runs in liblw's
host code or CUDA kernels.  Each tensor is checked (dtype, contiguity, size,
device) before its address crosses the ABI, since the C calls cannot see
them.  PyTorch is used for device memory and streams.  If the compiled
library is missing this module raises at load time -- there is no fallback.
Functions carry the C names; see include/lw.h for the contract of each.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "liblw.so")

LW_FMT_Q4_PAIR, LW_FMT_Q6, LW_FMT_BF16_EXP = 1, 2, 3
# device status codes (*d_status), as in include/lw.h
(LW_DEV_OK, LW_DEV_LANE_LENGTH, LW_DEV_BAD_CODE, LW_DEV_TILE_SIZE, LW_DEV_TIMEOUT,
 LW_DEV_BAD_TABLE, LW_DEV_BAD_STRIPS, LW_DEV_BAD_SLOT, LW_DEV_BAD_PAGE,
 LW_DEV_BAD_SEQ, LW_DEV_BAD_POSITION) = range(11)
(LW_OK, LW_ERR_INVALID_ARG, LW_ERR_SHAPE, LW_ERR_UNSUPPORTED, LW_ERR_ALLOC, LW_ERR_CORRUPT,
 LW_ERR_CUDA, LW_ERR_IO) = range(8)
SECTION_NAMES = ["words", "tile_off", "lane_bits", "table", "qparams", "signman",
                 "vflags", "vrow_off", "vexp", "lane_mid"]
STATUS_NAMES = {0: "LW_OK", 1: "LW_ERR_INVALID_ARG", 2: "LW_ERR_SHAPE", 3: "LW_ERR_UNSUPPORTED",
                4: "LW_ERR_ALLOC", 5: "LW_ERR_CORRUPT", 6: "LW_ERR_CUDA", 7: "LW_ERR_IO"}
DEV_STATUS = {0: "ok", 1: "lane length", 2: "bad code", 3: "tile size", 4: "timeout",
              5: "bad table", 6: "bad strips", 7: "bad slot", 8: "bad page", 9: "bad sequence",
              10: "bad position"}
TABLE_BYTES = 1024
EXPORTED = ["lw_encode_bundle", "lw_bundle_sections", "lw_bundle_free", "lw_table_from_lengths",
            "lw_validate_sections", "lw_workspace_bytes", "lw_decode", "lw_decode_gemv",
            "lw_decode_gemm", "lw_twin_gemv", "lw_twin_gemm", "lw_status_string",
            "lw_last_error", "lw_version", "lw_decode_gemv_noalloc", "lw_noalloc_scratch_bytes",
            "lw_decode_gemv_group", "lw_workspace_bytes_group", "lw_twin_gemv_group",
            "lw_bundle_desc", "lw_bundle_serialized_bytes", "lw_bundle_serialize",
            "lw_bundle_deserialize", "lw_bundle_save", "lw_bundle_load", "lw_transcode_twin",
            "lw_twin_tile_rows", "lw_decode_gemm_strips", "lw_graph_begin", "lw_graph_end",
            "lw_graph_launch", "lw_graph_free", "lw_decode_gemm_group", "lw_twin_gemm_group",
            "lw_table_lut_entries", "lw_test_stall_next", "lw_kv_tile_bytes", "lw_kv_page_bytes",
            "lw_kv_write", "lw_kv_read", "lw_kv_workspace_bytes", "lw_kv_attention",
            "lw_rotary_table", "lw_kv_write_rotary", "lw_kv_weigh_workspace_bytes", "lw_kv_weigh",
            "lw_kv_evict", "lw_kv_summary_bytes", "lw_kv_summarise",
            "lw_kv_blocks_workspace_bytes", "lw_kv_attention_blocks"]
LW_F32, LW_F16, LW_BF16 = 0, 1, 2
LW_KV_GROUP, LW_KV_TILE, LW_KV_LIMIT = 32, 16, 61440.0
(LW_ROTARY_PLAIN, LW_ROTARY_LINEAR, LW_ROTARY_NTK, LW_ROTARY_BANDS, LW_ROTARY_YARN) = range(5)


class LwError(RuntimeError):
    """A failing call: `status` is the lw_status code.  `detail` replaces the
    library's thread-local error text when the binding itself refused the
    call before reaching the library."""

    def __init__(self, status: int, what: str, detail: str | None = None):
        self.status = status
        text = _last_error() if detail is None else detail
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}: {text}")


class LwDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("twin", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class LwSections(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p * 10), ("bytes", ctypes.c_uint64 * 10),
                ("coded_bytes", ctypes.c_uint64), ("n_tiles", ctypes.c_uint64),
                ("n_verbatim", ctypes.c_int64), ("max_tile_rows", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("min_len", ctypes.c_int32),
                ("palette_size", ctypes.c_int32), ("bits_per_weight", ctypes.c_double),
                ("lut_entries", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LwDevBundle(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("twin", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("max_tile_rows", ctypes.c_int32), ("lmin", ctypes.c_int32),
                ("lmax", ctypes.c_int32), ("lut_entries", ctypes.c_int32),
                ("words", ctypes.c_void_p), ("tile_off", ctypes.c_void_p),
                ("lane_bits", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("qparams", ctypes.c_void_p), ("signman", ctypes.c_void_p),
                ("vflags", ctypes.c_void_p), ("vrow_off", ctypes.c_void_p),
                ("vexp", ctypes.c_void_p), ("lane_mid", ctypes.c_void_p)]


class LwKvCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_KV_ROWS = struct.Struct("@Pqqii")                    # lw_kv_rows
_KV_ATTN = struct.Struct("@PqqPqqPPPPqqiiiiiiif")      # lw_kv_attn
_ROTARY = struct.Struct("@iidddddd")                  # lw_rotary
_KV_ROTATED = struct.Struct("@PqqiiPqqiiPqqiiPqqiiPPPqqiiii")   # lw_kv_rotated
_KV_WEIGHTS = struct.Struct("@PqqPPPPqqPqqPqqqiiiiiiif")        # lw_kv_weights
_KV_EVICTION = struct.Struct("@PqqqPPqPqPPqqqPiiiiii")          # lw_kv_eviction
_KV_SUMMARIES = struct.Struct("@PPPPqii")             # lw_kv_summaries
_KV_BLOCKS = struct.Struct("@PPiiii")                 # lw_kv_blocks


_lib = None


def load():
    """Load liblw.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"liblw is not built ({LIB_PATH} missing): run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "lw_encode_bundle": ([P, P, P, P, P], i32),
        "lw_bundle_sections": ([P, P], i32),
        "lw_bundle_free": ([P], None),
        "lw_table_from_lengths": ([i32, P, i32, P, i32, P], i32),
        "lw_validate_sections": ([P, P], i32),
        "lw_workspace_bytes": ([P, i32], sz),
        "lw_decode": ([P, P, P, P], i32),
        "lw_decode_gemv": ([P, P, P, P, sz, P, P], i32),
        "lw_decode_gemm": ([P, P, i32, P, P, sz, P, P], i32),
        "lw_twin_gemv": ([P, P, P, P, sz, P, P], i32),
        "lw_twin_gemm": ([P, P, i32, P, P, sz, P, P], i32),
        "lw_status_string": ([i32], ctypes.c_char_p),
        "lw_last_error": ([], ctypes.c_char_p),
        "lw_version": ([], i32),
        "lw_decode_gemv_noalloc": ([P, P, P, P, P], i32),
        "lw_decode_gemv_group": ([P, i32, P, P, P, sz, P, P], i32),
        "lw_twin_gemv_group": ([P, i32, P, P, P, sz, P, P], i32),
        "lw_decode_gemm_group": ([P, i32, P, i32, P, P, sz, P, P], i32),
        "lw_twin_gemm_group": ([P, i32, P, i32, P, P, sz, P, P], i32),
        "lw_workspace_bytes_group": ([P, i32], sz),
        "lw_noalloc_scratch_bytes": ([], sz),
        "lw_bundle_desc": ([P, P], i32),
        "lw_bundle_serialized_bytes": ([P], sz),
        "lw_bundle_serialize": ([P, P, sz], i32),
        "lw_bundle_deserialize": ([P, sz, P], i32),
        "lw_bundle_save": ([P, ctypes.c_char_p], i32),
        "lw_bundle_load": ([ctypes.c_char_p, P], i32),
        "lw_transcode_twin": ([P, P, P, P], i32),
        "lw_decode_gemm_strips": ([P, P, i32, P, i32, P, P, sz, P, P], i32),
        "lw_twin_tile_rows": ([i32], i32),
        "lw_graph_begin": ([P], i32),
        "lw_graph_end": ([P, P], i32),
        "lw_graph_launch": ([P, P], i32),
        "lw_graph_free": ([P], None),
        "lw_table_lut_entries": ([P], i32),
        "lw_test_stall_next": ([i32], i32),
        "lw_kv_tile_bytes": ([i32], sz),
        "lw_kv_page_bytes": ([i32, i32, i32], sz),
        "lw_kv_write": ([P, P, P, P, i64, P, P], i32),
        "lw_kv_read": ([P, P, i64, P, P, P, P], i32),
        "lw_kv_workspace_bytes": ([P, i32, i64, i32], sz),
        "lw_kv_attention": ([P, P, P, sz, P, P], i32),
        "lw_rotary_table": ([P, i64, i64, P, P], i32),
        "lw_kv_write_rotary": ([P, P, P, P], i32),
        "lw_kv_weigh_workspace_bytes": ([P, i32, i64], sz),
        "lw_kv_weigh": ([P, P, P, sz, P, P], i32),
        "lw_kv_evict": ([P, P, P, P], i32),
        "lw_kv_summary_bytes": ([P], sz),
        "lw_kv_summarise": ([P, P, P, P], i32),
        "lw_kv_blocks_workspace_bytes": ([P, i32, i64, i32, i32], sz),
        "lw_kv_attention_blocks": ([P, P, P, P, sz, P, P], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _last_error() -> str:
    try:
        return load().lw_last_error().decode()
    except Exception:  # noqa: BLE001
        return ""


def _check(st: int, what: str):
    if st != 0:
        raise LwError(st, what)


def _np_ptr(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


# ----------------------------------------------------------------------------
# host bundles
# ----------------------------------------------------------------------------

@dataclass
class BundleStats:
    coded_bytes: int
    n_tiles: int
    n_verbatim: int
    max_tile_rows: int
    max_len: int
    min_len: int
    palette_size: int
    bits_per_weight: float
    lut_entries: int = 0


class HostBundle:
    """Owns an lw_bundle*; `sections` are numpy copies of its sections."""

    def __init__(self, handle, desc: LwDesc):
        self._h = handle
        self.desc = desc
        s = LwSections()
        _check(load().lw_bundle_sections(self._h, ctypes.byref(s)), "lw_bundle_sections")
        self.stats = BundleStats(int(s.coded_bytes), int(s.n_tiles), int(s.n_verbatim),
                                 int(s.max_tile_rows), int(s.max_len), int(s.min_len),
                                 int(s.palette_size), float(s.bits_per_weight),
                                 int(s.lut_entries))
        self.sections = {}
        for i, name in enumerate(SECTION_NAMES):
            n = int(s.bytes[i])
            if n:
                buf = (ctypes.c_uint8 * n).from_address(s.ptr[i])
                self.sections[name] = np.frombuffer(buf, dtype=np.uint8).copy()
        self._raw = s

    @property
    def fmt(self):
        return self.desc.fmt

    @property
    def twin(self):
        return bool(self.desc.twin)

    def view(self, name, dtype):
        return self.sections[name].view(dtype)

    def __del__(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.lw_bundle_free(self._h)
            self._h = None


def lw_encode_bundle(fmt: int, payload: np.ndarray, scales=None, mins=None,
                     twin: bool = False) -> HostBundle:
    """payload: uint8 codes [N][K] or uint16 bf16 bits [N][K]."""
    payload = np.ascontiguousarray(payload)
    n, k = payload.shape
    desc = LwDesc(fmt, int(twin), n, k)
    sc = None if scales is None else np.ascontiguousarray(scales, dtype=np.uint16)
    mn = None if mins is None else np.ascontiguousarray(mins, dtype=np.uint16)
    h = ctypes.c_void_p()
    _check(load().lw_encode_bundle(ctypes.byref(desc), _np_ptr(payload), _np_ptr(sc),
                                   _np_ptr(mn), ctypes.byref(h)), "lw_encode_bundle")
    return HostBundle(h, desc)


def _adopt(h) -> HostBundle:
    """Wrap a bundle handle returned by the library."""
    desc = LwDesc()
    st = load().lw_bundle_desc(h, ctypes.byref(desc))
    if st != 0:
        load().lw_bundle_free(h)
        raise LwError(st, "lw_bundle_desc")
    return HostBundle(h, desc)


def lw_bundle_serialize(hb: HostBundle) -> bytes:
    """The bundle as one byte string (the bundle file format)."""
    n = int(load().lw_bundle_serialized_bytes(hb._h))
    buf = ctypes.create_string_buffer(n)
    _check(load().lw_bundle_serialize(hb._h, buf, n), "lw_bundle_serialize")
    return buf.raw


def lw_bundle_deserialize(data: bytes) -> HostBundle:
    h = ctypes.c_void_p()
    _check(load().lw_bundle_deserialize(data, len(data), ctypes.byref(h)), "lw_bundle_deserialize")
    return _adopt(h)


def lw_bundle_save(hb: HostBundle, path) -> None:
    _check(load().lw_bundle_save(hb._h, os.fsencode(path)), "lw_bundle_save")


def lw_bundle_load(path) -> HostBundle:
    h = ctypes.c_void_p()
    _check(load().lw_bundle_load(os.fsencode(path), ctypes.byref(h)), "lw_bundle_load")
    return _adopt(h)


def lw_table_from_lengths(fmt: int, code_len, palette=None) -> np.ndarray:
    cl = np.ascontiguousarray(code_len, dtype=np.uint8)
    pal = None if palette is None else np.ascontiguousarray(palette, dtype=np.uint8)
    out = np.zeros(TABLE_BYTES, dtype=np.uint8)
    _check(load().lw_table_from_lengths(fmt, _np_ptr(cl), len(cl), _np_ptr(pal),
                                        0 if pal is None else len(pal), _np_ptr(out)),
           "lw_table_from_lengths")
    return out


def lw_table_lut_entries(table: np.ndarray) -> int:
    """Entries of the compact decode table the table-driven kernel builds from
    this lw_table (the lut_entries hint of a device bundle)."""
    t = np.ascontiguousarray(table, dtype=np.uint8)
    if t.size != TABLE_BYTES:
        raise LwError(1, "lw_table_lut_entries", f"a table is {TABLE_BYTES} bytes, got {t.size}")
    return int(load().lw_table_lut_entries(_np_ptr(t)))


def lw_test_stall_next(wait_us: int) -> None:
    """Testing hook: the next table-driven product launch leaves one stage
    unfilled and limits its waits to `wait_us` microseconds (it reports
    LW_DEV_TIMEOUT and finishes)."""
    _check(load().lw_test_stall_next(int(wait_us)), "lw_test_stall_next")


def table_fields(table: np.ndarray) -> dict:
    """Decode the documented lw_table layout (for tests and reports)."""
    t = np.asarray(table, dtype=np.uint8)
    i32 = t[:32].view(np.int32)
    return dict(fmt=int(i32[0]), alpha=int(i32[1]), n_sym=int(i32[2]), lmin=int(i32[3]),
                lmax=int(i32[4]), n_palette=int(i32[5]), phantom=int(i32[6]),
                lim_m1=t[32:80].view(np.uint32).copy(), off=t[80:128].view(np.int32).copy(),
                sym=t[128:640].view(np.uint16).copy(), code_len=t[640:896].copy(),
                palette=t[896:912].copy())


def lw_validate_sections(fmt: int, rows: int, cols: int, sections: dict, max_tile_rows: int,
                         twin: bool = False) -> None:
    desc = LwDesc(fmt, int(twin), rows, cols)
    s = LwSections()
    keep = []
    for i, name in enumerate(SECTION_NAMES):
        a = sections.get(name)
        if a is not None and a.size:
            a = np.ascontiguousarray(a).view(np.uint8)
            keep.append(a)
            s.ptr[i] = a.ctypes.data
            s.bytes[i] = a.nbytes
    s.max_tile_rows = max_tile_rows
    _check(load().lw_validate_sections(ctypes.byref(desc), ctypes.byref(s)),
           "lw_validate_sections")


# ----------------------------------------------------------------------------
# device bundles (caller-owned device memory: torch tensors)
# ----------------------------------------------------------------------------

class DeviceBundle:
    """Byte-for-byte device copies of a bundle's sections plus the
    lw_dev_bundle view that the C calls take."""

    def __init__(self, fmt, twin, rows, cols, sections: dict, max_tile_rows, lmin, lmax,
                 device="cuda", coded_bytes=None, lut_entries=None):
        """lut_entries: the compact decode table's size (lw_sections); None
        computes it from the host table section (lw_table_lut_entries)."""
        import torch
        if lut_entries is None:
            tab = sections.get("table")
            lut_entries = (lw_table_lut_entries(np.ascontiguousarray(tab).view(np.uint8).reshape(-1))
                           if tab is not None and not twin else 0)
        self.fmt, self.twin, self.rows, self.cols = fmt, bool(twin), rows, cols
        self.tensors = {}
        for name in SECTION_NAMES:
            a = sections.get(name)
            if a is not None and a.size:
                host = torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).copy())
                self.tensors[name] = host.to(device)
        self.coded_bytes = int(coded_bytes if coded_bytes is not None else
                               sum(t.numel() for t in self.tensors.values()))
        v = LwDevBundle()
        v.fmt, v.twin, v.rows, v.cols = fmt, int(twin), rows, cols
        v.max_tile_rows, v.lmin, v.lmax, v.lut_entries = max_tile_rows, lmin, lmax, lut_entries
        for name in SECTION_NAMES:
            t = self.tensors.get(name)
            setattr(v, name, t.data_ptr() if t is not None else None)
        self.view = v

    @classmethod
    def from_tensors(cls, fmt, twin, rows, cols, tensors: dict, max_tile_rows, lmin, lmax,
                     lut_entries=0):
        """A view over device tensors that already hold the sections."""
        self = cls.__new__(cls)
        self.fmt, self.twin, self.rows, self.cols = fmt, bool(twin), rows, cols
        self.tensors = dict(tensors)
        self.coded_bytes = int(sum(t.numel() * t.element_size() for t in self.tensors.values()))
        v = LwDevBundle()
        v.fmt, v.twin, v.rows, v.cols = fmt, int(twin), rows, cols
        v.max_tile_rows, v.lmin, v.lmax, v.lut_entries = max_tile_rows, lmin, lmax, lut_entries
        for name in SECTION_NAMES:
            t = self.tensors.get(name)
            setattr(v, name, t.data_ptr() if t is not None else None)
        self.view = v
        return self

    @classmethod
    def upload(cls, hb: HostBundle, device="cuda"):
        return cls(hb.desc.fmt, hb.desc.twin, hb.desc.rows, hb.desc.cols, hb.sections,
                   hb.stats.max_tile_rows, hb.stats.min_len, hb.stats.max_len, device,
                   hb.stats.coded_bytes, hb.stats.lut_entries)

    @property
    def ref(self):
        return ctypes.byref(self.view)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _tp(t):
    """A tensor's address, unchecked (for callers that drive the C functions
    directly and check their buffers themselves)."""
    return ctypes.c_void_p(t.data_ptr())


# ----------------------------------------------------------------------------
# device buffers, checked before their addresses cross the C ABI
# ----------------------------------------------------------------------------
# The C calls take bare device addresses: they cannot tell how large a buffer
# is, whether it lives on the device or how it is strided.  A tensor that is
# too small, on the host or strided would let a kernel read or write outside
# it, so every tensor is checked here first (LW_ERR_INVALID_ARG, nothing
# launched).  Sizes follow the view's shape; a shape the library refuses
# anyway (not a multiple of 64 x 256) is left for it to report.

def _refuse(fn: str, detail: str):
    raise LwError(LW_ERR_INVALID_ARG, fn, detail)


def _buf(fn: str, name: str, t, nbytes: int, dtypes=None):
    """Address of tensor `t` after checking that it is a torch.Tensor of one
    of `dtypes` (any if None), contiguous and at least `nbytes` bytes.  Its
    device is checked afterwards (_on), once every buffer has passed."""
    import torch
    if not isinstance(t, torch.Tensor):
        _refuse(fn, f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtypes is not None and t.dtype not in dtypes:
        want = ", ".join(str(d).replace("torch.", "") for d in dtypes)
        _refuse(fn, f"{name}: dtype {str(t.dtype).replace('torch.', '')}, expected {want}")
    if not t.is_contiguous():
        _refuse(fn, f"{name}: not contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        _refuse(fn, f"{name}: {have} bytes, the call needs {nbytes}")
    return ctypes.c_void_p(t.data_ptr())


def _bundle_device(fn: str, db, name: str = "bundle"):
    """The one CUDA device holding every section tensor of `db`."""
    devs = {t.device for t in db.tensors.values()}
    if len(devs) != 1:
        _refuse(fn, f"{name}: sections on {sorted(map(str, devs)) or 'no device'}, "
                    "expected one CUDA device")
    dev = devs.pop()
    if dev.type != "cuda":
        _refuse(fn, f"{name}: sections on {dev}, expected a CUDA device")
    if not all(t.is_contiguous() for t in db.tensors.values()):
        _refuse(fn, f"{name}: a section tensor is not contiguous")
    return dev


def _on(fn: str, dev, *named):
    """Every (name, tensor) pair is on the bundle's device `dev`."""
    for name, t in named:
        if t.device.type != "cuda":
            _refuse(fn, f"{name}: on {t.device}, expected a CUDA device")
        if t.device != dev:
            _refuse(fn, f"{name}: on {t.device}, the bundle is on {dev}")


def _dims(db):
    """(N, K) of the view when the library accepts that shape, else (0, 0)."""
    n, k = int(db.view.rows), int(db.view.cols)
    return (n, k) if n > 0 and k > 0 and n % 64 == 0 and k % 256 == 0 else (0, 0)


def _act_types(fmt: int):
    """Activation dtypes and element size of a format (fp32; BF16 as
    bfloat16 or its bits)."""
    import torch
    if fmt == LW_FMT_BF16_EXP:
        return (torch.bfloat16, torch.int16) + ((torch.uint16,) if hasattr(torch, "uint16") else ()), 2
    if fmt in (LW_FMT_Q4_PAIR, LW_FMT_Q6):
        return (torch.float32,), 4
    return None, 0


def _decoded_bytes(fmt: int, n: int, k: int) -> int:
    """Bytes lw_decode writes: packed pairs (4-bit), one byte per code
    (6-bit), BF16 bits."""
    return {LW_FMT_Q4_PAIR: n * k // 2, LW_FMT_Q6: n * k, LW_FMT_BF16_EXP: 2 * n * k}.get(fmt, 0)


def _status_ptr(fn: str, d_status):
    import torch
    return _buf(fn, "d_status", d_status, 4, (torch.int32,))


def _ws_ptr(fn: str, ws):
    return _buf(fn, "ws", ws, 0), ctypes.c_size_t(ws.numel() * ws.element_size())


def _product_bufs(fn: str, db, x, y, batch: int, xname="x", yname="y"):
    """Checked addresses of one matrix's activations [batch][K] and outputs
    fp32 [batch][N] (devices not yet checked)."""
    import torch
    n, k = _dims(db)
    b = max(int(batch), 0)
    types, esize = _act_types(int(db.view.fmt))
    return (_buf(fn, xname, x, b * k * esize, types),
            _buf(fn, yname, y, b * n * 4, (torch.float32,)))


def _checked(fn: str, dbs, xs, ys, batch: int, ws, d_status, names=("x", "y"), indexed=False,
             extra=()):
    """Check a product call's buffers in two passes -- first every buffer's
    type, dtype, layout and size, then that the bundles and every buffer sit
    on one CUDA device -- and return the addresses: (x list, y list, ws,
    ws bytes, d_status).  `extra`: further (name, tensor) pairs whose device
    is checked."""
    n = len(dbs)
    if n < 1 or len(xs) != n or len(ys) != n:
        _refuse(fn, f"{n} bundles, {len(xs)} activations, {len(ys)} outputs")
    label = (lambda i: (f"{names[0]}[{i}]", f"{names[1]}[{i}]")) if indexed else (lambda i: names)
    bufs = [_product_bufs(fn, d, x, y, batch, *label(i)) for i, (d, x, y) in enumerate(zip(dbs, xs, ys))]
    wp, wb = _ws_ptr(fn, ws) if ws is not None else (None, None)
    sp = _status_ptr(fn, d_status)
    dev = _bundle_device(fn, dbs[0], "bundle[0]" if indexed else "bundle")
    for i in range(1, n):
        if _bundle_device(fn, dbs[i], f"bundle[{i}]") != dev:
            _refuse(fn, f"bundle[{i}]: not on {dev} like bundle[0]")
    named = [p for i in range(n) for p in zip(label(i), (xs[i], ys[i]))]
    _on(fn, dev, *named, *((("ws", ws),) if ws is not None else ()), ("d_status", d_status), *extra)
    return [b[0] for b in bufs], [b[1] for b in bufs], wp, wb, sp


def lw_workspace_bytes(db: DeviceBundle, batch: int = 1) -> int:
    return int(load().lw_workspace_bytes(db.ref, batch))


def lw_decode(db: DeviceBundle, out, d_status, stream=None) -> None:
    fn = "lw_decode"
    n, k = _dims(db)
    o = _buf(fn, "out", out, _decoded_bytes(int(db.view.fmt), n, k))
    sp = _status_ptr(fn, d_status)
    _on(fn, _bundle_device(fn, db), ("out", out), ("d_status", d_status))
    _check(load().lw_decode(db.ref, o, sp, _stream_ptr(stream)), fn)


def lw_decode_gemm_strips(db: DeviceBundle, strips, X, batch, Y, ws, d_status, stream=None) -> None:
    """Y = W X on the 64-row strips listed in `strips` (device int32 tensor,
    ascending); the other rows of Y are left as they are."""
    import torch
    fn = "lw_decode_gemm_strips"
    n = int(strips.numel()) if strips is not None else 0
    lp = _buf(fn, "strips", strips, 4 * n, (torch.int32,)) if n else None
    (xp,), (yp,), wp, wb, sp = _checked(fn, [db], [X], [Y], batch, ws, d_status, ("X", "Y"),
                                        extra=(("strips", strips),) if n else ())
    _check(load().lw_decode_gemm_strips(db.ref, lp, n, xp, batch, yp, wp, wb, sp,
                                        _stream_ptr(stream)), fn)


class PreparedGemv:
    """lw_decode_gemv (one matrix) or lw_decode_gemv_group (several) -- or
    their twins -- with the arguments marshalled once, for calls repeated
    every step: each call() is one C call.  The tensors must stay alive and
    in place."""

    def __init__(self, dbs, xs, ys, ws, d_status, twin: bool = False):
        lib = load()
        fn = "PreparedGemv"
        self._keep = (list(dbs), list(xs), list(ys), ws, d_status)
        n = len(dbs)
        xps, yps, self._ws, self._wsb, self._st = _checked(fn, dbs, xs, ys, 1, ws, d_status,
                                                           indexed=True)
        if n == 1:
            self._fn = lib.lw_twin_gemv if twin else lib.lw_decode_gemv
            self._args = (dbs[0].ref, xps[0], yps[0])
        else:
            self._fn = lib.lw_twin_gemv_group if twin else lib.lw_decode_gemv_group
            self._views = _views(dbs)
            self._xa = (ctypes.c_void_p * n)(*xps)
            self._ya = (ctypes.c_void_p * n)(*yps)
            self._args = (self._views, n, self._xa, self._ya)

    def __call__(self, stream=None) -> None:
        _check(self._fn(*self._args, self._ws, self._wsb, self._st, _stream_ptr(stream)),
               "prepared gemv")


class StepGraph:
    """Library calls captured once on a stream and replayed as one CUDA
    graph (lw_graph_begin / lw_graph_end / lw_graph_launch).  Use as
        g = StepGraph(stream)
        with g.capture():
            ...library calls on `stream` (e.g. with torch.cuda.stream(stream))...
        g.launch()"""

    def __init__(self, stream):
        self.stream = stream
        self._h = ctypes.c_void_p()

    def capture(self):
        import contextlib
        import torch

        @contextlib.contextmanager
        def cm():
            with torch.cuda.stream(self.stream):
                _check(load().lw_graph_begin(_stream_ptr(self.stream)), "lw_graph_begin")
                try:
                    yield self
                finally:
                    _check(load().lw_graph_end(_stream_ptr(self.stream), ctypes.byref(self._h)),
                           "lw_graph_end")
        return cm()

    def launch(self, stream=None) -> None:
        _check(load().lw_graph_launch(self._h, _stream_ptr(stream if stream is not None else self.stream)),
               "lw_graph_launch")

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.lw_graph_free(self._h)
            self._h = ctypes.c_void_p()


def lw_twin_tile_rows(fmt: int) -> int:
    return int(load().lw_twin_tile_rows(fmt))


def lw_transcode_twin(db: DeviceBundle, d_status, stream=None) -> DeviceBundle:
    """Transcode a coded device bundle into its fixed-width twin on the
    device: new words, tile offsets and lane bit counts; every other section
    is the coded bundle's own tensor (shared, not copied)."""
    import torch
    dev = db.tensors["tile_off"].device
    n_tiles = (db.rows // 64) * (db.cols // 256)
    r2 = lw_twin_tile_rows(db.fmt)
    t = {"words": torch.empty(n_tiles * r2 * 128, dtype=torch.uint8, device=dev),
         "tile_off": torch.empty((n_tiles + 1) * 4, dtype=torch.uint8, device=dev),
         "lane_bits": torch.empty(n_tiles * 64, dtype=torch.uint8, device=dev)}
    for name in ("table", "qparams", "signman", "vflags", "vrow_off", "vexp"):
        if name in db.tensors:
            t[name] = db.tensors[name]
    tw = DeviceBundle.from_tensors(db.fmt, True, db.rows, db.cols, t, r2, 0, 0)
    fn = "lw_transcode_twin"
    sp = _status_ptr(fn, d_status)
    _on(fn, _bundle_device(fn, db), ("d_status", d_status))
    _check(load().lw_transcode_twin(db.ref, tw.ref, sp, _stream_ptr(stream)), fn)
    return tw


def _gemv(fn, db, x, y, ws, d_status, stream):
    (xp,), (yp,), wp, wb, sp = _checked(fn, [db], [x], [y], 1, ws, d_status)
    _check(getattr(load(), fn)(db.ref, xp, yp, wp, wb, sp, _stream_ptr(stream)), fn)


def _gemm(fn, db, X, batch, Y, ws, d_status, stream):
    (xp,), (yp,), wp, wb, sp = _checked(fn, [db], [X], [Y], batch, ws, d_status, ("X", "Y"))
    _check(getattr(load(), fn)(db.ref, xp, batch, yp, wp, wb, sp, _stream_ptr(stream)), fn)


def lw_decode_gemv(db: DeviceBundle, x, y, ws, d_status, stream=None) -> None:
    _gemv("lw_decode_gemv", db, x, y, ws, d_status, stream)


def lw_decode_gemm(db: DeviceBundle, X, batch, Y, ws, d_status, stream=None) -> None:
    _gemm("lw_decode_gemm", db, X, batch, Y, ws, d_status, stream)


def lw_twin_gemv(db: DeviceBundle, x, y, ws, d_status, stream=None) -> None:
    _gemv("lw_twin_gemv", db, x, y, ws, d_status, stream)


def lw_twin_gemm(db: DeviceBundle, X, batch, Y, ws, d_status, stream=None) -> None:
    _gemm("lw_twin_gemm", db, X, batch, Y, ws, d_status, stream)


def lw_decode_gemv_noalloc(db: DeviceBundle, x, y, d_status, stream=None) -> None:
    """lw_decode_gemv with the library's fixed device scratch instead of a
    caller workspace (allocates nothing)."""
    fn = "lw_decode_gemv_noalloc"
    (xp,), (yp,), _, _, sp = _checked(fn, [db], [x], [y], 1, None, d_status)
    _check(load().lw_decode_gemv_noalloc(db.ref, xp, yp, sp, _stream_ptr(stream)), fn)


def _views(dbs):
    arr = (ctypes.c_void_p * len(dbs))(*[ctypes.addressof(d.view) for d in dbs])
    return arr


def lw_workspace_bytes_group(dbs) -> int:
    return int(load().lw_workspace_bytes_group(_views(dbs), len(dbs)))


def _gemv_group(fn, dbs, xs, ys, ws, d_status, stream):
    xps, yps, wp, wb, sp = _checked(fn, dbs, xs, ys, 1, ws, d_status, indexed=True)
    n = len(dbs)
    xa, ya = (ctypes.c_void_p * n)(*xps), (ctypes.c_void_p * n)(*yps)
    _check(getattr(load(), fn)(_views(dbs), n, xa, ya, wp, wb, sp, _stream_ptr(stream)), fn)


def _gemm_group(fn, dbs, Xs, batch, Ys, ws, d_status, stream):
    xps, yps, wp, wb, sp = _checked(fn, dbs, Xs, Ys, batch, ws, d_status, indexed=True)
    n = len(dbs)
    xa, ya = (ctypes.c_void_p * n)(*xps), (ctypes.c_void_p * n)(*yps)
    _check(getattr(load(), fn)(_views(dbs), n, xa, batch, ya, wp, wb, sp, _stream_ptr(stream)), fn)


def lw_decode_gemm_group(dbs, Xs, batch, Ys, ws, d_status, stream=None) -> None:
    """One launch for several 4-/6-bit matrices, batch 1..8: Ys[i] = Xs[i] W_i^T."""
    _gemm_group("lw_decode_gemm_group", dbs, Xs, batch, Ys, ws, d_status, stream)


def lw_twin_gemm_group(dbs, Xs, batch, Ys, ws, d_status, stream=None) -> None:
    _gemm_group("lw_twin_gemm_group", dbs, Xs, batch, Ys, ws, d_status, stream)


def lw_decode_gemv_group(dbs, xs, ys, ws, d_status, stream=None) -> None:
    """One launch for several 4-/6-bit matrices: ys[i] = W_i xs[i]."""
    _gemv_group("lw_decode_gemv_group", dbs, xs, ys, ws, d_status, stream)


def lw_twin_gemv_group(dbs, xs, ys, ws, d_status, stream=None) -> None:
    """The fixed-width twin of lw_decode_gemv_group."""
    _gemv_group("lw_twin_gemv_group", dbs, xs, ys, ws, d_status, stream)


def lw_noalloc_scratch_bytes() -> int:
    return int(load().lw_noalloc_scratch_bytes())


# ----------------------------------------------------------------------------
# the 4-bit key/value cache
# ----------------------------------------------------------------------------

# These calls run once a layer and step, so their checks are written twice: one
# expression that a right call passes (a few microseconds), and, where it does
# not hold, the checks one by one, which say what is wrong.

class KvCache:
    """Pages of the 4-bit key/value cache (the layout of lw_kv_cache in
    include/lw.h) in a caller-owned tensor: any dtype and shape, contiguous,
    a whole number of pages."""

    def __init__(self, pages, kv_heads: int, head_dim: int, page_tokens: int):
        import torch
        fn = "KvCache"
        _kv_torch(torch)
        self.kv_heads, self.head_dim, self.page_tokens = int(kv_heads), int(head_dim), int(page_tokens)
        size = lw_kv_page_bytes(self.kv_heads, self.head_dim, self.page_tokens)
        if not size:
            _refuse(fn, f"{kv_heads} heads of {head_dim} values, pages of {page_tokens} tokens: head_dim "
                        f"is 64, 96 or 128, page_tokens a positive multiple of {LW_KV_TILE}")
        ptr = _buf(fn, "pages", pages, size)
        have = pages.numel() * pages.element_size()
        if have % size:
            _refuse(fn, f"pages: {have} bytes, not a multiple of the page size {size}")
        self.pages, self.device, self.n_pages = pages, pages.device, have // size
        self.index = pages.get_device()   # -1: not on a CUDA device, which the calls refuse
        self.view = LwKvCache(ptr, self.n_pages, self.kv_heads, self.head_dim, self.page_tokens, 0)
        self.ref = ctypes.byref(self.view)
        self.summary_bytes = int(load().lw_kv_summary_bytes(self.ref))

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, page_tokens: int, device="cuda"):
        """A cache in new memory, not initialised (keys past a sequence's
        length are never used)."""
        import torch
        size = lw_kv_page_bytes(kv_heads, head_dim, page_tokens)
        return cls(torch.empty(max(int(n_pages), 0) * size, dtype=torch.uint8, device=device),
                   kv_heads, head_dim, page_tokens)


def lw_kv_tile_bytes(head_dim: int) -> int:
    return int(load().lw_kv_tile_bytes(head_dim))


def lw_kv_page_bytes(kv_heads: int, head_dim: int, page_tokens: int) -> int:
    return int(load().lw_kv_page_bytes(kv_heads, head_dim, page_tokens))


def lw_kv_workspace_bytes(cache: KvCache, q_heads: int, q_tokens: int, batch: int) -> int:
    if cache.index >= 0 and _current_device() != cache.index:   # (sized by the current device)
        _kv_on("lw_kv_workspace_bytes", cache)
    return int(load().lw_kv_workspace_bytes(cache.ref, q_heads, q_tokens, batch))


_KV_TYPES = {}          # torch dtype -> lw_dtype
_I32 = _I64 = _F32 = None
_raw_stream = None      # device index -> its current stream's handle
_current_device = None  # () -> index of the current device, which the library launches on


def _kv_torch(torch):
    global _I32, _I64, _F32, _raw_stream, _current_device
    if _KV_TYPES:
        return
    _I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _KV_TYPES.update({torch.float32: LW_F32, torch.float16: LW_F16, torch.bfloat16: LW_BF16})


def _kv_distinct(t) -> bool:
    """Whether the rows [tokens][heads][dim] of `t` share no element."""
    (n, h, d), (st, sh, _) = t.shape, t.stride()
    if n == 0:
        return True
    if h == 1 or n == 1:
        return (n == 1 or st >= d) and (h == 1 or sh >= d)
    return (sh >= d and st >= (h - 1) * sh + d) or (st >= d and sh >= (n - 1) * st + d)


def _kv_apart(k, v) -> bool:
    """Whether the rows [tokens][heads][dim] of `k` and `v` (one shape and type, the last
    dimension contiguous) share no byte."""
    n, h, d = k.shape
    if n == 0 or h == 0:
        return True
    size, at, bt = k.element_size(), k.data_ptr(), v.data_ptr()
    (kt, kh, _), (vt, vh, _) = k.stride(), v.stride()
    row = d * size
    kspan, vspan = (n - 1) * kt + (h - 1) * kh, (n - 1) * vt + (h - 1) * vh
    if at + kspan * size + row <= bt or bt + vspan * size + row <= at:
        return True
    if kt == vt and kh == vh:   # interleaved in one buffer: a token's heads, then the other's, or head by head
        apart, heads = abs(bt - at), (h - 1) * kh * size + row
        if heads <= apart <= kt * size - heads or (row <= apart <= kh * size - row and apart + heads <= kt * size):
            return True
    starts = np.sort(np.concatenate([
        (p + size * (np.arange(n)[:, None] * t + np.arange(h) * s)).ravel()
        for p, t, s in ((at, kt, kh), (bt, vt, vh))]))
    return bool((np.diff(starts) >= row).all())


def _kv_heads(fn: str, name: str, t, tokens, heads, dim, written=False):
    """Refuse anything but rows of heads [tokens][heads][dim]."""
    import torch
    if not isinstance(t, torch.Tensor):
        _refuse(fn, f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _KV_TYPES:
        _refuse(fn, f"{name}: dtype {str(t.dtype).replace('torch.', '')}, expected float32, float16 "
                    "or bfloat16")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or \
            (tokens is not None and t.shape[0] != tokens):
        want = f"[{'tokens' if tokens is None else tokens}, {heads}, {dim}]"
        _refuse(fn, f"{name}: shape {list(t.shape)}, expected {want}")
    if t.numel() and t.stride(2) != 1:
        _refuse(fn, f"{name}: the last dimension is strided")
    if written and not _kv_distinct(t):
        _refuse(fn, f"{name}: rows that are written overlap")


def _kv_index(fn: str, name: str, t, dtype, n):
    """Refuse anything but a contiguous index vector of n entries."""
    import torch
    if not isinstance(t, torch.Tensor):
        _refuse(fn, f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        _refuse(fn, f"{name}: dtype {str(t.dtype).replace('torch.', '')}, expected "
                    f"{str(dtype).replace('torch.', '')}")
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        _refuse(fn, f"{name}: expected a contiguous vector" + ("" if n is None else f" of {n} entries"))


def _kv_on(fn: str, cache: KvCache, *named):
    if cache.index < 0:
        _refuse(fn, f"cache: pages on {cache.device}, expected a CUDA device")
    if _current_device() != cache.index:
        _refuse(fn, f"cache: pages on {cache.device}, the current device is cuda:{_current_device()}")
    for name, t in named:
        if t.device != cache.device:
            _refuse(fn, f"{name}: on {t.device}, the cache is on {cache.device}")


def _kv_rows_refuse(fn, cache, slots, k, v, d_status, written):
    _kv_index(fn, "slots", slots, _I64, None)
    for name, t in (("k", k), ("v", v)):
        _kv_heads(fn, name, t, slots.shape[0], cache.kv_heads, cache.head_dim, written)
    if k.dtype != v.dtype:
        _refuse(fn, f"v: dtype {v.dtype}, k has {k.dtype}")
    if written and not _kv_apart(k, v):
        _refuse(fn, "v: rows that are written overlap k's")
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, ("slots", slots), ("k", k), ("v", v), ("d_status", d_status))


def _kv_rows(fn, cache, slots, k, v, d_status, written):
    """The checked calls' arguments: slots, count, rows of k and v, status."""
    dev = cache.index
    try:
        n = slots.shape[0]
        shape = (n, cache.kv_heads, cache.head_dim)
        code, (kt, kh, kd), (vt, vh, vd) = _KV_TYPES.get(k.dtype), k.stride(), v.stride()
        ok = (code is not None and v.dtype is k.dtype and k.shape == shape and v.shape == shape
              and kd == 1 and vd == 1 and slots.dtype is _I64 and slots.dim() == 1
              and slots.is_contiguous() and d_status.dtype is _I32 and d_status.numel() >= 1
              and d_status.is_contiguous() and dev >= 0 and _current_device() == dev and k.get_device() == dev
              and v.get_device() == dev and slots.get_device() == dev and d_status.get_device() == dev
              and (not written or (_kv_distinct(k) and _kv_distinct(v) and _kv_apart(k, v))))
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        _kv_rows_refuse(fn, cache, slots, k, v, d_status, written)
        code, (kt, kh, kd), (vt, vh, vd) = _KV_TYPES[k.dtype], k.stride(), v.stride()
    return (slots.data_ptr(), n, _KV_ROWS.pack(k.data_ptr(), kt, kh, code, 0),
            _KV_ROWS.pack(v.data_ptr(), vt, vh, code, 0), d_status.data_ptr())


def lw_kv_write(cache: KvCache, k, v, slots, d_status, stream=None) -> None:
    """Quantise k, v [n, kv_heads, head_dim] (one dtype; the last dimension
    contiguous) into the slots int64 [n]; a negative slot is not stored."""
    sp, n, kr, vr, st = _kv_rows("lw_kv_write", cache, slots, k, v, d_status, False)
    r = _lib.lw_kv_write(cache.ref, kr, vr, sp, n, st,
                         _raw_stream(cache.index) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, "lw_kv_write")


def lw_kv_read(cache: KvCache, slots, k, v, d_status, stream=None) -> None:
    """Read the slots back into k, v [n, kv_heads, head_dim]; a negative slot
    reads as zeros."""
    sp, n, kr, vr, st = _kv_rows("lw_kv_read", cache, slots, k, v, d_status, True)
    r = _lib.lw_kv_read(cache.ref, sp, n, kr, vr, st,
                        _raw_stream(cache.index) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, "lw_kv_read")


def _kv_attention_refuse(cache, q, q_start, kv_len, page_table, out, ws, d_status, lse, max_q):
    import operator
    import torch
    fn = "lw_kv_attention"
    try:
        operator.index(max_q)
    except TypeError:
        _refuse(fn, f"max_q: expected a whole number, got {max_q!r}")
    heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    if isinstance(q, torch.Tensor) and (heads < 1 or heads % cache.kv_heads):
        _refuse(fn, f"q: shape {list(q.shape)}, expected [tokens, a multiple of {cache.kv_heads}, "
                    f"{cache.head_dim}]")
    _kv_heads(fn, "q", q, None, heads, cache.head_dim)
    _kv_heads(fn, "out", out, q.shape[0], heads, cache.head_dim, True)
    if out.dtype != q.dtype:
        _refuse(fn, f"out: dtype {out.dtype}, q has {q.dtype}")
    _kv_index(fn, "kv_len", kv_len, _I32, None)
    batch = kv_len.shape[0]
    _kv_index(fn, "q_start", q_start, _I32, batch + 1)
    if not isinstance(page_table, torch.Tensor) or page_table.dtype != torch.int32:
        _refuse(fn, "page_table: expected an int32 tensor")
    if page_table.dim() != 2 or page_table.shape[0] != batch or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        _refuse(fn, f"page_table: expected [{batch}, pages] with contiguous rows")
    named = (("q", q), ("out", out), ("q_start", q_start), ("kv_len", kv_len),
             ("page_table", page_table), ("ws", ws), ("d_status", d_status))
    if lse is not None:
        _buf(fn, "lse", lse, 4 * q.shape[0] * heads, (torch.float32,))
        named += (("lse", lse),)
    _ws_ptr(fn, ws)
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, *named)


def lw_kv_attention(cache: KvCache, q, q_start, kv_len, page_table, out, ws, d_status, *,
                    max_q: int, scale=None, causal: bool = True, window: int = 0, lse=None,
                    stream=None) -> None:
    """Attention of the packed query tokens q [tokens, q_heads, head_dim] over
    the cache: sequence b owns tokens q_start[b]..q_start[b+1]-1 and kv_len[b]
    keys in the pages page_table[b]; out as q, lse float32 [tokens, q_heads].
    scale: 1 / sqrt(head_dim) by default."""
    dev = cache.index
    try:
        tokens, heads, dim = shape = q.shape
        code, (qt, qh, qd), (ot, oh, od) = _KV_TYPES.get(q.dtype), q.stride(), out.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
        ok = (code is not None and out.dtype is q.dtype and out.shape == shape
              and dim == cache.head_dim and heads % cache.kv_heads == 0 and qd == 1 and od == 1
              and heads > 0 and (out.is_contiguous() or _kv_distinct(out))
              and q_start.dtype is _I32 and q_start.shape == (batch + 1,) and q_start.is_contiguous()
              and kv_len.dtype is _I32 and kv_len.shape == (batch,) and kv_len.is_contiguous()
              and page_table.dtype is _I32 and (td == 1 or width <= 1)
              and ws.is_contiguous() and d_status.dtype is _I32 and d_status.numel() >= 1
              and d_status.is_contiguous() and type(max_q) is int and dev >= 0 and _current_device() == dev
              and q.get_device() == dev
              and out.get_device() == dev and q_start.get_device() == dev
              and kv_len.get_device() == dev and page_table.get_device() == dev
              and ws.get_device() == dev and d_status.get_device() == dev
              and (lse is None or (lse.dtype is _F32 and lse.is_contiguous()
                                   and lse.numel() >= tokens * heads and lse.get_device() == dev)))
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        _kv_attention_refuse(cache, q, q_start, kv_len, page_table, out, ws, d_status, lse, max_q)
        tokens, heads, dim = q.shape
        code, (qt, qh, qd), (ot, oh, od) = _KV_TYPES[q.dtype], q.stride(), out.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
    try:
        a = _KV_ATTN.pack(q.data_ptr(), qt, qh, out.data_ptr(), ot, oh,
                          0 if lse is None else lse.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                          page_table.data_ptr(), ts, tokens, width, code, batch, heads, max_q,
                          1 if causal else 0, window, dim ** -0.5 if scale is None else scale)
    except struct.error as e:
        _refuse("lw_kv_attention", f"max_q {max_q!r}, window {window!r}, scale {scale!r}: {e}")
    r = _lib.lw_kv_attention(cache.ref, a, ws.data_ptr(), ws.numel() * ws.element_size(),
                             d_status.data_ptr(),
                             _raw_stream(cache.index) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, "lw_kv_attention")


# ---- rotary positions --------------------------------------------------------

def lw_rotary_table(table, *, first: int = 0, base: float = 10000.0, scaling: int = LW_ROTARY_PLAIN,
                    factor: float = 1.0, old_length: float = 0.0, low: float = 0.0, high: float = 0.0,
                    gain: float = 0.0, stream=None) -> None:
    """Fill table float32 [positions, rot] with the cosines and sines of positions first,
    first + 1, ...: what lw_kv_write_rotary rotates by."""
    import torch
    fn = "lw_rotary_table"
    _kv_torch(torch)
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or table.dim() != 2 or \
            not table.is_contiguous():
        _refuse(fn, "table: expected a contiguous float32 tensor [positions, rot]")
    if table.get_device() < 0 or table.get_device() != _current_device():
        _refuse(fn, f"table: on {table.device}, expected the current CUDA device")
    try:
        a = _ROTARY.pack(table.shape[1], scaling, base, factor, old_length, low, high, gain)
    except struct.error as e:
        _refuse(fn, f"rot {table.shape[1]}, scaling {scaling!r}, base {base!r}, factor {factor!r}, old_length "
                    f"{old_length!r}, low {low!r}, high {high!r}, gain {gain!r}: {e}")
    _kv_whole(fn, first=first)
    if not -1 << 63 <= first < 1 << 63:
        _refuse(fn, f"first: {first} is out of range")
    r = load().lw_rotary_table(a, first, table.shape[0], table.data_ptr(),
                               _raw_stream(table.get_device()) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, fn)


def _kv_beside(a, b) -> bool:
    """Whether the rows [tokens][heads][dim] of `a` and `b` (one type, the last dimension contiguous; as many
    tokens, any heads) share no byte."""
    (n, ha, d), (_, hb, e) = a.shape, b.shape
    if n == 0 or ha == 0 or hb == 0:
        return True
    if ha == hb and d == e:
        return _kv_apart(a, b)
    size, at, bt = a.element_size(), a.data_ptr(), b.data_ptr()
    (sa, ga, _), (sb, gb, _) = a.stride(), b.stride()
    heads_a, heads_b = ((ha - 1) * ga + d) * size, ((hb - 1) * gb + e) * size   # of a token
    if at + (n - 1) * sa * size + heads_a <= bt or bt + (n - 1) * sb * size + heads_b <= at:
        return True
    if sa == sb and sa > 0:   # interleaved in one buffer, token by token
        apart = (bt - at) % (sa * size)
        if heads_a <= apart and apart + heads_b <= sa * size:
            return True
    rows = [(p + size * (np.arange(n)[:, None] * t + np.arange(h) * g)).ravel()
            for p, t, h, g in ((at, sa, ha, ga), (bt, sb, hb, gb))]
    start = np.concatenate(rows)
    end = start + np.repeat([d * size, e * size], [len(rows[0]), len(rows[1])])
    order = np.argsort(start, kind="stable")
    return bool((start[order][1:] >= end[order][:-1]).all())


def _kv_same_rows(a, b) -> bool:
    return a.data_ptr() == b.data_ptr() and a.stride() == b.stride()


def _kv_written_beside(q_out, qp, k, v) -> bool:
    """A quick yes to what the usual call needs: q_out's rows are distinct, are q's (at `qp`, of q_out's strides) or
    share no byte with them, and share none with k's and v's."""
    if q_out.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        at, n = q_out.data_ptr(), q_out.nbytes
        kp, vp, kn = k.data_ptr(), v.data_ptr(), k.nbytes
        return ((at == qp or at + n <= qp or qp + n <= at) and (at + n <= kp or kp + kn <= at)
                and (at + n <= vp or vp + kn <= at))
    return False


def _kv_rotary_refuse(fn, cache, k, v, slots, positions, table, d_status, q, q_out):
    import torch
    _kv_index(fn, "slots", slots, _I64, None)
    n = slots.shape[0]
    _kv_index(fn, "positions", positions, _I64, n)
    for name, t in (("k", k), ("v", v)):
        _kv_heads(fn, name, t, n, cache.kv_heads, cache.head_dim)
    if k.dtype != v.dtype:
        _refuse(fn, f"v: dtype {v.dtype}, k has {k.dtype}")
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or table.dim() != 2 or \
            not table.is_contiguous():
        _refuse(fn, "table: expected a contiguous float32 tensor [positions, rot]")
    named = (("slots", slots), ("positions", positions), ("k", k), ("v", v), ("table", table),
             ("d_status", d_status))
    if (q is None) != (q_out is None):
        _refuse(fn, "q and q_out come together")
    if q is not None:
        heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        if isinstance(q, torch.Tensor) and heads < 1:
            _refuse(fn, f"q: shape {list(q.shape)}, expected [{n}, heads, {cache.head_dim}]")
        _kv_heads(fn, "q", q, n, heads, cache.head_dim)
        _kv_heads(fn, "q_out", q_out, n, heads, cache.head_dim, True)
        if q.dtype != k.dtype or q_out.dtype != q.dtype:
            _refuse(fn, f"q, q_out: dtypes {q.dtype}, {q_out.dtype}, k has {k.dtype}")
        if not (_kv_same_rows(q, q_out) or _kv_apart(q, q_out)):
            _refuse(fn, "q_out: rows that are written overlap q's (it may be q itself)")
        for name, t in (("k", k), ("v", v)):
            if not _kv_beside(q_out, t):
                _refuse(fn, f"q_out: rows that are written overlap {name}'s")
        named += (("q", q), ("q_out", q_out))
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, *named)


def lw_kv_write_rotary(cache: KvCache, k, v, slots, positions, table, d_status, *, q=None, q_out=None,
                       interleaved: bool = False, stream=None) -> None:
    """lw_kv_write of keys rotated by their tokens' positions int64 [n], and the queries
    q [n, q_heads, head_dim] of the same tokens rotated into q_out (which may be q).  table float32
    [positions, rot] (lw_rotary_table): the first rot elements of a head are rotated, in pairs of
    neighbours (interleaved) or of elements rot / 2 apart."""
    dev = cache.index
    try:
        n = slots.shape[0]
        shape = (n, cache.kv_heads, cache.head_dim)
        code, (kt, kh, kd), (vt, vh, vd) = _KV_TYPES.get(k.dtype), k.stride(), v.stride()
        rows, rot = table.shape
        ok = (code is not None and v.dtype is k.dtype and k.shape == shape and v.shape == shape
              and kd == 1 and vd == 1 and slots.dtype is _I64 and slots.dim() == 1
              and slots.is_contiguous() and positions.dtype is _I64 and positions.shape == (n,)
              and positions.is_contiguous() and table.dtype is _F32 and table.is_contiguous()
              and d_status.dtype is _I32 and d_status.numel() >= 1 and d_status.is_contiguous()
              and dev >= 0 and _current_device() == dev and k.get_device() == dev
              and v.get_device() == dev and slots.get_device() == dev
              and positions.get_device() == dev and table.get_device() == dev
              and d_status.get_device() == dev)
        if q is None:
            ok = ok and q_out is None
            qp = op = heads = qt = qh = ot = oh = 0
        else:
            heads = q.shape[1]
            qp, op, (qt, qh, qd), (ot, oh, od) = q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
            ok = (ok and q.dtype is k.dtype and q_out.dtype is k.dtype and heads > 0
                  and q.shape == (n, heads, cache.head_dim) and q_out.shape == q.shape and qd == 1
                  and od == 1 and q.get_device() == dev and q_out.get_device() == dev
                  and ((qt == ot and qh == oh and _kv_written_beside(q_out, qp, k, v))
                       or (_kv_distinct(q_out) and ((qp == op and qt == ot and qh == oh) or _kv_apart(q, q_out))
                           and _kv_beside(q_out, k) and _kv_beside(q_out, v))))
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        _kv_rotary_refuse("lw_kv_write_rotary", cache, k, v, slots, positions, table, d_status, q, q_out)
        n, (rows, rot) = slots.shape[0], table.shape
        code, (kt, kh, kd), (vt, vh, vd) = _KV_TYPES[k.dtype], k.stride(), v.stride()
        qp = op = heads = qt = qh = ot = oh = 0
        if q is not None:
            heads = q.shape[1]
            qp, op, (qt, qh, qd), (ot, oh, od) = q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
    a = _KV_ROTATED.pack(k.data_ptr(), kt, kh, code, 0, v.data_ptr(), vt, vh, code, 0, qp, qt, qh, code, 0,
                         op, ot, oh, code, 0, slots.data_ptr(), positions.data_ptr(), table.data_ptr(),
                         rows, n, heads, rot, 1 if interleaved else 0, 0)
    r = _lib.lw_kv_write_rotary(cache.ref, a, d_status.data_ptr(),
                                _raw_stream(dev) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, "lw_kv_write_rotary")


# ---- eviction by accumulated attention weight ----------------------------------

def _kv_weight_rows(fn, name, t, batch, heads, keys, written):
    """Refuse anything but rows of weights float32 [batch, kv_heads, keys]."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        _refuse(fn, f"{name}: expected a float32 tensor")
    if t.dim() != 3 or t.shape[0] != batch or t.shape[1] != heads or (keys is not None and t.shape[2] != keys):
        _refuse(fn, f"{name}: shape {list(t.shape)}, expected "
                    f"[{batch}, {heads}, {'keys' if keys is None else keys}]")
    if t.numel() and t.shape[2] > 1 and t.stride(2) != 1:
        _refuse(fn, f"{name}: the last dimension is strided")
    if written and not _kv_distinct(t):
        _refuse(fn, f"{name}: rows that are written overlap")


def _kv_table(fn, name, t, batch):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        _refuse(fn, f"{name}: expected an int32 tensor")
    if t.dim() != 2 or t.shape[0] != batch or (t.shape[1] > 1 and t.stride(1) != 1):
        _refuse(fn, f"{name}: expected [{batch}, pages] with contiguous rows")


def _kv_clear(a, b) -> bool:
    """Whether the weights `b`, written, are `a` itself, entry for entry, or share no byte with it."""
    if a.data_ptr() == b.data_ptr() and a.stride()[:2] == b.stride()[:2]:
        return True
    def end(t):
        return t.data_ptr() + 4 * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    return (a.numel() == 0 or b.numel() == 0 or end(a) <= b.data_ptr() or end(b) <= a.data_ptr()
            or _kv_beside(a, b))   # (interleaved in one buffer)


def lw_kv_weigh_workspace_bytes(cache: KvCache, q_heads: int, q_tokens: int) -> int:
    if cache.index >= 0 and _current_device() != cache.index:   # (sized by the current device)
        _kv_on("lw_kv_weigh_workspace_bytes", cache)
    return int(load().lw_kv_weigh_workspace_bytes(cache.ref, q_heads, q_tokens))


def _kv_weigh_refuse(cache, q, lse, q_start, kv_len, page_table, weights, ws, d_status, max_q, add_to):
    import operator
    import torch
    fn = "lw_kv_weigh"
    try:
        operator.index(max_q)
    except TypeError:
        _refuse(fn, f"max_q: expected a whole number, got {max_q!r}")
    heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    if isinstance(q, torch.Tensor) and (heads < 1 or heads % cache.kv_heads):
        _refuse(fn, f"q: shape {list(q.shape)}, expected [tokens, a multiple of {cache.kv_heads}, "
                    f"{cache.head_dim}]")
    _kv_heads(fn, "q", q, None, heads, cache.head_dim)
    _kv_index(fn, "kv_len", kv_len, _I32, None)
    batch = kv_len.shape[0]
    _kv_index(fn, "q_start", q_start, _I32, batch + 1)
    _kv_table(fn, "page_table", page_table, batch)
    _buf(fn, "lse", lse, 4 * q.shape[0] * heads, (torch.float32,))
    _kv_weight_rows(fn, "weights", weights, batch, cache.kv_heads, None, True)
    named = (("q", q), ("lse", lse), ("q_start", q_start), ("kv_len", kv_len), ("page_table", page_table),
             ("weights", weights), ("ws", ws), ("d_status", d_status))
    if add_to is not None:
        _kv_weight_rows(fn, "add_to", add_to, batch, cache.kv_heads, weights.shape[2], False)
        if not _kv_clear(add_to, weights):
            _refuse(fn, "add_to: overlaps weights (it may be weights itself)")
        named += (("add_to", add_to),)
    _ws_ptr(fn, ws)
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, *named)


def lw_kv_weigh(cache: KvCache, q, lse, q_start, kv_len, page_table, weights, ws, d_status, *, max_q: int,
                add_to=None, scale=None, causal: bool = True, window: int = 0, stream=None) -> None:
    """The softmax weight that each cached key was given, summed over the query tokens and the query
    heads of its key/value head: weights float32 [batch, kv_heads, keys] = add_to (none, or weights
    itself to go on summing) + those sums.  The other arguments as lw_kv_attention had them, lse
    [tokens, q_heads] as it left it."""
    dev = cache.index
    try:
        tokens, heads, dim = q.shape
        code, (qt, qh, qd) = _KV_TYPES.get(q.dtype), q.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
        shape, (wb, wh, wd) = weights.shape, weights.stride()
        keys = shape[2]
        ap = ab = ah = 0
        ok = (code is not None and dim == cache.head_dim and heads % cache.kv_heads == 0 and heads > 0
              and qd == 1 and shape == (batch, cache.kv_heads, keys) and weights.dtype is _F32
              and (wd == 1 or keys <= 1) and _kv_distinct(weights)
              and lse.dtype is _F32 and lse.is_contiguous() and lse.numel() >= tokens * heads
              and q_start.dtype is _I32 and q_start.shape == (batch + 1,) and q_start.is_contiguous()
              and kv_len.dtype is _I32 and kv_len.shape == (batch,) and kv_len.is_contiguous()
              and page_table.dtype is _I32 and (td == 1 or width <= 1)
              and ws.is_contiguous() and d_status.dtype is _I32 and d_status.numel() >= 1
              and d_status.is_contiguous() and type(max_q) is int and dev >= 0 and _current_device() == dev
              and q.get_device() == dev and lse.get_device() == dev and q_start.get_device() == dev
              and kv_len.get_device() == dev and page_table.get_device() == dev
              and weights.get_device() == dev and ws.get_device() == dev and d_status.get_device() == dev)
        if add_to is not None:
            ap, (ab, ah, ad) = add_to.data_ptr(), add_to.stride()
            ok = (ok and add_to.dtype is _F32 and add_to.shape == shape and (ad == 1 or keys <= 1)
                  and add_to.get_device() == dev and _kv_clear(add_to, weights))
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        _kv_weigh_refuse(cache, q, lse, q_start, kv_len, page_table, weights, ws, d_status, max_q, add_to)
        tokens, heads, dim = q.shape
        code, (qt, qh, qd) = _KV_TYPES[q.dtype], q.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
        keys, (wb, wh, wd) = weights.shape[2], weights.stride()
        ap, (ab, ah, ad) = (0, (0, 0, 0)) if add_to is None else (add_to.data_ptr(), add_to.stride())
    try:
        a = _KV_WEIGHTS.pack(q.data_ptr(), qt, qh, lse.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                             page_table.data_ptr(), ts, tokens, ap, ab, ah, weights.data_ptr(), wb, wh, keys,
                             width, code, batch, heads, max_q, 1 if causal else 0, window,
                             dim ** -0.5 if scale is None else scale)
    except struct.error as e:
        _refuse("lw_kv_weigh", f"max_q {max_q!r}, window {window!r}, scale {scale!r}: {e}")
    r = _lib.lw_kv_weigh(cache.ref, a, ws.data_ptr(), ws.numel() * ws.element_size(), d_status.data_ptr(),
                         _raw_stream(dev) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, "lw_kv_weigh")


def _kv_whole(fn, **named):
    import operator
    for name, x in named.items():
        try:
            operator.index(x)
        except TypeError:
            _refuse(fn, f"{name}: expected a whole number, got {x!r}")


def _kv_evict_refuse(cache, weights, kv_len, page_table, out_table, out_len, out_weights, kept, d_status, keep, first,
                     recent):
    import torch
    fn = "lw_kv_evict"
    _kv_whole(fn, keep=keep, first=first, recent=recent)
    _kv_index(fn, "kv_len", kv_len, _I32, None)
    batch, heads = kv_len.shape[0], cache.kv_heads
    _kv_index(fn, "out_len", out_len, _I32, batch)
    _kv_table(fn, "page_table", page_table, batch)
    _kv_table(fn, "out_table", out_table, batch)
    _kv_weight_rows(fn, "weights", weights, batch, heads, None, False)
    named = (("weights", weights), ("kv_len", kv_len), ("page_table", page_table), ("out_table", out_table),
             ("out_len", out_len), ("kept", kept), ("d_status", d_status))
    if not isinstance(kept, torch.Tensor) or kept.dtype != torch.int32 or not kept.is_contiguous() or \
            tuple(kept.shape) != (batch, heads, keep):
        _refuse(fn, f"kept: expected a contiguous int32 tensor [{batch}, {heads}, {keep}]")
    if batch and abs(out_len.data_ptr() - kv_len.data_ptr()) < 4 * batch:
        _refuse(fn, "out_len: overlaps kv_len")
    if out_weights is not None:
        _kv_weight_rows(fn, "out_weights", out_weights, batch, heads, None, True)
        if not _kv_clear(weights, out_weights):
            _refuse(fn, "out_weights: overlaps weights (it may be weights itself)")
        named += (("out_weights", out_weights),)
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, *named)


def lw_kv_evict(cache: KvCache, weights, kv_len, page_table, out_table, out_len, out_weights, kept, d_status, *,
                keep: int, first: int = 0, recent: int = 0, stream=None) -> None:
    """Keep at most `keep` keys of each head of a sequence: the first `first`, the last `recent`, and
    of the others those of the largest weights float32 [batch, kv_heads, keys].  They move together to the
    front of out_table's pages (page_table itself, or other pages); kept int32 [batch, kv_heads, keep]
    lists them (-1: none), out_len int32 [batch] says how many there are, out_weights (None, weights
    itself, or other rows of at least `keep`) gets their weights."""
    dev = cache.index
    try:
        batch, width = page_table.shape
        out_batch, out_width = out_table.shape
        ts, td = page_table.stride()
        so, od = out_table.stride()
        heads, (wb, wh, wd), keys = cache.kv_heads, weights.stride(), weights.shape[2]
        kp, lp = kv_len.data_ptr(), out_len.data_ptr()
        ok = (out_batch == batch and page_table.dtype is _I32 and out_table.dtype is _I32
              and (td == 1 or width <= 1) and (od == 1 or out_width <= 1)
              and weights.dtype is _F32 and weights.shape == (batch, heads, keys) and (wd == 1 or keys <= 1)
              and kv_len.dtype is _I32 and kv_len.shape == (batch,) and kv_len.is_contiguous()
              and out_len.dtype is _I32 and out_len.shape == (batch,) and out_len.is_contiguous()
              and abs(kp - lp) >= 4 * batch and type(keep) is int and type(first) is int and type(recent) is int
              and kept.dtype is _I32 and kept.shape == (batch, heads, keep) and kept.is_contiguous()
              and d_status.dtype is _I32 and d_status.numel() >= 1 and d_status.is_contiguous()
              and dev >= 0 and _current_device() == dev and weights.get_device() == dev
              and kv_len.get_device() == dev and page_table.get_device() == dev and out_table.get_device() == dev
              and out_len.get_device() == dev and kept.get_device() == dev and d_status.get_device() == dev)
        op = ob = oh = on = 0
        if out_weights is not None:
            op, (ob, oh, od), on = out_weights.data_ptr(), out_weights.stride(), out_weights.shape[2]
            ok = (ok and out_weights.dtype is _F32 and out_weights.shape == (batch, heads, on)
                  and (od == 1 or on <= 1) and _kv_distinct(out_weights) and _kv_clear(weights, out_weights)
                  and out_weights.get_device() == dev)
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    fn = "lw_kv_evict"
    if not ok:
        _kv_evict_refuse(cache, weights, kv_len, page_table, out_table, out_len, out_weights, kept, d_status, keep,
                         first, recent)
        (batch, width), out_width = page_table.shape, out_table.shape[1]
        ts, so, (wb, wh, _), keys = page_table.stride(0), out_table.stride(0), weights.stride(), weights.shape[2]
        kp, lp, op, ob, oh, on = kv_len.data_ptr(), out_len.data_ptr(), 0, 0, 0, 0
        if out_weights is not None:
            op, (ob, oh, _), on = out_weights.data_ptr(), out_weights.stride(), out_weights.shape[2]
    try:
        a = _KV_EVICTION.pack(weights.data_ptr(), wb, wh, keys, kp, page_table.data_ptr(), ts, out_table.data_ptr(),
                              so, lp, op, ob, oh, on, kept.data_ptr(), width, out_width, batch, keep, first, recent)
    except struct.error as e:
        _refuse(fn, f"keep {keep!r}, first {first!r}, recent {recent!r}: {e}")
    r = _lib.lw_kv_evict(cache.ref, a, d_status.data_ptr(),
                         _raw_stream(dev) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, fn)


# ---- sparse attention ----------------------------------------------------------

def lw_kv_summary_bytes(cache: KvCache) -> int:
    return cache.summary_bytes


def _kv_summary(fn, cache, summary):
    _buf(fn, "summary", summary, lw_kv_summary_bytes(cache))


def lw_kv_summarise(cache: KvCache, summary, start, kv_len, page_table, d_status, stream=None) -> None:
    """Bring the summaries of the pages that hold tokens start[b] .. kv_len[b] - 1 up to date: summary is
    memory of lw_kv_summary_bytes(cache) bytes, start and kv_len int32 [batch]."""
    dev = cache.index
    try:
        batch, width = page_table.shape
        ts, td = page_table.stride()
        ok = (start.dtype is _I32 and start.shape == (batch,) and start.is_contiguous()
              and kv_len.dtype is _I32 and kv_len.shape == (batch,) and kv_len.is_contiguous()
              and page_table.dtype is _I32 and (td == 1 or width <= 1) and summary.is_contiguous()
              and summary.nbytes >= cache.summary_bytes
              and d_status.dtype is _I32 and d_status.numel() >= 1 and d_status.is_contiguous()
              and dev >= 0 and _current_device() == dev and summary.get_device() == dev
              and start.get_device() == dev and kv_len.get_device() == dev
              and page_table.get_device() == dev and d_status.get_device() == dev)
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    fn = "lw_kv_summarise"
    if not ok:
        _kv_index(fn, "kv_len", kv_len, _I32, None)
        batch = kv_len.shape[0]
        _kv_index(fn, "start", start, _I32, batch)
        _kv_table(fn, "page_table", page_table, batch)
        _kv_summary(fn, cache, summary)
        _status_ptr(fn, d_status)
        _kv_on(fn, cache, ("summary", summary), ("start", start), ("kv_len", kv_len),
               ("page_table", page_table), ("d_status", d_status))
        width, ts = page_table.shape[1], page_table.stride(0)
    a = _KV_SUMMARIES.pack(summary.data_ptr(), start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), ts,
                           width, batch)
    r = _lib.lw_kv_summarise(cache.ref, a, d_status.data_ptr(),
                             _raw_stream(dev) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, fn)


def lw_kv_blocks_workspace_bytes(cache: KvCache, q_heads: int, q_tokens: int, table_width: int, blocks: int) -> int:
    if cache.index >= 0 and _current_device() != cache.index:   # (sized by the current device)
        _kv_on("lw_kv_blocks_workspace_bytes", cache)
    return int(load().lw_kv_blocks_workspace_bytes(cache.ref, q_heads, q_tokens, table_width, blocks))


def _kv_blocks_refuse(cache, summary, q, q_start, kv_len, page_table, out, ws, d_status, blocks, first, recent,
                      lse, chosen):
    import torch
    fn = "lw_kv_attention_blocks"
    _kv_whole(fn, blocks=blocks, first=first, recent=recent)
    heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    if isinstance(q, torch.Tensor) and (heads < 1 or heads % cache.kv_heads):
        _refuse(fn, f"q: shape {list(q.shape)}, expected [tokens, a multiple of {cache.kv_heads}, "
                    f"{cache.head_dim}]")
    _kv_heads(fn, "q", q, None, heads, cache.head_dim)
    _kv_heads(fn, "out", out, q.shape[0], heads, cache.head_dim, True)
    if out.dtype != q.dtype:
        _refuse(fn, f"out: dtype {out.dtype}, q has {q.dtype}")
    _kv_index(fn, "kv_len", kv_len, _I32, None)
    batch = kv_len.shape[0]
    _kv_index(fn, "q_start", q_start, _I32, batch + 1)
    _kv_table(fn, "page_table", page_table, batch)
    _kv_summary(fn, cache, summary)
    named = (("summary", summary), ("q", q), ("out", out), ("q_start", q_start), ("kv_len", kv_len),
             ("page_table", page_table), ("ws", ws), ("d_status", d_status))
    if lse is not None:
        _buf(fn, "lse", lse, 4 * q.shape[0] * heads, (torch.float32,))
        named += (("lse", lse),)
    if chosen is not None:
        want = (q.shape[0], cache.kv_heads, blocks)
        if not isinstance(chosen, torch.Tensor) or chosen.dtype != torch.int32 or \
                not chosen.is_contiguous() or tuple(chosen.shape) != want:
            _refuse(fn, f"chosen: expected a contiguous int32 tensor {list(want)}")
        named += (("chosen", chosen),)
    _ws_ptr(fn, ws)
    _status_ptr(fn, d_status)
    _kv_on(fn, cache, *named)


def lw_kv_attention_blocks(cache: KvCache, summary, q, q_start, kv_len, page_table, out, ws, d_status, *,
                           blocks: int, first: int = 1, recent: int = 1, scale=None, lse=None, chosen=None,
                           stream=None) -> None:
    """lw_kv_attention (causal) in which every query token and key/value head reads at most `blocks` pages:
    the first `first`, the last `recent`, and those that score highest against `summary`
    (lw_kv_summarise).  chosen int32 [tokens, kv_heads, blocks]: the pages' places in the page table, -1
    where there are fewer.  ws: lw_kv_blocks_workspace_bytes, zeroed once."""
    dev = cache.index
    try:
        tokens, heads, dim = shape = q.shape
        code, (qt, qh, qd), (ot, oh, od) = _KV_TYPES.get(q.dtype), q.stride(), out.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
        ok = (code is not None and out.dtype is q.dtype and out.shape == shape
              and dim == cache.head_dim and heads % cache.kv_heads == 0 and qd == 1 and od == 1
              and heads > 0 and (out.is_contiguous() or _kv_distinct(out))
              and q_start.dtype is _I32 and q_start.shape == (batch + 1,) and q_start.is_contiguous()
              and kv_len.dtype is _I32 and kv_len.shape == (batch,) and kv_len.is_contiguous()
              and page_table.dtype is _I32 and (td == 1 or width <= 1) and summary.is_contiguous()
              and summary.nbytes >= cache.summary_bytes
              and ws.is_contiguous() and d_status.dtype is _I32 and d_status.numel() >= 1
              and d_status.is_contiguous() and type(blocks) is int and type(first) is int
              and type(recent) is int and dev >= 0 and _current_device() == dev
              and q.get_device() == dev and out.get_device() == dev and q_start.get_device() == dev
              and kv_len.get_device() == dev and page_table.get_device() == dev
              and summary.get_device() == dev and ws.get_device() == dev and d_status.get_device() == dev
              and (lse is None or (lse.dtype is _F32 and lse.is_contiguous()
                                   and lse.numel() >= tokens * heads and lse.get_device() == dev))
              and (chosen is None or (chosen.dtype is _I32 and chosen.is_contiguous()
                                      and chosen.shape == (tokens, cache.kv_heads, blocks)
                                      and chosen.get_device() == dev)))
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    fn = "lw_kv_attention_blocks"
    if not ok:
        _kv_blocks_refuse(cache, summary, q, q_start, kv_len, page_table, out, ws, d_status, blocks, first,
                          recent, lse, chosen)
        tokens, heads, dim = q.shape
        code, (qt, qh, qd), (ot, oh, od) = _KV_TYPES[q.dtype], q.stride(), out.stride()
        batch, width = page_table.shape
        ts, td = page_table.stride()
    try:
        a = _KV_ATTN.pack(q.data_ptr(), qt, qh, out.data_ptr(), ot, oh,
                          0 if lse is None else lse.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                          page_table.data_ptr(), ts, tokens, width, code, batch, heads, 1, 1, 0,
                          dim ** -0.5 if scale is None else scale)
        b = _KV_BLOCKS.pack(summary.data_ptr(), 0 if chosen is None else chosen.data_ptr(), blocks, first,
                            recent, 0)
    except struct.error as e:
        _refuse(fn, f"blocks {blocks!r}, first {first!r}, recent {recent!r}, scale {scale!r}: {e}")
    r = _lib.lw_kv_attention_blocks(cache.ref, a, b, ws.data_ptr(), ws.numel() * ws.element_size(),
                                    d_status.data_ptr(),
                                    _raw_stream(dev) if stream is None else stream.cuda_stream)
    if r:
        raise LwError(r, fn)
