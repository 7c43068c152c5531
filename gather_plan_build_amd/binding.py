"""ctypes binding of libgpb.so (the C ABI in include/gpb.h).

Argument marshalling only: every step of the compose path runs in the HIP
kernels behind the C calls.  torch provides device memory and streams.  The
functions keep the C names without the ``gpb_`` prefix.

There is no fallback: if libgpb.so is missing or fails to load, importing this
module raises.
"""
import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("GPB_LIB", os.path.join(HERE, "libgpb.so"))

MAX_SOURCES = 64
STATUS_BAD_DESCRIPTOR = 1
STATUS_BAD_STAGING_ROW = 2
STATUS_BAD_PLAN_INPUT = 4
STATUS_LAYER_MISMATCH = 8

OK, EINVAL, EALIGN, EPAGE, ECAPACITY, ERANGE, EHIP, ESCRATCH = 0, -1, -2, -3, -4, -5, -6, -7
ENOMEM = -8
SCRATCH_BYTES = 64 * 1024 * 1024  # GPB_SCRATCH_BYTES

_I32P = ctypes.POINTER(ctypes.c_int32)


class gpb_batch(ctypes.Structure):
    _fields_ = [("bs", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("row_bytes", ctypes.c_int32), ("n_pool_pages", ctypes.c_int32),
                ("n_pool_entries", ctypes.c_int32), ("n_writers", ctypes.c_int32),
                ("staging_cap_pages", ctypes.c_int32),
                ("h_prefix_pages", ctypes.c_void_p), ("h_cur_tokens", ctypes.c_void_p),
                ("h_req_pages", ctypes.c_void_p), ("d_prefix_pages", ctypes.c_void_p),
                ("d_cur_tokens", ctypes.c_void_p), ("d_req_pages", ctypes.c_void_p)]


PLAN_FIELDS = ("slot_base", "prefix_span", "current_span", "q_lens", "kv_lens",
               "q_starts", "k_bases", "q_bases", "current_bases", "slot_pages",
               "owner", "src", "page_inverse", "staging_page_inverse", "writer",
               "staging_rows", "mixed_locs", "token_req", "topk_offsets", "segments",
               "prefix_slots", "current_slots", "pool_locs", "cur_page_token0",
               "cur_page_ntok", "prefix_desc", "current_desc", "writer_offsets",
               "writer_tokens", "writer_rows", "writer_page_row0")


class gpb_plan(ctypes.Structure):
    _fields_ = [("d_" + f, ctypes.c_void_p) for f in PLAN_FIELDS] + \
        [("d_status", ctypes.c_void_p)]


class gpb_sources(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32),
                ("base", ctypes.c_void_p * MAX_SOURCES),
                ("n_pages", ctypes.c_int64 * MAX_SOURCES)]


MAX_GROUPS = 4
MAX_GROUP_SOURCES = 16


class gpb_row_group(ctypes.Structure):
    _fields_ = [("d_staging", ctypes.c_void_p), ("n_staging_rows", ctypes.c_int64),
                ("d_cur_rows", ctypes.c_void_p), ("row_bytes", ctypes.c_int32)]


class gpb_gather_group(ctypes.Structure):
    _fields_ = [("d_dense", ctypes.c_void_p), ("table", ctypes.POINTER(gpb_sources)),
                ("row_bytes", ctypes.c_int32)]


class gpb_layer_group(ctypes.Structure):
    _fields_ = [("d_dense", ctypes.c_void_p), ("table", ctypes.POINTER(gpb_sources)),
                ("d_staging", ctypes.c_void_p), ("n_staging_rows", ctypes.c_int64),
                ("d_cur_rows", ctypes.c_void_p), ("row_bytes", ctypes.c_int32)]


MAX_AXES = 4
BF16, FP16, HELD_E4M3 = 1, 2, 16


class gpb_row_format(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("dtype", "n_kv_heads", "k_dim", "v_dim", "values_in_key", "row_bytes")]


class gpb_append(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("d_pool", ctypes.c_void_p), ("n_pool_rows", ctypes.c_int64),
                ("d_pool_locs", ctypes.c_void_p), ("d_rows", ctypes.c_void_p),
                ("d_q", ctypes.c_void_p), ("d_q_out", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("qo_token_stride", ctypes.c_int64), ("qo_head_stride", ctypes.c_int64),
                ("rot_start", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("section", ctypes.c_int32 * MAX_AXES),
                ("d_inv_freq", ctypes.c_void_p), ("d_positions", ctypes.c_void_p),
                ("positions_stride", ctypes.c_int64)]


class gpb_attend_shape(ctypes.Structure):
    _fields_ = [("bs", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("page_rows", ctypes.c_int32), ("h_q_lens", ctypes.c_void_p),
                ("h_kv_lens", ctypes.c_void_p), ("n_groups", ctypes.c_int32),
                ("h_groups", ctypes.c_void_p)]


class gpb_attend_plan(ctypes.Structure):
    _fields_ = [("format", gpb_row_format)] + [(n, ctypes.c_int32) for n in (
        "bs", "n_heads", "window", "sinks", "page_rows", "n_groups", "n_tokens", "max_keys",
        "n_items", "n_wide", "n_joins", "n_refs", "n_partial_rows", "joins_at", "refs_at",
        "positions_at", "list_ints")] + [("workspace_bytes", ctypes.c_int64)]


class gpb_attend_io(ctypes.Structure):
    _fields_ = [("d_q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("d_out", ctypes.c_void_p),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("d_lse", ctypes.c_void_p), ("scale", ctypes.c_float)]


def _hip_runtimes():
    """Distinct libamdhip64 files mapped into this process."""
    found = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                path = line.split()[-1] if len(line.split()) >= 6 else ""
                if "libamdhip64" in os.path.basename(path):
                    found.add(os.path.realpath(path))
    except OSError:
        pass
    return found


def _load(path):
    if not os.path.exists(path):
        raise ImportError("libgpb.so not built at %s: run python "
                          "gather_plan_build_amd/build.py (no fallback exists)" % path)
    # torch provides device memory and streams; its HIP runtime must be the
    # one libgpb.so binds to (same SONAME, loaded first), or the process would
    # hold two runtimes whose streams and devices do not mix.
    import torch  # noqa: F401
    import torch.cuda  # noqa: F401
    lib = ctypes.CDLL(path)
    runtimes = _hip_runtimes()
    if len(runtimes) > 1:
        raise ImportError("two HIP runtimes are loaded (%s): load torch before "
                          "libgpb.so" % ", ".join(sorted(runtimes)))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.gpb_plan_sizes.argtypes = [ctypes.POINTER(gpb_batch), _I32P, _I32P, _I32P]
    lib.gpb_plan_build.argtypes = [ctypes.POINTER(gpb_batch), ctypes.POINTER(gpb_plan), vp]
    lib.gpb_plan_build_clear.argtypes = [ctypes.POINTER(gpb_batch), ctypes.POINTER(gpb_plan),
                                         vp, i64, vp]
    lib.gpb_writer_counts.argtypes = [ctypes.POINTER(gpb_batch), _I32P]
    lib.gpb_compose_gather_records.argtypes = [vp, ctypes.POINTER(gpb_sources), vp, i32, i32,
                                               i32, i32, vp, vp]
    lib.gpb_compose_layer.argtypes = [vp, ctypes.POINTER(gpb_sources),
                                      ctypes.POINTER(gpb_plan), i32, i32, vp, i64, vp, i32,
                                      i32, i32, vp, vp]
    lib.gpb_compose_consume.argtypes = lib.gpb_compose_layer.argtypes
    lib.gpb_compose_layer_noalloc.argtypes = [vp, ctypes.POINTER(gpb_sources), i32, i32,
                                              ctypes.POINTER(gpb_plan), i32, i32, vp, i32,
                                              i32, i32, vp, vp]
    lib.gpb_compose_layer_fill.argtypes = [vp, ctypes.POINTER(gpb_sources),
                                           ctypes.POINTER(gpb_plan), i32, i32, vp, i64, vp,
                                           i64, vp, i32, i32, i32, vp, vp]
    lib.gpb_compose_layer_ahead.argtypes = [vp] + list(lib.gpb_compose_layer.argtypes)
    lib.gpb_compose_consume_fill.argtypes = lib.gpb_compose_layer_fill.argtypes
    lib.gpb_compose_layer_ahead_fill.argtypes = [vp] + list(lib.gpb_compose_layer_fill.argtypes)
    lib.gpb_staging_clear.argtypes = [vp, i64, vp]
    lib.gpb_current_row_scatter.argtypes = [vp, i64, vp, vp, i32, i32, vp, vp]
    lib.gpb_compose_gather.argtypes = [vp, ctypes.POINTER(gpb_sources), vp, vp, i32,
                                       i32, i32, vp, vp]
    lib.gpb_compose_gather_slots.argtypes = [vp, ctypes.POINTER(gpb_sources), vp, i32, vp,
                                             vp, i32, i32, i32, vp, vp]
    lib.gpb_current_row_fill.argtypes = [vp, i64, vp, vp, i64, vp, vp, i32, i32, vp, vp]
    lib.gpb_current_row_scatter_groups.argtypes = [ctypes.POINTER(gpb_row_group), i32, vp,
                                                   i32, vp, vp]
    lib.gpb_compose_gather_groups.argtypes = [ctypes.POINTER(gpb_gather_group), i32, vp, vp,
                                              i32, i32, vp, vp]
    lib.gpb_compose_layer_groups.argtypes = [ctypes.POINTER(gpb_layer_group), i32,
                                             ctypes.POINTER(gpb_plan), i32, i32, i32, i32,
                                             vp, vp]
    lib.gpb_row_append.argtypes = [ctypes.POINTER(gpb_row_format), ctypes.POINTER(gpb_append),
                                   vp, vp]
    lib.gpb_rows_read.argtypes = [ctypes.POINTER(gpb_row_format), vp, i64, vp, i32, vp, i32, vp,
                                  vp]
    lib.gpb_rows_read.restype = i32
    lib.gpb_attend_plan_build.argtypes = [ctypes.POINTER(gpb_row_format),
                                          ctypes.POINTER(gpb_attend_shape),
                                          ctypes.POINTER(gpb_attend_plan), vp, i64]
    lib.gpb_attend_dense.argtypes = [ctypes.POINTER(gpb_attend_plan), vp,
                                     ctypes.POINTER(gpb_attend_io), vp, i64, vp, vp, i64, vp,
                                     vp]
    lib.gpb_attend_paged.argtypes = [ctypes.POINTER(gpb_attend_plan), vp,
                                     ctypes.POINTER(gpb_attend_io), vp, i64, vp, i64, vp, i64,
                                     vp, i64, vp, vp]
    lib.gpb_strerror.argtypes = [ctypes.c_int]
    lib.gpb_strerror.restype = ctypes.c_char_p
    for f in EXPORTS:
        if f != "gpb_strerror":
            getattr(lib, f).restype = ctypes.c_int
    return lib


EXPORTS = ("gpb_plan_sizes", "gpb_plan_build", "gpb_plan_build_clear",
           "gpb_writer_counts", "gpb_staging_clear", "gpb_current_row_scatter",
           "gpb_compose_gather", "gpb_compose_gather_slots", "gpb_compose_gather_records",
           "gpb_compose_layer", "gpb_compose_layer_fill", "gpb_compose_consume",
           "gpb_compose_layer_ahead", "gpb_compose_layer_noalloc",
           "gpb_compose_consume_fill", "gpb_compose_layer_ahead_fill",
           "gpb_current_row_fill", "gpb_current_row_scatter_groups",
           "gpb_compose_gather_groups", "gpb_compose_layer_groups", "gpb_row_append",
           "gpb_rows_read", "gpb_attend_plan_build", "gpb_attend_dense", "gpb_attend_paged",
           "gpb_strerror")

lib = _load(LIB_PATH)


class GpbError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__("%s: %s (%d)" % (what, strerror(code), code))


def strerror(code):
    return lib.gpb_strerror(int(code)).decode()


def _check(rc, what):
    if rc != OK:
        raise GpbError(rc, what)


def _ptr(x):
    """Device address of a GPU torch tensor, or an int address (taken as a
    device address), or None.  A tensor in host memory is refused: its address
    would reach a kernel."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("a %s tensor in host memory was passed where device memory "
                         "is required" % (tuple(x.shape),))
    return x.data_ptr()


def _gpu_device(device):
    import torch
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("the compose runs on the GPU: device %s is not a GPU device" % dev)
    return dev


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _host_i32(a):
    """Contiguous int32 copy of host metadata; values outside int32 raise
    instead of wrapping."""
    v = np.asarray(a, dtype=np.int64).reshape(-1)
    if v.size and (v.min() < np.iinfo(np.int32).min or v.max() > np.iinfo(np.int32).max):
        raise ValueError("batch metadata value outside int32")
    return np.ascontiguousarray(v.astype(np.int32))


class BatchMeta:
    """Host side of a gpb_batch: geometry plus the three host arrays."""

    def __init__(self, bs, page_size, row_bytes, n_pool_pages, n_pool_entries,
                 n_writers, staging_cap_pages, prefix_pages, cur_tokens, req_pages):
        self.h_prefix = _host_i32(prefix_pages)
        self.h_cur = _host_i32(cur_tokens)
        self.h_req = _host_i32(req_pages)
        self.c = gpb_batch(bs, page_size, row_bytes, n_pool_pages, n_pool_entries,
                           n_writers, staging_cap_pages,
                           self.h_prefix.ctypes.data if self.h_prefix.size else None,
                           self.h_cur.ctypes.data if self.h_cur.size else None,
                           self.h_req.ctypes.data if self.h_req.size else None,
                           None, None, None)

    @classmethod
    def of(cls, b):
        """From any object with the workload attributes (workloads.Batch)."""
        return cls(b.bs, b.page_size, b.row_bytes, b.n_pool_pages, b.n_pool_entries,
                   b.n_writers, b.staging_cap_pages, b.prefix_pages, b.cur_tokens,
                   b.req_pages)

    def plan_key(self):
        """What a plan depends on (page 0d87bc5, commit "descriptor cache on
        the slot-remap objects": descriptors are cached for one batch and
        never reused across a different page layout, slot spans, table
        layout, device or capacity; page d63fbd4, commit "counting barrier +
        CUDA-IPC gather": the plan cache lives on the batch's slot remap): the
        geometry except the row size, and the three metadata arrays.  Two
        batches with equal keys have identical plans; the device is checked
        beside the key."""
        import hashlib
        c = self.c
        h = hashlib.sha256()
        for a in (self.h_prefix, self.h_cur, self.h_req):
            h.update(np.int64(a.size).tobytes())
            h.update(a.tobytes())
        return (c.bs, c.page_size, c.n_pool_pages, c.n_pool_entries, c.n_writers,
                c.staging_cap_pages, h.hexdigest())


def writer_counts(meta):
    """Entries of every writer's scatter list (host only, no device read)."""
    out = np.zeros(max(meta.c.n_writers, 1), np.int32)
    _check(lib.gpb_writer_counts(ctypes.byref(meta.c), out.ctypes.data_as(_I32P)),
           "gpb_writer_counts")
    return out[:meta.c.n_writers]


def plan_sizes(meta):
    """(S, T, NCP) after host validation; raises GpbError on a bad batch."""
    S, T, NCP = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib.gpb_plan_sizes(ctypes.byref(meta.c), ctypes.byref(S), ctypes.byref(T),
                              ctypes.byref(NCP)), "gpb_plan_sizes")
    return S.value, T.value, NCP.value


class Plan:
    """Device inputs and outputs of gpb_plan_build for one batch.

    Construction validates the batch on the host, copies the three metadata
    arrays to the device once and allocates every output (torch int32).
    ``build`` launches the plan kernels; the outputs are ``self.t[name]``."""

    def __init__(self, meta, device="cuda"):
        import torch
        self.meta = meta
        self.S, self.T, self.NCP = plan_sizes(meta)
        b = meta.c
        dev = _gpu_device(device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.key = meta.plan_key()
        self.d_prefix = torch.from_numpy(meta.h_prefix).to(dev)
        self.d_cur = torch.from_numpy(meta.h_cur).to(dev)
        self.d_req = torch.from_numpy(meta.h_req).to(dev)
        b.d_prefix_pages = self.d_prefix.data_ptr() if self.d_prefix.numel() else None
        b.d_cur_tokens = self.d_cur.data_ptr() if self.d_cur.numel() else None
        b.d_req_pages = self.d_req.data_ptr() if self.d_req.numel() else None
        bs, npp = b.bs, b.n_pool_pages
        sizes = {"slot_base": bs, "prefix_span": 2 * bs, "current_span": 2 * bs,
                 "q_lens": bs, "kv_lens": bs, "q_starts": bs, "k_bases": bs,
                 "q_bases": bs, "current_bases": bs, "slot_pages": self.S,
                 "owner": self.S, "src": self.S, "page_inverse": npp,
                 "staging_page_inverse": npp, "writer": self.NCP,
                 "staging_rows": self.T, "mixed_locs": self.T, "token_req": self.T,
                 "topk_offsets": self.T, "segments": 4 * bs,
                 "prefix_slots": self.S - self.NCP, "current_slots": self.NCP,
                 "pool_locs": self.T, "cur_page_token0": self.NCP,
                 "cur_page_ntok": self.NCP, "prefix_desc": 4 * (self.S - self.NCP),
                 "current_desc": 4 * self.NCP, "writer_offsets": b.n_writers + 1,
                 "writer_tokens": self.T, "writer_rows": self.T,
                 "writer_page_row0": self.NCP}
        self.t = {k: torch.empty(sizes[k], dtype=torch.int32, device=dev)
                  for k in PLAN_FIELDS}
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.c = gpb_plan(*[(self.t[k].data_ptr() if sizes[k] else None)
                            for k in PLAN_FIELDS], self.status.data_ptr())

    def build(self, stream=None, clear=None):
        """Launch the plan kernels; with ``clear`` (a uint8 device tensor) the
        same launches also zero it (gpb_plan_build_clear)."""
        if clear is None:
            _check(lib.gpb_plan_build(ctypes.byref(self.meta.c), ctypes.byref(self.c),
                                      _stream(stream)), "gpb_plan_build")
        else:
            _check(lib.gpb_plan_build_clear(ctypes.byref(self.meta.c), ctypes.byref(self.c),
                                            _ptr(clear), clear.numel() * clear.element_size(),
                                            _stream(stream)), "gpb_plan_build_clear")
        return self


def plan_build(meta, device="cuda", stream=None):
    """Validate, allocate and launch: returns the Plan (outputs in .t)."""
    return Plan(meta, device).build(stream)


class Sources:
    """A gpb_sources pointer table: [(base, n_pages), ...] with base a tensor
    or a device address.  Built once, passed by reference to every gather."""

    def __init__(self, entries):
        if not 1 <= len(entries) <= MAX_SOURCES:
            raise GpbError(EINVAL, "Sources")
        self.keep = [e[0] for e in entries]
        self.c = gpb_sources()
        self.c.n = len(entries)
        for i, (base, n_pages) in enumerate(entries):
            self.c.base[i] = _ptr(base)
            self.c.n_pages[i] = int(n_pages)


def staging_clear(buf, n_bytes=None, stream=None):
    """Zero a staging region (tensor, or address with n_bytes)."""
    if n_bytes is None:
        n_bytes = buf.numel() * buf.element_size()
    _check(lib.gpb_staging_clear(_ptr(buf), int(n_bytes), _stream(stream)),
           "gpb_staging_clear")


def current_row_scatter(staging, n_staging_rows, staging_rows, cur_rows, n_rows,
                        row_bytes, status=None, stream=None):
    _check(lib.gpb_current_row_scatter(_ptr(staging), int(n_staging_rows),
                                       _ptr(staging_rows), _ptr(cur_rows), int(n_rows),
                                       int(row_bytes), _ptr(status), _stream(stream)),
           "gpb_current_row_scatter")


def compose_gather(dense, sources, owner, src, n_slots, page_rows, row_bytes,
                   status=None, stream=None):
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_gather(_ptr(dense), ctypes.byref(sources.c), _ptr(owner),
                                  _ptr(src), int(n_slots), int(page_rows),
                                  int(row_bytes), _ptr(status), _stream(stream)),
           "gpb_compose_gather")


def compose_gather_slots(dense, sources, slots, n_list, owner, src, n_slots, page_rows,
                         row_bytes, status=None, stream=None):
    """Gather only the listed dense slots (prefetch or consume half)."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_gather_slots(_ptr(dense), ctypes.byref(sources.c), _ptr(slots),
                                        int(n_list), _ptr(owner), _ptr(src), int(n_slots),
                                        int(page_rows), int(row_bytes), _ptr(status),
                                        _stream(stream)),
           "gpb_compose_gather_slots")


def compose_gather_records(dense, sources, records, n_records, n_slots, page_rows,
                           row_bytes, status=None, stream=None):
    """Gather the pages named by (slot, owner, src, 0) records."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_gather_records(_ptr(dense), ctypes.byref(sources.c),
                                          _ptr(records), int(n_records), int(n_slots),
                                          int(page_rows), int(row_bytes), _ptr(status),
                                          _stream(stream)),
           "gpb_compose_gather_records")


def compose_layer(dense, sources, plan, n_slots, n_cur_pages, staging, n_staging_rows,
                  cur_rows, n_rows, page_rows, row_bytes, status=None, stream=None):
    """Scatter and gather of one layer in one launch (``plan`` a Plan)."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_layer(_ptr(dense), ctypes.byref(sources.c), ctypes.byref(plan.c),
                                 int(n_slots), int(n_cur_pages), _ptr(staging),
                                 int(n_staging_rows), _ptr(cur_rows), int(n_rows),
                                 int(page_rows), int(row_bytes), _ptr(status),
                                 _stream(stream)),
           "gpb_compose_layer")


def compose_layer_noalloc(dense, pools, n_writers, staging_cap_pages, plan, n_slots,
                          n_cur_pages, cur_rows, n_rows, page_rows, row_bytes, status=None,
                          stream=None):
    """The one-launch layer with staging in the library's static array:
    ``pools`` lists the pool entries only, the library adds the slabs."""
    if not isinstance(pools, Sources):
        pools = Sources(pools)
    _check(lib.gpb_compose_layer_noalloc(_ptr(dense), ctypes.byref(pools.c), int(n_writers),
                                         int(staging_cap_pages), ctypes.byref(plan.c),
                                         int(n_slots), int(n_cur_pages), _ptr(cur_rows),
                                         int(n_rows), int(page_rows), int(row_bytes),
                                         _ptr(status), _stream(stream)),
           "gpb_compose_layer_noalloc")


def compose_layer_fill(dense, sources, plan, n_slots, n_cur_pages, staging, n_staging_rows,
                       pool, n_pool_rows, cur_rows, n_rows, page_rows, row_bytes, status=None,
                       stream=None):
    """The one-launch layer with the fused fill (current rows also to their
    pool rows)."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_layer_fill(_ptr(dense), ctypes.byref(sources.c),
                                      ctypes.byref(plan.c), int(n_slots), int(n_cur_pages),
                                      _ptr(staging), int(n_staging_rows), _ptr(pool),
                                      int(n_pool_rows), _ptr(cur_rows), int(n_rows),
                                      int(page_rows), int(row_bytes), _ptr(status),
                                      _stream(stream)),
           "gpb_compose_layer_fill")


def compose_consume(dense, sources, plan, n_slots, n_cur_pages, staging, n_staging_rows,
                    cur_rows, n_rows, page_rows, row_bytes, status=None, stream=None):
    """The consume half in one launch: scatter and current-page gather."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_consume(_ptr(dense), ctypes.byref(sources.c), ctypes.byref(plan.c),
                                   int(n_slots), int(n_cur_pages), _ptr(staging),
                                   int(n_staging_rows), _ptr(cur_rows), int(n_rows),
                                   int(page_rows), int(row_bytes), _ptr(status),
                                   _stream(stream)),
           "gpb_compose_consume")


def compose_layer_ahead(dense, dense_next, sources, plan, n_slots, n_cur_pages, staging,
                        n_staging_rows, cur_rows, n_rows, page_rows, row_bytes, status=None,
                        stream=None):
    """This layer's consume and the next layer's prefix pages in one launch."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_layer_ahead(_ptr(dense), _ptr(dense_next), ctypes.byref(sources.c),
                                       ctypes.byref(plan.c), int(n_slots), int(n_cur_pages),
                                       _ptr(staging), int(n_staging_rows), _ptr(cur_rows),
                                       int(n_rows), int(page_rows), int(row_bytes),
                                       _ptr(status), _stream(stream)),
           "gpb_compose_layer_ahead")


def compose_consume_fill(dense, sources, plan, n_slots, n_cur_pages, staging, n_staging_rows,
                         pool, n_pool_rows, cur_rows, n_rows, page_rows, row_bytes, status=None,
                         stream=None):
    """The consume half in one launch with the fused fill (current rows also
    to their pool rows)."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_consume_fill(_ptr(dense), ctypes.byref(sources.c),
                                        ctypes.byref(plan.c), int(n_slots), int(n_cur_pages),
                                        _ptr(staging), int(n_staging_rows), _ptr(pool),
                                        int(n_pool_rows), _ptr(cur_rows), int(n_rows),
                                        int(page_rows), int(row_bytes), _ptr(status),
                                        _stream(stream)),
           "gpb_compose_consume_fill")


def compose_layer_ahead_fill(dense, dense_next, sources, plan, n_slots, n_cur_pages, staging,
                             n_staging_rows, pool, n_pool_rows, cur_rows, n_rows, page_rows,
                             row_bytes, status=None, stream=None):
    """This layer's consume with the fused fill and the next layer's prefix
    pages in one launch."""
    if not isinstance(sources, Sources):
        sources = Sources(sources)
    _check(lib.gpb_compose_layer_ahead_fill(_ptr(dense), _ptr(dense_next),
                                            ctypes.byref(sources.c), ctypes.byref(plan.c),
                                            int(n_slots), int(n_cur_pages), _ptr(staging),
                                            int(n_staging_rows), _ptr(pool), int(n_pool_rows),
                                            _ptr(cur_rows), int(n_rows), int(page_rows),
                                            int(row_bytes), _ptr(status), _stream(stream)),
           "gpb_compose_layer_ahead_fill")


def current_row_fill(staging, n_staging_rows, staging_rows, pool, n_pool_rows, pool_locs,
                     cur_rows, n_rows, row_bytes, status=None, stream=None):
    """Each current row to its staging row and to its pool row, one pass."""
    _check(lib.gpb_current_row_fill(_ptr(staging), int(n_staging_rows), _ptr(staging_rows),
                                    _ptr(pool), int(n_pool_rows), _ptr(pool_locs),
                                    _ptr(cur_rows), int(n_rows), int(row_bytes),
                                    _ptr(status), _stream(stream)),
           "gpb_current_row_fill")


def current_row_scatter_groups(groups, staging_rows, n_rows, status=None, stream=None):
    """One launch scattering the current rows of every group:
    groups = [(staging, n_staging_rows, cur_rows, row_bytes), ...]."""
    arr = (gpb_row_group * max(len(groups), 1))(
        *[gpb_row_group(_ptr(st), int(n), _ptr(cur), int(rb)) for st, n, cur, rb in groups])
    _check(lib.gpb_current_row_scatter_groups(arr, len(groups), _ptr(staging_rows),
                                              int(n_rows), _ptr(status), _stream(stream)),
           "gpb_current_row_scatter_groups")


def compose_gather_groups(groups, owner, src, n_slots, page_rows, status=None, stream=None):
    """One launch gathering every group: groups = [(dense, Sources, row_bytes), ...]."""
    keep = [g[1] if isinstance(g[1], Sources) else Sources(g[1]) for g in groups]
    arr = (gpb_gather_group * max(len(groups), 1))(
        *[gpb_gather_group(_ptr(d), ctypes.pointer(t.c), int(rb))
          for (d, _, rb), t in zip(groups, keep)])
    _check(lib.gpb_compose_gather_groups(arr, len(groups), _ptr(owner), _ptr(src),
                                         int(n_slots), int(page_rows), _ptr(status),
                                         _stream(stream)),
           "gpb_compose_gather_groups")


def compose_layer_groups(groups, plan, n_slots, n_cur_pages, n_rows, page_rows, status=None,
                         stream=None):
    """One launch composing one layer of every group: groups = [(dense, Sources, staging,
    n_staging_rows, cur_rows, row_bytes), ...] on one plan (a Plan)."""
    keep = [g[1] if isinstance(g[1], Sources) else Sources(g[1]) for g in groups]
    arr = (gpb_layer_group * max(len(groups), 1))(
        *[gpb_layer_group(_ptr(d), ctypes.pointer(t.c), _ptr(st), int(n), _ptr(cur), int(rb))
          for (d, _, st, n, cur, rb), t in zip(groups, keep)])
    _check(lib.gpb_compose_layer_groups(arr, len(groups), ctypes.byref(plan.c), int(n_slots),
                                        int(n_cur_pages), int(n_rows), int(page_rows),
                                        _ptr(status), _stream(stream)),
           "gpb_compose_layer_groups")


# ---- making the rows, and reading them ---------------------------------------


def _in_32_bits(n, what):
    """n, which the C call takes as int32: ctypes would cut it without a word."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError("%s: %d does not fit in 32 bits" % (what, n))
    return n


class RowFormat:
    """What a token row holds: ``n_kv_heads`` key heads of ``k_dim`` values, then
    as many value heads of ``v_dim``; with ``values_in_key`` one key head whose
    first ``v_dim`` values are the value (a latent row).  ``dtype`` is "bf16" or
    "fp16" (or the torch dtype), ``row_bytes`` the distance between rows.  With
    ``held="e4m3"`` a row holds a byte for a value and a scale for a head (of a
    latent row, the value; the rest of its key stays in 16 bits): half the memory,
    and values off by up to 1/16.  Keys, values and queries are given, and results
    come, in ``dtype``; the rows' tensors are of any type, uint8 [rows, row_bytes]
    say.  The layout is this library's (gpb.h); other caches' rows in 8 bits, which
    may be of the same size, cannot be told from them and come out as wrong numbers."""

    def __init__(self, dtype, n_kv_heads, k_dim, v_dim, values_in_key=False, row_bytes=None,
                 held=None):
        import torch
        codes = {"bf16": BF16, "fp16": FP16, torch.bfloat16: BF16, torch.float16: FP16}
        if dtype not in codes:
            raise ValueError("a row's type is bf16 or fp16, not %r" % (dtype,))
        self.dtype = torch.bfloat16 if codes[dtype] == BF16 else torch.float16
        self.n_kv_heads = _in_32_bits(int(n_kv_heads), "n_kv_heads")
        self.k_dim, self.v_dim = _in_32_bits(int(k_dim), "k_dim"), _in_32_bits(int(v_dim), "v_dim")
        self.values_in_key = bool(values_in_key)
        if held not in (None, "e4m3"):
            raise ValueError("rows are held in their type (None) or in e4m3, not in %r" % (held,))
        self.held = held
        # values of a row, and bytes of the row without padding
        self.values = self.n_kv_heads * (self.k_dim + (0 if values_in_key else self.v_dim))
        if held is None:
            payload = 2 * self.values
        elif self.values_in_key:
            payload = self.v_dim + 2 * (self.k_dim - self.v_dim) + 1
        else:
            payload = self.values + 2 * self.n_kv_heads
        self.row_bytes = _in_32_bits(
            (payload + 15) // 16 * 16 if row_bytes is None else int(row_bytes), "row_bytes")
        self.c = gpb_row_format(codes[dtype] | (HELD_E4M3 if held else 0), self.n_kv_heads,
                                self.k_dim, self.v_dim, int(self.values_in_key), self.row_bytes)
        self.ref = ctypes.byref(self.c)


class Rotation:
    """Rotation of the values [start, start + 2 * len(inv_freq)) of every key and
    query head (``inv_freq`` float32 device tensor, one entry per pair).
    ``interleaved``: pairs are neighbours, else half the rotated values apart.
    ``sections``: pairs per position axis (their sum the number of pairs); one
    axis by default."""

    def __init__(self, inv_freq, start=0, interleaved=False, sections=None):
        import torch
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: a contiguous float32 vector, got %s %s"
                             % (inv_freq.dtype, tuple(inv_freq.shape)))
        self.inv_freq, self.interleaved = inv_freq, int(bool(interleaved))
        self.start = _in_32_bits(int(start), "start")
        self.pairs = pairs = inv_freq.numel()
        self.index_dtype = torch.int32
        self.sections = [pairs] if sections is None else [int(n) for n in sections]
        if not 1 <= len(self.sections) <= MAX_AXES or sum(self.sections) != pairs:
            raise ValueError("sections %s do not name the axis of %d pairs (at most %d axes)"
                             % (self.sections, pairs, MAX_AXES))
        self.c_sections = (ctypes.c_int32 * MAX_AXES)(*self.sections)


def _same_device(index, **tensors):
    """Every tensor on GPU ``index``: the launch goes there, whatever the current
    device is."""
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s is on %s, the call runs on GPU %d" % (name, t.device, index))


def _heads(t, n_tokens, n_heads, dim, dtype, what):
    """Strides (token, head) in elements of a [tokens, heads, dim] tensor whose
    last dimension is contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype != dtype or shape[0] < n_tokens or shape[1] != n_heads \
            or shape[2] != dim or stride[2] != 1:
        raise ValueError("%s: need %s [>= %d, %d, %d] with its last dimension contiguous, got "
                         "%s %s, strides %s" % (what, dtype, n_tokens, n_heads, dim, t.dtype,
                                                tuple(shape), stride))
    return stride[0], stride[1]


def _int32(t, numel, what):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < numel:
        raise ValueError("%s: need a contiguous int32 tensor of %d, got %s %s"
                         % (what, numel, t.dtype, tuple(t.shape)))
    return t.data_ptr()


def _rows_of(t, row_bytes, what):
    """Number of whole rows in a contiguous tensor of any type."""
    if not t.is_contiguous():
        raise ValueError("%s: need a contiguous tensor" % what)
    return t.numel() * t.element_size() // row_bytes


def _device_index(t, what):
    if not t.is_cuda:
        raise ValueError("%s is in host memory: the rows are made and read on the GPU" % what)
    return t.get_device()


class _on:
    """The device of a call made current (where it is not), and the stream."""

    def __init__(self, index, stream):
        import torch
        self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(index)
        self.other = None   # a stream that is not the device's current one
        self.used = torch.cuda.current_stream(index)   # the one the kernels run on
        if stream is None:
            self.raw = self.used.cuda_stream
        elif isinstance(stream, int):
            self.raw = stream
            if stream != self.used.cuda_stream:
                self.other = self.used = torch.cuda.ExternalStream(stream, device=index) \
                    if stream else torch.cuda.default_stream(index)
        else:
            if stream.device.index != index:
                raise ValueError("the stream is on %s, the tensors on GPU %d"
                                 % (stream.device, index))
            self.raw = stream.cuda_stream
            self.other = self.used = stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.raw

    def __exit__(self, *a):
        if self.guard is not None:
            return self.guard.__exit__(*a)


def row_append(fmt, k, v, pool, pool_locs, rotation=None, positions=None, rows=None, q=None,
               q_out=None, status=None, stream=None):
    """Make rows from keys ``k`` [T, n_kv_heads, k_dim] and values ``v`` (None where
    they are in the key), rotate the keys at ``positions`` (int32 [T], or [axes, T])
    and store row t at pool row ``pool_locs[t]`` (int32 [T]; -1 stores none) and, with
    ``rows``, at row t there.  ``pool`` may be None (then pool_locs too).  Queries
    ``q`` [T, heads, k_dim] are rotated into ``q_out`` (``q`` itself by default).
    A held format quantises the rows as it writes them.  One launch.  T is the length
    of ``pool_locs`` (of ``k`` without a pool)."""
    T = _in_32_bits(k.shape[0] if pool_locs is None else pool_locs.numel(), "rows to append")
    dev = _device_index(k, "k")
    if q is not None and q_out is None:
        q_out = q
    _same_device(dev, v=v, pool=pool, pool_locs=pool_locs, rows=rows, q=q, q_out=q_out,
                 positions=positions, status=status,
                 inv_freq=None if rotation is None else rotation.inv_freq)
    dtype, kd = fmt.dtype, fmt.k_dim
    k_ts, k_hs = _heads(k, T, fmt.n_kv_heads, kd, dtype, "k")
    v_ptr = v_ts = v_hs = 0
    if not fmt.values_in_key:
        if v is None:
            raise ValueError("v: the row format holds values apart from the keys")
        v_ts, v_hs = _heads(v, T, fmt.n_kv_heads, fmt.v_dim, dtype, "v")
        v_ptr = v.data_ptr()
    elif v is not None:
        raise ValueError("v: the row format holds the values in the keys")
    pool_ptr = locs_ptr = n_pool_rows = rows_ptr = 0
    if pool is not None:
        if pool_locs is None:
            raise ValueError("pool_locs: a pool needs the rows to store at")
        pool_ptr, n_pool_rows = pool.data_ptr(), _rows_of(pool, fmt.row_bytes, "pool")
        locs_ptr = _int32(pool_locs, T, "pool_locs")
    elif pool_locs is not None:
        raise ValueError("pool_locs without a pool")
    if rows is not None:
        if _rows_of(rows, fmt.row_bytes, "rows") < T:
            raise ValueError("rows: %d rows of %d bytes do not fit" % (T, fmt.row_bytes))
        rows_ptr = rows.data_ptr()
    heads = q_ptr = qo_ptr = q_ts = q_hs = qo_ts = qo_hs = 0
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        q_ts, q_hs = _heads(q, T, heads, kd, dtype, "q")
        qo_ts, qo_hs = _heads(q_out, T, heads, kd, dtype, "q_out")
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
    if rotation is not None and rotation.pairs:
        if positions is None:
            raise ValueError("positions: a rotation needs them")
        n, shape = len(rotation.sections), positions.shape
        stride = positions.stride()
        if positions.dtype != rotation.index_dtype or len(shape) not in (1, 2) or \
                (shape[0] if len(shape) == 2 else 1) != n or shape[-1] < T or \
                (T > 1 and stride[-1] != 1):
            raise ValueError("positions: need int32 [%d, >= %d], got %s %s"
                             % (n, T, positions.dtype, tuple(shape)))
        turn = (rotation.start, 2 * rotation.pairs, rotation.interleaved, n, rotation.c_sections,
                rotation.inv_freq.data_ptr(), positions.data_ptr(),
                stride[0] if len(shape) == 2 else 0)
    else:
        turn = ()
    a = gpb_append(T, heads, k.data_ptr(), v_ptr, k_ts, k_hs, v_ts, v_hs, pool_ptr, n_pool_rows,
                   locs_ptr, rows_ptr, q_ptr, qo_ptr, q_ts, q_hs, qo_ts, qo_hs, *turn)
    with _on(dev, stream) as st:
        rc = lib.gpb_row_append(fmt.ref, ctypes.byref(a),
                                None if status is None else status.data_ptr(), st)
    if rc != OK:
        _check(rc, "gpb_row_append")


def rows_read(fmt, rows, locs=None, n_rows=None, out=None, status=None, stream=None):
    """Rows held in 8 bits back as rows of ``fmt.dtype``: row i of ``out`` [n, values]
    is what row ``locs[i]`` of ``rows`` (a pool, a dense buffer, packed rows) stands
    for, a row of zeros where ``locs[i]`` is -1; without ``locs`` (int32) row i of
    ``rows``, all of them or the first ``n_rows``.  Exact.  ``out``'s rows may lie
    apart, by less than 2^31 bytes; without ``out`` one is allocated.  One launch.
    Returns ``out``."""
    import torch
    if fmt.held is None:
        raise ValueError("rows of 16 bits a value need no reading back")
    dev = _device_index(rows, "rows")
    _same_device(dev, locs=locs, out=out, status=status)
    n_src = _rows_of(rows, fmt.row_bytes, "rows")
    n = (n_src if locs is None else locs.numel()) if n_rows is None else int(n_rows)
    if n < 0 or (locs is None and n > n_src):
        raise ValueError("%d rows of %d" % (n, n_src))
    locs_ptr = None if locs is None else _int32(locs, _in_32_bits(n, "rows to read"), "locs")
    on = _on(dev, stream)
    with on as st:
        if out is None:
            with torch.cuda.stream(on.used):   # it belongs to the stream the kernel runs on
                out = torch.empty(n, fmt.values, dtype=fmt.dtype, device=rows.device)
        if out.dim() != 2 or out.dtype != fmt.dtype or out.shape[0] < n or \
                out.shape[1] != fmt.values or out.stride(1) != 1:
            raise ValueError("out: need %s [>= %d, %d] with its last dimension contiguous, got "
                             "%s %s, strides %s" % (fmt.dtype, n, fmt.values, out.dtype,
                                                    tuple(out.shape), out.stride()))
        apart = _in_32_bits(2 * (out.stride(0) if out.shape[0] > 1 else fmt.values),
                            "bytes from one row of out to the next")
        rc = lib.gpb_rows_read(fmt.ref, rows.data_ptr(), n_src, locs_ptr, n, out.data_ptr(), apart,
                               None if status is None else status.data_ptr(), st)
    if rc != OK:
        _check(rc, "gpb_rows_read")
    return out


# Lists of dropped plans that streams made elsewhere may still read, each with the
# events that say when they have been.
_lists_in_use = []


class AttendPlan:
    """The work list of an attention over one batch, on the device: request r has
    ``q_lens[r]`` queries, the last of its ``kv_lens[r]`` keys.  A query sees the
    keys up to its own position, with ``window`` only the last ``window`` of them
    and the first ``sinks`` of the sequence.  ``groups`` lists (first request,
    number of requests, shared keys): consecutive requests that begin with the same
    whole pages, read once for all of them (paged attention only).  One plan serves
    every layer of the batch, on any stream, and may be dropped while calls with it
    are under way; a captured graph needs it for as long as it is replayed, and
    serves its lengths alone.  Making one takes 40 to 90 us for a decode batch, which
    needs a new one every step, to 0.7 ms for 44,600 queries, and waits for the
    current stream (the list is copied to the device from ordinary memory)."""

    def __init__(self, fmt, n_heads, q_lens, kv_lens, window=0, sinks=0, page_size=64,
                 groups=(), device="cuda"):
        import torch
        h_q, h_kv, h_g = _host_i32(q_lens), _host_i32(kv_lens), _host_i32(list(groups))
        if h_q.size != h_kv.size:
            raise ValueError("%d q_lens, %d kv_lens" % (h_q.size, h_kv.size))
        if h_g.size % 3:
            raise ValueError("groups: (first request, number of requests, shared keys) each")
        shape = gpb_attend_shape(h_q.size, _in_32_bits(int(n_heads), "n_heads"),
                                 _in_32_bits(int(window), "window"),
                                 _in_32_bits(int(sinks), "sinks"),
                                 _in_32_bits(int(page_size), "page_size"), h_q.ctypes.data if h_q.size else None,
                                 h_kv.ctypes.data if h_q.size else None, h_g.size // 3,
                                 h_g.ctypes.data if h_g.size else None)
        _lists_in_use[:] = [x for x in _lists_in_use if any(not e.query() for e in x[1].values())]
        self.fmt, self.n_heads, self.readers = fmt, int(n_heads), {}
        self.c = gpb_attend_plan()
        _check(lib.gpb_attend_plan_build(ctypes.byref(fmt.c), ctypes.byref(shape),
                                         ctypes.byref(self.c), None, 0),
               "gpb_attend_plan_build")
        self.list_host = np.zeros(max(self.c.list_ints, 4), np.int32)
        _check(lib.gpb_attend_plan_build(ctypes.byref(fmt.c), ctypes.byref(shape),
                                         ctypes.byref(self.c), self.list_host.ctypes.data,
                                         self.list_host.size), "gpb_attend_plan_build")
        self.n_tokens, self.bs = self.c.n_tokens, self.c.bs
        self.workspace_bytes = self.c.workspace_bytes
        dev = _gpu_device(device)
        self.device = torch.device("cuda", torch.cuda.current_device()) \
            if dev.index is None else dev
        self.list = torch.from_numpy(self.list_host).to(self.device)
        self.list_stream = torch.cuda.current_stream(self.device).cuda_stream
        self.list_ptr, self.ref = self.list.data_ptr(), ctypes.byref(self.c)

    def read_on(self, on):
        """Kernels on the stream of ``on`` read the list: should the plan go before
        they end, its memory is not handed out until they have.  The allocator sees
        to that on streams of torch.  It would do so by an event on the stream when
        the list goes, and a stream made elsewhere may be gone by then, so there the
        event is recorded now (not into a capture: a graph needs its plan anyway)."""
        if on.raw == self.list_stream:
            return
        if on.raw == 0 or on.used.stream_id != on.raw:
            self.list.record_stream(on.used)
            return
        import torch
        with torch.cuda.stream(on.used):
            if not torch.cuda.is_current_stream_capturing():
                self.readers.setdefault(on.raw, torch.cuda.Event()).record()

    readers = {}   # events of streams made elsewhere, by handle

    def __del__(self):
        if self.readers and _lists_in_use is not None:   # (at exit it may be gone)
            _lists_in_use.append((self.list, self.readers))

    def room(self, out, lse, own_lse, workspace):
        """Results and workspace of one call, where the caller has none."""
        import torch
        if out is None:
            out = torch.empty(self.n_tokens, self.n_heads, self.fmt.v_dim, dtype=self.fmt.dtype,
                              device=self.device)
        if own_lse:
            lse = torch.empty(self.n_tokens, self.n_heads, dtype=torch.float32,
                              device=self.device)
        if workspace is None and self.workspace_bytes:
            workspace = self.workspace()
        return out, lse, workspace

    def workspace(self):
        """A workspace for one call at a time."""
        import torch
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)


def _attend(plan, q, scale, out, lse, workspace, status, stream, call, what, **tensors):
    import torch
    fmt, T, dev = plan.fmt, plan.n_tokens, plan.device
    own_lse = lse is True
    if lse is True or lse is False:
        lse = None
    _same_device(dev.index, q=q, out=out, lse=lse, workspace=workspace, status=status, **tensors)
    q_ts, q_hs = _heads(q, T, plan.n_heads, fmt.k_dim, fmt.dtype, "q")
    on = _on(dev.index, stream)
    with on as st:
        if out is None or own_lse or (workspace is None and plan.workspace_bytes):
            if on.other is None:
                out, lse, workspace = plan.room(out, lse, own_lse, workspace)
            else:   # what is allocated here belongs to the stream the kernels run on
                with torch.cuda.stream(on.other):
                    out, lse, workspace = plan.room(out, lse, own_lse, workspace)
        o_ts, o_hs = _heads(out, T, plan.n_heads, fmt.v_dim, fmt.dtype, "out")
        if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or
                                lse.dim() != 2 or lse.shape[0] < T or
                                lse.shape[1] != plan.n_heads):
            raise ValueError("lse: need a contiguous float32 [>= %d, %d], got %s %s"
                             % (T, plan.n_heads, lse.dtype, tuple(lse.shape)))
        n = 0
        if workspace is not None:
            n = _rows_of(workspace, 1, "workspace")
        io = gpb_attend_io(q.data_ptr(), q_ts, q_hs, out.data_ptr(), o_ts, o_hs,
                           0 if lse is None else lse.data_ptr(), scale)
        rc = call(ctypes.byref(io), workspace.data_ptr() if n else None, n,
                  None if status is None else status.data_ptr(), st)
        plan.read_on(on)
    if rc != OK:
        _check(rc, what)
    return out, lse


def attend_dense(plan, q, dense, k_bases, scale, out=None, lse=True, workspace=None,
                 status=None, stream=None):
    """Attention of the packed queries ``q`` [T, heads, k_dim] over the dense buffer of
    a compose: key x of request r is row ``k_bases[r] + x`` of ``dense``.  Returns
    (out [T, heads, v_dim], lse [T, heads] float32, or None with ``lse=None``).
    Without a workspace one is allocated for the call."""
    rows, bases = _rows_of(dense, plan.fmt.row_bytes, "dense"), _int32(k_bases, plan.bs, "k_bases")
    return _attend(plan, q, scale, out, lse, workspace, status, stream,
                   lambda io, ws, n, word, st: lib.gpb_attend_dense(
                       plan.ref, plan.list_ptr, io, dense.data_ptr(), rows, bases, ws, n, word,
                       st),
                   "gpb_attend_dense", dense=dense, k_bases=k_bases)


def attend_paged(plan, q, pool, pages, scale, page_base=None, out=None, lse=True,
                 workspace=None, status=None, stream=None):
    """Attention of the packed queries over the paged pool.  ``pages`` is a table
    [bs, pages] of int32 pool pages, or with ``page_base`` (int32 [bs]) one list in
    which request r's pages start at entry ``page_base[r]`` (a compose plan's
    slot_pages and slot_base).  Returns as attend_dense."""
    rows = _rows_of(pool, plan.fmt.row_bytes, "pool")
    stride = base = 0
    if page_base is None:
        if pages.dim() != 2 or pages.shape[0] < plan.bs:
            raise ValueError("pages: need a table [>= %d, pages], got %s"
                             % (plan.bs, tuple(pages.shape)))
        stride = pages.shape[1]
    else:
        base = _int32(page_base, plan.bs, "page_base")
    listed, table = pages.numel(), _int32(pages, 0, "pages")
    return _attend(plan, q, scale, out, lse, workspace, status, stream,
                   lambda io, ws, n, word, st: lib.gpb_attend_paged(
                       plan.ref, plan.list_ptr, io, pool.data_ptr(), rows, table, listed,
                       base or None, stride, ws, n, word, st),
                   "gpb_attend_paged", pool=pool, pages=pages, page_base=page_base)
