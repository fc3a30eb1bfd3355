"""ctypes binding of libfpstok (include/fpstok.h).

Argument marshalling only: PyTorch supplies device memory and the current
HIP stream; every step of the tokenizer runs in the library's gfx950 kernels.
The library must have been built (``__graft_entry__.build()`` or
``python -m point_cloud_tokenization_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfpstok.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "fpstok.h")

OK, EINVAL, EWORKSPACE, EUNSUPPORTED, EHIP, EDEVICE = 0, 1, 2, 3, 4, 5
VORONOI, KNN = 0, 1
F32, F16, BF16, I32 = 0, 1, 2, 3  # fpstok_dtype
MAX_PATCHES, MAX_K, MAX_LLOYD = 1024, 64, 1000
NOALLOC_MAX_WORKSPACE = 64 << 20  # FPSTOK_NOALLOC_MAX_WORKSPACE
MAX_HEAD_DIM, MAX_SINKS, MAX_AXES = 128, 64, 4
MAX_WIDTH, MAX_BUCKETS = 8192, 128
NORMS = {"none": 0, "rms": 1, "layer": 2}  # fpstok_norm
GATES = {"none": 0, "row": 1, "sequence": 2}  # fpstok_gate
ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2}  # fpstok_act


class FpstokError(RuntimeError):
    def __init__(self, status, where, detail):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (where, _STATUS.get(status, status), detail))


_STATUS = {OK: "ok", EINVAL: "invalid argument", EWORKSPACE: "workspace too small",
           EUNSUPPORTED: "unsupported", EHIP: "HIP runtime error",
           EDEVICE: "device-side failure"}


class Batch(ctypes.Structure):
    _fields_ = [("coords", ctypes.c_void_p), ("features", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("num_events", ctypes.c_int64),
                ("num_points", ctypes.c_int64), ("num_features", ctypes.c_int32),
                ("charge_col", ctypes.c_int32), ("max_event_points", ctypes.c_int64),
                ("coords_dtype", ctypes.c_int32), ("features_dtype", ctypes.c_int32)]


class Params(ctypes.Structure):
    _fields_ = [("num_patches", ctypes.c_int32), ("k", ctypes.c_int32),
                ("lloyd_iters", ctypes.c_int32), ("assign_mode", ctypes.c_int32),
                ("pool_weighted", ctypes.c_int32)]


class Seqs(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int64), ("num_rows", ctypes.c_int64),
                ("cu_seqlens", ctypes.c_void_p), ("token_count", ctypes.c_void_p),
                ("capacity", ctypes.c_int32), ("max_len", ctypes.c_int32)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class AttnParams(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("window_left", ctypes.c_int32), ("window_right", ctypes.c_int32),
                ("num_sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


class RopeParams(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("positions_dtype", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("pairs", ctypes.c_int32 * 4), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32)]


class RelBias(ctypes.Structure):
    _fields_ = [("q_positions", ctypes.c_void_p), ("k_positions", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("positions_dtype", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("buckets", ctypes.c_int32 * 4),
                ("log_steps", ctypes.c_int32 * 4), ("rate", ctypes.c_float * 4),
                ("shift", ctypes.c_float * 4)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class ResidualParams(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("stream_dtype", ctypes.c_int32),
                ("branch_dtype", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("pre_norm", ctypes.c_int32), ("gate_per", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("eps", ctypes.c_float)]


class ResidualWeights(ctypes.Structure):
    """fpstok_residual_weights, and with the gradients' pointers
    fpstok_residual_weight_grads."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("post_weight", "post_bias", "scale", "pre_weight",
                                               "pre_bias")]


_lib = None


def lib():
    """The loaded libfpstok (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfpstok.so is not built (%s); run __graft_entry__.build()"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        B, Pp = ctypes.POINTER(Batch), ctypes.POINTER(Params)
        L.fpstok_workspace_size.argtypes = [B, Pp]
        L.fpstok_workspace_size.restype = sz
        L.fpstok_sample.argtypes = [B, Pp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fpstok_assign.argtypes = [B, Pp, vp, vp, vp, vp, sz, vp]
        L.fpstok_knn.argtypes = [B, Pp, vp, vp, vp, vp, sz, vp]
        L.fpstok_lloyd.argtypes = [B, Pp, vp, vp, vp, vp, sz, vp]
        L.fpstok_pool.argtypes = [B, Pp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fpstok_tokenize.argtypes = [B, Pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fpstok_tokenize_noalloc.argtypes = [B, Pp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.fpstok_validate.argtypes = [B, vp]
        i64, i32 = ctypes.c_int64, ctypes.c_int32
        L.fpstok_pack.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, vp]
        L.fpstok_unpack.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp]
        L.fpstok_pool_backward.argtypes = [B, Pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fpstok_random_start.argtypes = [vp, i64, ctypes.c_uint64, ctypes.c_uint64, vp, vp]
        L.fpstok_device_status.argtypes = [vp, sz, vp]
        L.fpstok_debug_set_spin_limit.argtypes = [ctypes.c_uint32]
        L.fpstok_debug_set_spin_limit.restype = None
        L.fpstok_upcast.argtypes = [vp, i64, i32, vp, vp]
        S, A = ctypes.POINTER(Seqs), ctypes.POINTER(AttnParams)
        L.fpstok_attention.argtypes = [S, S, A] + [ctypes.POINTER(Heads)] * 4 + [vp, vp, sz, vp]
        L.fpstok_attention_backward.argtypes = [S, S, A] + [ctypes.POINTER(Heads)] * 4 + [vp] + \
            [ctypes.POINTER(Heads)] * 4 + [vp, sz, vp]
        L.fpstok_attention_workspace_size.argtypes = [S, S, A, i32]
        L.fpstok_attention_workspace_size.restype = sz
        L.fpstok_rope.argtypes = [S, ctypes.POINTER(RopeParams), vp, vp] + \
            [ctypes.POINTER(Heads)] * 4 + [vp]
        RB = ctypes.POINTER(RelBias)
        L.fpstok_attention_bias.argtypes = [S, S, A, RB] + [ctypes.POINTER(Heads)] * 4 + \
            [vp, vp, sz, vp]
        L.fpstok_attention_bias_backward.argtypes = [S, S, A, RB] + \
            [ctypes.POINTER(Heads)] * 4 + [vp] + [ctypes.POINTER(Heads)] * 4 + [vp, vp, sz, vp]
        L.fpstok_attention_bias_workspace_size.argtypes = [S, S, A, RB, i32]
        L.fpstok_attention_bias_workspace_size.restype = sz
        RP, RW = ctypes.POINTER(ResidualParams), ctypes.POINTER(ResidualWeights)
        R = ctypes.POINTER(Rows)
        L.fpstok_residual.argtypes = [S, RP, RW] + [R] * 5 + [vp, vp]
        L.fpstok_residual_backward.argtypes = [S, RP, RW] + [R] * 3 + [vp] + [R] * 5 + \
            [RW, vp, sz, vp]
        L.fpstok_residual_workspace_size.argtypes = [S, RP]
        L.fpstok_residual_workspace_size.restype = sz
        for f in ("fpstok_attention", "fpstok_attention_backward", "fpstok_rope",
                  "fpstok_attention_bias", "fpstok_attention_bias_backward",
                  "fpstok_residual", "fpstok_residual_backward",
                  "fpstok_sample", "fpstok_assign", "fpstok_knn", "fpstok_lloyd",
                  "fpstok_pool", "fpstok_tokenize", "fpstok_validate", "fpstok_pack",
                  "fpstok_unpack", "fpstok_pool_backward", "fpstok_random_start",
                  "fpstok_device_status", "fpstok_tokenize_noalloc", "fpstok_upcast"):
            getattr(L, f).restype = ctypes.c_int
        L.fpstok_status_string.argtypes = [ctypes.c_int]
        L.fpstok_status_string.restype = ctypes.c_char_p
        L.fpstok_last_error.argtypes = []
        L.fpstok_last_error.restype = ctypes.c_char_p
        L.fpstok_version.argtypes = []
        L.fpstok_version.restype = ctypes.c_int
        _lib = L
    return _lib


def declared_functions():
    """Names of the functions include/fpstok.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fpstok_[a-z_]+)\s*\(", text)))


def _check(rc, where):
    if rc != OK:
        raise FpstokError(rc, where, lib().fpstok_last_error().decode())


def version():
    return lib().fpstok_version()


# ------------------------------------------------------------ tensor helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, dev=None):
    import torch

    if t is None:
        raise ValueError("%s is required" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if dev is not None and t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _dtype_code(t, name):
    import torch

    codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    if t.dtype not in codes:
        raise TypeError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    return codes[t.dtype]


def make_batch(coords, offsets, features=None, charge_col=-1, max_event_points=0):
    """A Batch struct over the given tensors (which the caller keeps alive).
    coords and features may each be float32, float16 or bfloat16; the library
    upcasts 16-bit inputs exactly to float32 before using them.
    max_event_points: optional host-side bound on the pulses of any event (0:
    unknown); see fpstok_batch in include/fpstok.h."""
    import torch

    cd = _dtype_code(coords, "coords")
    _need(coords, coords.dtype, "coords")
    _need(offsets, torch.int64, "offsets", coords.device)
    if coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be [N,4]")
    C, fd = 0, F32
    if features is not None:
        fd = _dtype_code(features, "features")
        _need(features, features.dtype, "features", coords.device)
        if features.dim() != 2 or features.shape[0] != coords.shape[0]:
            raise ValueError("features must be [N,C]")
        C = features.shape[1]
    bt = Batch(coords.data_ptr(), features.data_ptr() if features is not None else None,
               offsets.data_ptr(), offsets.numel() - 1, coords.shape[0], C, charge_col,
               int(max_event_points), cd, fd)
    return bt


def upcast(src, out, stream=None):
    """out[i] = float32 value of the float16 / bfloat16 src[i] (exact)."""
    import torch

    code = _dtype_code(src, "src")
    if code == F32:
        raise TypeError("src must be float16 or bfloat16")
    _need(src, src.dtype, "src")
    _need(out, torch.float32, "out", src.device)
    if out.numel() != src.numel():
        raise ValueError("out must have as many elements as src")
    _check(lib().fpstok_upcast(_ptr(src), src.numel(), code, _ptr(out),
                               _stream_handle(stream)), "fpstok_upcast")


def make_params(num_patches=128, k=16, lloyd_iters=0, assign_mode=VORONOI, pool_weighted=1):
    return Params(num_patches, k, lloyd_iters, assign_mode, pool_weighted)


def workspace_size(bt, pr):
    return lib().fpstok_workspace_size(ctypes.byref(bt), ctypes.byref(pr))


def alloc_workspace(bt, pr, device):
    import torch

    n = workspace_size(bt, pr)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


# ----------------------------------------------------------- the five calls

def sample(bt, pr, centroid_idx, centroids, token_count, assign, ws, start_idx=None,
           stream=None):
    _check(lib().fpstok_sample(ctypes.byref(bt), ctypes.byref(pr), _ptr(start_idx),
                               _ptr(centroid_idx), _ptr(centroids), _ptr(token_count),
                               _ptr(assign), _ptr(ws), ws.numel(), _stream_handle(stream)),
           "fpstok_sample")


def assign(bt, pr, centroids, token_count, out, ws, stream=None):
    _check(lib().fpstok_assign(ctypes.byref(bt), ctypes.byref(pr), _ptr(centroids),
                               _ptr(token_count), _ptr(out), _ptr(ws), ws.numel(),
                               _stream_handle(stream)), "fpstok_assign")


def knn(bt, pr, centroids, token_count, knn_idx, ws, stream=None):
    _check(lib().fpstok_knn(ctypes.byref(bt), ctypes.byref(pr), _ptr(centroids),
                            _ptr(token_count), _ptr(knn_idx), _ptr(ws), ws.numel(),
                            _stream_handle(stream)), "fpstok_knn")


def lloyd(bt, pr, centroids, token_count, assign_, ws, stream=None):
    _check(lib().fpstok_lloyd(ctypes.byref(bt), ctypes.byref(pr), _ptr(centroids),
                              _ptr(token_count), _ptr(assign_), _ptr(ws), ws.numel(),
                              _stream_handle(stream)), "fpstok_lloyd")


def pool(bt, pr, token_count, assign_, knn_idx, pooled, cell_count, ws, stream=None):
    _check(lib().fpstok_pool(ctypes.byref(bt), ctypes.byref(pr), _ptr(token_count),
                             _ptr(assign_), _ptr(knn_idx), _ptr(pooled), _ptr(cell_count),
                             _ptr(ws), ws.numel(), _stream_handle(stream)), "fpstok_pool")


def pool_backward(bt, pr, token_count, assign_, knn_idx, pooled, grad_pooled, grad_features,
                  ws, stream=None):
    """fpstok_pool_backward: gradient of the pooling with respect to the features."""
    _check(lib().fpstok_pool_backward(ctypes.byref(bt), ctypes.byref(pr), _ptr(token_count),
                                      _ptr(assign_), _ptr(knn_idx), _ptr(pooled),
                                      _ptr(grad_pooled), _ptr(grad_features), _ptr(ws),
                                      ws.numel(), _stream_handle(stream)), "fpstok_pool_backward")


def random_start(offsets, start_idx, seed, step=0, stream=None):
    """fpstok_random_start: a random FPS start per event into start_idx [B]
    int32 (offsets [B+1] int64), from Philox4x32-10 with the given seed and
    step."""
    import torch

    _need(offsets, torch.int64, "offsets")
    _need(start_idx, torch.int32, "start_idx")
    B = offsets.numel() - 1
    _check(lib().fpstok_random_start(_ptr(offsets), B, int(seed) & (2**64 - 1),
                                     int(step) & (2**64 - 1), _ptr(start_idx),
                                     _stream_handle(stream)), "fpstok_random_start")


def pack(token_count, rows, packed, doc_id, cu_seqlens, stream=None):
    """fpstok_pack on device tensors: token_count [B] int32, rows [B,P,D]
    float32; packed [B*P,D] float32, doc_id [B*P] int32 (or None) and
    cu_seqlens [B+1] int32 are written."""
    import torch

    B, P, D = rows.shape
    _need(token_count, torch.int32, "token_count")
    _need(rows, torch.float32, "rows")
    _need(packed, torch.float32, "packed")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    if doc_id is not None:
        _need(doc_id, torch.int32, "doc_id")
    _check(lib().fpstok_pack(B, P, D, _ptr(token_count), _ptr(rows), _ptr(packed), _ptr(doc_id),
                             _ptr(cu_seqlens), _stream_handle(stream)), "fpstok_pack")


def unpack(token_count, cu_seqlens, packed, rows, stream=None):
    """fpstok_unpack: rows [B,P,D] float32 from the packed rows."""
    import torch

    B, P, D = rows.shape
    for t, dt, name in ((token_count, torch.int32, "token_count"),
                        (cu_seqlens, torch.int32, "cu_seqlens"),
                        (packed, torch.float32, "packed"), (rows, torch.float32, "rows")):
        _need(t, dt, name)
    _check(lib().fpstok_unpack(B, P, D, _ptr(token_count), _ptr(cu_seqlens), _ptr(packed),
                               _ptr(rows), _stream_handle(stream)), "fpstok_unpack")


def tokenize_call(bt, pr, centroid_idx, centroids, token_count, assign_, knn_idx, pooled,
                  cell_count, ws, start_idx=None, stream=None):
    """fpstok_tokenize: the whole tokenizer in one call."""
    _check(lib().fpstok_tokenize(ctypes.byref(bt), ctypes.byref(pr), _ptr(start_idx),
                                 _ptr(centroid_idx), _ptr(centroids), _ptr(token_count),
                                 _ptr(assign_), _ptr(knn_idx), _ptr(pooled), _ptr(cell_count),
                                 _ptr(ws), ws.numel(), _stream_handle(stream)), "fpstok_tokenize")


def tokenize_noalloc_call(bt, pr, centroid_idx, centroids, token_count, assign_, knn_idx,
                          pooled, cell_count, start_idx=None, stream=None):
    """fpstok_tokenize_noalloc: the whole tokenizer with the library's fixed
    scratch region as its workspace (no allocation)."""
    _check(lib().fpstok_tokenize_noalloc(ctypes.byref(bt), ctypes.byref(pr), _ptr(start_idx),
                                         _ptr(centroid_idx), _ptr(centroids), _ptr(token_count),
                                         _ptr(assign_), _ptr(knn_idx), _ptr(pooled),
                                         _ptr(cell_count), _stream_handle(stream)),
           "fpstok_tokenize_noalloc")


def validate(bt, stream=None):
    _check(lib().fpstok_validate(ctypes.byref(bt), _stream_handle(stream)), "fpstok_validate")


def device_status(ws, stream=None):
    """fpstok_device_status: raises FpstokError (status EDEVICE) if a bounded
    wait between workgroups gave up in the last sample / tokenize call on the
    workspace tensor `ws`.  Synchronizes the stream."""
    _check(lib().fpstok_device_status(_ptr(ws), ws.numel(), _stream_handle(stream)),
           "fpstok_device_status")


def debug_set_spin_limit(polls):
    """Testing only: polls before a wait between workgroups gives up (0: the
    default)."""
    lib().fpstok_debug_set_spin_limit(int(polls))


# ------------------------------------------------------------- convenience

def offsets_from_batch_ids(batch_ids, num_events):
    """CSR offsets [B+1] from sorted per-pulse event ids (device-side; pass
    num_events to avoid a host sync)."""
    import torch

    counts = torch.bincount(batch_ids, minlength=num_events)
    off = torch.zeros(num_events + 1, dtype=torch.int64, device=batch_ids.device)
    torch.cumsum(counts, 0, out=off[1:])
    return off


class Tokenizer:
    """Preallocated outputs and workspace for one batch shape; call() runs the
    whole tokenizer (sample -> [Lloyd] -> [kNN] -> pool) on the current
    stream without host synchronization."""

    def __init__(self, coords, features, offsets, num_patches=128, assign_mode="voronoi", k=16,
                 lloyd_iters=0, pool="charge", charge_col=-1, max_event_points=0):
        import torch

        self.mode = {"voronoi": VORONOI, "knn": KNN}[assign_mode]
        self.coords, self.features, self.offsets = coords, features, offsets
        self.bt = make_batch(coords, offsets, features, charge_col, max_event_points)
        self.pr = make_params(num_patches, k, lloyd_iters, self.mode,
                              1 if pool == "charge" else 0)
        dev = coords.device
        B, N, P = offsets.numel() - 1, coords.shape[0], num_patches
        C = features.shape[1]
        self.out = dict(
            centroid_idx=torch.empty((B, P), dtype=torch.int32, device=dev),
            centroids=torch.empty((B, P, 4), dtype=torch.float32, device=dev),
            token_count=torch.empty(B, dtype=torch.int32, device=dev),
            # the Voronoi slots are computed in Voronoi mode and for Lloyd
            assign=torch.empty(N, dtype=torch.int32, device=dev)
            if self.mode == VORONOI or lloyd_iters > 0 else None,
            knn_idx=torch.empty((B, P, k), dtype=torch.int32, device=dev)
            if self.mode == KNN else None,
            pooled=torch.empty((B, P, C), dtype=torch.float32, device=dev),
            cell_count=torch.empty((B, P), dtype=torch.int32, device=dev),
        )
        self.ws = alloc_workspace(self.bt, self.pr, dev)
        # the call's fixed arguments, marshalled once; only the stream is
        # looked up per call (torch's current stream on this device)
        o = self.out
        self._fn = lib().fpstok_tokenize
        self._head = (ctypes.byref(self.bt), ctypes.byref(self.pr))
        self._tail = (_ptr(o["centroid_idx"]), _ptr(o["centroids"]), _ptr(o["token_count"]),
                      _ptr(o["assign"]), _ptr(o["knn_idx"]), _ptr(o["pooled"]),
                      _ptr(o["cell_count"]), _ptr(self.ws), self.ws.numel())
        self._dev = dev.index if dev.index is not None else torch.cuda.current_device()
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def __call__(self, start_idx=None, stream=None):
        """fpstok_tokenize on the preallocated buffers."""
        if stream is None and self._raw_stream is not None:
            rc = self._fn(*self._head, _ptr(start_idx), *self._tail,
                          ctypes.c_void_p(self._raw_stream(self._dev)))
            if rc != OK:
                _check(rc, "fpstok_tokenize")
            return self.out
        o = self.out
        tokenize_call(self.bt, self.pr, o["centroid_idx"], o["centroids"], o["token_count"],
                      o["assign"], o["knn_idx"], o["pooled"], o["cell_count"], self.ws,
                      start_idx, stream)
        return o

    def check(self, stream=None):
        """Raise if the last call's outputs are not valid (fpstok_device_status;
        synchronizes)."""
        device_status(self.ws, stream)

    def stepwise(self, start_idx=None, stream=None):
        """The same result through the five separate calls."""
        o = self.out
        sample(self.bt, self.pr, o["centroid_idx"], o["centroids"], o["token_count"],
               o["assign"], self.ws, start_idx, stream)
        if self.pr.lloyd_iters > 0:
            lloyd(self.bt, self.pr, o["centroids"], o["token_count"], o["assign"], self.ws,
                  stream)
        if self.mode == KNN:
            knn(self.bt, self.pr, o["centroids"], o["token_count"], o["knn_idx"], self.ws,
                stream)
        pool(self.bt, self.pr, o["token_count"], o["assign"], o["knn_idx"], o["pooled"],
             o["cell_count"], self.ws, stream)
        return o


def tokenize(coords, features, offsets=None, batch_ids=None, num_events=None, num_patches=128,
             assign_mode="voronoi", k=16, lloyd_iters=0, pool="charge", charge_col=-1,
             start_idx=None, stream=None):
    """Tokenize one batch: returns a dict of device tensors (centroid_idx,
    centroids, token_count, assign, knn_idx or None, pooled, cell_count)."""
    if offsets is None:
        if batch_ids is None or num_events is None:
            raise ValueError("give offsets, or batch_ids with num_events")
        offsets = offsets_from_batch_ids(batch_ids, num_events)
    t = Tokenizer(coords, features, offsets, num_patches, assign_mode, k, lloyd_iters, pool,
                  charge_col)
    return t(start_idx, stream)


# --------------------------------------------- attention over the tokens

def make_seqs(num_rows, cu_seqlens=None, token_count=None, capacity=0, max_len=0):
    """A Seqs struct (fpstok_seqs): the rows of a batch of sequences, packed
    (cu_seqlens [B+1] int32, as pack writes it) or padded (token_count [B]
    int32 with `capacity` slots per sequence).  max_len: optional host-side
    bound on any length (0: unknown).  The struct keeps its tensor alive."""
    import torch

    if (cu_seqlens is None) == (token_count is None):
        raise ValueError("give cu_seqlens or token_count")
    t = cu_seqlens if token_count is None else token_count
    _need(t, torch.int32, "cu_seqlens" if token_count is None else "token_count")
    if t.dim() != 1 or (token_count is None and t.numel() < 1):
        raise ValueError("cu_seqlens must be [B+1], token_count [B]")
    if token_count is None:
        s = Seqs(t.numel() - 1, int(num_rows), t.data_ptr(), None, 0, int(max_len))
    else:
        s = Seqs(t.numel(), int(num_rows), None, t.data_ptr(), int(capacity), int(max_len))
    s.tensor = t
    return s


def make_heads(t, name, heads=None, rows=None, like=None):
    """A Heads struct over a [rows, heads, D] device tensor (any row and head
    stride, adjacent elements), which the caller keeps alive."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError("%s must be [rows, heads, D] with adjacent elements" % name)
    if (heads is not None and t.shape[1] != heads) or (rows is not None and t.shape[0] != rows):
        raise ValueError("%s must hold %s rows of %s heads, got %s" % (name, rows, heads,
                                                                     tuple(t.shape)))
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
        if t.device != like.device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, like.device))
        if t.shape[2] != like.shape[2]:
            raise ValueError("%s must have heads of %d elements" % (name, like.shape[2]))
    # (the stride of a single row or head is not used, and may be anything)
    return Heads(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0,
                 t.stride(1) if t.shape[1] > 1 else 0)


class _DeviceCall:
    """Calls a library function on the stream of one device.  Buffers that the
    constructor allocates are for calls on any stream: a stream other than the
    one they were filled on waits for that before its first call, and the
    allocator does not give them to others before that stream is done with
    them."""

    def __init__(self, device):
        import torch

        self.device = device
        self._index = device.index if device.index is not None else torch.cuda.current_device()
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._filled, self._ready, self._own = None, set(), ()

    def _allocated(self, *own):
        """The constructor's own buffers, filled on its current stream."""
        import torch

        self._own = own

        with torch.cuda.device(self._index):
            stream = torch.cuda.current_stream()
            self._ready.add(stream.cuda_stream)
            if not torch.cuda.is_current_stream_capturing():
                self._filled = torch.cuda.Event()
                self._filled.record(stream)

    def _wait_for_fills(self, stream):
        import torch

        with torch.cuda.stream(torch.cuda.current_stream() if stream is None else stream):
            # (work before a capture is no part of it: who captures has waited)
            if not torch.cuda.is_current_stream_capturing():
                here = torch.cuda.current_stream()
                here.wait_event(self._filled)
                for t in self._own:
                    t.record_stream(here)
                self._ready.add(here.cuda_stream)

    def _call(self, fn, where, args, stream):
        import torch

        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self._call(fn, where, args, stream)
        if stream is not None:
            s = stream.cuda_stream
        elif self._raw_stream is not None:
            s = self._raw_stream(self._index)
        else:
            s = torch.cuda.current_stream(self.device).cuda_stream
        if self._filled is not None and s not in self._ready:
            self._wait_for_fills(stream)
        rc = fn(*args, ctypes.c_void_p(s))
        if rc != OK:
            _check(rc, where)


class BiasAxis:
    """One axis of a RelativeBias: its buckets, the rate that turns positions
    into units, the shift, and the buckets per doubling of a log axis (0:
    linear).  Without a shift distance 0 is in the middle."""

    def __init__(self, buckets, rate=1.0, shift=None, log_steps=0):
        self.buckets, self.rate, self.log_steps = int(buckets), float(rate), int(log_steps)
        if shift is None:
            shift = self.buckets // 2 if self.log_steps else self.buckets / 2
        self.shift = float(shift)


class RelativeBias:
    """A learned bias for Attention (fpstok_rel_bias): table [H, buckets of all
    axes] float32, and the rows' positions [rows, axes], float32 or int32
    (k_positions None: the queries')."""

    def __init__(self, table, axes, q_positions, k_positions=None):
        import torch

        A = len(axes)
        if not 1 <= A <= MAX_AXES:
            raise ValueError("axes must name 1 to %d axes" % MAX_AXES)
        _need(table, torch.float32, "table")
        if table.dim() != 2 or table.shape[1] != sum(a.buckets for a in axes):
            raise ValueError("table must be [heads, %d]" % sum(a.buckets for a in axes))
        if q_positions.dtype not in (torch.float32, torch.int32):
            raise TypeError("positions must be float32 or int32, got %s" % q_positions.dtype)
        for name, p in (("q_positions", q_positions), ("k_positions", k_positions)):
            if p is not None:
                _need(p, q_positions.dtype, name, table.device)
                if p.dim() != 2 or p.shape[1] != A:
                    raise ValueError("%s must be [rows, %d]" % (name, A))
        self.table, self.q_positions, self.k_positions = table, q_positions, k_positions
        pad = lambda v: list(v) + [0] * (4 - A)  # noqa: E731
        i4, f4 = ctypes.c_int32 * 4, ctypes.c_float * 4
        self.struct = RelBias(
            q_positions.data_ptr(), None if k_positions is None else k_positions.data_ptr(),
            table.data_ptr(), I32 if q_positions.dtype == torch.int32 else F32, A,
            i4(*pad(a.buckets for a in axes)), i4(*pad(a.log_steps for a in axes)),
            f4(*pad(a.rate for a in axes)), f4(*pad(a.shift for a in axes)))


class Attention(_DeviceCall):
    """fpstok_attention on given tensors, with its outputs and workspace
    allocated once, and with training=True fpstok_attention_backward; with a bias
    (RelativeBias) fpstok_attention_bias and fpstok_attention_bias_backward.

    q [q rows, H, D]; k, v [k rows, Hk, D] (float32, float16 or bfloat16, any
    row and head stride); q_seqs, k_seqs: make_seqs (k_seqs None: q_seqs).
    window = (left, right), -1 for unbounded; right = 0 is causal.  A call
    takes what the tensors hold by then; it returns (out, lse), the same
    buffers each time, and rows behind the last packed sequence keep what they
    held (0 after construction).  out and, in training, grads = (grad_q, grad_k,
    grad_v) may be given; other buffers assigned to .grads take the place of
    those before.  With a bias, grads ends with grad_table (None: the table
    gets no gradient)."""

    def __init__(self, q, k, v, q_seqs, k_seqs=None, window=(-1, -1), num_sinks=0, scale=None,
                 training=False, out=None, grads=None, bias=None):
        import torch

        super().__init__(q.device)
        qh = make_heads(q, "q", rows=q_seqs.num_rows)
        ks = q_seqs if k_seqs is None else k_seqs
        kh = make_heads(k, "k", rows=ks.num_rows, like=q)
        vh = make_heads(v, "v", rows=ks.num_rows, heads=k.shape[1], like=q)
        for s in (q_seqs, ks):
            if s.tensor.device != q.device:
                raise ValueError("the sequences are on %s, expected %s" % (s.tensor.device,
                                                                        q.device))
        D = q.shape[2]
        self.q, self.k, self.v, self.q_seqs, self.k_seqs = q, k, v, q_seqs, k_seqs
        self.params = AttnParams(q.shape[1], k.shape[1], D, _dtype_code(q, "q"), int(window[0]),
                                 int(window[1]), int(num_sinks),
                                 1.0 / D ** 0.5 if scale is None else float(scale))
        self.out = torch.zeros(q.shape, dtype=q.dtype, device=q.device) if out is None else out
        self.lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
        oh = make_heads(self.out, "out", rows=q.shape[0], heads=q.shape[1], like=q)
        self.bias, name, fixed = bias, "fpstok_attention", 3
        call = (ctypes.byref(q_seqs), None if k_seqs is None else ctypes.byref(k_seqs),
                ctypes.byref(self.params))
        if bias is not None:
            self._check_bias(bias, ks)
            name, fixed = "fpstok_attention_bias", 4
            call += (ctypes.byref(bias.struct),)
        self._head = call + (ctypes.byref(qh), ctypes.byref(kh), ctypes.byref(vh),
                             ctypes.byref(oh), _ptr(self.lse))
        size = getattr(lib(), name + "_workspace_size")
        need = [size(*self._head[:fixed], b) for b in ((0, 1) if training else (0,))]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device=q.device) if max(need) else None
        self._ws = (_ptr(self.ws), 0 if self.ws is None else self.ws.numel())
        self._name, self._fwd = name, getattr(lib(), name)
        self._bwd = getattr(lib(), name + "_backward")
        self._training, self._grads = bool(training), None
        own = [t for t in (self.lse, self.ws, self.out if out is None else None) if t is not None]
        if grads is not None:
            self.grads = grads
        elif training:
            leaves = (q, k, v) if bias is None else (q, k, v, bias.table)
            self.grads = tuple(torch.zeros(t.shape, dtype=t.dtype, device=t.device)
                               for t in leaves)
            own += self.grads
        self._allocated(*own)

    def _check_bias(self, bias, ks):
        q = self.q
        if bias.table.device != q.device:
            raise ValueError("the bias is on %s, expected %s" % (bias.table.device, q.device))
        if bias.table.shape[0] != q.shape[1]:
            raise ValueError("the bias's table must hold %d heads" % q.shape[1])
        if bias.q_positions.shape[0] != q.shape[0]:
            raise ValueError("q_positions must hold %d rows" % q.shape[0])
        if bias.k_positions is None and ks is not self.q_seqs:
            raise ValueError("k_seqs need k_positions")
        if bias.k_positions is not None and bias.k_positions.shape[0] != ks.num_rows:
            raise ValueError("k_positions must hold %d rows" % ks.num_rows)

    @property
    def grads(self):
        """(grad_q, grad_k, grad_v), with a bias also grad_table, where backward
        writes; None if not training."""
        return self._grads

    @grads.setter
    def grads(self, grads):
        if not self._training:
            raise ValueError("construct with training=True")
        grads = tuple(grads)
        if len(grads) != (3 if self.bias is None else 4):
            raise ValueError("grads must be (grad_q, grad_k, grad_v%s)" % (
                "" if self.bias is None else ", grad_table"))
        table = ()
        if self.bias is not None:
            if grads[3] is not None:
                _need(grads[3], self.bias.table.dtype, "grad_table", self.device)
                if grads[3].shape != self.bias.table.shape:
                    raise ValueError("grad_table must be %s" % (tuple(self.bias.table.shape),))
            table = (_ptr(grads[3]),)
        views = [make_heads(g, name, rows=t.shape[0], heads=t.shape[1], like=t)
                 for name, g, t in zip(("grad_q", "grad_k", "grad_v"), grads,
                                       (self.q, self.k, self.v))]
        self._grads = grads
        self._tail = tuple(ctypes.byref(h) for h in views) + table + self._ws

    def __call__(self, stream=None):
        """fpstok_attention (with a bias fpstok_attention_bias): (out, lse)."""
        self._call(self._fwd, self._name, self._head + self._ws, stream)
        return self.out, self.lse

    def backward(self, grad_out, stream=None):
        """fpstok_attention_backward after a call on the same inputs:
        (grad_q, grad_k, grad_v), with a bias also grad_table."""
        if self._grads is None:
            raise ValueError("construct with training=True")
        gh = make_heads(grad_out, "grad_out", rows=self.q.shape[0], heads=self.q.shape[1],
                        like=self.q)
        self._call(self._bwd, self._name + "_backward",
                   self._head + (ctypes.byref(gh),) + self._tail, stream)
        return self._grads


def rope_frequencies(pairs, base=10000.0, top=1.0, device=None):
    """[sum(pairs)] float32 frequencies: on every axis a geometric row from
    `top` down to top / base (excluded)."""
    import torch

    f = [top * float(base) ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in pairs]
    return torch.cat(f).to(torch.float32).to(device)


class Rope(_DeviceCall):
    """fpstok_rope on given tensors: q [rows, H, D] and, unless None, k
    [rows, Hk, D] turned by positions [rows, A] (float32 or int32), pairs[a]
    pairs by axis a with freqs [sum(pairs)] float32.  Outputs are allocated
    once unless given (q_out=q, k_out=k turn in place); a call returns
    (q_out, k_out)."""

    def __init__(self, q, k, positions, freqs, pairs, seqs, interleaved=False, q_out=None,
                 k_out=None):
        import torch

        super().__init__(q.device)
        pairs = [int(x) for x in pairs]
        A = len(pairs)
        if not 1 <= A <= MAX_AXES:
            raise ValueError("pairs must name 1 to %d axes" % MAX_AXES)
        if positions.dtype not in (torch.float32, torch.int32):
            raise TypeError("positions must be float32 or int32, got %s" % positions.dtype)
        _need(positions, positions.dtype, "positions", q.device)
        _need(freqs, torch.float32, "freqs", q.device)
        if tuple(positions.shape) != (q.shape[0], A):
            raise ValueError("positions must be [%d, %d]" % (q.shape[0], A))
        if freqs.numel() != sum(pairs):
            raise ValueError("freqs must hold %d values" % sum(pairs))
        if seqs.tensor.device != q.device:
            raise ValueError("the sequences are on %s, expected %s" % (seqs.tensor.device,
                                                                    q.device))
        qh = make_heads(q, "q", rows=seqs.num_rows)
        self.q_out = torch.zeros(q.shape, dtype=q.dtype, device=q.device) if q_out is None \
            else q_out
        qo = make_heads(self.q_out, "q_out", rows=q.shape[0], heads=q.shape[1], like=q)
        kh = ko = self.k_out = None
        if k is not None:
            kh = make_heads(k, "k", rows=seqs.num_rows, like=q)
            self.k_out = torch.zeros(k.shape, dtype=k.dtype, device=k.device) if k_out is None \
                else k_out
            ko = make_heads(self.k_out, "k_out", rows=k.shape[0], heads=k.shape[1], like=q)
        self._keep = (q, k, positions, freqs, seqs)
        code = I32 if positions.dtype == torch.int32 else F32
        views = tuple(None if h is None else ctypes.byref(h) for h in (qh, qo, kh, ko))
        self._args = []
        for inverse in (0, 1):
            pr = RopeParams(q.shape[1], 0 if k is None else k.shape[1], q.shape[2],
                            _dtype_code(q, "q"), code, A,
                            (ctypes.c_int32 * 4)(*(pairs + [0] * (4 - A))),
                            1 if interleaved else 0, inverse)
            self._args.append((ctypes.byref(seqs), ctypes.byref(pr), _ptr(positions), _ptr(freqs))
                              + views)
        self._fn = lib().fpstok_rope
        own = [self.q_out] if q_out is None else []
        if k is not None and k_out is None:
            own.append(self.k_out)
        if own:
            self._allocated(*own)

    def __call__(self, inverse=False, stream=None):
        """fpstok_rope; inverse=True turns back (the gradient)."""
        self._call(self._fn, "fpstok_rope", self._args[1 if inverse else 0], stream)
        return self.q_out, self.k_out


def make_rows(t, name, rows=None, width=None, dtype=None, device=None):
    """A Rows struct over a [rows, C] device tensor (any row stride, adjacent
    elements), which the caller keeps alive."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be [rows, C] with adjacent elements" % name)
    if (rows is not None and t.shape[0] != rows) or (width is not None and t.shape[1] != width):
        raise ValueError("%s must hold %s rows of %s elements, got %s" % (name, rows, width,
                                                                        tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    # (the stride of a single row is not used, and may be anything)
    return Rows(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0)


def _rows_overlap(a, b):
    """Whether two [rows, C] views (any row stride, adjacent elements) share a byte."""
    def span(t):
        n, step = t.shape[0], (t.stride(0) if t.shape[0] > 1 else 0) * t.element_size()
        return t.data_ptr(), (n if step else min(n, 1)), step, t.shape[1] * t.element_size()

    if a.numel() == 0 or b.numel() == 0:
        return False
    (pa, na, sa, wa), (pb, nb, sb, wb) = sorted((span(a), span(b)), key=lambda x: x[1])
    if pb >= pa + (na - 1) * sa + wa or pa >= pb + (nb - 1) * sb + wb:
        return False
    if nb == 1:
        return True
    if na == 1 or sa == sb:  # side by side in wider rows
        at = (pa - pb) % sb
        return not (at >= wb and at + wa <= sb)
    for start in range(pa - pb, pa - pb + na * sa, sa):
        k = 0 if start < wb else (start - wb) // sb + 1  # the first row that ends behind it
        if k < nb and k * sb < start + wa:
            return True
    return False


class Residual(_DeviceCall):
    """fpstok_residual on given tensors, with its outputs allocated once, and
    with training=True fpstok_residual_backward.

    x [rows, C] the stream; y [rows, C] the block's result, or None; gate
    [rows, C] (gate_per="row") or [sequences, C] (gate_per="sequence");
    post_norm, pre_norm: "none", "rms" or "layer"; activation of the gate:
    "none", "sigmoid" or "silu"; the weights [C] float32 or None.  A call takes
    what the tensors hold by then; it returns (x_out, h), the same buffers each
    time (h None without pre_norm); rows behind the last packed sequence keep
    what they held (0 after construction).  x_out=x and h=y work in place (not
    with training=True, whose gradients read x and y)."""

    def __init__(self, x, y, seqs, gate=None, gate_per="none", activation="none",
                 post_norm="none", pre_norm="rms", post_weight=None, post_bias=None, scale=None,
                 pre_weight=None, pre_bias=None, eps=1e-6, training=False, x_out=None, h=None):
        import torch

        super().__init__(x.device)
        for value, known, name in ((post_norm, NORMS, "post_norm"), (pre_norm, NORMS, "pre_norm"),
                                   (gate_per, GATES, "gate_per"),
                                   (activation, ACTIVATIONS, "activation")):
            if value not in known:
                raise ValueError("%s must be one of %s" % (name, ", ".join(known)))
        n, dev = seqs.num_rows, x.device
        if seqs.tensor.device != dev:
            raise ValueError("the sequences are on %s, expected %s" % (seqs.tensor.device, dev))
        xr = make_rows(x, "x", rows=n)
        C = x.shape[1]
        branch = y if y is not None else h
        bd = x.dtype if branch is None else branch.dtype
        yr = None if y is None else make_rows(y, "y", n, C, bd, dev)
        if (gate is None) != (gate_per == "none"):
            raise ValueError("give gate with gate_per, or neither")
        gate_rows = n if gate_per == "row" else seqs.num_seqs
        gr = None if gate is None else make_rows(gate, "gate", gate_rows, C, bd, dev)
        for name, t in (("x_out", x_out), ("h", h)):
            if training and t is not None and t.dim() == 2 and \
                    any(i is not None and _rows_overlap(t, i) for i in (x, y, gate)):
                raise ValueError("training=True reads x, y and gate again: give %s rows of its own"
                                 % name)
        weights = dict(post_weight=post_weight, post_bias=post_bias, scale=scale,
                       pre_weight=pre_weight, pre_bias=pre_bias)
        for name, w in weights.items():
            if w is not None:
                _need(w, torch.float32, name, dev)
                if tuple(w.shape) != (C,):
                    raise ValueError("%s must be [%d]" % (name, C))
        self._rows, self._C, self._sd, self._bd = n, C, x.dtype, bd
        own = []

        def buffer(given, name, shape, dtype):
            if given is not None:
                return given, make_rows(given, name, shape[0], shape[1], dtype, dev)
            t = torch.zeros(shape, dtype=dtype, device=dev)
            own.append(t)
            return t, make_rows(t, name)

        self.x_out, xo = buffer(x_out, "x_out", (n, C), x.dtype)
        self.h = ho = None
        if pre_norm != "none":
            self.h, ho = buffer(h, "h", (n, C), bd)
        elif h is not None:
            raise ValueError("h without pre_norm")
        self.stats = None
        if training:
            self.stats = torch.zeros((n, 4), dtype=torch.float32, device=dev)
            own.append(self.stats)
        self.params = ResidualParams(C, _dtype_code(x, "x"),
                                     _dtype_code(x if branch is None else branch, "y"),
                                     NORMS[post_norm], NORMS[pre_norm], GATES[gate_per],
                                     ACTIVATIONS[activation], float(eps))
        self._keep = (x, y, gate, seqs, weights)
        view = lambda r: None if r is None else ctypes.byref(r)  # noqa: E731
        w = ResidualWeights(*[_ptr(weights[k]) for k, _ in ResidualWeights._fields_])
        self._head = (ctypes.byref(seqs), ctypes.byref(self.params), ctypes.byref(w), view(xr),
                      view(yr), view(gr))
        self._out = (view(xo), view(ho), _ptr(self.stats))
        self._fwd, self._bwd = lib().fpstok_residual, lib().fpstok_residual_backward
        self.grads = None
        if training:
            grads = {"x": torch.zeros((n, C), dtype=x.dtype, device=dev)}
            if y is not None:
                grads["y"] = torch.zeros((n, C), dtype=bd, device=dev)
            if gate is not None:
                grads["gate"] = torch.zeros((gate_rows, C), dtype=bd, device=dev)
            for name, t in weights.items():
                if t is not None:
                    grads[name] = torch.zeros(C, dtype=torch.float32, device=dev)
            need = lib().fpstok_residual_workspace_size(*self._head[:2])
            self.ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            out = [None if grads.get(k) is None else make_rows(grads[k], k)
                   for k in ("x", "y", "gate")]
            gw = ResidualWeights(*[_ptr(grads.get(k)) for k, _ in ResidualWeights._fields_])
            self._tail = tuple(view(r) for r in out) + (
                ctypes.byref(gw), _ptr(self.ws), 0 if self.ws is None else self.ws.numel())
            self.grads = grads
            own += list(grads.values()) + ([] if self.ws is None else [self.ws])
        if own:
            self._allocated(*own)

    def __call__(self, stream=None):
        """fpstok_residual: (x_out, h)."""
        self._call(self._fwd, "fpstok_residual", self._head + self._out, stream)
        return self.x_out, self.h

    def backward(self, grad_x_out=None, grad_h=None, stream=None):
        """fpstok_residual_backward after a call on the same inputs: a dict of
        the gradients of x, y, gate and the weights that are given (a gradient
        that is None counts as 0)."""
        if self.grads is None:
            raise ValueError("construct with training=True")
        gx = gh = None
        if grad_x_out is not None:
            gx = make_rows(grad_x_out, "grad_x_out", self._rows, self._C, self._sd, self.device)
        if grad_h is not None:
            gh = make_rows(grad_h, "grad_h", self._rows, self._C, self._bd, self.device)
        view = lambda r: None if r is None else ctypes.byref(r)  # noqa: E731
        self._call(self._bwd, "fpstok_residual_backward",
                   self._head + (self._out[2], view(gx), view(gh)) + self._tail, stream)
        return self.grads
