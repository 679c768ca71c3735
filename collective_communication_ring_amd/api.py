"""Python binding of libar (C ABI declared in include/ar.h).

Argument marshalling only: every step of the collectives and operators runs in
libar's HIP kernels.  The low-level functions carry the C names (``ar_init``,
``ar_allreduce``, ...) and take plain integers (device pointers, sizes,
stream handles).  ``Comm`` is a convenience wrapper over torch tensors:
PyTorch provides device memory and streams, nothing else.

The operators' torch wrappers marshal in C++ (``_binding.so``).

There is no fallback: if ``libar.so`` has not been built, ``lib()`` raises, and
so does ``binding()`` without ``_binding.so``.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libar.so")

# ---- constants mirrored from include/ar.h --------------------------------
AR_INT32, AR_FLOAT32, AR_BF16, AR_E4M3 = 0, 1, 2, 3
AR_RING, AR_TREE, AR_AUTO = 0, 1, 2
AR_SIMPLE, AR_LL, AR_PROTO_AUTO = 0, 1, 2
AR_SUCCESS, AR_ERR_INVALID_ARG, AR_ERR_INVALID_USAGE, AR_ERR_UNSUPPORTED = 0, 1, 2, 3
AR_ERR_HIP, AR_ERR_TIMEOUT, AR_ERR_INTERNAL = 4, 5, 6
AR_LAUNCH_AUTO, AR_LAUNCH_STEP, AR_LAUNCH_FUSED, AR_LAUNCH_PIPELINED = 0, 1, 2, 3
(AR_OPT_CHUNK_BYTES, AR_OPT_LAUNCH, AR_OPT_GRID, AR_OPT_TIMEOUT_US, AR_OPT_DEBUG,
 AR_OPT_ALGO, AR_OPT_PROTO, AR_OPT_TREE_MAX_BYTES, AR_OPT_DEBUG_MUTE_RANK, AR_OPT_REDOP,
 AR_OPT_CHANNELS, AR_OPT_DEBUG_LL_LAUNCHES) = range(12)
AR_SUM, AR_MAX, AR_MIN, AR_AVG = 0, 1, 2, 3
(AR_COST_TREE_LL, AR_COST_RING_FUSED, AR_COST_RING_PIPELINED, AR_COST_RING_STEP,
 AR_COST_RING_LL, AR_COST_TREE_FUSED) = range(6)
COST_FORMS = {"tree-ll": AR_COST_TREE_LL, "ring-fused": AR_COST_RING_FUSED,
              "ring-pipelined": AR_COST_RING_PIPELINED, "ring-step": AR_COST_RING_STEP,
              "ring-ll": AR_COST_RING_LL, "tree-fused": AR_COST_TREE_FUSED}
AR_ROTARY_HALVES, AR_ROTARY_PAIRS = 0, 1
(AR_SCALING_NONE, AR_SCALING_LINEAR, AR_SCALING_BASE, AR_SCALING_BANDS,
 AR_SCALING_RAMP) = range(5)
ROTARY_LAYOUTS = {"halves": AR_ROTARY_HALVES, "pairs": AR_ROTARY_PAIRS}
SCALINGS = {None: AR_SCALING_NONE, "linear": AR_SCALING_LINEAR, "base": AR_SCALING_BASE,
            "bands": AR_SCALING_BANDS, "ramp": AR_SCALING_RAMP}
REDOPS = {"sum": AR_SUM, "max": AR_MAX, "min": AR_MIN, "avg": AR_AVG}

DTYPES = {"int32": AR_INT32, "float32": AR_FLOAT32, "bf16": AR_BF16}
ALGOS = {"ring": AR_RING, "tree": AR_TREE, "auto": AR_AUTO}
PROTOS = {"simple": AR_SIMPLE, "ll": AR_LL, "auto": AR_PROTO_AUTO}
LAUNCHES = {"auto": AR_LAUNCH_AUTO, "step": AR_LAUNCH_STEP, "fused": AR_LAUNCH_FUSED,
            "pipelined": AR_LAUNCH_PIPELINED}
ELEM_SIZE = {AR_INT32: 4, AR_FLOAT32: 4, AR_BF16: 2}

_lib = None


class ar_span_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_size_t), ("dtype", ctypes.c_int)]


class ar_rmsnorm_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("rows", ctypes.c_size_t), ("cols", ctypes.c_size_t), ("group", ctypes.c_size_t),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_size_t),
                ("weight", ctypes.c_void_p),
                ("sum", ctypes.c_void_p), ("sum_stride", ctypes.c_size_t),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_size_t),
                ("scale", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class ar_rmsnorm_backward_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int), ("ranks", ctypes.c_int),
                ("rows", ctypes.c_size_t), ("cols", ctypes.c_size_t),
                ("dy", ctypes.c_void_p), ("dy_stride", ctypes.c_size_t),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t),
                ("weight", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dsum", ctypes.c_void_p), ("dsum_stride", ctypes.c_size_t),
                ("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_size_t),
                ("dweight", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class ar_rotary_scheme_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_size_t), ("scaling", ctypes.c_int)] + [
        (n, ctypes.c_double) for n in ("base", "scale", "original", "low", "high", "fast", "slow")]


class ar_rotation_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_size_t), ("layout", ctypes.c_int), ("factor", ctypes.c_float),
                ("frequencies", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("position_bytes", ctypes.c_int), ("position_stride", ctypes.c_size_t)]


class ar_heads_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_size_t),
                ("token_stride", ctypes.c_size_t), ("head_stride", ctypes.c_size_t)]


_HEAD_SIZES = [(n, ctypes.c_size_t) for n in ("batch", "tokens", "q_heads", "k_heads", "dim")]


class ar_rotary_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("inverse", ctypes.c_int)] + _HEAD_SIZES + [
        ("rotation", ar_rotation_t)] + [(n, ar_heads_t) for n in ("q", "k", "q_out", "k_out")]


class ar_head_rmsnorm_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)] + _HEAD_SIZES + [("rotation", ar_rotation_t)] + [
        (n, ar_heads_t) for n in ("q", "k", "q_out", "k_out")] + [
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class ar_head_rmsnorm_backward_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int), ("ranks", ctypes.c_int),
                ("eps", ctypes.c_float)] + _HEAD_SIZES + [("rotation", ar_rotation_t)] + [
        (n, ar_heads_t) for n in ("dq_out", "dk_out", "q", "k", "dq", "dk")] + [
        (n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "q_dweight", "k_dweight", "workspace")
    ] + [("workspace_bytes", ctypes.c_size_t)]


class ar_orthogonalize_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("steps", ctypes.c_int), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("count", ctypes.c_size_t), ("rows", ctypes.c_size_t),
                ("cols", ctypes.c_size_t), ("x", ctypes.POINTER(ctypes.c_void_p)),
                ("x_stride", ctypes.c_size_t), ("out", ctypes.POINTER(ctypes.c_void_p)),
                ("out_stride", ctypes.c_size_t), ("coefficients", ctypes.POINTER(ctypes.c_float)),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class ArError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, ar_status_string(status), status))


def lib():
    """Load libar.so; raise if it is not built (no fallback path exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libar.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    sig = {
        "ar_init": ([ctypes.POINTER(vp), i, sz, i, i, i], i),
        "ar_destroy": ([vp], i),
        "ar_workspace_bytes": ([vp], sz),
        "ar_set_workspace": ([vp, vp, sz, vp], i),
        "ar_allreduce": ([vp, vp, vp, sz, vp], i),
        "ar_allreduce_noalloc": ([vp, vp, vp, sz, vp], i),
        "ar_reduce_scatter": ([vp, vp, vp, sz, vp], i),
        "ar_all_gather": ([vp, vp, vp, sz, vp], i),
        "ar_check": ([vp], i),
        "ar_set_option": ([vp, i, i64], i),
        "ar_get_option": ([vp, i, ctypes.POINTER(i64)], i),
        "ar_plan": ([vp, sz, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i)], i),
        "ar_set_cost": ([vp, i, ctypes.c_double, ctypes.c_double], i),
        "ar_get_cost": ([vp, i, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)], i),
        "ar_auto_tree_max_bytes": ([vp], i64),
        "ar_ring_segment": ([vp, sz, i, ctypes.POINTER(sz), ctypes.POINTER(sz)], i),
        "ar_tree_parent": ([vp, i, i], i),
        "ar_ring_channel_stride": ([vp, i], i),
        "ar_status_string": ([i], ctypes.c_char_p),
        "ar_last_hip_error": ([vp], i),
        "ar_stream_add": ([vp, vp, vp, sz, vp], i),
        "ar_stream_copy": ([vp, vp, sz, vp], i),
        "ar_stream_rows": ([vp, vp, i, sz, vp], i),
        "ar_ll_pingpong": ([vp, vp, i, i, i64, vp], i),
        "ar_stream_create_cu_masked": ([ctypes.POINTER(vp), ctypes.c_uint32,
                                        ctypes.POINTER(ctypes.c_uint32)], i),
        "ar_stream_destroy": ([vp], i),
        "ar_rmsnorm": ([ctypes.POINTER(ar_rmsnorm_t), vp], i),
        "ar_reduce_scatter_rmsnorm": ([vp, vp, ctypes.POINTER(ar_rmsnorm_t), vp], i),
        "ar_rmsnorm_backward": ([ctypes.POINTER(ar_rmsnorm_backward_t), vp], i),
        "ar_rmsnorm_backward_workspace": ([i, sz, sz], sz),
        "ar_grad_norm": ([vp, ctypes.POINTER(ar_span_t), sz, vp, vp], i),
        "ar_grad_clip": ([ctypes.POINTER(ar_span_t), ctypes.POINTER(ar_span_t), sz, vp,
                          ctypes.c_float, vp], i),
        "ar_rotary_frequencies": ([ctypes.POINTER(ar_rotary_scheme_t),
                                   ctypes.POINTER(ctypes.c_double),
                                   ctypes.POINTER(ctypes.c_double)], i),
        "ar_rotary": ([ctypes.POINTER(ar_rotary_t), vp], i),
        "ar_head_rmsnorm": ([ctypes.POINTER(ar_head_rmsnorm_t), vp], i),
        "ar_head_rmsnorm_backward": ([ctypes.POINTER(ar_head_rmsnorm_backward_t), vp], i),
        "ar_head_rmsnorm_backward_workspace": ([i, sz], sz),
        "ar_orthogonalize": ([ctypes.POINTER(ar_orthogonalize_t), vp], i),
        "ar_orthogonalize_workspace": ([sz, sz, sz], sz),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _ok(status, what):
    if status != AR_SUCCESS:
        raise ArError(status, what)


# ---- the C entry points, same names ----------------------------------------

def ar_init(R, count, dtype, algo=AR_RING, proto=AR_SIMPLE):
    h = ctypes.c_void_p()
    _ok(lib().ar_init(ctypes.byref(h), R, count, dtype, algo, proto), "ar_init")
    return h.value


def ar_destroy(comm):
    return lib().ar_destroy(comm)


def ar_workspace_bytes(comm):
    return lib().ar_workspace_bytes(comm)


def ar_set_workspace(comm, dev_ptr, nbytes, stream=0):
    _ok(lib().ar_set_workspace(comm, dev_ptr, nbytes, stream), "ar_set_workspace")


def ar_allreduce(comm, send_ptr, recv_ptr, count, stream=0):
    _ok(lib().ar_allreduce(comm, send_ptr, recv_ptr, count, stream), "ar_allreduce")


def ar_allreduce_noalloc(comm, send_ptr, recv_ptr, count, stream=0):
    _ok(lib().ar_allreduce_noalloc(comm, send_ptr, recv_ptr, count, stream),
        "ar_allreduce_noalloc")


def ar_reduce_scatter(comm, send_ptr, recv_ptr, recvcount, stream=0):
    _ok(lib().ar_reduce_scatter(comm, send_ptr, recv_ptr, recvcount, stream), "ar_reduce_scatter")


def ar_all_gather(comm, send_ptr, recv_ptr, sendcount, stream=0):
    _ok(lib().ar_all_gather(comm, send_ptr, recv_ptr, sendcount, stream), "ar_all_gather")


def ar_check(comm):
    """Returns the status code (AR_SUCCESS or AR_ERR_TIMEOUT ...)."""
    return lib().ar_check(comm)


def ar_set_option(comm, option, value):
    _ok(lib().ar_set_option(comm, option, int(value)), "ar_set_option")


def ar_get_option(comm, option):
    v = ctypes.c_int64()
    _ok(lib().ar_get_option(comm, option, ctypes.byref(v)), "ar_get_option")
    return v.value


def ar_plan(comm, count):
    a, p, l = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _ok(lib().ar_plan(comm, count, ctypes.byref(a), ctypes.byref(p), ctypes.byref(l)), "ar_plan")
    return a.value, p.value, l.value


def ar_set_cost(comm, form, alpha_us, bw_gbps):
    _ok(lib().ar_set_cost(comm, form, alpha_us, bw_gbps), "ar_set_cost")


def ar_get_cost(comm, form):
    a, b = ctypes.c_double(), ctypes.c_double()
    _ok(lib().ar_get_cost(comm, form, ctypes.byref(a), ctypes.byref(b)), "ar_get_cost")
    return a.value, b.value


def ar_auto_tree_max_bytes(comm):
    return int(lib().ar_auto_tree_max_bytes(comm))


def ar_ring_segment(comm, count, c):
    lo, hi = ctypes.c_size_t(), ctypes.c_size_t()
    _ok(lib().ar_ring_segment(comm, count, c, ctypes.byref(lo), ctypes.byref(hi)),
        "ar_ring_segment")
    return lo.value, hi.value


def ar_tree_parent(comm, tree, r):
    return lib().ar_tree_parent(comm, tree, r)


def ar_ring_channel_stride(comm, k):
    return lib().ar_ring_channel_stride(comm, k)


def ar_status_string(status):
    return lib().ar_status_string(status).decode()


def ar_last_hip_error(comm):
    return lib().ar_last_hip_error(comm)


def ar_stream_add(a_ptr, b_ptr, c_ptr, n, stream=0):
    _ok(lib().ar_stream_add(a_ptr, b_ptr, c_ptr, n, stream), "ar_stream_add")


def ar_stream_copy(src_ptr, dst_ptr, nbytes, stream=0):
    _ok(lib().ar_stream_copy(src_ptr, dst_ptr, nbytes, stream), "ar_stream_copy")


def ar_stream_rows(src_ptr, dst_ptr, rows, row_bytes, stream=0):
    _ok(lib().ar_stream_rows(src_ptr, dst_ptr, rows, row_bytes, stream), "ar_stream_rows")


def ar_ll_pingpong(lines_ptr, result_ptr, iters, xcd_apart, timeout_us=2_000_000, stream=0):
    _ok(lib().ar_ll_pingpong(lines_ptr, result_ptr, iters, int(bool(xcd_apart)), timeout_us, stream),
        "ar_ll_pingpong")


def ar_stream_create_cu_masked(cus, num_cus):
    """A stream restricted to the CUs in `cus` (an iterable of CU indices);
    returns the raw hipStream_t as an integer."""
    words = (num_cus + 31) // 32
    mask = (ctypes.c_uint32 * words)()
    for c in cus:
        mask[c // 32] |= 1 << (c % 32)
    h = ctypes.c_void_p()
    rc = lib().ar_stream_create_cu_masked(ctypes.byref(h), words, mask)
    if rc != AR_SUCCESS:
        raise ArError(rc, "ar_stream_create_cu_masked (hipError %d)" % ar_last_hip_error(None))
    return h.value


def ar_stream_destroy(stream):
    _ok(lib().ar_stream_destroy(stream), "ar_stream_destroy")


def ar_rmsnorm(args, stream=0):
    """args: an ar_rmsnorm_t."""
    _ok(lib().ar_rmsnorm(ctypes.byref(args), stream), "ar_rmsnorm")


def ar_reduce_scatter_rmsnorm(comm, send_ptr, args, stream=0):
    _ok(lib().ar_reduce_scatter_rmsnorm(comm, send_ptr, ctypes.byref(args), stream),
        "ar_reduce_scatter_rmsnorm")


def ar_rmsnorm_backward(args, stream=0):
    """args: an ar_rmsnorm_backward_t."""
    _ok(lib().ar_rmsnorm_backward(ctypes.byref(args), stream), "ar_rmsnorm_backward")


def ar_rmsnorm_backward_workspace(ranks, rows, cols):
    """Bytes; 0 for sizes that ar_rmsnorm_backward refuses."""
    return lib().ar_rmsnorm_backward_workspace(ranks, rows, cols)


def ar_grad_norm(comm, spans, n, norm_ptr, stream=0):
    """spans: a ctypes array of ar_span_t."""
    _ok(lib().ar_grad_norm(comm, spans, n, norm_ptr, stream), "ar_grad_norm")


def ar_grad_clip(spans, out_spans, n, norm_ptr, max_norm, stream=0):
    _ok(lib().ar_grad_clip(spans, out_spans, n, norm_ptr, max_norm, stream), "ar_grad_clip")


def ar_rotary_frequencies(scheme):
    """scheme: an ar_rotary_scheme_t.  (frequencies, a ctypes array of rot_dim /
    2 radians a position, and the factor)"""
    f = (ctypes.c_double * max(1, scheme.rot_dim // 2))()
    factor = ctypes.c_double()
    _ok(lib().ar_rotary_frequencies(ctypes.byref(scheme), f, ctypes.byref(factor)),
        "ar_rotary_frequencies")
    return f, factor.value


def ar_rotary(args, stream=0):
    """args: an ar_rotary_t."""
    _ok(lib().ar_rotary(ctypes.byref(args), stream), "ar_rotary")


def ar_head_rmsnorm(args, stream=0):
    """args: an ar_head_rmsnorm_t."""
    _ok(lib().ar_head_rmsnorm(ctypes.byref(args), stream), "ar_head_rmsnorm")


def ar_head_rmsnorm_backward(args, stream=0):
    """args: an ar_head_rmsnorm_backward_t."""
    _ok(lib().ar_head_rmsnorm_backward(ctypes.byref(args), stream), "ar_head_rmsnorm_backward")


def ar_head_rmsnorm_backward_workspace(ranks, dim):
    """Bytes; 0 for sizes that ar_head_rmsnorm_backward refuses."""
    return lib().ar_head_rmsnorm_backward_workspace(ranks, dim)


def ar_orthogonalize(args, stream=0):
    """args: an ar_orthogonalize_t."""
    _ok(lib().ar_orthogonalize(ctypes.byref(args), stream), "ar_orthogonalize")


def ar_orthogonalize_workspace(count, rows, cols):
    """Bytes; 0 for sizes that ar_orthogonalize refuses, or for nothing."""
    return lib().ar_orthogonalize_workspace(count, rows, cols)


# ---- torch convenience wrapper ---------------------------------------------

def _torch_dtype(dt):
    import torch
    return {AR_INT32: torch.int32, AR_FLOAT32: torch.float32, AR_BF16: torch.bfloat16}[dt]


_bound = None  # the marshalling module, and the library whose entry points it has


def binding():
    """The operators' argument marshalling (_binding.so), calling lib()'s
    entry points; raises if it is not built."""
    global _bound
    L = lib()
    if _bound is not None and _bound[1] is L:
        return _bound[0]
    import torch  # noqa: F401  (its libraries come first)
    if not os.path.exists(os.path.join(HERE, "_binding.so")):
        raise RuntimeError("_binding.so is not built (in %s); run __graft_entry__.build()" % HERE)
    from . import _binding
    _binding.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                    (L.ar_rmsnorm, L.ar_reduce_scatter_rmsnorm, L.ar_rmsnorm_backward)))
    _binding.init_heads(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                          (L.ar_rotary, L.ar_head_rmsnorm, L.ar_head_rmsnorm_backward,
                           L.ar_orthogonalize)))
    _bound = (_binding, L)
    return _binding


_current_raw_stream = None


def _raw_stream(index):
    """The handle of a device's current stream."""
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        # without the Stream object that the public call makes, where this torch has it
        _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_raw_stream(index)


def _stream_of(t, stream):
    """The given stream's handle, or that of the current one on t's GPU."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(t.get_device()) if t.is_cuda else None


def rmsnorm(x, weight, y, eps=1e-6, residual=None, sum=None, scale=None, group=0, rstd=None,
            stream=None):
    """RMS norm of x + residual (``ar_rmsnorm``): y = h / sqrt(mean(h^2) + eps)
    * weight with h = x + residual, written to ``y``; h to ``sum`` and
    1 / sqrt(mean(h^2) + eps) to ``rstd`` [rows] where given.

    x, residual, sum: [rows, cols] of float32 or bfloat16, rows any distance
    apart; y the same, or float8_e4m3fn with ``scale`` [rows, ceil(cols /
    group)] float32, one scale for each ``group`` (32, 64, 128, 256; 0: all)
    columns.  sum or y may be x or residual.  Asynchronous on the current
    torch stream (or the given one)."""
    rc = (_bound and _bound[0] or binding()).rmsnorm(
        x, weight, y, eps, residual, sum, scale, group, rstd, _stream_of(x, stream))
    if rc:
        raise ArError(rc, "ar_rmsnorm")
    return y


def _own_workspace(stream, make, *sizes):
    """A workspace that a call makes for itself."""
    if stream is None:
        return make(*sizes)
    # from that stream's memory: what was freed on the current one may still be
    # in use there
    import torch
    with torch.cuda.stream(stream):
        return make(*sizes)


def rmsnorm_backward_workspace(ranks, rows, cols, device="cuda"):
    """A workspace for ``rmsnorm_backward`` calls of these sizes (a tensor the
    caller keeps; one call at a time may use it)."""
    import torch
    return torch.empty(max(256, ar_rmsnorm_backward_workspace(ranks, rows, cols)),
                       dtype=torch.uint8, device=device)


def rmsnorm_backward(dy, x, weight, rstd, dx, dweight, dsum=None, workspace=None, stream=None):
    """Backward pass of ``rmsnorm`` (``ar_rmsnorm_backward``): dx [rows, cols]
    is the gradient of x + residual (x here is the forward's ``sum``, or its x
    where it had no residual), plus ``dsum``, the gradient that reaches the
    sum from elsewhere; dweight is [ranks, cols] float32, a row for each of
    ``ranks`` equal shards of the rows.  dx may be dy, x or dsum.  Without
    ``workspace`` (``rmsnorm_backward_workspace``) one is allocated."""
    if workspace is None:
        workspace = _own_workspace(stream, rmsnorm_backward_workspace, dweight.shape[0], x.shape[0],
                                   x.shape[-1], x.device)
    rc = (_bound and _bound[0] or binding()).rmsnorm_backward(
        dy, x, weight, rstd, dx, dweight, dsum, workspace, _stream_of(x, stream))
    if rc:
        raise ArError(rc, "ar_rmsnorm_backward")
    return dx


class Rotation:
    """How heads are rotated by their tokens' positions: the first ``rot_dim``
    elements of each, in pairs (i, i + rot_dim / 2) (layout "halves") or (2i, 2i
    + 1) ("pairs"), pair i by base^(-2i / rot_dim) radians a position.

    scaling, for contexts ``scale`` times the ``original`` length: None,
    "linear", "base", "bands" (with ``low`` and ``high``) or "ramp" (with
    ``fast`` and ``slow``, and a ``factor`` of the rotated values), as ar.h's
    AR_SCALING_* define them.  ``frequencies`` is a float64 tensor [rot_dim / 2]
    on the device; it and ``factor`` may be given other values."""

    def __init__(self, rot_dim, base=10000.0, layout="halves", scaling=None, scale=1.0, original=0,
                 low=1.0, high=4.0, fast=32.0, slow=1.0, device="cuda"):
        import torch
        if scaling not in SCALINGS:
            raise ValueError("scaling must be one of %s, got %r" % (list(SCALINGS), scaling))
        if layout not in ROTARY_LAYOUTS:
            raise ValueError("layout must be one of %s, got %r" % (list(ROTARY_LAYOUTS), layout))
        frequencies, self.factor = ar_rotary_frequencies(ar_rotary_scheme_t(
            rot_dim, SCALINGS[scaling], base, scale, original, low, high, fast, slow))
        self.layout = ROTARY_LAYOUTS[layout]
        self.frequencies = torch.frombuffer(frequencies, dtype=torch.float64).to(device)


def rotary(q, positions, rotation, q_out, k=None, k_out=None, inverse=False, stream=None):
    """Rotates heads by their tokens' positions (``ar_rotary``): q [batch,
    tokens, heads, dim] or [tokens, heads, dim], float32 or bfloat16, any
    distances between batches, tokens and heads (``x.transpose(1, 2)`` of heads
    ahead of tokens), to ``q_out``, and k (with a head count of its own) to
    ``k_out``.  positions: int32 or int64, [batch, tokens], or [tokens] for all
    batches.  ``rotation``: a ``Rotation``.  inverse: the transpose, for the
    outputs' gradients in the backward pass.  Outputs may be their inputs."""
    rc = (_bound and _bound[0] or binding()).rotary(
        q, q_out, k, k_out, positions, rotation.frequencies, rotation.layout, rotation.factor,
        bool(inverse), _stream_of(q, stream))
    if rc:
        raise ArError(rc, "ar_rotary")
    return q_out


def _turn(positions, rotation):
    if rotation is None:
        return positions, None, 0, 1.0
    return positions, rotation.frequencies, rotation.layout, rotation.factor


def head_rmsnorm(q, q_weight, q_out, eps=1e-6, k=None, k_weight=None, k_out=None, positions=None,
                 rotation=None, stream=None):
    """RMS norm of each head of q, by ``q_weight`` [dim], and of k, by
    ``k_weight``, and with ``positions`` and ``rotation`` the rotation of what
    comes out (``ar_head_rmsnorm``).  Arrays as ``rotary``'s; the weights are of
    their type or float32.  Outputs may be their inputs."""
    rc = (_bound and _bound[0] or binding()).head_rmsnorm(
        q, q_weight, q_out, eps, k, k_weight, k_out, *_turn(positions, rotation),
        _stream_of(q, stream))
    if rc:
        raise ArError(rc, "ar_head_rmsnorm")
    return q_out


def head_rmsnorm_backward_workspace(ranks, dim, device="cuda"):
    """A workspace for ``head_rmsnorm_backward`` calls of these sizes (a tensor
    the caller keeps; one call at a time may use it)."""
    import torch
    return torch.empty(max(256, ar_head_rmsnorm_backward_workspace(ranks, dim)), dtype=torch.uint8,
                       device=device)


def head_rmsnorm_backward(dq_out, q, q_weight, dq, q_dweight, eps=1e-6, dk_out=None, k=None,
                          k_weight=None, dk=None, k_dweight=None, positions=None, rotation=None,
                          workspace=None, stream=None):
    """Backward pass of ``head_rmsnorm`` (``ar_head_rmsnorm_backward``): from
    the outputs' gradients and the forward's inputs, dq and dk, and the weights'
    gradients [ranks, dim] float32, a row for each of ``ranks`` equal shards of
    the batches.  dq may be dq_out or q, dk dk_out or k.  Without ``workspace``
    (``head_rmsnorm_backward_workspace``) one is allocated."""
    if workspace is None:
        workspace = _own_workspace(stream, head_rmsnorm_backward_workspace, q_dweight.shape[0],
                                   q.shape[-1], q.device)
    rc = (_bound and _bound[0] or binding()).head_rmsnorm_backward(
        dq_out, q, q_weight, dq, q_dweight, eps, dk_out, k, k_weight, dk, k_dweight,
        *_turn(positions, rotation), workspace, _stream_of(q, stream))
    if rc:
        raise ArError(rc, "ar_head_rmsnorm_backward")
    return dq


# Newton-Schulz coefficients that take singular values of 0.002 and more to
# about 0.7 .. 1.2 in five steps.
ORTHOGONALIZE_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize_workspace(count, rows, cols, dtype=None, device="cuda"):
    """A workspace for ``orthogonalize`` calls of ``count`` matrices (a tensor
    the caller keeps; one call at a time may use it; its size is the same for
    every dtype)."""
    import torch
    return torch.empty(max(256, ar_orthogonalize_workspace(count, rows, cols)), dtype=torch.uint8,
                       device=device)


# The most that orthogonalize takes for a workspace of its own, in bytes, where one
# matrix needs no more: some 90 million elements at once fill the GPU many times over.
_ORTHOGONALIZE_OWN = 2 << 30


def _orthogonalize_room(count, rows, cols):
    """How many matrices that workspace holds."""
    m, n = (-(-side // 32) * 32 for side in sorted((rows, cols)))
    if m * n <= 16384 and 4 * m * (2 * n + m) <= 163584:
        return min(count, 1)  # they stay in LDS
    one = ar_orthogonalize_workspace(1, rows, cols)
    each = ar_orthogonalize_workspace(2, rows, cols) - one
    return min(count, 1 + max(0, _ORTHOGONALIZE_OWN - one) // each) if each else count


def orthogonalize(x, y, steps=5, coefficients=ORTHOGONALIZE_COEFFICIENTS, eps=1e-7, scale=1.0,
                  workspace=None, stream=None):
    """Orthogonalises matrices of one shape by Newton-Schulz steps
    (``ar_orthogonalize``): X = x / (norm(x) + eps), ``steps`` times X = a X +
    (b A + c A^2) X with A = X X^T, and scale * X to ``y``.

    x, y: float32 or bfloat16, [rows, cols], [count, rows, cols], or a list of
    [rows, cols] (rows equally far apart in all); y may be x.  coefficients:
    (a, b, c), or three for each step.  Without ``workspace``
    (``orthogonalize_workspace``) one is allocated, of 2 GiB or one matrix's; a
    smaller one, down to that of one matrix, takes the matrices in parts."""
    (xs, count, first), (ys, count_y, _) = _matrices(x), _matrices(y)
    if not count and not count_y:
        return y
    if count != count_y:
        raise ValueError("x are %d matrices, y %d" % (count, count_y))
    rows = [k.tolist() if hasattr(k, "tolist") else k for k in coefficients]  # also of a tensor or array
    flat = [float(c) for row in rows for c in (row if hasattr(row, "__len__") else (row,))]
    if len(flat) == 3:
        flat = flat * steps
    if len(flat) != 3 * steps:
        raise ValueError("coefficients must be three, or three for each of %d steps" % steps)
    if workspace is None:
        sizes = first.shape[-2], first.shape[-1]
        workspace = _own_workspace(stream, orthogonalize_workspace, _orthogonalize_room(count, *sizes),
                                   *sizes, first.dtype, first.device)
    rc = (_bound and _bound[0] or binding()).orthogonalize(xs, ys, flat, eps, scale, workspace,
                                                           _stream_of(first, stream))
    if rc:
        raise ArError(rc, "ar_orthogonalize")
    return y


def _matrices(x):
    """What the binding takes, how many matrices, and a tensor of their sizes."""
    if isinstance(x, (list, tuple)):
        for t in x[:1]:
            if t.dim() != 2:
                raise ValueError("a matrix must have shape (rows, cols), got %s" % (tuple(t.shape),))
        return list(x), len(x), x[0] if len(x) else None
    if x.dim() not in (2, 3):
        raise ValueError("matrices must have shape ([count,] rows, cols), got %s" % (tuple(x.shape),))
    return x, 1 if x.dim() == 2 else x.shape[0], x


class TensorList:
    """Gradient tensors of one GPU as ``Comm.grad_norm`` / ``Comm.grad_clip``
    take them: float32 or bfloat16, each dense in memory (in any order of its
    dimensions).  Keeps the tensors; each call reads their addresses anew."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self._array = (ar_span_t * len(self.tensors))()
        self._address = ctypes.addressof(self._array)
        self.spans()

    def __len__(self):
        return len(self.tensors)

    def spans(self):
        """The tensors as a ctypes array of ar_span_t."""
        self.index = (_bound and _bound[0] or binding()).spans(
            self.tensors, self._address, len(self._array))  # their GPU; -1 without tensors
        return self._array


def _tensor_list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


class Comm:
    """A communicator of R logical ranks on one GPU, with its workspace.

    Buffers are rank-major torch tensors on the device: ``send`` of shape
    [R, n] etc.  Calls are asynchronous on the current torch stream (or the
    given one)."""

    def __init__(self, R, count, dtype="float32", algo="ring", proto="simple", device=None,
                 launch=None, **options):
        import torch
        self.R = R
        self.count = count
        self.dtype = DTYPES[dtype] if isinstance(dtype, str) else dtype
        self.device = torch.device(device if device is not None else "cuda")
        self.handle = ar_init(R, count, self.dtype,
                              ALGOS[algo] if isinstance(algo, str) else algo,
                              PROTOS[proto] if isinstance(proto, str) else proto)
        if launch is not None:
            self.set_option(AR_OPT_LAUNCH, LAUNCHES[launch] if isinstance(launch, str) else launch)
        for k, v in options.items():
            if k == "redop" and isinstance(v, str):
                v = REDOPS[v]
            self.set_option(globals()["AR_OPT_" + k.upper()], v)
        nbytes = ar_workspace_bytes(self.handle)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        self._ws_stream = torch.cuda.current_stream(self.device).cuda_stream
        ar_set_workspace(self.handle, self.workspace.data_ptr(), self.workspace.numel(),
                         self._stream(None))

    def _stream(self, stream):
        if stream is None and self.workspace is not None:
            raw = _raw_stream(self.workspace.get_device())
            if raw == self._ws_stream:
                return raw
        import torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if getattr(self, "workspace", None) is not None and \
                s.cuda_stream != self._ws_stream and not torch.cuda.is_current_stream_capturing():
            # the workspace may still be in use on this stream when the comm is
            # dropped: keep torch's allocator from reusing it too early
            self.workspace.record_stream(s)
        return s.cuda_stream

    def _check_tensor(self, t, rows, cols, what):
        if t.device != self.device and not (t.is_cuda and self.device.index is None):
            raise ValueError("%s must be on %s" % (what, self.device))
        if t.dtype != _torch_dtype(self.dtype):
            raise ValueError("%s has dtype %s, comm has %s" % (what, t.dtype, _torch_dtype(self.dtype)))
        if tuple(t.shape) != (rows, cols):
            raise ValueError("%s must have shape (%d, %d), got %s" % (what, rows, cols, tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous (rank-major rows)" % what)

    def allreduce(self, send, recv, stream=None):
        n = send.shape[1]
        self._check_tensor(send, self.R, n, "send")
        self._check_tensor(recv, self.R, n, "recv")
        ar_allreduce(self.handle, send.data_ptr(), recv.data_ptr(), n, self._stream(stream))
        return recv

    def reduce_scatter(self, send, recv, stream=None):
        n = recv.shape[1]
        self._check_tensor(send, self.R, n * self.R, "send")
        self._check_tensor(recv, self.R, n, "recv")
        ar_reduce_scatter(self.handle, send.data_ptr(), recv.data_ptr(), n, self._stream(stream))
        return recv

    def all_gather(self, send, recv, stream=None):
        n = send.shape[1]
        self._check_tensor(send, self.R, n, "send")
        self._check_tensor(recv, self.R, n * self.R, "recv")
        ar_all_gather(self.handle, send.data_ptr(), recv.data_ptr(), n, self._stream(stream))
        return recv

    def reduce_scatter_rmsnorm(self, send, weight, y, eps=1e-6, residual=None, sum=None,
                               scale=None, group=0, rstd=None, stream=None):
        """Reduce-scatter of ``send`` [R, R * tokens * cols] with an RMS norm
        behind it, in one pass (``ar_reduce_scatter_rmsnorm``).  Rank q's row
        of residual, sum and y ([R, tokens * cols]) holds its own tokens;
        weight [cols] gives the row length; rstd is [R, tokens] and scale
        [R, tokens * ceil(cols / group)].  Otherwise as ``rmsnorm``."""
        if self.workspace is None:  # closed
            raise ArError(AR_ERR_INVALID_ARG, "ar_reduce_scatter_rmsnorm")
        rc = (_bound and _bound[0] or binding()).reduce_scatter_rmsnorm(
            self.handle, send, weight, y, eps, residual, sum, scale, group, rstd,
            self._stream(stream), self.R, self.dtype, self.workspace.get_device())
        if rc:
            raise ArError(rc, "ar_reduce_scatter_rmsnorm")
        return y

    def grad_norm(self, grads, norm, stream=None):
        """Global 2-norm of the tensors of ``grads`` (a sequence, or a
        ``TensorList`` kept for many calls) to ``norm``, one float32 on the
        device (``ar_grad_norm``), all on the comm's GPU.  Uses the comm's
        workspace: ordered with its collectives on one stream."""
        grads = _tensor_list(grads)
        spans = grads.spans()
        self._check_norm(grads, norm)
        ar_grad_norm(self.handle, spans, len(grads), norm.data_ptr(), self._stream(stream))
        return norm

    def grad_clip(self, grads, norm, max_norm, out=None, stream=None):
        """Scales the tensors of ``grads`` to a norm of at most ``max_norm``,
        ``norm`` being theirs on the device (``ar_grad_clip``): in place, or
        into the tensors of ``out``."""
        grads = _tensor_list(grads)
        spans = grads.spans()
        self._check_norm(grads, norm)
        to = spans
        if out is not None:
            out = _tensor_list(out)
            to = out.spans()
            if out.index != grads.index or not binding().same_layout(grads.tensors, out.tensors):
                raise ValueError("out must have the shapes, dtypes, strides and device of grads")
        ar_grad_clip(spans, to, len(grads), norm.data_ptr(), max_norm, self._stream(stream))
        return norm

    def _check_norm(self, grads, norm):
        import torch
        if norm.numel() != 1 or norm.dtype != torch.float32 or not norm.is_cuda or \
                (grads.index >= 0 and grads.index != norm.get_device()):
            raise ValueError("norm must be one float32 on the gradients' device")
        # the stream and the partial sums are those of the communicator's GPU
        if self.workspace is not None and norm.get_device() != self.workspace.get_device():
            raise ValueError("norm is on cuda:%d, the comm on cuda:%d" %
                             (norm.get_device(), self.workspace.get_device()))

    def check(self):
        return ar_check(self.handle)

    def set_option(self, option, value):
        ar_set_option(self.handle, option, value)

    def get_option(self, option):
        return ar_get_option(self.handle, option)

    def plan(self, count):
        return ar_plan(self.handle, count)

    def channel_strides(self):
        """Ring stride of each channel this comm runs."""
        K = self.get_option(AR_OPT_CHANNELS)
        return [ar_ring_channel_stride(self.handle, k) for k in range(K)]

    def close(self):
        """Destroy the communicator and release its workspace.  A comm used on
        a stream that the caller destroys itself (ar_stream_destroy) must be
        closed, and that stream's work finished, before the stream goes: the
        workspace is recorded on every stream the comm ran on."""
        if getattr(self, "handle", None):
            ar_destroy(self.handle)
            self.handle = None
        self.workspace = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
