"""Fused equivariant message passing (l <= 3) for GB300: Python binding.

A thin ctypes layer over the C ABI of ``libeqmp.so`` (declared in
include/eqmp.h).  Each function takes torch CUDA tensors, checks dtypes and
shapes, passes raw device pointers and the current CUDA stream, and raises
``EqmpError`` on a non-OK status.  All arithmetic happens in the library's
CUDA kernels; there is no CPU path.  PyTorch supplies device memory and
streams only.

Entry points (same names as the C ABI):
  eqmp_sh(vec, Y=None)                         -> Y [E, 16]
  eqmp_tp_scatter(Y, x, row_offsets, src, ...)  -> out [N, C, 16]
  eqmp_fused(vec, x, row_offsets, src, ...)     -> out [N, C, 16]
  eqmp_fused_staged(h_in, d_in, ..., out, h_out) -> h_out: copy in, layer, copy out
                                                (prepare=True: a prepared call for a step loop)
  eqmp_plan_staged(h_in, d_in, ..., out, h_out)  -> plan; plan.launch(stream): the same step as one
                                                CUDA graph launch
  eqmp_fused_so2(...)                           -> out, aligned-frame schedule
  eqmp_validate_graph(row_offsets, src, n_src, n_edges)
  eqmp_device_error()                           -> int (watchdog code)
  eqmp_fused_backward(vec, x, row_offsets, src, dst, send_offsets, send_edges, grad_out, ...)
                                                -> dict of gradients
  eqmp_fused_backward_noalloc(...)              -> the same, no workspace
  eqmp_radius_graph(pos, cutoff, box=None)      -> (dict(off, src, vec[, img, dst, rev]), E)
  eqmp_fused_lmax(l_max, vec, x, row_offsets, src, ...) -> out, degree 4..6
  eqmp_path_table()                             -> list of (l1, l2, l3)
  eqmp_dropout(x, drop)                         -> out; drop = Dropout(p, seed, offset, group)
  eqmp_layer_norm(x, w, b, residual=, drop=)    -> dict(y[, s][, stats])
  eqmp_layer_norm_backward(grad_y, s, stats, w, grad_s=, drop=) -> dict of gradients
  eqmp_degree_norm(x, w, b, residual=, drop=)   -> dict, on node features [N, C, (l_max+1)^2]
  eqmp_degree_norm_backward(grad_y, s, stats, w, grad_s=, drop=) -> dict of gradients
  eqmp_head_norm(q, k, wq, wk, pos=, freq=)     -> dict(q, k[, rstd]): norm of each head, rotation by position
  eqmp_head_norm_backward(grad_q, grad_k, q, k, rstd, wq, wk, pos=, freq=) -> dict of gradients
  eqmp_edge_bias(vec, borders, table)           -> dict(bias, bucket) by the edges' lengths
  eqmp_edge_bias_backward(grad_bias, bucket, n_buckets) -> dict(table)
  eqmp_edge_attention(q, k, v, row_offsets, src, bias=) -> dict(out[, stats])
  eqmp_edge_attention_backward(grad_out, q, k, v, stats, row_offsets, src, dst, send_offsets, send_edges, bias=)
                                                -> dict of gradients

stream= (default: torch's current stream) is the stream that a call's kernels run on.  The inputs must be ready there.
Results that the call allocates come from that stream's pool and are recorded on the current stream as well, so they may
be used and freed on either; the current stream has to wait for the call's stream before it reads them.
"""
import ctypes
import os

__all__ = [
    "EqmpError", "load_library", "library_path", "eqmp_num_paths", "eqmp_path_table",
    "eqmp_status_string", "eqmp_sh", "eqmp_tp_scatter", "eqmp_fused", "eqmp_fused_staged", "eqmp_plan_staged",
    "eqmp_fused_so2",
    "eqmp_validate_graph",
    "eqmp_device_error", "eqmp_fused_backward", "eqmp_fused_backward_noalloc", "eqmp_radius_graph", "eqmp_fused_lmax",
    "eqmp_num_paths_lmax", "eqmp_watchdog_selftest", "eqmp_fp32_peak_probe", "sender_view",
    "Dropout", "eqmp_dropout", "eqmp_layer_norm", "eqmp_layer_norm_backward", "eqmp_layer_norm_backward_workspace_size",
    "eqmp_degree_norm", "eqmp_degree_norm_backward", "eqmp_degree_norm_backward_workspace_size",
    "eqmp_head_norm", "eqmp_head_norm_backward", "eqmp_head_norm_backward_workspace_size",
    "eqmp_edge_bias", "eqmp_edge_bias_backward", "eqmp_edge_bias_backward_workspace_size",
    "eqmp_edge_attention", "eqmp_edge_attention_workspace_size",
    "eqmp_edge_attention_backward", "eqmp_edge_attention_backward_workspace_size", "EQMP_OK", "EQMP_ERR_INVALID_ARG", "EQMP_ERR_UNSUPPORTED",
    "EQMP_ERR_CUDA", "EQMP_ERR_DEVICE_TIMEOUT", "EQMP_ERR_GRAPH",
]

EQMP_OK, EQMP_ERR_INVALID_ARG, EQMP_ERR_UNSUPPORTED, EQMP_ERR_CUDA = 0, 1, 2, 3
EQMP_ERR_DEVICE_TIMEOUT, EQMP_ERR_GRAPH = 4, 5
EQMP_F32, EQMP_BF16 = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
# EQMP_LIB selects another build of the library (e.g. a tuning variant).
_LIB_PATH = os.environ.get("EQMP_LIB") or os.path.join(_HERE, "_build", "libeqmp.so")
_lib = None


class EqmpError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_status_text(status)} (status {status})")


class Weights(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("R", ctypes.c_void_p), ("M", ctypes.c_void_p),
                ("K", ctypes.c_int32)]


class Dropout(ctypes.Structure):
    """Dropout of one call (eqmp_drop): rate p, seed and offset of the counter-based generator, and how many
    consecutive columns share a draw (group).  The same Dropout gives the same mask, in the forward and in the
    backward pass; another offset (a step or a layer) gives another one.  step: an int64 CUDA tensor of one
    value that is added to offset when the kernel runs (for recorded CUDA graphs)."""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step_ptr", ctypes.c_void_p), ("group", ctypes.c_int32)]
    step = None

    def __init__(self, p, seed, offset=0, group=1, step=None):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
            raise ValueError("seed and offset must be unsigned 64-bit")
        if not 1 <= group < 1 << 31:
            raise ValueError("group must be at least 1")
        super().__init__(p, seed, offset, None, group)
        if step is not None:
            import torch

            _require(step, "step", torch.int64)
            if step.numel() != 1:
                raise ValueError("step must hold one value")
            self.step, self.step_ptr = step, step.data_ptr()  # keeps the tensor alive


_NO_DROP = Dropout(0.0, 0)


def library_path():
    return _LIB_PATH


def load_library():
    """Load libeqmp.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libeqmp.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.eqmp_num_paths.restype = i32
    lib.eqmp_path_table.argtypes = [ctypes.POINTER(i32)]
    lib.eqmp_path_table.restype = i32
    lib.eqmp_status_string.argtypes = [i32]
    lib.eqmp_status_string.restype = ctypes.c_char_p
    lib.eqmp_sh.argtypes = [vp, i64, vp, vp]
    lib.eqmp_sh.restype = i32
    layer = [vp, vp, i64, i32, vp, vp, i64, i64, i32, Weights, vp, i32, vp]
    lib.eqmp_tp_scatter.argtypes = layer
    lib.eqmp_tp_scatter.restype = i32
    lib.eqmp_fused.argtypes = layer
    lib.eqmp_fused.restype = i32
    lib.eqmp_fused_so2.argtypes = layer
    lib.eqmp_fused_so2.restype = i32
    sz = ctypes.c_size_t
    lib.eqmp_fused_staged.argtypes = [vp, vp, sz] + layer[:-1] + [vp, sz, vp]
    lib.eqmp_fused_staged.restype = i32
    lib.eqmp_plan_staged.argtypes = [vp, vp, sz] + layer[:-1] + [vp, sz, ctypes.POINTER(vp)]
    lib.eqmp_plan_staged.restype = i32
    lib.eqmp_plan_launch.argtypes = [vp, vp]
    lib.eqmp_plan_launch.restype = i32
    lib.eqmp_plan_destroy.argtypes = [vp]
    lib.eqmp_plan_destroy.restype = i32
    lib.eqmp_validate_graph.argtypes = [vp, vp, i64, i64, i64, vp]
    lib.eqmp_validate_graph.restype = i32
    lib.eqmp_device_error.argtypes = [ctypes.POINTER(i32)]
    lib.eqmp_device_error.restype = i32
    lib.eqmp_fused_backward_workspace_size.argtypes = [i64, i64, i32, i32]
    lib.eqmp_fused_backward_workspace_size.restype = i64
    lib.eqmp_fused_backward.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, i32, Weights,
                                        vp, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.eqmp_fused_backward.restype = i32
    lib.eqmp_fused_backward_noalloc.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, i64, i32, Weights,
                                                vp, vp, vp, vp, vp, vp, vp]
    lib.eqmp_fused_backward_noalloc.restype = i32
    lib.eqmp_fused_backward_noalloc_max_bytes.restype = i64
    lib.eqmp_watchdog_selftest.argtypes = [i32, vp]
    lib.eqmp_watchdog_selftest.restype = i32
    lib.eqmp_fp32_peak_probe.argtypes = [i32, i32, vp, ctypes.POINTER(ctypes.c_double), vp]
    lib.eqmp_fp32_peak_probe.restype = i32
    lib.eqmp_num_paths_lmax.argtypes = [i32]
    lib.eqmp_num_paths_lmax.restype = i32
    lib.eqmp_fused_lmax.argtypes = [i32, vp, vp, i64, vp, vp, i64, i64, i32, Weights, vp, vp]
    lib.eqmp_fused_lmax.restype = i32
    lib.eqmp_radius_graph_workspace_size.argtypes = [i64]
    lib.eqmp_radius_graph_workspace_size.restype = ctypes.c_size_t
    lib.eqmp_radius_graph.argtypes = [vp, i64, ctypes.c_float, vp, vp, vp, vp, vp, i64, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.eqmp_radius_graph.restype = i32
    lib.eqmp_radius_graph_pbc.argtypes = [vp, i64, ctypes.c_float, ctypes.POINTER(ctypes.c_float), vp, vp, vp, vp,
                                          vp, vp, i64, vp, vp, ctypes.c_size_t, vp]
    lib.eqmp_radius_graph_pbc.restype = i32
    f32 = ctypes.c_float
    lib.eqmp_dropout.argtypes = [vp, i64, i32, i64, i64, Dropout, vp, vp]
    lib.eqmp_layer_norm.argtypes = [vp, i64, vp, i64, i32, i64, i64, Dropout, vp, vp, f32, vp, vp, vp, vp]
    lib.eqmp_degree_norm.argtypes = [vp, vp, i32, i64, i32, i32, Dropout, vp, vp, f32, vp, vp, vp, vp]
    lib.eqmp_layer_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, i32, i64, i64, Dropout, vp, vp, vp, vp, vp,
                                             vp, vp, i64, vp]
    lib.eqmp_degree_norm_backward.argtypes = [vp, vp, vp, i32, i64, i32, i32, Dropout, vp, vp, vp, vp, vp, vp, vp,
                                              i64, vp]
    for name in ("dropout", "layer_norm", "degree_norm", "layer_norm_backward", "degree_norm_backward"):
        getattr(lib, "eqmp_" + name).restype = i32
    lib.eqmp_layer_norm_backward_workspace_size.argtypes = [i64, i64]
    lib.eqmp_layer_norm_backward_workspace_size.restype = i64
    lib.eqmp_degree_norm_backward_workspace_size.argtypes = [i64, i32, i32]
    lib.eqmp_degree_norm_backward_workspace_size.restype = i64
    lib.eqmp_head_norm.argtypes = [vp, i64, i32, vp, i64, i32, i32, i64, i32, vp, vp, f32, vp, vp, i32, vp, vp, vp, vp]
    lib.eqmp_head_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, i64, i32, i32, i64, i32, vp, vp, vp, vp, vp,
                                            i32, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.eqmp_edge_bias.argtypes = [vp, i64, vp, i32, vp, i32, vp, vp, vp]
    lib.eqmp_edge_bias_backward.argtypes = [vp, vp, i64, i32, i32, vp, vp, i64, vp]
    rows = [vp, i64, vp, i64, vp, i64]
    lib.eqmp_edge_attention.argtypes = rows + [i32, i64, i64, i64, i32, i32, i32, vp, vp, vp, f32, vp, vp, vp, i64, vp]
    lib.eqmp_edge_attention_backward.argtypes = [vp, i64] + rows + [i32, i64, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, i64,
                                                                    vp, f32, vp, vp, vp, vp, vp, vp, i64, vp]
    for name in ("head_norm", "edge_bias", "edge_attention"):
        getattr(lib, "eqmp_" + name).restype = getattr(lib, f"eqmp_{name}_backward").restype = i32
    lib.eqmp_head_norm_backward_workspace_size.argtypes = [i64, i32]
    lib.eqmp_edge_bias_backward_workspace_size.argtypes = [i64, i32, i32]
    lib.eqmp_edge_attention_workspace_size.argtypes = [i64, i32, i32]
    lib.eqmp_edge_attention_backward_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    for name in ("head_norm_backward", "edge_bias_backward", "edge_attention", "edge_attention_backward"):
        getattr(lib, f"eqmp_{name}_workspace_size").restype = i64
    _lib = lib
    return lib


def _status_text(status):
    try:
        return load_library().eqmp_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - library absent
        return "status"


def _check(status, where):
    if status != EQMP_OK:
        raise EqmpError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _torch_stream(stream):
    import torch

    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream)


def _empty(shape, dtype, device, stream, temporary=False, zero=False):
    """Memory for kernels on `stream` (None: the current one), filled with zeros there if asked for.

    The allocator hands freed memory out again in the order of the stream that it was allocated on, so it is allocated
    on the stream of the kernels; a result is recorded on the current stream as well, where the caller will use it."""
    import torch

    make = torch.zeros if zero else torch.empty
    if stream is None or stream.cuda_stream == (current := torch.cuda.current_stream()).cuda_stream:
        return make(shape, dtype=dtype, device=device)
    torch.cuda.set_stream(_torch_stream(stream))
    try:
        t = make(shape, dtype=dtype, device=device)
    finally:
        torch.cuda.set_stream(current)
    if not temporary:
        t.record_stream(current)
    return t


def _require(t, name, dtype=None, cuda=True):
    import torch

    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def eqmp_num_paths():
    return int(load_library().eqmp_num_paths())


def eqmp_path_table():
    lib = load_library()
    buf = (ctypes.c_int32 * (3 * 34))()
    _check(lib.eqmp_path_table(buf), "eqmp_path_table")
    return [tuple(buf[3 * p:3 * p + 3]) for p in range(lib.eqmp_num_paths())]


def eqmp_status_string(status):
    return load_library().eqmp_status_string(int(status)).decode()


def eqmp_sh(vec, Y=None, stream=None):
    """Y[E, 16] = real SH (l <= 3) of vec[E, 3] (fp32, CUDA)."""
    import torch

    _require(vec, "vec", torch.float32)
    E = vec.shape[0] if vec.dim() == 2 else -1
    if vec.dim() != 2 or vec.shape[1] != 3:
        raise ValueError("vec must be [E, 3]")
    if Y is None:
        Y = _empty((E, 16), torch.float32, vec.device, stream)
    _require(Y, "Y", torch.float32)
    if tuple(Y.shape) != (E, 16):
        raise ValueError("Y must be [E, 16]")
    _check(load_library().eqmp_sh(_ptr(vec), E, _ptr(Y), _stream(stream)), "eqmp_sh")
    return Y


def _layer(fn_name, edge_in, x, row_offsets, src, w, R, M, out, stream, n_edges):
    import torch

    _require(x, "x", (torch.float32, torch.bfloat16))
    _require(row_offsets, "row_offsets", torch.int32)
    _require(src, "src", torch.int32)
    for name, t in (("w", w), ("R", R), ("M", M)):
        _require(t, name, torch.float32)
    if x.dim() != 3 or x.shape[2] != 16:
        raise ValueError("x must be [N_src, C, 16]")
    n_src, C = x.shape[0], x.shape[1]
    N = row_offsets.shape[0] - 1
    E = n_edges if n_edges is not None else edge_in.shape[0]
    if out is None:
        out = _empty((N, C, 16), x.dtype, x.device, stream)
    _require(out, "out", x.dtype)
    if tuple(out.shape) != (N, C, 16):
        raise ValueError("out must be [N, C, 16]")
    dt = EQMP_BF16 if x.dtype == torch.bfloat16 else EQMP_F32
    if w is not None:
        wt = Weights(ctypes.c_void_p(w.data_ptr()), None, None, 0)
    else:
        wt = Weights(None, ctypes.c_void_p(R.data_ptr()) if R is not None else None,
                     ctypes.c_void_p(M.data_ptr()) if M is not None else None,
                     R.shape[1] if R is not None and R.dim() == 2 else 0)
    fn = getattr(load_library(), fn_name)
    st = fn(_ptr(edge_in), _ptr(x), n_src, dt, _ptr(row_offsets), _ptr(src), N, E, C, wt,
            _ptr(out), dt, _stream(stream))
    _check(st, fn_name)
    return out


def eqmp_tp_scatter(Y, x, row_offsets, src, w=None, R=None, M=None, out=None, stream=None,
                    n_edges=None):
    """out[N, C, 16] = receiver sum of CG(x[src], Y) with shared w or radial (R, M)."""
    import torch

    _require(Y, "Y", torch.float32)
    return _layer("eqmp_tp_scatter", Y, x, row_offsets, src, w, R, M, out, stream, n_edges)


def eqmp_fused(vec, x, row_offsets, src, w=None, R=None, M=None, out=None, stream=None,
               n_edges=None):
    """out[N, C, 16] = receiver sum of CG(x[src], SH(vec)), one fused kernel."""
    import torch

    _require(vec, "vec", torch.float32)
    return _layer("eqmp_fused", vec, x, row_offsets, src, w, R, M, out, stream, n_edges)


def eqmp_fused_staged(h_in, d_in, vec, x, row_offsets, src, out, h_out, w=None, R=None, M=None, stream=None,
                      n_edges=None, prepare=False):
    """One step from host memory: h_in (pinned CPU uint8) -> d_in (CUDA
    uint8, same size), eqmp_fused on the CUDA tensors given (views into
    d_in), out -> h_out (pinned CPU, out's size).  Asynchronous on the
    stream; synchronise before reading h_out.

    prepare=True checks and marshals the arguments once and returns a
    function of no arguments that issues the same C call (for a loop that
    repeats the step on the same buffers; the tensors must stay alive and
    unmoved while it is used).  It raises EqmpError on a non-OK status."""
    import torch

    _require(h_in, "h_in", torch.uint8, cuda=False)
    _require(d_in, "d_in", torch.uint8)
    _require(h_out, "h_out", out.dtype, cuda=False)
    _require(vec, "vec", torch.float32)
    _require(x, "x", (torch.float32, torch.bfloat16))
    _require(row_offsets, "row_offsets", torch.int32)
    _require(src, "src", torch.int32)
    for name, t in (("w", w), ("R", R), ("M", M)):
        _require(t, name, torch.float32)
    if h_in.is_cuda or h_out.is_cuda:
        raise ValueError("h_in and h_out are host tensors")
    if h_in.numel() != d_in.numel():
        raise ValueError("h_in and d_in must have the same size")
    if x.dim() != 3 or x.shape[2] != 16:
        raise ValueError("x must be [N_src, C, 16]")
    n_src, C = x.shape[0], x.shape[1]
    N = row_offsets.shape[0] - 1
    E = n_edges if n_edges is not None else vec.shape[0]
    _require(out, "out", x.dtype)
    if tuple(out.shape) != (N, C, 16) or tuple(h_out.shape) != (N, C, 16):
        raise ValueError("out and h_out must be [N, C, 16]")
    dt = EQMP_BF16 if x.dtype == torch.bfloat16 else EQMP_F32
    if w is not None:
        wt = Weights(ctypes.c_void_p(w.data_ptr()), None, None, 0)
    else:
        wt = Weights(None, ctypes.c_void_p(R.data_ptr()) if R is not None else None,
                     ctypes.c_void_p(M.data_ptr()) if M is not None else None,
                     R.shape[1] if R is not None and R.dim() == 2 else 0)
    fn = load_library().eqmp_fused_staged
    args = (_ptr(h_in), _ptr(d_in), h_in.numel(), _ptr(vec), _ptr(x), n_src, dt, _ptr(row_offsets), _ptr(src),
            N, E, C, wt, _ptr(out), dt, _ptr(h_out), h_out.numel() * h_out.element_size(), _stream(stream))
    if prepare == "plan":
        return _Plan(args[:-1], (h_in, d_in, vec, x, row_offsets, src, out, h_out, w, R, M))
    if prepare:
        keep = (h_in, d_in, vec, x, row_offsets, src, out, h_out, w, R, M, stream)

        def run(_keep=keep):
            st = fn(*args)
            if st != EQMP_OK:
                raise EqmpError(st, "eqmp_fused_staged")
            return h_out
        return run
    _check(fn(*args), "eqmp_fused_staged")
    return h_out


class _Plan:
    """A staged step recorded once as a CUDA graph (eqmp_plan_staged);
    launch(stream) replays it with one graph launch."""

    def __init__(self, args, keep):
        lib = load_library()
        h = ctypes.c_void_p()
        _check(lib.eqmp_plan_staged(*args, ctypes.byref(h)), "eqmp_plan_staged")
        self._h, self._keep, self._lib = h, keep, lib
        self.h_out = keep[7]

    def launch(self, stream=None):
        st = self._lib.eqmp_plan_launch(self._h, _stream(stream))
        if st != EQMP_OK:
            raise EqmpError(st, "eqmp_plan_launch")
        return self.h_out

    def destroy(self):
        if self._h:
            self._lib.eqmp_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # pragma: no cover - interpreter shutdown
            pass


def eqmp_plan_staged(h_in, d_in, vec, x, row_offsets, src, out, h_out, w=None, R=None, M=None, n_edges=None):
    """The step of eqmp_fused_staged recorded once as a CUDA graph: returns a
    plan whose launch(stream=None) replays the input copy, the layer and the
    result copy with one graph launch.  The tensors must stay alive and
    unmoved while the plan is used (the plan holds references to them);
    h_in and h_out must be pinned."""
    if not (h_in.is_pinned() and h_out.is_pinned()):
        raise ValueError("h_in and h_out must be pinned for a plan")
    return eqmp_fused_staged(h_in, d_in, vec, x, row_offsets, src, out, h_out, w=w, R=R, M=M, n_edges=n_edges,
                             prepare="plan")


def eqmp_fused_so2(vec, x, row_offsets, src, w=None, R=None, M=None, out=None, stream=None,
                   n_edges=None):
    """eqmp_fused computed in the aligned (SO(2)) edge frame; same result."""
    import torch

    _require(vec, "vec", torch.float32)
    return _layer("eqmp_fused_so2", vec, x, row_offsets, src, w, R, M, out, stream, n_edges)


def eqmp_validate_graph(row_offsets, src, n_src, n_edges, stream=None):
    """Raise EqmpError(EQMP_ERR_GRAPH) if the CSR preconditions do not hold."""
    N = row_offsets.shape[0] - 1
    st = load_library().eqmp_validate_graph(_ptr(row_offsets), _ptr(src), N, int(n_src),
                                            int(n_edges), _stream(stream))
    _check(st, "eqmp_validate_graph")


def eqmp_device_error():
    """Watchdog code since the last call (0 = no device wait gave up)."""
    code = ctypes.c_int32(0)
    st = load_library().eqmp_device_error(ctypes.byref(code))
    if st not in (EQMP_OK, EQMP_ERR_DEVICE_TIMEOUT):
        _check(st, "eqmp_device_error")
    return int(code.value)


def eqmp_watchdog_selftest(wait_ms=20, stream=None):
    """Launch the watchdog self-test (a wait that must give up); read the code with eqmp_device_error()."""
    _check(load_library().eqmp_watchdog_selftest(int(wait_ms), _stream(stream)), "eqmp_watchdog_selftest")


def eqmp_fp32_peak_probe(iters, out, blocks_per_sm=4, stream=None):
    """Launch the FP32 throughput probe (out: one-float CUDA tensor); returns its flop count."""
    flops = ctypes.c_double(0.0)
    _check(load_library().eqmp_fp32_peak_probe(int(iters), int(blocks_per_sm), _ptr(out), ctypes.byref(flops),
                                                _stream(stream)), "eqmp_fp32_peak_probe")
    return flops.value


def eqmp_num_paths_lmax(l_max):
    return int(load_library().eqmp_num_paths_lmax(int(l_max)))


def eqmp_fused_lmax(l_max, vec, x, row_offsets, src, w=None, R=None, M=None, out=None, stream=None):
    """The layer at degree l_max = 4..6: x [N_src, C, (l_max+1)^2] fp32 -> out [N, C, (l_max+1)^2]."""
    import torch

    l_max = int(l_max)
    nc = (l_max + 1) ** 2
    for name, t in (("vec", vec), ("x", x), ("w", w), ("R", R), ("M", M)):
        _require(t, name, torch.float32)
    _require(row_offsets, "row_offsets", torch.int32)
    _require(src, "src", torch.int32)
    if x.dim() != 3 or x.shape[2] != nc:
        raise ValueError(f"x must be [N_src, C, {nc}]")
    n_src, C = x.shape[0], x.shape[1]
    N = row_offsets.shape[0] - 1
    if out is None:
        out = _empty((N, C, nc), torch.float32, x.device, stream)
    _require(out, "out", torch.float32)
    if tuple(out.shape) != (N, C, nc):
        raise ValueError(f"out must be [N, C, {nc}]")
    if w is not None:
        wt = Weights(ctypes.c_void_p(w.data_ptr()), None, None, 0)
    else:
        wt = Weights(None, ctypes.c_void_p(R.data_ptr()) if R is not None else None,
                     ctypes.c_void_p(M.data_ptr()) if M is not None else None,
                     R.shape[1] if R is not None and R.dim() == 2 else 0)
    st = load_library().eqmp_fused_lmax(l_max, _ptr(vec), _ptr(x), n_src, _ptr(row_offsets), _ptr(src), N,
                                        vec.shape[0], C, wt, _ptr(out), _stream(stream))
    _check(st, "eqmp_fused_lmax")
    return out


def eqmp_radius_graph(pos, cutoff, e_cap=None, dst=False, rev=False, stream=None, box=None):
    """Radius graph of pos [N, 3] fp32 (CUDA): dict(off, src, vec[, img][, dst][, rev]), E.

    Edges j -> i for i != j with the float32 squared distance below
    cutoff^2, CSR by receiver with senders ascending.  With box = (Lx, Ly, Lz)
    the boundaries are periodic (eqmp_radius_graph_pbc): positions inside the
    box, every image within one box length per direction, and "img" holds
    each edge's image index.  When the edge count exceeds the capacity
    (e_cap, default 64 N), the call is repeated once with the exact count,
    which costs one device-to-host read of E.
    """
    import torch

    _require(pos, "pos", torch.float32)
    if pos.dim() != 2 or pos.shape[1] != 3:
        raise ValueError("pos must be [N, 3]")
    lib = load_library()
    N = pos.shape[0]
    dev = pos.device
    ws = _empty(max(int(lib.eqmp_radius_graph_workspace_size(N)), 256), torch.uint8, dev, stream, temporary=True)
    off = _empty(N + 1, torch.int32, dev, stream)
    e_total = _empty(1, torch.int64, dev, stream, temporary=True)
    cap = int(64 * N if e_cap is None else e_cap)
    st = _stream(stream)
    for _ in range(2):
        out = dict(off=off, src=_empty(cap, torch.int32, dev, stream),
                   vec=_empty((cap, 3), torch.float32, dev, stream))
        if dst:
            out["dst"] = _empty(cap, torch.int32, dev, stream)
        if rev:
            out["rev"] = _empty(cap, torch.int32, dev, stream)
        if box is None:
            _check(lib.eqmp_radius_graph(_ptr(pos), N, float(cutoff), _ptr(off), _ptr(out["src"]),
                                         _ptr(out["vec"]), _ptr(out.get("dst")), _ptr(out.get("rev")), cap,
                                         _ptr(e_total), _ptr(ws), ws.numel(), st), "eqmp_radius_graph")
        else:
            out["img"] = _empty(cap, torch.int32, dev, stream)
            lengths = (ctypes.c_float * 3)(*[float(v) for v in box])
            _check(lib.eqmp_radius_graph_pbc(_ptr(pos), N, float(cutoff), lengths, _ptr(off), _ptr(out["src"]),
                                             _ptr(out["vec"]), _ptr(out["img"]), _ptr(out.get("dst")),
                                             _ptr(out.get("rev")), cap, _ptr(e_total), _ptr(ws), ws.numel(), st),
                   "eqmp_radius_graph_pbc")
        with torch.cuda.stream(_torch_stream(stream)):  # the count is read behind the kernels that write it
            E = int(e_total.item())
        if E < 0:
            raise EqmpError(EQMP_ERR_INVALID_ARG, "eqmp_radius_graph: positions non-finite or out of range"
                            " (outside the box, with periodic boundaries)"
                            if E == -1 else "eqmp_radius_graph: 2^31 edges or more")
        if E <= cap:
            break
        cap = E
    for k in ("src", "vec", "img", "dst", "rev"):
        if k in out:
            out[k] = out[k][:E]
    return out, E


def sender_view(src, n_src):
    """(send_offsets [n_src+1], send_edges [E]) grouping edge ids by sender
    (stable, edge order kept within a sender); host-side graph preparation
    for eqmp_fused_backward (numpy or torch CPU int arrays in, numpy out)."""
    import numpy as np

    src = np.asarray(src, dtype=np.int64)
    order = np.argsort(src, kind="stable").astype(np.int32)
    offs = np.searchsorted(src[order], np.arange(int(n_src) + 1), side="left").astype(np.int32)
    return offs, order


def _backward_prepare(vec, x, row_offsets, src, dst, send_offsets, send_edges, grad_out, w, R, M, need, stream):
    """Checks of the backward's inputs and its requested output tensors."""
    import torch

    spec = (("vec", vec, torch.float32), ("x", x, torch.float32),
            ("row_offsets", row_offsets, torch.int32), ("src", src, torch.int32),
            ("dst", dst, torch.int32), ("send_offsets", send_offsets, torch.int32),
            ("send_edges", send_edges, torch.int32), ("grad_out", grad_out, torch.float32),
            ("w", w, torch.float32), ("R", R, torch.float32), ("M", M, torch.float32))
    for name, t, dt in spec:  # every dtype first, then placement and layout
        _require(t, name, dt, cuda=False)
    for name, t, dt in spec:
        _require(t, name, dt)
    if (w is None) == (R is None or M is None):
        raise ValueError("give exactly one of w or (R, M)")
    n_src, C = x.shape[0], x.shape[1]
    N = row_offsets.shape[0] - 1
    E = vec.shape[0]
    radial = w is None
    dev = x.device
    out = {}
    if "x" in need:
        out["x"] = _empty((n_src, C, 16), torch.float32, dev, stream)
    if "vec" in need:
        out["vec"] = _empty((E, 3), torch.float32, dev, stream, zero=True)
    if radial:
        if "R" in need:
            out["R"] = _empty((E, 8), torch.float32, dev, stream, zero=True)
        if "M" in need:
            out["M"] = _empty((8, 34 * C), torch.float32, dev, stream)
    elif "w" in need:
        out["w"] = _empty((34, C), torch.float32, dev, stream)
    wt = (Weights(ctypes.c_void_p(w.data_ptr()), None, None, 0) if not radial else
          Weights(None, ctypes.c_void_p(R.data_ptr()), ctypes.c_void_p(M.data_ptr()), R.shape[1]))
    head = (_ptr(vec), _ptr(x), n_src, _ptr(row_offsets), _ptr(src), _ptr(dst), _ptr(send_offsets),
            _ptr(send_edges), send_edges.shape[0], N, E, C, wt, _ptr(grad_out), _ptr(out.get("x")),
            _ptr(out.get("w")), _ptr(out.get("R")), _ptr(out.get("M")), _ptr(out.get("vec")))
    return out, head, (N, E, C, radial)


def eqmp_fused_backward(vec, x, row_offsets, src, dst, send_offsets, send_edges, grad_out,
                        w=None, R=None, M=None, need=("x", "w", "vec"), stream=None):
    """Gradients of the fused layer; returns {"x", "w" | "R", "M", "vec"} as requested."""
    import torch

    out, head, (N, E, C, radial) = _backward_prepare(vec, x, row_offsets, src, dst, send_offsets,
                                                     send_edges, grad_out, w, R, M, need, stream)
    lib = load_library()
    nbytes = int(lib.eqmp_fused_backward_workspace_size(N, E, C, 1 if radial else 0))
    if nbytes < 0:
        raise EqmpError(EQMP_ERR_CUDA, "eqmp_fused_backward_workspace_size")
    ws = _empty(max(nbytes // 4, 4), torch.float32, x.device, stream, temporary=True)
    _check(lib.eqmp_fused_backward(*head, _ptr(ws), ws.numel() * 4, _stream(stream)), "eqmp_fused_backward")
    return out


def eqmp_fused_backward_noalloc(vec, x, row_offsets, src, dst, send_offsets, send_edges, grad_out,
                                w=None, R=None, M=None, need=("x", "w", "vec"), stream=None):
    """eqmp_fused_backward with the library's static scratch instead of a
    workspace (the C entry point allocates no device memory; this wrapper
    only allocates the requested output tensors through torch)."""
    out, head, _ = _backward_prepare(vec, x, row_offsets, src, dst, send_offsets, send_edges, grad_out,
                                     w, R, M, need, stream)
    _check(load_library().eqmp_fused_backward_noalloc(*head, _stream(stream)), "eqmp_fused_backward_noalloc")
    return out


# ------------------------------------------------------------------ norms and dropout
_OUT_NAMES = {k: f"out[{k!r}]" for k in ("y", "s", "stats", "x", "r", "w", "b", "q", "k", "v", "wq", "wk", "pos", "rstd",
                                               "bias", "bucket", "table", "out")}
_L_MAX = {16: 3, 25: 4, 36: 5, 49: 6}  # components of a channel -> degree


def _refuse(t, name, dtype, shape, dev):
    """The error of a tensor that is not what an entry point needs."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _packed(t, name, dtype, shape, dev, torch):
    """Checks a packed tensor and returns its address."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev, torch):
    """Checks an input of rows and returns its address and row stride.  A row (everything behind the first dimension)
    is packed; the rows of a matrix may be any distance apart."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    if t.is_contiguous() or (len(shape) == 2 and (t.stride(1) == 1 or shape[1] == 1)):
        return t.data_ptr(), t.stride(0)
    raise ValueError(f"{name} must have contiguous rows" if len(shape) == 2 else f"{name} must be contiguous")


def _result(out, k, like, dtype, shape, dev, torch, stream):
    """The result tensor k: the caller's own from `out`, or a new one on the device of `like`."""
    if out is None or (t := out.get(k)) is None:
        if stream is None:
            t = torch.empty(shape, dtype=dtype, device=like.device)
        else:
            t = _empty(shape, dtype, like.device, stream)
        return t, t.data_ptr()
    return t, _packed(t, _OUT_NAMES[k], dtype, shape, dev, torch)


def _main_input(x, name, degree, torch):
    """Checks the type and the form of a norm's main input; returns the current device and the degree."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not torch.float32 and x.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = x.shape
    if degree:
        l_max = _L_MAX.get(shape[2], 0) if len(shape) == 3 else 0
        if not l_max or shape[1] < 1:
            raise ValueError(f"{name} must be [N, C, (l_max+1)^2] with l_max in 3..6 and C >= 1")
        return torch.cuda.current_device(), l_max
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be [rows, cols] with cols >= 1")
    return torch.cuda.current_device(), 0


def _drop(drop, dev):
    if not isinstance(drop, Dropout):
        raise TypeError(f"drop must be a Dropout, not {type(drop).__name__}")
    if drop.step is not None and drop.step.get_device() != dev:
        raise ValueError("drop's step must be a CUDA tensor on the current device")
    return drop


def _raw_stream(stream, dev, torch):
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _unknown(need, allowed):
    for k in need:
        if k not in allowed:
            raise ValueError(f"need has {k!r}; allowed are {', '.join(allowed)}")


def _norm_forward(entry, degree, x, w, b, eps, residual, drop, need, out, stream):
    import torch

    f32 = torch.float32
    dev, l_max = _main_input(x, "x", degree, torch)
    dtype, shape = x.dtype, x.shape
    n, c = shape[0], shape[1]
    xp, x_ld = _rows(x, "x", dtype, shape, dev, torch)
    rp, r_ld = (None, 0) if residual is None else _rows(residual, "residual", dtype, shape, dev, torch)
    wp = None if w is None else _packed(w, "w", f32, (l_max + 1, c) if degree else (c,), dev, torch)
    bp = None if b is None else _packed(b, "b", f32, (c,), dev, torch)
    if need is None:
        need = ("y",) if residual is None else ("y", "s")
    got, sp, yp, tp = {}, None, None, None
    if "y" in need:
        got["y"], yp = _result(out, "y", x, dtype, shape, dev, torch, stream)
    if "s" in need:
        got["s"], sp = _result(out, "s", x, dtype, shape, dev, torch, stream)
    if "stats" in need:
        got["stats"], tp = _result(out, "stats", x, f32, (n, l_max + 2), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("y", "s", "stats"))
    dt = EQMP_F32 if dtype is f32 else EQMP_BF16
    dr = _NO_DROP if drop is None else _drop(drop, dev)
    lib, st = load_library(), _raw_stream(stream, dev, torch)
    if degree:
        status = lib.eqmp_degree_norm(xp, rp, dt, n, c, l_max, dr, wp, bp, eps, sp, yp, tp, st)
    else:
        status = lib.eqmp_layer_norm(xp, x_ld, rp, r_ld, dt, n, c, dr, wp, bp, eps, sp, yp, tp, st)
    if status:
        raise EqmpError(status, entry)
    return got


def _norm_backward(entry, degree, grad_y, s, stats, w, grad_s, drop, need, out, workspace, stream):
    import torch

    f32 = torch.float32
    dev, l_max = _main_input(s, "s", degree, torch)
    dtype, shape = s.dtype, s.shape
    n, c = shape[0], shape[1]
    w_shape = (l_max + 1, c) if degree else (c,)
    xp, x_ld = _rows(s, "s", dtype, shape, dev, torch)
    gp, g_ld = _rows(grad_y, "grad_y", dtype, shape, dev, torch)
    rp, r_ld = (None, 0) if grad_s is None else _rows(grad_s, "grad_s", dtype, shape, dev, torch)
    wp = None if w is None else _packed(w, "w", f32, w_shape, dev, torch)
    tp = _packed(stats, "stats", f32, (n, l_max + 2), dev, torch)
    got, grp, gxp, gwp, gbp, ws, nbytes = {}, None, None, None, None, None, 0
    if "x" in need:
        got["x"], gxp = _result(out, "x", s, dtype, shape, dev, torch, stream)
    if "r" in need:
        got["r"], grp = _result(out, "r", s, dtype, shape, dev, torch, stream)
    if "w" in need:
        got["w"], gwp = _result(out, "w", s, f32, w_shape, dev, torch, stream)
    if "b" in need:
        got["b"], gbp = _result(out, "b", s, f32, (c,), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("x", "r", "w", "b"))
    lib, st = load_library(), _raw_stream(stream, dev, torch)
    if gwp is not None or gbp is not None:
        if workspace is None:
            nbytes = (lib.eqmp_degree_norm_backward_workspace_size(n, c, l_max) if degree else
                      lib.eqmp_layer_norm_backward_workspace_size(n, c))
            if nbytes < 0:
                raise EqmpError(EQMP_ERR_UNSUPPORTED, entry)
            workspace = _empty(nbytes // 4 + 4, f32, s.device, stream, temporary=True)
        else:
            _require(workspace, "workspace", torch.uint8)
            if workspace.get_device() != dev:
                raise ValueError("workspace must be a CUDA tensor on the current device")
            nbytes = workspace.numel()
        ws = workspace.data_ptr()
    dt = EQMP_F32 if dtype is f32 else EQMP_BF16
    dr = _NO_DROP if drop is None else _drop(drop, dev)
    if degree:
        status = lib.eqmp_degree_norm_backward(gp, xp, rp, dt, n, c, l_max, dr, wp, tp, grp, gxp, gwp, gbp, ws, nbytes, st)
    else:
        status = lib.eqmp_layer_norm_backward(gp, g_ld, xp, x_ld, rp, r_ld, dt, n, c, dr, wp, tp, grp, gxp, gwp, gbp, ws,
                                              nbytes, st)
    if status:
        raise EqmpError(status, entry)
    return got


def eqmp_dropout(x, drop, out=None, stream=None):
    """dropout(x), fp32 or bf16, by a Dropout.  x: [rows, ...]; the row of an element and its place in the row choose
    its draw.  The backward pass is the same call on the gradient.  out may be x (in place)."""
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dtype, shape = x.dtype, x.shape
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"x has dtype {dtype}")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    cols = 1
    for n in shape[1:]:
        cols *= n
    if not shape or cols < 1:
        raise ValueError("x must be [rows, ...] with values in a row")
    dev = torch.cuda.current_device()
    xp, ld = _rows(x, "x", dtype, shape, dev, torch)
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
    op = _packed(out, "out", dtype, shape, dev, torch)
    dr = _NO_DROP if drop is None else _drop(drop, dev)
    status = load_library().eqmp_dropout(xp, cols if out is x else ld, EQMP_F32 if dtype is torch.float32 else EQMP_BF16,
                                         shape[0], cols, dr, op,
                                         _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_dropout")
    return out


def eqmp_layer_norm(x, w=None, b=None, eps=1e-5, residual=None, drop=None, need=None, out=None, stream=None):
    """Layer norm of the rows of x [rows, cols] (fp32 or bf16; w, b fp32 [cols] or None), behind an optional dropout
    and residual sum: s = residual + dropout(x), y = norm(s).

    Returns a dict of what `need` names: "y", "s" (default with a residual) and "stats" ([rows, 2], for the backward
    pass).  `out` may hold tensors to write into, by the same names.  x and residual may be slices of wider
    matrices (contiguous rows, any distance apart)."""
    return _norm_forward("eqmp_layer_norm", False, x, w, b, eps, residual, drop, need, out, stream)


def eqmp_layer_norm_backward(grad_y, s, stats, w=None, grad_s=None, drop=None, need=("x", "w", "b"), out=None,
                             workspace=None, stream=None):
    """Gradients of eqmp_layer_norm from dL/dy, the forward pass's s (x where there was neither residual nor dropout)
    and stats, and grad_s = dL/ds from other uses of s.

    Returns a dict of what `need` names: "x" (behind the dropout), "r" (dL/ds in all: of the residual), "w", "b"."""
    return _norm_backward("eqmp_layer_norm_backward", False, grad_y, s, stats, w, grad_s, drop, need, out, workspace,
                          stream)


def eqmp_degree_norm(x, w=None, b=None, eps=1e-5, residual=None, drop=None, need=None, out=None, stream=None):
    """The layer norm by degree of node features x [N, C, (l_max+1)^2], l_max 3..6, which commutes with rotations:
    degree 0 as a layer norm over the channels, each degree l > 0 divided by its root mean square over channels and
    orders.  w [l_max+1, C] and b [C] fp32 or None; drop.group must be (l_max+1)^2.  Otherwise as eqmp_layer_norm,
    with stats [N, l_max+2]; tensors are contiguous."""
    return _norm_forward("eqmp_degree_norm", True, x, w, b, eps, residual, drop, need, out, stream)


def eqmp_degree_norm_backward(grad_y, s, stats, w=None, grad_s=None, drop=None, need=("x", "w", "b"), out=None,
                              workspace=None, stream=None):
    """Gradients of eqmp_degree_norm; as eqmp_layer_norm_backward, with "w" [l_max+1, C] and "b" [C]."""
    return _norm_backward("eqmp_degree_norm_backward", True, grad_y, s, stats, w, grad_s, drop, need, out, workspace,
                          stream)


def eqmp_layer_norm_backward_workspace_size(rows, cols):
    """Bytes of workspace that eqmp_layer_norm_backward needs for grad_w and grad_b."""
    return int(load_library().eqmp_layer_norm_backward_workspace_size(int(rows), int(cols)))


def eqmp_degree_norm_backward_workspace_size(n, channels, l_max):
    """Bytes of workspace that eqmp_degree_norm_backward needs for grad_w and grad_b."""
    return int(load_library().eqmp_degree_norm_backward_workspace_size(int(n), int(channels), int(l_max)))


# ------------------------------------------------------------------ attention over a receiver's edges
def _heads(t, name, dtype, shape, dev, torch):
    """Checks a tensor [N, H, D] and returns its address and the distance between nodes.  A node's heads are packed; the
    nodes may be any distance apart."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    n, h, d = shape
    node, head, one = t.stride()
    if (one == 1 or d == 1) and (head == d or h == 1):
        return t.data_ptr(), node if n > 1 else h * d
    raise ValueError(f"{name} must have contiguous heads")


def _head_input(x, name, torch):
    """Checks the type and the form of a main input [N, H, D]; returns the current device."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not torch.float32 and x.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() != 3 or x.shape[1] < 1 or x.shape[2] < 1:
        raise ValueError(f"{name} must be [N, H, D] with H >= 1 and D >= 1")
    return torch.cuda.current_device()


def _workspace(workspace, nbytes, entry, like, dev, stream, torch):
    """Address and size of a call's workspace: the caller's, or a temporary one."""
    if nbytes < 0:
        raise EqmpError(EQMP_ERR_UNSUPPORTED, entry)
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = _empty(nbytes, torch.uint8, like.device, stream, temporary=True)
        return workspace.data_ptr(), nbytes, workspace
    _require(workspace, "workspace", torch.uint8)
    if workspace.get_device() != dev:
        raise ValueError("workspace must be a CUDA tensor on the current device")
    return workspace.data_ptr(), workspace.numel(), workspace


def _positions(pos, freq, n, d, dev, torch):
    """Addresses of positions and frequencies and the number of axes; 0 axes without them."""
    if pos is None and freq is None:
        return None, None, 0
    if pos is None or freq is None:
        raise ValueError("give pos and freq together")
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2 or not 1 <= pos.shape[1] <= 3:
        raise ValueError("pos must be a tensor [N, axes] with 1 to 3 axes")
    if d % 2:
        raise ValueError("a rotation needs an even head size")
    axes, f32 = pos.shape[1], torch.float32
    return _packed(pos, "pos", f32, (n, axes), dev, torch), _packed(freq, "freq", f32, (d // 2, axes), dev, torch), axes


def eqmp_head_norm(q, k=None, wq=None, wk=None, eps=1e-6, pos=None, freq=None, need=None, out=None, stream=None):
    """Norm of each head of the queries q [N, Hq, D] and keys k [N, Hk, D] (fp32 or bf16) by its root mean square, times
    wq, wk (fp32 [D] or None), then the rotation of its pairs (2p, 2p+1) by the angles
    theta[n, p] = sum_a pos[n, a] freq[p, a] (pos [N, axes], freq [D/2, axes], fp32; None: no rotation).

    Returns a dict of what `need` names: "q", "k" (the default) and "rstd" ([N, Hq + Hk], for the backward pass).  `out`
    may hold tensors to write into, by the same names.  q and k may be slices of one projection (packed heads, nodes any
    distance apart)."""
    import torch

    f32 = torch.float32
    dev = _head_input(q, "q", torch)
    dtype, (n, hq, d) = q.dtype, q.shape
    hk = 0
    if k is not None:
        _head_input(k, "k", torch)
        hk = k.shape[1]
    qp, q_ld = _heads(q, "q", dtype, q.shape, dev, torch)
    kp, k_ld = (None, 0) if k is None else _heads(k, "k", dtype, (n, hk, d), dev, torch)
    wqp = None if wq is None else _packed(wq, "wq", f32, (d,), dev, torch)
    wkp = None if wk is None else _packed(wk, "wk", f32, (d,), dev, torch)
    pp, fp, axes = _positions(pos, freq, n, d, dev, torch)
    if need is None:
        need = ("q",) if k is None else ("q", "k")
    got, oq, ok, rp = {}, None, None, None
    if "q" in need:
        got["q"], oq = _result(out, "q", q, dtype, (n, hq, d), dev, torch, stream)
    if "k" in need:
        if k is None:
            raise ValueError("need has 'k', and there are no keys")
        got["k"], ok = _result(out, "k", q, dtype, (n, hk, d), dev, torch, stream)
    if "rstd" in need:
        got["rstd"], rp = _result(out, "rstd", q, f32, (n, hq + hk), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("q", "k", "rstd"))
    status = load_library().eqmp_head_norm(qp, q_ld, hq, kp, k_ld, hk, EQMP_F32 if dtype is f32 else EQMP_BF16, n, d, wqp, wkp,
                                           eps, pp, fp, axes, oq, ok, rp, _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_head_norm")
    return got


def eqmp_head_norm_backward(grad_q, grad_k, q, k, rstd, wq=None, wk=None, pos=None, freq=None, need=None, out=None,
                            workspace=None, stream=None):
    """Gradients of eqmp_head_norm from those of its results, its inputs and its rstd (grad_k and k None: queries alone).

    Returns a dict of what `need` names: "q", "k", "wq", "wk" (the default, keys' where there are keys) and "pos"."""
    import torch

    f32 = torch.float32
    dev = _head_input(q, "q", torch)
    dtype, (n, hq, d) = q.dtype, q.shape
    if (k is None) != (grad_k is None):
        raise ValueError("give k and grad_k together")
    hk = 0
    if k is not None:
        _head_input(k, "k", torch)
        hk = k.shape[1]
    qp, q_ld = _heads(q, "q", dtype, q.shape, dev, torch)
    gqp, gq_ld = _heads(grad_q, "grad_q", dtype, q.shape, dev, torch)
    kp, k_ld = (None, 0) if k is None else _heads(k, "k", dtype, (n, hk, d), dev, torch)
    gkp, gk_ld = (None, 0) if k is None else _heads(grad_k, "grad_k", dtype, (n, hk, d), dev, torch)
    wqp = None if wq is None else _packed(wq, "wq", f32, (d,), dev, torch)
    wkp = None if wk is None else _packed(wk, "wk", f32, (d,), dev, torch)
    rp = _packed(rstd, "rstd", f32, (n, hq + hk), dev, torch)
    pp, fp, axes = _positions(pos, freq, n, d, dev, torch)
    allowed = ("q", "wq") + (("k", "wk") if hk else ()) + (("pos",) if axes else ())
    if need is None:
        need = ("q", "k", "wq", "wk") if hk else ("q", "wq")
    _unknown(need, allowed)
    got, oq, ok, owq, owk, op = {}, None, None, None, None, None
    if "q" in need:
        got["q"], oq = _result(out, "q", q, dtype, (n, hq, d), dev, torch, stream)
    if "k" in need:
        got["k"], ok = _result(out, "k", q, dtype, (n, hk, d), dev, torch, stream)
    if "wq" in need:
        got["wq"], owq = _result(out, "wq", q, f32, (d,), dev, torch, stream)
    if "wk" in need:
        got["wk"], owk = _result(out, "wk", q, f32, (d,), dev, torch, stream)
    if "pos" in need:
        got["pos"], op = _result(out, "pos", q, f32, (n, axes), dev, torch, stream)
    lib = load_library()
    ws, nbytes, held = None, 0, None
    if owq is not None or owk is not None:
        ws, nbytes, held = _workspace(workspace, lib.eqmp_head_norm_backward_workspace_size(n, d), "eqmp_head_norm_backward", q,
                                      dev, stream, torch)
    status = lib.eqmp_head_norm_backward(gqp, gq_ld, gkp, gk_ld, qp, q_ld, hq, kp, k_ld, hk,
                                         EQMP_F32 if dtype is f32 else EQMP_BF16, n, d, wqp, wkp, rp, pp, fp, axes, oq, ok, owq,
                                         owk, op, ws, nbytes, _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_head_norm_backward")
    return got


def eqmp_head_norm_backward_workspace_size(n, head_size):
    """Bytes of workspace that eqmp_head_norm_backward needs for the weights' gradients."""
    return int(load_library().eqmp_head_norm_backward_workspace_size(int(n), int(head_size)))


def eqmp_edge_bias(vec, borders, table, need=("bias", "bucket"), out=None, stream=None):
    """The learned bias of each edge and head by the bucket of the edge's length: bucket[e] = the number of borders
    [B-1] (fp32, ascending) that are at most |vec[e]| (vec [E, 3] fp32), bias[e] = table[bucket[e]] (table [B, H] fp32).

    Returns a dict of what `need` names: "bias" [E, H] and "bucket" [E] int32 (for the backward pass).  `out` may hold
    tensors to write into."""
    import torch

    f32 = torch.float32
    for t, name in ((vec, "vec"), (table, "table")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if vec.dim() != 2 or table.dim() != 2 or table.shape[0] < 1 or table.shape[1] < 1:
        raise ValueError("vec must be [E, 3], table [B, H] with B, H >= 1")
    dev = torch.cuda.current_device()
    n, (b, h) = vec.shape[0], table.shape
    vp = _packed(vec, "vec", f32, (n, 3), dev, torch)
    tp = _packed(table, "table", f32, (b, h), dev, torch)
    bp = _packed(borders, "borders", f32, (b - 1,), dev, torch)
    got, op, kp = {}, None, None
    if "bias" in need:
        got["bias"], op = _result(out, "bias", vec, f32, (n, h), dev, torch, stream)
    if "bucket" in need:
        got["bucket"], kp = _result(out, "bucket", vec, torch.int32, (n,), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("bias", "bucket"))
    status = load_library().eqmp_edge_bias(vp, n, bp, b, tp, h, op, kp, _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_edge_bias")
    return got


def eqmp_edge_bias_backward(grad_bias, bucket, n_buckets, out=None, workspace=None, stream=None):
    """Gradient of eqmp_edge_bias's table, dict(table=[n_buckets, H]): the sums of grad_bias [E, H] (fp32) over the edges of
    each bucket."""
    import torch

    f32 = torch.float32
    if not isinstance(grad_bias, torch.Tensor):
        raise TypeError("grad_bias must be a torch.Tensor")
    if grad_bias.dim() != 2 or grad_bias.shape[1] < 1:
        raise ValueError("grad_bias must be [E, H] with H >= 1")
    if n_buckets < 1:
        raise ValueError("n_buckets must be at least 1")
    dev = torch.cuda.current_device()
    n, h = grad_bias.shape
    gp = _packed(grad_bias, "grad_bias", f32, (n, h), dev, torch)
    kp = _packed(bucket, "bucket", torch.int32, (n,), dev, torch)
    table, tp = _result(out, "table", grad_bias, f32, (n_buckets, h), dev, torch, stream)
    lib = load_library()
    ws, nbytes, held = _workspace(workspace, lib.eqmp_edge_bias_backward_workspace_size(n, n_buckets, h),
                                  "eqmp_edge_bias_backward", grad_bias, dev, stream, torch)
    status = lib.eqmp_edge_bias_backward(gp, kp, n, n_buckets, h, tp, ws, nbytes, _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_edge_bias_backward")
    return dict(table=table)


def eqmp_edge_bias_backward_workspace_size(n_edges, n_buckets, heads):
    """Bytes of workspace that eqmp_edge_bias_backward needs."""
    return int(load_library().eqmp_edge_bias_backward_workspace_size(int(n_edges), int(n_buckets), int(heads)))


def _attention_inputs(q, k, v, row_offsets, src, bias, torch):
    """Checks of what both passes of the attention take; the sizes and the arguments in the order of the C call."""
    f32, i32 = torch.float32, torch.int32
    dev = _head_input(q, "q", torch)
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.dim() == 3 and v.dim() == 3 and v.shape[2] > 0):
        _head_input(k, "k", torch)
        _head_input(v, "v", torch)
    dtype, (n, h, d), n_src, dv = q.dtype, q.shape, k.shape[0], v.shape[2]
    qp, q_ld = _heads(q, "q", dtype, (n, h, d), dev, torch)
    kp, k_ld = _heads(k, "k", dtype, (n_src, h, d), dev, torch)
    vp, v_ld = _heads(v, "v", dtype, (n_src, h, dv), dev, torch)
    op = _packed(row_offsets, "row_offsets", i32, (n + 1,), dev, torch)
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be a tensor [E]")
    e = src.shape[0]
    sp = _packed(src, "src", i32, (e,), dev, torch)
    bp = None if bias is None else _packed(bias, "bias", f32, (e, h), dev, torch)
    rows = (qp, q_ld, kp, k_ld, vp, v_ld, EQMP_F32 if dtype is f32 else EQMP_BF16, n, n_src, e, h, d, dv, op, sp)
    return dev, dtype, (n, n_src, e, h, d, dv), rows, bp


def eqmp_edge_attention(q, k, v, row_offsets, src, bias=None, scale=None, need=("out",), out=None, workspace=None, stream=None):
    """Attention over a receiver's edges: softmax over the edges e of receiver i of scale q[i].k[src[e]] + bias[e], and the
    sum of v[src[e]] by it, for each head.  q [N, H, D], k [N_src, H, D], v [N_src, H, Dv] (fp32 or bf16, one type; packed
    heads, nodes any distance apart), bias [E, H] fp32 or None, scale 1 / sqrt(D) by default.  v may be node features
    [N_src, C, K] as features.view(N_src, H, C // H * K).

    An edge whose bias is -inf is left out; a receiver without an edge gets zeros.  Returns a dict of what `need` names:
    "out" [N, H, Dv] and "stats" ([N, H, 2], for the backward pass).  `out` may hold tensors to write into."""
    import torch

    dev, dtype, (n, n_src, e, h, d, dv), rows, bp = _attention_inputs(q, k, v, row_offsets, src, bias, torch)
    got, op, tp = {}, None, None
    if "out" in need:
        got["out"], op = _result(out, "out", q, dtype, (n, h, dv), dev, torch, stream)
    if "stats" in need:
        got["stats"], tp = _result(out, "stats", q, torch.float32, (n, h, 2), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("out", "stats"))
    lib = load_library()
    ws, nbytes, held = _workspace(workspace, lib.eqmp_edge_attention_workspace_size(e, h, dv), "eqmp_edge_attention", q, dev,
                                  stream, torch)
    status = lib.eqmp_edge_attention(*rows, bp, d ** -0.5 if scale is None else scale, op, tp, ws, nbytes,
                                     _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_edge_attention")
    return got


def eqmp_edge_attention_backward(grad_out, q, k, v, stats, row_offsets, src, dst, send_offsets, send_edges, bias=None,
                                 scale=None, need=("q", "k", "v"), out=None, workspace=None, stream=None):
    """Gradients of eqmp_edge_attention from grad_out [N, H, Dv], the forward call's inputs and its stats.  dst, send_offsets
    and send_edges: the sender view of the edges, as eqmp_fused_backward (None where neither "k" nor "v" is asked for).

    Returns a dict of what `need` names: "q", "k", "v" and "bias" ([E, H])."""
    import torch

    f32, i32 = torch.float32, torch.int32
    dev, dtype, (n, n_src, e, h, d, dv), rows, bp = _attention_inputs(q, k, v, row_offsets, src, bias, torch)
    gp, g_ld = _heads(grad_out, "grad_out", dtype, (n, h, dv), dev, torch)
    tp = _packed(stats, "stats", f32, (n, h, 2), dev, torch)
    dp, sop, sep, e_send = None, None, None, 0
    if "k" in need or "v" in need:
        if not isinstance(send_edges, torch.Tensor) or send_edges.dim() != 1:
            raise ValueError("send_edges must be a tensor [E_send]")
        e_send = send_edges.shape[0]
        dp = _packed(dst, "dst", i32, (e,), dev, torch)
        sop = _packed(send_offsets, "send_offsets", i32, (n_src + 1,), dev, torch)
        sep = _packed(send_edges, "send_edges", i32, (e_send,), dev, torch)
    got, gq, gk, gv, gb = {}, None, None, None, None
    if "q" in need:
        got["q"], gq = _result(out, "q", q, dtype, (n, h, d), dev, torch, stream)
    if "k" in need:
        got["k"], gk = _result(out, "k", q, dtype, (n_src, h, d), dev, torch, stream)
    if "v" in need:
        got["v"], gv = _result(out, "v", q, dtype, (n_src, h, dv), dev, torch, stream)
    if "bias" in need:
        got["bias"], gb = _result(out, "bias", q, f32, (e, h), dev, torch, stream)
    if len(got) != len(need):
        _unknown(need, ("q", "k", "v", "bias"))
    lib = load_library()
    ws, nbytes, held = _workspace(workspace, lib.eqmp_edge_attention_backward_workspace_size(n, e, e_send, h, d, dv),
                                  "eqmp_edge_attention_backward", q, dev, stream, torch)
    status = lib.eqmp_edge_attention_backward(gp, g_ld, *rows, dp, sop, sep, e_send, bp, d ** -0.5 if scale is None else scale, tp,
                                              gq, gk, gv, gb, ws, nbytes, _raw_stream(stream, dev, torch))
    if status:
        raise EqmpError(status, "eqmp_edge_attention_backward")
    return got


def eqmp_edge_attention_workspace_size(n_edges, heads, value_size):
    """Bytes of workspace that eqmp_edge_attention needs (0: none)."""
    return int(load_library().eqmp_edge_attention_workspace_size(int(n_edges), int(heads), int(value_size)))


def eqmp_edge_attention_backward_workspace_size(n, n_edges, n_send_edges, heads, head_size, value_size):
    """Bytes of workspace that eqmp_edge_attention_backward needs."""
    return int(load_library().eqmp_edge_attention_backward_workspace_size(int(n), int(n_edges), int(n_send_edges), int(heads),
                                                                           int(head_size), int(value_size)))
