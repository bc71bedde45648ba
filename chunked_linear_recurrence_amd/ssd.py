"""ctypes binding of libssdscan (include/libssdscan.h): argument marshalling only.

Every step of the computation runs in the library's HIP kernels.  torch is used for
device memory (output and workspace tensors) and for the current HIP stream.  If the
built library is missing the first call raises; there is no fallback path.
"""
import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libssdscan.so")

SSD_F32, SSD_BF16 = 0, 1
SSD_FLAG_RESIDUAL = 1
SSD_FLAG_WAVEFRONT = 2
SSD_FLAG_SCAN_FORM = 4
SSD_FLAG_SILU = 8
SSD_FLAG_SOFTPLUS = 16

STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL_ARG", 2: "SSD_ERR_BAD_SHAPE", 3: "SSD_ERR_BAD_DTYPE",
          4: "SSD_ERR_UNSUPPORTED", 5: "SSD_ERR_MISALIGNED", 6: "SSD_ERR_WORKSPACE",
          7: "SSD_ERR_HIP", 8: "SSD_ERR_ALIAS"}

# Every symbol the header declares.
EXPORTS = ["ssd_chunk_scan_workspace_bytes", "ssd_chunk_scan_fwd", "ssd_segmented_workspace_bytes",
           "ssd_chunk_scan_segmented", "ssd_chunk_scan_stages", "ssd_workspace_layout",
           "ssd_shape_supported", "ssd_status_string", "ssd_last_error_message", "ssd_version", "ssd_step",
           "ssd_scan_form_supported", "ssd_chunk_scan_fwd_noalloc",
           "ssd_conv_fwd", "ssd_conv_step", "ssd_conv_bwd", "ssd_conv_bwd_workspace_bytes",
           "ssd_selective_fwd", "ssd_selective_step", "ssd_selective_bwd", "ssd_selective_kept_bytes",
           "ssd_selective_fwd_workspace_bytes", "ssd_selective_bwd_workspace_bytes",
           "ssd_norm_fwd", "ssd_norm_bwd", "ssd_norm_bwd_workspace_bytes"]

# Workspace limit of ssd_chunk_scan_fwd_noalloc (SSD_NOALLOC_SCRATCH_BYTES in the header).
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ConvDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x_batch_stride", ctypes.c_int64), ("x_token_stride", ctypes.c_int64),
                ("dy_batch_stride", ctypes.c_int64), ("dy_token_stride", ctypes.c_int64)]


class SelectiveDims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "seqlen", "channels", "dstate", "ngroups")] +
                [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)] +
                [(n + s, ctypes.c_int64) for n in ("u", "delta", "z", "B", "C", "dy")
                 for s in ("_batch_stride", "_token_stride")])


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_row_stride", ctypes.c_int64), ("dy_row_stride", ctypes.c_int64)]


class SSDError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__("%s: %s" % (STATUS.get(status, status), message))


_lib = None


def lib():
    """Load libssdscan.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libssdscan.so is not built (%s); run __graft_entry__.build() "
                               "or python chunked_linear_recurrence_amd/build.py" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32, i64, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
        dp = ctypes.POINTER(Dims)
        L.ssd_chunk_scan_workspace_bytes.argtypes = [dp, i32]
        L.ssd_chunk_scan_workspace_bytes.restype = sz
        L.ssd_chunk_scan_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, u32, vp, sz, vp]
        L.ssd_chunk_scan_fwd.restype = ctypes.c_int
        L.ssd_chunk_scan_fwd_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, u32, vp]
        L.ssd_chunk_scan_fwd_noalloc.restype = ctypes.c_int
        L.ssd_chunk_scan_stages.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, u32, vp, sz, vp, i32, i32]
        L.ssd_chunk_scan_stages.restype = ctypes.c_int
        L.ssd_segmented_workspace_bytes.argtypes = [dp, i32, i64, i32, u32]
        L.ssd_segmented_workspace_bytes.restype = sz
        L.ssd_chunk_scan_segmented.argtypes = [dp, i32, i64, vp, vp, vp, vp, vp, vp, vp, i32, u32, vp, vp, sz, vp]
        L.ssd_chunk_scan_segmented.restype = ctypes.c_int
        L.ssd_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, u32, vp]
        L.ssd_step.restype = ctypes.c_int
        L.ssd_workspace_layout.argtypes = [dp, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.ssd_workspace_layout.restype = ctypes.c_int
        L.ssd_scan_form_supported.argtypes = [i32, i32, i64, i64]
        L.ssd_scan_form_supported.restype = i32
        L.ssd_shape_supported.argtypes = [i32, i32, i64, i64]
        L.ssd_shape_supported.restype = i32
        cp, sp, np_ = ctypes.POINTER(ConvDims), ctypes.POINTER(SelectiveDims), ctypes.POINTER(NormDims)
        f32 = ctypes.c_float
        for name, args in (("ssd_conv_fwd", [cp] + [vp] * 7 + [u32, vp]),
                           ("ssd_conv_step", [cp] + [vp] * 6 + [u32, vp]),
                           ("ssd_conv_bwd", [cp] + [vp] * 11 + [u32, vp, sz, vp]),
                           ("ssd_selective_fwd", [sp] + [vp] * 13 + [u32, vp, sz, vp]),
                           ("ssd_selective_step", [sp] + [vp] * 11 + [u32, vp]),
                           ("ssd_selective_bwd", [sp] + [vp] * 21 + [u32, vp, sz, vp]),
                           ("ssd_norm_fwd", [np_, vp, vp, vp, f32, vp, vp, vp, vp]),
                           ("ssd_norm_bwd", [np_] + [vp] * 9 + [sz, vp])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        for name, arg in (("ssd_conv_bwd_workspace_bytes", cp), ("ssd_selective_kept_bytes", sp),
                          ("ssd_selective_fwd_workspace_bytes", sp), ("ssd_selective_bwd_workspace_bytes", sp),
                          ("ssd_norm_bwd_workspace_bytes", np_)):
            getattr(L, name).argtypes = [arg]
            getattr(L, name).restype = sz
        L.ssd_status_string.argtypes = [ctypes.c_int]
        L.ssd_status_string.restype = ctypes.c_char_p
        L.ssd_last_error_message.argtypes = []
        L.ssd_last_error_message.restype = ctypes.c_char_p
        L.ssd_version.argtypes = []
        L.ssd_version.restype = i32
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise SSDError(status, lib().ssd_last_error_message().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()      # ctypes passes ints as void *


# Moves the versions of the tensors of a sequence on (torch.autograd.graph.increment_version
# without its own checks: a single-token call counts in tenths of a microsecond).
_move_on = torch._C._increment_version


def _wrote(*tensors):
    """The caller's tensors that a call has written (None: not given).  Autograd does not see a
    write behind a pointer; with its version moved on, a backward that saved such a tensor raises
    instead of reading the new values."""
    _move_on([t for t in tensors if t is not None])


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_ACT_DTYPES = (torch.float32, torch.bfloat16)


def _expect(name, t, shape, dtypes, allow_none=False):
    """Raise ValueError unless tensor `t` has exactly `shape` (None entries match any
    size), one of `dtypes` and a contiguous layout.  The C side sees only raw pointers,
    so this is the one place where a wrong dtype, shape or stride can be caught."""
    if t is None:
        if allow_none:
            return
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor (got %s)" % (name, type(t).__name__))
    ts = t.shape
    ok = len(ts) == len(shape)
    if ok:
        for s, d in zip(shape, ts):     # a plain loop: this runs on every call of every entry point
            if s is not None and s != d:
                ok = False
                break
    if not ok:
        raise ValueError("%s has shape %s; expected %s" % (
            name, tuple(ts), tuple("*" if s is None else s for s in shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s; expected %s" % (
            name, t.dtype, " or ".join(str(d) for d in dtypes)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _same_device(**tensors):
    """All tensors on one CUDA device (checked after shapes and dtypes)."""
    first = None
    for n, t in tensors.items():
        if t is None:
            continue
        d = t.device
        if d.type != "cuda":
            raise ValueError("%s is on %s; every tensor must be on a CUDA device" % (n, d))
        if first is None:
            first = d
        elif d != first:
            raise ValueError("tensors are on different devices: %s" % (
                ", ".join("%s %s" % (m, u.device) for m, u in tensors.items() if u is not None)))


def check_layer_args(x, dt, A, B, C, D=None, init_state=None, y=None, final_state=None, workspace=None):
    """Shapes, dtypes, contiguity and device of one layer's tensors (ssd_chunk_scan_fwd):
    x [b, L, H, P], dt [b, L, H], B and C [b, L, G, N], all of one activation dtype
    (float32 or bfloat16), y like x; A and D [H] float32; init_state and final_state
    [b, H, P, N] float32; all contiguous and on one CUDA device."""
    _expect("x", x, (None, None, None, None), _ACT_DTYPES)
    b, L, H, P = x.shape
    _expect("B", B, (b, L, None, None), (x.dtype,))
    G, N = B.shape[2], B.shape[3]
    _expect("dt", dt, (b, L, H), (x.dtype,))
    _expect("C", C, (b, L, G, N), (x.dtype,))
    _expect("A", A, (H,), (torch.float32,))
    _expect("D", D, (H,), (torch.float32,), allow_none=True)
    _expect("init_state", init_state, (b, H, P, N), (torch.float32,), allow_none=True)
    _expect("y", y, (b, L, H, P), (x.dtype,), allow_none=True)
    _expect("final_state", final_state, (b, H, P, N), (torch.float32,), allow_none=True)
    _expect("workspace", workspace, (None,), (torch.uint8,), allow_none=True)
    _same_device(x=x, dt=dt, A=A, B=B, C=C, D=D, init_state=init_state, y=y,
                 final_state=final_state, workspace=workspace)


def check_stack_args(x0, dt, A, B, C, D, layer_states, y=None, workspace=None):
    """As check_layer_args for the stack (ssd_chunk_scan_segmented): A and D are
    [n_layers, H] float32 and layer_states [n_layers, b, H, P, N] float32."""
    _expect("x0", x0, (None, None, None, None), _ACT_DTYPES)
    b, L, H, P = x0.shape
    _expect("B", B, (b, L, None, None), (x0.dtype,))
    G, N = B.shape[2], B.shape[3]
    _expect("dt", dt, (b, L, H), (x0.dtype,))
    _expect("C", C, (b, L, G, N), (x0.dtype,))
    _expect("A", A, (None, H), (torch.float32,))
    nl = A.shape[0]
    _expect("D", D, (nl, H), (torch.float32,), allow_none=True)
    _expect("layer_states", layer_states, (nl, b, H, P, N), (torch.float32,))
    _expect("y", y, (b, L, H, P), (x0.dtype,), allow_none=True)
    _expect("workspace", workspace, (None,), (torch.uint8,), allow_none=True)
    _same_device(x0=x0, dt=dt, A=A, B=B, C=C, D=D, layer_states=layer_states, y=y,
                 workspace=workspace)


def check_step_args(x, dt, A, B, C, D, state, y=None):
    """As check_layer_args for one decode token (ssd_step): x [b, H, P], dt [b, H],
    B and C [b, G, N], A and D [H], state [b, H, P, N] float32."""
    _expect("x", x, (None, None, None), _ACT_DTYPES)
    b, H, P = x.shape
    _expect("B", B, (b, None, None), (x.dtype,))
    G, N = B.shape[1], B.shape[2]
    _expect("dt", dt, (b, H), (x.dtype,))
    _expect("C", C, (b, G, N), (x.dtype,))
    _expect("A", A, (H,), (torch.float32,))
    _expect("D", D, (H,), (torch.float32,), allow_none=True)
    _expect("state", state, (b, H, P, N), (torch.float32,))
    _expect("y", y, (b, H, P), (x.dtype,), allow_none=True)
    _same_device(x=x, dt=dt, A=A, B=B, C=C, D=D, state=state, y=y)


def dims_of(x, B, dtype=None):
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if dtype is None:
        dtype = SSD_BF16 if x.dtype == torch.bfloat16 else SSD_F32
    return Dims(b, L, H, P, N, G, dtype, 0)


def shape_supported(dtype, chunk, headdim, dstate) -> bool:
    return bool(lib().ssd_shape_supported(dtype, chunk, headdim, dstate))


def scan_form_supported(dtype, chunk, headdim, dstate) -> bool:
    return bool(lib().ssd_scan_form_supported(dtype, chunk, headdim, dstate))


def workspace_bytes(dims, chunk) -> int:
    return lib().ssd_chunk_scan_workspace_bytes(ctypes.byref(dims), chunk)


def segmented_workspace_bytes(dims, chunk, V, n_layers=1, wavefront=False) -> int:
    flags = SSD_FLAG_WAVEFRONT if wavefront else 0
    return lib().ssd_segmented_workspace_bytes(ctypes.byref(dims), chunk, V, n_layers, flags)


NSTAGES = 4   # chunk_cumsum, chunk_state, state_pass, chunk_scan


def workspace_layout(dims, chunk):
    offs = (ctypes.c_size_t * 4)()
    _check(lib().ssd_workspace_layout(ctypes.byref(dims), chunk, offs))
    return list(offs)


def alloc_workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def fwd(x, dt, A, B, C, D=None, init_state=None, chunk=256, *, y=None, final_state=None,
        residual=False, workspace=None, stream=None, want_final=True, first_stage=1, last_stage=NSTAGES,
        scan_form=False):
    """One layer over the whole sequence (ssd_chunk_scan_fwd).  Returns (y, final_state).
    scan_form=True computes the chunk outputs with the associative-scan kernel.

    The decay a_t = exp(dt A) must lie in [0, 1]: dt >= 0 and A <= 0 (the library's
    contract; other values give unspecified results).  Tensor shapes, dtypes, contiguity
    and device are checked here (ValueError), values are not."""
    lib()                  # fails loudly when the library is not built
    check_layer_args(x, dt, A, B, C, D, init_state, y, final_state, workspace)
    dims = dims_of(x, B)
    nbytes = workspace_bytes(dims, chunk)
    if nbytes == 0:
        _check(lib().ssd_chunk_scan_fwd(ctypes.byref(dims), None, None, None, None, None, None, None,
                                        chunk, None, None, 0, None, 0, None))
    if workspace is None:
        workspace = alloc_workspace(nbytes, x.device)
    given = (y, final_state)
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and want_final:
        final_state = torch.empty(x.shape[0], x.shape[2], x.shape[3], B.shape[3], dtype=torch.float32,
                                  device=x.device)
    flags = (SSD_FLAG_RESIDUAL if residual else 0) | (SSD_FLAG_SCAN_FORM if scan_form else 0)
    args = (ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state),
            chunk, _ptr(y), _ptr(final_state), flags, _ptr(workspace), workspace.numel(), _stream(stream))
    if first_stage == 1 and last_stage == NSTAGES:
        _check(lib().ssd_chunk_scan_fwd(*args))
    else:
        _check(lib().ssd_chunk_scan_stages(*args, first_stage, last_stage))
    _wrote(*given)
    return y, final_state


def fwd_noalloc(x, dt, A, B, C, D=None, init_state=None, chunk=256, *, y, final_state=None,
                residual=False, stream=None):
    """ssd_chunk_scan_fwd_noalloc: one layer with the library's own scratch as workspace
    (nothing is allocated; y and final_state are caller tensors).  The workspace this call
    needs (workspace_bytes) must not exceed NOALLOC_SCRATCH_BYTES.  Calls that overlap on
    one GPU share that scratch and must be serialised by the caller.  Returns (y, final_state)."""
    lib()                  # fails loudly when the library is not built
    check_layer_args(x, dt, A, B, C, D, init_state, y, final_state)
    dims = dims_of(x, B)
    flags = SSD_FLAG_RESIDUAL if residual else 0
    _check(lib().ssd_chunk_scan_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                            _ptr(D), _ptr(init_state), chunk, _ptr(y), _ptr(final_state),
                                            flags, _stream(stream)))
    _wrote(y, final_state)
    return y, final_state


def segmented(x0, dt, A, B, C, D, layer_states, V, chunk=256, *, y=None, residual=True,
              wavefront=True, workspace=None, stream=None):
    """Vertical layer stack (ssd_chunk_scan_segmented); layer_states is updated in place.
    wavefront=False runs the (segment, layer) steps strictly one at a time.  As for fwd,
    dt >= 0 and A <= 0."""
    lib()                  # fails loudly when the library is not built
    check_stack_args(x0, dt, A, B, C, D, layer_states, y, workspace)
    dims = dims_of(x0, B)
    n_layers = A.shape[0]
    nbytes = segmented_workspace_bytes(dims, chunk, V, n_layers, wavefront)
    if workspace is None:
        workspace = alloc_workspace(nbytes, x0.device)
    given = y
    if y is None:
        y = torch.empty_like(x0)
    flags = (SSD_FLAG_RESIDUAL if residual else 0) | (SSD_FLAG_WAVEFRONT if wavefront else 0)
    _check(lib().ssd_chunk_scan_segmented(ctypes.byref(dims), n_layers, V, _ptr(x0), _ptr(dt), _ptr(A),
                                          _ptr(B), _ptr(C), _ptr(D), _ptr(layer_states), chunk, flags,
                                          _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)))
    _wrote(given, layer_states)
    return y, layer_states


def horizontal(x0, dt, A, B, C, D, layer_states, chunk=256, *, residual=True, stream=None):
    """Layer-serial stack: ssd_chunk_scan_fwd once per layer over the whole sequence."""
    lib()                  # fails loudly when the library is not built
    check_stack_args(x0, dt, A, B, C, D, layer_states)
    u = x0
    dims = dims_of(x0, B)
    ws = alloc_workspace(workspace_bytes(dims, chunk), x0.device)
    bufs = [torch.empty_like(x0), torch.empty_like(x0)]
    for l in range(A.shape[0]):
        out = bufs[l % 2]
        fwd(u, dt, A[l], B, C, None if D is None else D[l], layer_states[l], chunk, y=out,
            final_state=layer_states[l], residual=residual, workspace=ws, stream=stream)
        u = out
    return u.clone(), layer_states


def step(x, dt, A, B, C, D, state, *, y=None, residual=False, stream=None):
    """One decode step (ssd_step): x [b, H, P], dt [b, H], B/C [b, G, N]; state [b, H, P, N]
    float32 is updated in place.  Returns y [b, H, P].  As for fwd, dt >= 0 and A <= 0."""
    lib()                  # fails loudly when the library is not built
    check_step_args(x, dt, A, B, C, D, state, y)
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dtype = SSD_BF16 if x.dtype == torch.bfloat16 else SSD_F32
    dims = Dims(b, 1, H, P, N, G, dtype, 0)
    given = y
    if y is None:
        y = torch.empty_like(x)
    flags = SSD_FLAG_RESIDUAL if residual else 0
    _check(lib().ssd_step(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                          _ptr(state), _ptr(y), flags, _stream(stream)))
    _move_on((state,) if given is None else (state, given))
    return y


def tile_order_to_pn(t, P, N):
    """Re-index states stored in the library's tile order ([..., P*N]) to [..., P, N].

    Tile (nt, pt), lane l, value r holds (p = 16 pt + l % 16, n = 16 nt + 4 (l // 16) + r).
    """
    lead = t.shape[:-1]
    v = t.reshape(*lead, N // 16, P // 16, 4, 16, 4)          # nt, pt, g, col, r
    nd = len(lead)
    perm = list(range(nd)) + [nd + 1, nd + 3, nd + 0, nd + 2, nd + 4]   # pt, col, nt, g, r
    return v.permute(*perm).reshape(*lead, P, N)


# ---------------------------------------------------------------- operators around a scan
# These take views (rows of contiguous channels at any batch and token stride) for their
# activation inputs, and run on the tensors' own device.  With `stream`, outputs and
# workspaces are allocated for that stream, so that the allocator reuses their memory in its
# order.

_DTYPE_CODE = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


def _param(name, t, shape, device, dtype=torch.float32):
    """A contiguous tensor of this shape and dtype on `device`, or None; its pointer."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError("%s has shape %s; expected %s" % (name, tuple(t.shape), shape))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s; expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s; expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(name, t, shape, dtype, device):
    """An activation view with contiguous channels.  Its pointer, batch stride and token stride
    (0 where the shape has no tokens)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor (got %s)" % (name, type(t).__name__))
    if t.shape != shape:
        raise ValueError("%s has shape %s; expected %s" % (name, tuple(t.shape), shape))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s; expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s; expected %s" % (name, t.device, device))
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s must have contiguous channels" % name)
    return t.data_ptr(), st[0], (st[1] if len(shape) == 3 else 0)


def _coef_rows(name, t, lead, dtype, device):
    """B or C [*lead, G, N]: as _rows, with [G, N] contiguous together."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor (got %s)" % (name, type(t).__name__))
    shape = t.shape
    if len(shape) != len(lead) + 2 or shape[:-2] != lead:
        raise ValueError("%s has shape %s; expected %s" % (name, tuple(shape), tuple(lead) + ("*", "*")))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s; expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s; expected %s" % (name, t.device, device))
    st = t.stride()
    if st[-1] != 1 or (st[-2] != shape[-1] and shape[-2] != 1):
        raise ValueError("%s must have contiguous groups of states" % name)
    return t.data_ptr(), st[0], (st[1] if len(lead) == 2 else 0)


def _activation(name, t, dim):
    """The tensor whose dtype, device and shape the others follow."""
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor (got %s)" % (name, type(t).__name__))
    if t.dim() != dim:
        raise ValueError("%s has shape %s; expected %d dimensions" % (name, tuple(t.shape), dim))
    if t.dtype not in _DTYPE_CODE:
        raise ValueError("%s has dtype %s; expected torch.float32 or torch.bfloat16" % (name, t.dtype))
    return _DTYPE_CODE[t.dtype]


def _elsewhere(t, stream):
    """The context in which a call on tensor t has to run, or None when it is the current one:
    the given stream's, or t's device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors are on %s; every tensor must be on a CUDA device" % t.device)
    if stream is not None:
        if stream.device != t.device:
            raise ValueError("the stream is on %s and the tensors are on %s" % (stream.device, t.device))
        return torch.cuda.stream(stream)
    return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _current(t):
    """The current stream of t's device as an integer.  (torch.cuda.current_stream builds a
    Stream object: 2.7 us, where a single-token kernel takes 3.)"""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _out(name, t, shape, dtype, device):
    """A caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _param(name, t, shape, device, dtype)
    return t


def _out_like(name, t, x):
    """The same for an output of x's shape and type (the quicker of torch's allocations where x
    is contiguous, whose layout it takes)."""
    if t is None and x.is_contiguous():
        return torch.empty_like(x)
    return _out(name, t, tuple(x.shape), x.dtype, x.device)


_NO_WORKSPACE = torch.empty(0, dtype=torch.uint8)


def _workspace(t, nbytes, device):
    """A caller's workspace or, where one is needed, a fresh one."""
    if t is None and nbytes == 0:
        return _NO_WORKSPACE
    if t is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != device:
        raise ValueError("workspace must be a contiguous torch.uint8 tensor on %s" % device)
    return t


def _taps(weight):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a torch.Tensor [channels, taps]")
    return weight.shape[1]


def conv_fwd(x, weight, bias=None, init_state=None, *, lengths=None, silu=True, y=None, final_state=None,
             want_final=True, stream=None):
    """Short causal convolution with an optional SiLU (ssd_conv_fwd): x [b, L, C], weight
    [C, W] and bias [C] float32, init_state [b, W-1, C] (the inputs before the first token),
    lengths [b] int32 (each row's own tokens).  Returns (y [b, L, C], final_state [b, W-1, C]);
    final_state may be init_state, which is then updated in place."""
    L_ = lib()
    code = _activation("x", x, 3)
    b, L, C = x.shape
    W = _taps(weight)
    dev = x.device
    xp, xb, xt = _rows("x", x, (b, L, C), x.dtype, dev)
    wp = _param("weight", weight, (C, W), dev)
    bp = _param("bias", bias, (C,), dev)
    ip = _param("init_state", init_state, (b, W - 1, C), dev, x.dtype)
    lp = _param("lengths", lengths, (b,), dev, torch.int32)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return conv_fwd(x, weight, bias, init_state, lengths=lengths, silu=silu, y=y, final_state=final_state,
                            want_final=want_final)
    given = (y, final_state)
    y = _out_like("y", y, x)
    if final_state is not None or (want_final and W > 1):
        final_state = _out("final_state", final_state, (b, W - 1, C), x.dtype, dev)
    dims = ConvDims(b, L, C, W, code, xb, xt, 0, 0)
    _check(L_.ssd_conv_fwd(dims, xp, wp, bp, ip, lp, y.data_ptr(), _ptr(final_state), SSD_FLAG_SILU if silu else 0,
                           _current(x)))
    _wrote(*given)
    return y, final_state


def conv_step(x, weight, bias, state, *, silu=True, y=None, state_out=None, stream=None):
    """One token of the convolution (ssd_conv_step): x [b, C], state [b, W-1, C], updated in
    place unless state_out is given.  Returns y [b, C]."""
    L_ = lib()
    code = _activation("x", x, 2)
    b, C = x.shape
    W = _taps(weight)
    dev, shape = x.device, (b, W - 1, C)
    xp, xb, _ = _rows("x", x, (b, C), x.dtype, dev)
    wp = _param("weight", weight, (C, W), dev)
    bp = _param("bias", bias, (C,), dev)
    ip = _param("state", state, shape, dev, x.dtype)
    op = ip if state_out is None else _param("state_out", state_out, shape, dev, x.dtype)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return conv_step(x, weight, bias, state, silu=silu, y=y, state_out=state_out)
    given = y
    y = _out_like("y", y, x)
    dims = ConvDims(b, 1, C, W, code, xb, 0, 0, 0)
    _check(L_.ssd_conv_step(dims, xp, wp, bp, ip, op, y.data_ptr(), SSD_FLAG_SILU if silu else 0, _current(x)))
    moved = state if state_out is None else state_out
    _move_on((moved,) if given is None else (moved, given))
    return y


class ConvGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]
    dinit: Optional[torch.Tensor]


def conv_bwd(dy, x, weight, bias=None, init_state=None, *, dfinal=None, lengths=None, silu=True, workspace=None,
             stream=None):
    """Gradients of conv_fwd (ssd_conv_bwd) from dy [b, L, C] and dfinal [b, W-1, C], the
    gradient of final_state.  dbias and dinit are None where the forward had no bias or
    init_state."""
    L_ = lib()
    code = _activation("x", x, 3)
    b, L, C = x.shape
    W = _taps(weight)
    dev, st = x.device, (b, W - 1, C)
    xp, xb, xt = _rows("x", x, (b, L, C), x.dtype, dev)
    gp, gb, gt = _rows("dy", dy, (b, L, C), x.dtype, dev)
    wp = _param("weight", weight, (C, W), dev)
    bp = _param("bias", bias, (C,), dev)
    ip = _param("init_state", init_state, st, dev, x.dtype)
    fp = _param("dfinal", dfinal, st, dev, x.dtype)
    lp = _param("lengths", lengths, (b,), dev, torch.int32)
    dims = ConvDims(b, L, C, W, code, xb, xt, gb, gt)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return conv_bwd(dy, x, weight, bias, init_state, dfinal=dfinal, lengths=lengths, silu=silu,
                            workspace=workspace)
    ws = _workspace(workspace, L_.ssd_conv_bwd_workspace_bytes(dims), dev)
    g = ConvGrads(torch.empty((b, L, C), dtype=x.dtype, device=dev),
                  torch.empty((C, W), dtype=torch.float32, device=dev),
                  None if bias is None else torch.empty((C,), dtype=torch.float32, device=dev),
                  None if init_state is None else torch.empty(st, dtype=x.dtype, device=dev))
    _check(L_.ssd_conv_bwd(dims, gp, xp, wp, bp, ip, fp, lp, _ptr(g.dx), _ptr(g.dweight), _ptr(g.dbias),
                           _ptr(g.dinit), SSD_FLAG_SILU if silu else 0, ws.data_ptr(), ws.numel(), _current(x)))
    return g


def _selective_inputs(u, delta, A, B, C, D, z, delta_bias, step, dy=None):
    """Checks of the selective scan's inputs; (dims, pointers in the C ABI's order up to
    delta_bias, pointer of dy)."""
    code = _activation("u", u, 2 if step else 3)
    shape, dtype, dev = tuple(u.shape), u.dtype, u.device
    lead, d = shape[:-1], shape[-1]
    up, ub, ut = _rows("u", u, shape, dtype, dev)
    ep, eb, et = _rows("delta", delta, shape, dtype, dev)
    Bp, Bb, Bt = _coef_rows("B", B, lead, dtype, dev)
    Cp, Cb, Ct = _coef_rows("C", C, lead, dtype, dev)
    G, N = B.shape[-2:]
    if C.shape[-2:] != (G, N):
        raise ValueError("C has shape %s; expected %s" % (tuple(C.shape), tuple(B.shape)))
    zp, zb, zt = _rows("z", z, shape, dtype, dev) if z is not None else (None, 0, 0)
    gp, gb, gt = _rows("dy", dy, shape, dtype, dev) if dy is not None else (None, 0, 0)
    ptrs = (up, ep, _param("A", A, (d, N), dev), Bp, Cp, _param("D", D, (d,), dev), zp,
            _param("delta_bias", delta_bias, (d,), dev))
    dims = SelectiveDims(lead[0], 1 if step else lead[1], d, N, G, code, 0, ub, ut, eb, et, zb, zt, Bb, Bt, Cb, Ct,
                         gb, gt)
    return dims, ptrs, gp


def selective_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, init_state=None, *, lengths=None,
                  softplus=True, y=None, final_state=None, keep=False, workspace=None, stream=None):
    """Selective scan with a decay for every channel and state (ssd_selective_fwd):
        dt = softplus(delta + delta_bias);  h = exp(dt A) h + dt u B;  y = (C.h + D u) silu(z)
    u, delta, z [b, L, D], A [D, N], B and C [b, L, G, N], D and delta_bias [D], init_state
    [b, D, N] float32, lengths [b] int32.  Returns (y, final_state), or with keep=True
    (y, final_state, kept), where kept is what selective_bwd needs.  final_state may be
    init_state, which is then updated in place.  Unlike fwd, the input term carries dt."""
    L_ = lib()
    dims, ptrs, _ = _selective_inputs(u, delta, A, B, C, D, z, delta_bias, False)
    b, L, d = u.shape
    dev, st = u.device, (b, d, B.shape[3])
    ip = _param("init_state", init_state, st, dev)
    lp = _param("lengths", lengths, (b,), dev, torch.int32)
    ctx = _elsewhere(u, stream)
    if ctx is not None:
        with ctx:
            return selective_fwd(u, delta, A, B, C, D, z, delta_bias, init_state, lengths=lengths, softplus=softplus,
                                 y=y, final_state=final_state, keep=keep, workspace=workspace)
    ws = _workspace(workspace, L_.ssd_selective_fwd_workspace_bytes(dims), dev)
    given = (y, final_state)
    y = _out_like("y", y, u)
    final_state = _out("final_state", final_state, st, torch.float32, dev)
    kept = torch.empty(L_.ssd_selective_kept_bytes(dims), dtype=torch.uint8, device=dev) if keep else None
    _check(L_.ssd_selective_fwd(dims, *ptrs, ip, lp, y.data_ptr(), final_state.data_ptr(), _ptr(kept),
                                SSD_FLAG_SOFTPLUS if softplus else 0, ws.data_ptr(), ws.numel(), _current(u)))
    _wrote(*given)
    return (y, final_state, kept) if keep else (y, final_state)


def selective_step(u, delta, A, B, C, D, z, delta_bias, state, *, softplus=True, y=None, state_out=None, stream=None):
    """One token of the selective scan (ssd_selective_step): u, delta, z [b, D], B and C
    [b, G, N], state [b, D, N] float32, updated in place unless state_out is given.
    Returns y [b, D]."""
    L_ = lib()
    dims, ptrs, _ = _selective_inputs(u, delta, A, B, C, D, z, delta_bias, True)
    b, d = u.shape
    dev, st = u.device, (b, d, B.shape[2])
    ip = _param("state", state, st, dev)
    op = ip if state_out is None else _param("state_out", state_out, st, dev)
    ctx = _elsewhere(u, stream)
    if ctx is not None:
        with ctx:
            return selective_step(u, delta, A, B, C, D, z, delta_bias, state, softplus=softplus, y=y,
                                  state_out=state_out)
    given = y
    y = _out_like("y", y, u)
    _check(L_.ssd_selective_step(dims, *ptrs, ip, op, y.data_ptr(), SSD_FLAG_SOFTPLUS if softplus else 0,
                                 _current(u)))
    moved = state if state_out is None else state_out
    _move_on((moved,) if given is None else (moved, given))
    return y


class SelectiveGrads(NamedTuple):
    du: torch.Tensor
    ddelta: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddelta_bias: Optional[torch.Tensor]
    dinit: torch.Tensor


def selective_bwd(dy, u, delta, A, B, C, D, z, delta_bias, kept, *, dfinal=None, lengths=None, softplus=True,
                  workspace=None, stream=None):
    """Gradients of selective_fwd (ssd_selective_bwd) from dy [b, L, D] and dfinal [b, D, N]
    (the gradient of final_state), with the kept states of a selective_fwd(keep=True) on the
    same arguments.  dD, dz and ddelta_bias are None where the forward had no such input."""
    L_ = lib()
    dims, ptrs, gp = _selective_inputs(u, delta, A, B, C, D, z, delta_bias, False, dy)
    b, L, d = u.shape
    G, N = B.shape[2:]
    dev = u.device
    fp = _param("dfinal", dfinal, (b, d, N), dev)
    lp = _param("lengths", lengths, (b,), dev, torch.int32)
    kp = _param("kept", kept, (L_.ssd_selective_kept_bytes(dims),), dev, torch.uint8)
    ctx = _elsewhere(u, stream)
    if ctx is not None:
        with ctx:
            return selective_bwd(dy, u, delta, A, B, C, D, z, delta_bias, kept, dfinal=dfinal, lengths=lengths,
                                 softplus=softplus, workspace=workspace)
    ws = _workspace(workspace, L_.ssd_selective_bwd_workspace_bytes(dims), dev)

    def act(*shape):
        return torch.empty(shape, dtype=u.dtype, device=dev)

    def f32(*shape):
        return torch.empty(shape, dtype=torch.float32, device=dev)
    g = SelectiveGrads(act(b, L, d), act(b, L, d), f32(d, N), act(b, L, G, N), act(b, L, G, N),
                       None if D is None else f32(d), None if z is None else act(b, L, d),
                       None if delta_bias is None else f32(d), f32(b, d, N))
    _check(L_.ssd_selective_bwd(dims, gp, *ptrs, kp, fp, lp, _ptr(g.du), _ptr(g.ddelta), _ptr(g.dA), _ptr(g.dB),
                                _ptr(g.dC), _ptr(g.dD), _ptr(g.dz), _ptr(g.ddelta_bias), _ptr(g.dinit),
                                SSD_FLAG_SOFTPLUS if softplus else 0, ws.data_ptr(), ws.numel(), _current(u)))
    return g


def norm_fwd(x, weight=None, bias=None, eps=1e-5, *, y=None, want_stats=False, stream=None):
    """Layer norm of the rows of x [rows, D] (ssd_norm_fwd), weight and bias [D] float32.
    Returns y, or (y, mean, rstd) with want_stats=True, which norm_bwd needs."""
    L_ = lib()
    code = _activation("x", x, 2)
    rows, d = x.shape
    dev = x.device
    xp, xs, _ = _rows("x", x, (rows, d), x.dtype, dev)
    wp = _param("weight", weight, (d,), dev)
    bp = _param("bias", bias, (d,), dev)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return norm_fwd(x, weight, bias, eps, y=y, want_stats=want_stats)
    given = y
    y = _out_like("y", y, x)
    mean = rstd = None
    if want_stats:
        mean = torch.empty((rows,), dtype=torch.float32, device=dev)
        rstd = torch.empty((rows,), dtype=torch.float32, device=dev)
    dims = NormDims(rows, d, code, 0, xs, 0)
    _check(L_.ssd_norm_fwd(dims, xp, wp, bp, eps, y.data_ptr(), _ptr(mean), _ptr(rstd), _current(x)))
    if given is not None:
        _wrote(given)
    return (y, mean, rstd) if want_stats else y


class NormGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: torch.Tensor


def norm_bwd(dy, x, weight, mean, rstd, *, workspace=None, stream=None):
    """Gradients of norm_fwd (ssd_norm_bwd) from dy [rows, D] and the forward's mean and rstd."""
    L_ = lib()
    code = _activation("x", x, 2)
    rows, d = x.shape
    dev = x.device
    xp, xs, _ = _rows("x", x, (rows, d), x.dtype, dev)
    gp, gs, _ = _rows("dy", dy, (rows, d), x.dtype, dev)
    wp = _param("weight", weight, (d,), dev)
    mp = _param("mean", mean, (rows,), dev)
    rp = _param("rstd", rstd, (rows,), dev)
    dims = NormDims(rows, d, code, 0, xs, gs)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return norm_bwd(dy, x, weight, mean, rstd, workspace=workspace)
    ws = _workspace(workspace, L_.ssd_norm_bwd_workspace_bytes(dims), dev)
    g = NormGrads(torch.empty((rows, d), dtype=x.dtype, device=dev),
                  torch.empty((d,), dtype=torch.float32, device=dev),
                  torch.empty((d,), dtype=torch.float32, device=dev))
    _check(L_.ssd_norm_bwd(dims, gp, xp, wp, mp, rp, _ptr(g.dx), _ptr(g.dweight), _ptr(g.dbias), ws.data_ptr(),
                           ws.numel(), _current(x)))
    return g
