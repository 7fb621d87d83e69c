"""ctypes binding of the gated linear recurrence (include/ssm_gated.h).

Argument marshalling only, as in binding.py: the argument structs are packed with struct (one call
instead of a ctypes object per field, which is most of the host time of a one-token step).  Calls
go to the tensors' own device, on its current stream unless another stream is given.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import binding
from .binding import SSM_BF16, SSM_F32, _check

# The layouts of ssm_gated_args_t, ssm_gated_grads_t, ssm_gated_step_t and ssm_gated_out_t.
_ARGS = struct.Struct("@Pqq Pqq Pqq Pqq PPP PPP q iiif")
_GRADS = struct.Struct("@Pqq P Pqq Pqq Pqq Pqq PPPP")
_STEP = struct.Struct("@Pq P PPPP P qqqqq PPP iiiif 4x")
_OUT = struct.Struct("@Pqq")


def declare(lib: ctypes.CDLL) -> None:
    """Declare the argument and result types of this header's entry points."""
    vp, ci, i64, sz, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_char_p
    lib.ssm_gated_checkpoint_size.argtypes = [ci, ci, i64]
    lib.ssm_gated_checkpoint_size.restype = sz
    lib.ssm_gated_bwd_workspace_size.argtypes = [ci, ci, i64, ci]
    lib.ssm_gated_bwd_workspace_size.restype = sz
    lib.ssm_gated_scan_fwd.argtypes = [st, st, vp, vp, sz, vp]
    lib.ssm_gated_scan_fwd.restype = ci
    lib.ssm_gated_scan_bwd.argtypes = [st, st, vp, sz, vp, sz, vp]
    lib.ssm_gated_scan_bwd.restype = ci
    lib.ssm_gated_state_update.argtypes = [st, vp]
    lib.ssm_gated_state_update.restype = ci


_IO = {torch.bfloat16: SSM_BF16, torch.float32: SSM_F32}

# The current stream's handle and the current device without building torch's objects for them, which
# takes longer than the rest of a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev, stream, fn, *args):
    """fn(*args, stream) with device `dev` (an index) current."""
    if stream is None:
        raw = _raw_stream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev == _current_device():
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def _lib():
    return binding._lib or binding.load()


@contextlib.contextmanager
def _allocating(tensor, stream):
    """Allocations inside belong to the tensor's device and to the stream that the call runs on, so that
    torch neither hands out memory still in use on it nor reuses theirs before it is done."""
    if not tensor.is_cuda:
        raise ValueError("x: not a CUDA tensor")
    with torch.cuda.device(tensor.device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=tensor.device)
        with torch.cuda.stream(stream):
            yield


def _dense(t, name, shape, dtypes, dev):
    """Address of an optional dense tensor on device `dev` (an index)."""
    if t is None:
        return 0
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype} (expected {' or '.join(str(d) for d in dtypes)})")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a dense tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    return t.data_ptr()


_F32 = (torch.float32,)
_I32 = (torch.int32,)
_FLAG = (torch.uint8, torch.bool)


def _like(t, name, x, dtype, shape, dev):
    """Address of an operand of x's type and shape."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {t.dtype} (x is {dtype})")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} (x has {tuple(shape)})")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    return t.data_ptr()


def _seq(t, name, x, dtype, shape, dev):
    """Address, batch stride and dim stride of a (batch, dim, seqlen) operand."""
    if t is None:
        return 0, 0, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _like(t, name, x, dtype, shape, dev)
    sb, sd, sl = t.stride()
    if sl != 1 and shape[2] > 1:
        raise ValueError(f"{name}: consecutive steps must be next to each other (stride {sl})")
    return t.data_ptr(), sb, sd


def _io(x, dims):
    """io_dtype, dtype, shape and device index of the leading operand."""
    dtype = x.dtype
    io = _IO.get(dtype)
    if io is None:
        raise TypeError(f"unsupported I/O dtype {dtype}")
    dev, shape = x.get_device(), x.shape
    if dev < 0:
        raise ValueError("x: not a CUDA tensor")
    if len(shape) != dims:
        raise ValueError(f"x: expected {'(batch, dim, seqlen)' if dims == 3 else '(batch, dim)'}, got {tuple(shape)}")
    return io, dtype, shape, dev


def _args(like, r, i, lam, r_bias, i_bias, z, initial_state, lengths, reset, c):
    x, dtype, shape, dev, io = like
    if lam is None:
        raise ValueError("lam is required")
    # (written out rather than through _seq: a small call's host time is mostly this)
    if r.dtype is not dtype or r.shape != shape or r.get_device() != dev:
        _like(r, "r", x, dtype, shape, dev)
    if i.dtype is not dtype or i.shape != shape or i.get_device() != dev:
        _like(i, "i", x, dtype, shape, dev)
    xb, xd, xl = x.stride()
    rb, rd, rl = r.stride()
    ib, id_, il = i.stride()
    b, d, L = shape
    if not xl == rl == il == 1 and L > 1:
        raise ValueError("x, r, i: consecutive steps must be next to each other (stride 1)")
    zp, zb, zd = _seq(z, "z", x, dtype, shape, dev)
    ch = (d,)
    return _ARGS.pack(x.data_ptr(), xb, xd, r.data_ptr(), rb, rd, i.data_ptr(), ib, id_, zp, zb, zd,
                      _dense(lam, "lam", ch, _F32, dev), _dense(r_bias, "r_bias", ch, _F32, dev),
                      _dense(i_bias, "i_bias", ch, _F32, dev), _dense(initial_state, "initial_state", (b, d), _F32, dev),
                      _dense(lengths, "lengths", (b,), _I32, dev), _dense(reset, "reset", (b, L), _FLAG, dev), L, b, d, io, c)


def _buffer(t, name, dev):
    """Address and bytes of an optional dense buffer."""
    if t is None:
        return 0, 0
    if not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: expected a dense tensor on cuda:{dev}")
    return t.data_ptr(), t.nbytes


def ssm_gated_checkpoint_size(batch: int, dim: int, seqlen: int) -> int:
    return int(_lib().ssm_gated_checkpoint_size(batch, dim, seqlen))


def ssm_gated_bwd_workspace_size(batch: int, dim: int, seqlen: int, have_checkpoints: bool = False) -> int:
    return int(_lib().ssm_gated_bwd_workspace_size(batch, dim, seqlen, int(bool(have_checkpoints))))


def new_gated_checkpoints(batch, dim, seqlen, device="cuda"):
    """Allocate (with torch) the checkpoints that a forward call stores for its backward."""
    return torch.empty(ssm_gated_checkpoint_size(batch, dim, seqlen), dtype=torch.uint8, device=device)


def new_gated_workspace(batch, dim, seqlen, have_checkpoints=False, device="cuda"):
    """Allocate (with torch) a workspace of the backward for these sizes."""
    return torch.empty(max(ssm_gated_bwd_workspace_size(batch, dim, seqlen, have_checkpoints), 256), dtype=torch.uint8,
                       device=device)


def ssm_gated_scan_fwd(x, r, i, lam, r_bias, i_bias, z, y, last_state, initial_state=None, lengths=None, reset=None,
                       checkpoints=None, c=8.0, stream=None, check=True):
    """Marshal a forward call.  x/r/i/z/y: (b, d, L), any batch and channel strides; lam/r_bias/i_bias: (d)
    fp32 (biases may be None); z may be None; last_state/initial_state: (b, d) fp32 or None; lengths: (b)
    int32 or None; reset: (b, L) uint8 or bool or None; checkpoints: from new_gated_checkpoints, or None."""
    io, dtype, shape, dev = _io(x, 3)
    args = _args((x, dtype, shape, dev, io), r, i, lam, r_bias, i_bias, z, initial_state, lengths, reset, c)
    if y is None:
        raise ValueError("y is required")
    code = _call(dev, stream, _lib().ssm_gated_scan_fwd, args, _OUT.pack(*_seq(y, "y", x, dtype, shape, dev)),
                 _dense(last_state, "last_state", shape[:2], _F32, dev), *_buffer(checkpoints, "checkpoints", dev))
    if check:
        _check(code, "ssm_gated_scan_fwd")
    return code


def ssm_gated_scan_bwd(x, r, i, lam, r_bias, i_bias, z, dy, dx, dr, di, dlam, dr_bias, di_bias, dz, workspace,
                       initial_state=None, dlast_state=None, dinitial_state=None, lengths=None, reset=None,
                       checkpoints=None, c=8.0, stream=None, check=True):
    """Marshal a backward call (shapes as the forward; dlam/dr_bias/di_bias (d) fp32 or None, dinitial_state
    (b, d) fp32 or None; dz required with z; checkpoints: the forward's, or None)."""
    io, dtype, shape, dev = _io(x, 3)
    like = (x, dtype, shape, dev)
    args = _args((*like, io), r, i, lam, r_bias, i_bias, z, initial_state, lengths, reset, c)
    ch, rows = (shape[1],), shape[:2]
    grads = _GRADS.pack(*_seq(dy, "dy", *like), _dense(dlast_state, "dlast_state", rows, _F32, dev), *_seq(dx, "dx", *like),
                        *_seq(dr, "dr", *like), *_seq(di, "di", *like), *_seq(dz, "dz", *like), _dense(dlam, "dlam", ch, _F32, dev),
                        _dense(dr_bias, "dr_bias", ch, _F32, dev), _dense(di_bias, "di_bias", ch, _F32, dev),
                        _dense(dinitial_state, "dinitial_state", rows, _F32, dev))
    code = _call(dev, stream, _lib().ssm_gated_scan_bwd, args, grads, *_buffer(checkpoints, "checkpoints", dev),
                 *_buffer(workspace, "workspace", dev))
    if check:
        _check(code, "ssm_gated_scan_bwd")
    return code


def ssm_gated_state_update(state, x, r, i, lam, r_bias, i_bias, z, y, slots=None, c=8.0, stream=None, check=True):
    """Marshal a one-token step.  state: (slots, d) fp32 in/out, rows of any stride; x/r/i/z/y: (b, d), rows of
    any stride; slots: (b) int32, the state of each row (outside the pool: the row is skipped), or None."""
    # (the checks are written out here: this call's host time is most of a small step)
    io, dtype, shape, dev = _io(x, 2)
    b, d = shape
    xs, xc = x.stride()
    if r.dtype is not dtype or r.shape != shape or r.get_device() != dev:
        _like(r, "r", x, dtype, shape, dev)
    rs, rc = r.stride()
    if i.dtype is not dtype or i.shape != shape or i.get_device() != dev:
        _like(i, "i", x, dtype, shape, dev)
    is_, ic = i.stride()
    if y.dtype is not dtype or y.shape != shape or y.get_device() != dev:
        _like(y, "y", x, dtype, shape, dev)
    ys, yc = y.stride()
    zp = zs = 0
    zc = 1
    if z is not None:
        zp = _like(z, "z", x, dtype, shape, dev)
        zs, zc = z.stride()
    if state.dtype is not torch.float32 or state.dim() != 2 or state.shape[1] != d or state.get_device() != dev:
        raise ValueError(f"state: expected (slots, {d}) torch.float32 on cuda:{dev}")
    ss, sc = state.stride()
    if not xc == rc == ic == zc == yc == sc == 1 and d > 1:
        raise ValueError("channels must be next to each other (stride 1) in x, r, i, z, y and state")
    if lam is None:
        raise ValueError("lam is required")
    ch = (d,)
    args = _STEP.pack(state.data_ptr(), ss, _dense(slots, "slots", (b,), _I32, dev), x.data_ptr(), r.data_ptr(), i.data_ptr(), zp,
                      y.data_ptr(), xs, rs, is_, zs, ys, _dense(lam, "lam", ch, _F32, dev),
                      _dense(r_bias, "r_bias", ch, _F32, dev), _dense(i_bias, "i_bias", ch, _F32, dev), b, d, state.shape[0], io, c)
    code = _call(dev, stream, _lib().ssm_gated_state_update, args)
    if check:
        _check(code, "ssm_gated_state_update")
    return code


def gated_scan_fwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, initial_state=None, lengths=None, reset=None,
                   return_last_state=True, checkpoints=None, c=8.0, stream=None):
    """Convenience wrapper: allocates y (x's dtype; zeros behind the rows' lengths) and last_state (fp32) and
    calls ssm_gated_scan_fwd.  Returns (y, last_state)."""
    with _allocating(x, stream):
        y = (torch.empty if lengths is None else torch.zeros)(x.shape, dtype=x.dtype, device=x.device)
        last = torch.empty(x.shape[:2], dtype=torch.float32, device=x.device) if return_last_state else None
        ssm_gated_scan_fwd(x, r, i, lam, r_bias, i_bias, z, y, last, initial_state=initial_state, lengths=lengths, reset=reset,
                           checkpoints=checkpoints, c=c, stream=stream)
    return y, last


def gated_scan_bwd(x, r, i, lam, r_bias=None, i_bias=None, z=None, dy=None, initial_state=None, dlast_state=None,
                   lengths=None, reset=None, checkpoints=None, workspace=None, c=8.0, stream=None):
    """Convenience wrapper: allocates every gradient and, if not given, a workspace, then calls
    ssm_gated_scan_bwd.  Returns a dict dx, dr, di, dz (or None), dlam, dr_bias, di_bias, dinitial_state."""
    b, d, L = x.shape
    f32 = dict(dtype=torch.float32, device=x.device)
    with _allocating(x, stream):
        out = {k: torch.empty(x.shape, dtype=x.dtype, device=x.device) for k in ("dx", "dr", "di")}
        out["dz"] = None if z is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        out.update({k: torch.empty(d, **f32) for k in ("dlam", "dr_bias", "di_bias")}, dinitial_state=torch.empty((b, d), **f32))
        if workspace is None:
            workspace = new_gated_workspace(b, d, L, checkpoints is not None, device=x.device)
        ssm_gated_scan_bwd(x, r, i, lam, r_bias, i_bias, z, dy, out["dx"], out["dr"], out["di"], out["dlam"], out["dr_bias"],
                           out["di_bias"], out["dz"], workspace, initial_state=initial_state, dlast_state=dlast_state,
                           dinitial_state=out["dinitial_state"], lengths=lengths, reset=reset, checkpoints=checkpoints, c=c,
                           stream=stream)
    return out
