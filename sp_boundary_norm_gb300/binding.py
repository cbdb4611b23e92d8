"""Thin Python binding of ``libspboundary.so`` (ctypes; marshalling only).

The functions carry the C entry points' names.  They take torch tensors for
device memory, check shapes, dtypes and devices (the C ABI trusts the sizes
it is given), and pass raw pointers and the current CUDA stream.  Every step
of the boundary runs in the library's CUDA kernels; there is no fallback: if
the library is not built, ``load()`` raises.
"""
import contextlib
import ctypes
import importlib.util
import os

import torch

from . import _build

SP_OK = 0
STATUS_NAMES = {0: "SP_OK", 1: "SP_ERR_INVALID_ARG", 2: "SP_ERR_MISALIGNED",
                3: "SP_ERR_UNSUPPORTED", 4: "SP_ERR_CUDA", 5: "SP_ERR_TIMEOUT",
                6: "SP_ERR_DEVICE_CHECK", 7: "SP_ERR_OVERLAP"}
NORMS = {"layernorm": 0, "rmsnorm": 1}
MAX_RANKS = 16

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_u64 = ctypes.c_uint64
_PP = ctypes.POINTER(ctypes.c_void_p)

_lib = None

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTS = {"none": 0, "silu": 1}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}
SCAN_RUN = 16               # tokens per saved state of the gated recurrence


class RopeTable(ctypes.Structure):
    """Frequencies of a head's rotated pairs, made by sp_rope_table."""
    _fields_ = [("pairs", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 256)]


class SpError(RuntimeError):
    def __init__(self, code, message):
        self.code = code
        self.name = STATUS_NAMES.get(code, str(code))
        super().__init__(f"{self.name}: {message}")


def load():
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    lib.sp_rs_norm_fwd.restype = _i32
    lib.sp_rs_norm_fwd.argtypes = [
        _PP, _PP, _vp, _vp, _vp, _i64, _i64, _i64, _i32, ctypes.c_float, ctypes.c_double,
        _u64, _u64, _vp, _i32, _i32, _PP, _PP, _PP, _PP, _PP, _i32, _vp, _vp]
    lib.sp_allgather_seq.restype = _i32
    lib.sp_allgather_seq.argtypes = [_PP, _i64, _i64, _i64, _i32, _vp, _i32, _PP, _i32, _vp, _vp]
    lib.sp_reduce_scatter_seq.restype = _i32
    lib.sp_reduce_scatter_seq.argtypes = [_PP, _i64, _i64, _i64, _i32, _vp, _i32, _PP, _vp, _vp]
    lib.sp_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.sp_norm_bwd_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32, _i32]
    lib.sp_norm_bwd.restype = _i32
    lib.sp_norm_bwd.argtypes = [
        _PP, _PP, _PP, _PP, _PP, _vp, _PP, _i64, _i64, _i64, _i32, ctypes.c_double, _vp, _i32,
        _i32, _PP, _PP, _i32, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
    lib.sp_shard_norm_fwd.restype = _i32
    lib.sp_shard_norm_fwd.argtypes = [
        _PP, _PP, _vp, _vp, _vp, _i64, _i64, _i64, _i32, ctypes.c_float, ctypes.c_double,
        _u64, _u64, _vp, _i32, _i32, _PP, _PP, _PP, _PP, _PP, _vp, _vp]
    lib.sp_rs_norm_bwd.restype = _i32
    lib.sp_rs_norm_bwd.argtypes = list(lib.sp_norm_bwd.argtypes)
    lib.sp_rs_norm_bwd_bitmask.restype = _i32
    lib.sp_rs_norm_bwd_bitmask.argtypes = list(lib.sp_norm_bwd.argtypes)
    lib.sp_norm_bwd_bitmask.restype = _i32
    lib.sp_norm_bwd_bitmask.argtypes = list(lib.sp_norm_bwd.argtypes)
    lib.sp_rs_norm_fwd_bitmask.restype = _i32
    lib.sp_rs_norm_fwd_bitmask.argtypes = list(lib.sp_rs_norm_fwd.argtypes)
    lib.sp_norm_bwd_philox.restype = _i32
    lib.sp_norm_bwd_philox.argtypes = [
        _PP, _PP, _PP, _PP, _vp, _PP, _i64, _i64, _i64, _i32, ctypes.c_double, _u64, _u64, _vp,
        _i32, _i32, _PP, _PP, _i32, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
    lib.sp_norm_bwd_noalloc.restype = _i32
    lib.sp_norm_bwd_noalloc.argtypes = [
        _PP, _PP, _PP, _PP, _PP, _vp, _PP, _i64, _i64, _i64, _i32, ctypes.c_double, _vp, _i32,
        _i32, _PP, _PP, _i32, _vp, _vp, _vp, _vp, _vp]
    tab = ctypes.POINTER(RopeTable)
    lib.sp_rope_table.restype = _i32
    lib.sp_rope_table.argtypes = [_i32, ctypes.c_double, _i32, ctypes.c_double, _i64,
                                  ctypes.c_double, ctypes.c_double, ctypes.c_double, tab]
    for fn in (lib.sp_rope_fwd, lib.sp_rope_bwd):
        fn.restype = _i32
        fn.argtypes = [_vp, _i64, _i64, _i64, _i64, _i64, _i64, _i32, _i32, tab, _i32, _vp, _i64,
                       _vp, _i32, _vp, _i64, _i64, _vp, _vp]
    lib.sp_gated_scan_fwd.restype = _i32
    lib.sp_gated_scan_fwd.argtypes = [
        _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _i64,
        _vp, _vp, _vp, _vp]
    lib.sp_gated_scan_bwd.restype = _i32
    lib.sp_gated_scan_bwd.argtypes = [
        _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp,
        _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp]
    lib.sp_group_norm_fwd.restype = _i32
    lib.sp_group_norm_fwd.argtypes = [
        _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _i32, ctypes.c_float, _i32, _i32, _vp,
        _i64, _vp, _vp, _vp]
    lib.sp_group_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.sp_group_norm_bwd_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32]
    lib.sp_group_norm_bwd.restype = _i32
    lib.sp_group_norm_bwd.argtypes = [
        _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _i32, _i32, _i32,
        _vp, _i64, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.sp_last_error.restype = ctypes.c_char_p
    lib.sp_last_error.argtypes = []
    lib.sp_abi_version.restype = _i32
    lib.sp_abi_version.argtypes = []
    lib.sp_debug_inject.restype = _i32
    lib.sp_debug_inject.argtypes = [_i32]
    lib.sp_debug_scan_withhold.restype = _i32
    lib.sp_debug_scan_withhold.argtypes = [_i32]
    lib.sp_debug_group_norm_shape.restype = _i32
    lib.sp_debug_group_norm_shape.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32, _i32,
                                              ctypes.POINTER(_i64)]
    lib.sp_debug_tune.restype = _i32
    lib.sp_debug_tune.argtypes = [_i32, _i32, _i32, _i32, _i32]
    lib.sp_debug_last_shape.restype = _i32
    lib.sp_debug_last_shape.argtypes = [_i32, _vp]
    lib.sp_debug_philox.restype = _i32
    lib.sp_debug_philox.argtypes = [_vp, _vp, _i64, _vp]
    _lib = lib
    return lib


def _check(code):
    if code != SP_OK:
        msg = load().sp_last_error()
        raise SpError(code, msg.decode() if msg else "")


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _ptr_array(ts):
    if ts is None:
        return None
    arr = (ctypes.c_void_p * max(1, len(ts)))()
    for i, x in enumerate(ts):
        arr[i] = x.data_ptr()
    return ctypes.cast(arr, _PP)


def _on_device(device):
    """The calls launch on the current CUDA device: make it the tensors' own."""
    return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(x, shape, dtype, device, what):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(x.shape)} != {tuple(shape)}")
    if x.dtype != dtype:
        raise ValueError(f"{what}: dtype {x.dtype} != {dtype}")
    if x.device != device:
        raise ValueError(f"{what}: on {x.device}, expected {device}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def shard_sizes(s, t):
    """Tokens per shard along s: o_k = floor(k*s/t)."""
    o = [(k * s) // t for k in range(t + 1)]
    return [o[k + 1] - o[k] for k in range(t)]


_status = {}


def device_status(device):
    """The binding's device status word for ``device`` (an int32 tensor); a
    bare "cuda" means the current CUDA device, as it does for tensors."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if device not in _status:
        _status[device] = torch.zeros(1, dtype=torch.int32, device=device)
    return _status[device]


def check_device_status(device, reset=True):
    """Raise SpError if a kernel flagged a device-side failure (synchronises)."""
    st = device_status(device)
    code = int(st.item())
    if reset:
        st.zero_()
    if code != SP_OK:
        raise SpError(code, "device-side check failed")


def _seq_meta(cu_seqlens, b, device):
    if cu_seqlens is None:
        return None, 0
    _need(cu_seqlens, (cu_seqlens.numel(),), torch.int32, device, "cu_seqlens")
    if b != 1:
        raise ValueError("cu_seqlens requires b == 1")
    return _ptr(cu_seqlens), cu_seqlens.numel() - 1


def sp_rs_norm_fwd(partials, residual, bias, gamma, beta, *, eps, p, seed, offset=0,
                   cu_seqlens=None, norm="layernorm", z_out, mask_out, mean_out, rstd_out,
                   gathered, status=None):
    """Fused g* + bias + dropout + residual + norm + g (writes the given outputs;
    mask_out=None stores no mask: the backward is then sp_norm_bwd_philox)."""
    _rs_norm_fwd_call("sp_rs_norm_fwd", 1, partials, residual, bias, gamma, beta, eps, p, seed,
                      offset, cu_seqlens, norm, z_out, mask_out, mean_out, rstd_out, gathered,
                      status)


def sp_rs_norm_fwd_bitmask(partials, residual, bias, gamma, beta, *, eps, p, seed, offset=0,
                           cu_seqlens=None, norm="layernorm", z_out, mask_bits_out, mean_out,
                           rstd_out, gathered, status=None):
    """sp_rs_norm_fwd storing the mask one bit per element
    (mask_bits_out[k]: (b, s_k, h / 8) uint8, bit e of byte j = channel 8j + e)."""
    if mask_bits_out is None:
        raise ValueError("mask_bits_out is required")
    _rs_norm_fwd_call("sp_rs_norm_fwd_bitmask", 8, partials, residual, bias, gamma, beta, eps,
                      p, seed, offset, cu_seqlens, norm, z_out, mask_bits_out, mean_out,
                      rstd_out, gathered, status)


def _rs_norm_fwd_call(entry, mask_div, partials, residual, bias, gamma, beta, eps, p, seed,
                      offset, cu_seqlens, norm, z_out, mask_out, mean_out, rstd_out, gathered,
                      status):
    lib = load()
    t = len(partials)
    if not 1 <= t <= MAX_RANKS:
        raise ValueError("1 <= t <= 16")
    b, s, h = partials[0].shape
    dev = partials[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    for r in range(t):
        _need(partials[r], (b, s, h), bf, dev, f"partials[{r}]")
    ln = norm == "layernorm"
    for k in range(t):
        _need(residual[k], (b, sizes[k], h), bf, dev, f"residual[{k}]")
        _need(z_out[k], (b, sizes[k], h), bf, dev, f"z_out[{k}]")
        if mask_out is not None:
            _need(mask_out[k], (b, sizes[k], h // mask_div), torch.uint8, dev, f"mask_out[{k}]")
        _need(rstd_out[k], (b, sizes[k]), torch.float32, dev, f"rstd_out[{k}]")
        if ln:
            _need(mean_out[k], (b, sizes[k]), torch.float32, dev, f"mean_out[{k}]")
    for j, g in enumerate(gathered):
        _need(g, (b, s, h), bf, dev, f"gathered[{j}]")
    for name, v in (("bias", bias), ("gamma", gamma)):
        _need(v, (h,), bf, dev, name)
    if ln:
        _need(beta, (h,), bf, dev, "beta")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        code = getattr(lib, entry)(
            _ptr_array(partials), _ptr_array(residual), _ptr(bias), _ptr(gamma),
            _ptr(beta) if ln else None, b, s, h, t, float(eps), float(p), int(seed), int(offset),
            cu, n_seqs, NORMS[norm], _ptr_array(z_out), _ptr_array(mask_out),
            _ptr_array(mean_out) if ln else None, _ptr_array(rstd_out), _ptr_array(gathered),
            len(gathered), _ptr(st), _stream(dev))
    _check(code)


def sp_shard_norm_fwd(y_shards, residual, bias, gamma, beta, *, s, eps, p, seed, offset=0,
                      cu_seqlens=None, norm="layernorm", z_out, mask_out, mean_out, rstd_out,
                      o_shards, status=None):
    """Unfused middle step: bias + dropout + residual + norm on reduced shards
    (mask_out=None: no mask stored, as for sp_rs_norm_fwd)."""
    lib = load()
    t = len(y_shards)
    b, _, h = y_shards[0].shape
    dev = y_shards[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    ln = norm == "layernorm"
    for k in range(t):
        for name, x in (("y_shards", y_shards), ("residual", residual), ("z_out", z_out),
                        ("o_shards", o_shards)):
            _need(x[k], (b, sizes[k], h), bf, dev, f"{name}[{k}]")
        if mask_out is not None:
            _need(mask_out[k], (b, sizes[k], h), torch.uint8, dev, f"mask_out[{k}]")
        _need(rstd_out[k], (b, sizes[k]), torch.float32, dev, f"rstd_out[{k}]")
        if ln:
            _need(mean_out[k], (b, sizes[k]), torch.float32, dev, f"mean_out[{k}]")
    for name, v in (("bias", bias), ("gamma", gamma)):
        _need(v, (h,), bf, dev, name)
    if ln:
        _need(beta, (h,), bf, dev, "beta")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        _check(lib.sp_shard_norm_fwd(
            _ptr_array(y_shards), _ptr_array(residual), _ptr(bias), _ptr(gamma),
            _ptr(beta) if ln else None, b, s, h, t, float(eps), float(p), int(seed), int(offset),
            cu, n_seqs, NORMS[norm], _ptr_array(z_out), _ptr_array(mask_out),
            _ptr_array(mean_out) if ln else None, _ptr_array(rstd_out), _ptr_array(o_shards),
            _ptr(st), _stream(dev)))


def sp_allgather_seq(shards, gathered, *, s, cu_seqlens=None, status=None):
    """g alone: gathered[j][:, o_k:o_{k+1}, :] = shards[k] for every j."""
    lib = load()
    t = len(shards)
    b, _, h = shards[0].shape
    dev = shards[0].device
    sizes = shard_sizes(s, t)
    for k in range(t):
        _need(shards[k], (b, sizes[k], h), torch.bfloat16, dev, f"shards[{k}]")
    for j, g in enumerate(gathered):
        _need(g, (b, s, h), torch.bfloat16, dev, f"gathered[{j}]")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        _check(lib.sp_allgather_seq(_ptr_array(shards), b, s, h, t, cu, n_seqs,
                                    _ptr_array(gathered), len(gathered), _ptr(st), _stream(dev)))


def sp_reduce_scatter_seq(partials, shards, *, cu_seqlens=None, status=None):
    """g* alone: shards[k] = bf16(sum_r partials[r][:, o_k:o_{k+1}, :])."""
    lib = load()
    t = len(partials)
    b, s, h = partials[0].shape
    dev = partials[0].device
    sizes = shard_sizes(s, t)
    for r in range(t):
        _need(partials[r], (b, s, h), torch.bfloat16, dev, f"partials[{r}]")
        _need(shards[r], (b, sizes[r], h), torch.bfloat16, dev, f"shards[{r}]")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        _check(lib.sp_reduce_scatter_seq(_ptr_array(partials), b, s, h, t, cu, n_seqs,
                                         _ptr_array(shards), _ptr(st), _stream(dev)))


def sp_norm_bwd_workspace_bytes(b, s, h, t, norm="layernorm"):
    return int(load().sp_norm_bwd_workspace_bytes(b, s, h, t, NORMS[norm]))


def sp_norm_bwd(dy, z, mask, mean, rstd, gamma, dz_skip=None, *, s, p, cu_seqlens=None,
                norm="layernorm", dresidual, dgathered, dgamma=None, dbeta=None, dbias=None,
                workspace, status=None):
    """Backward of the boundary (writes the given outputs)."""
    _norm_bwd_call("sp_norm_bwd", 1, dy, z, mask, mean, rstd, gamma, dz_skip, s, p,
                   cu_seqlens, norm, dresidual, dgathered, dgamma, dbeta, dbias, workspace,
                   status)


def sp_norm_bwd_bitmask(dy, z, mask_bits, mean, rstd, gamma, dz_skip=None, *, s, p,
                        cu_seqlens=None, norm="layernorm", dresidual, dgathered, dgamma=None,
                        dbeta=None, dbias=None, workspace, status=None):
    """sp_norm_bwd reading the mask stored one bit per element
    (mask_bits[k]: (b, s_k, h / 8) uint8, bit e of byte j = channel 8j + e)."""
    _norm_bwd_call("sp_norm_bwd_bitmask", 8, dy, z, mask_bits, mean, rstd, gamma, dz_skip, s,
                   p, cu_seqlens, norm, dresidual, dgathered, dgamma, dbeta, dbias, workspace,
                   status)


def _norm_bwd_call(entry, mask_div, dy, z, mask, mean, rstd, gamma, dz_skip, s, p, cu_seqlens,
                   norm, dresidual, dgathered, dgamma, dbeta, dbias, workspace, status):
    lib = load()
    t = len(dy)
    b, _, h = dy[0].shape
    dev = dy[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    ln = norm == "layernorm"
    for k in range(t):
        _need(dy[k], (b, sizes[k], h), bf, dev, f"dy[{k}]")
        _need(z[k], (b, sizes[k], h), bf, dev, f"z[{k}]")
        _need(mask[k], (b, sizes[k], h // mask_div), torch.uint8, dev, f"mask[{k}]")
        _need(rstd[k], (b, sizes[k]), torch.float32, dev, f"rstd[{k}]")
        if ln:
            _need(mean[k], (b, sizes[k]), torch.float32, dev, f"mean[{k}]")
        if dz_skip is not None:
            _need(dz_skip[k], (b, sizes[k], h), bf, dev, f"dz_skip[{k}]")
        _need(dresidual[k], (b, sizes[k], h), bf, dev, f"dresidual[{k}]")
    for j, g in enumerate(dgathered):
        _need(g, (b, s, h), bf, dev, f"dgathered[{j}]")
    _need(gamma, (h,), bf, dev, "gamma")
    for name, v in (("dgamma", dgamma), ("dbeta", dbeta), ("dbias", dbias)):
        if v is not None:
            _need(v, (h,), torch.float32, dev, name)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        code = getattr(lib, entry)(
            _ptr_array(dy), _ptr_array(z), _ptr_array(mask), _ptr_array(mean) if ln else None,
            _ptr_array(rstd), _ptr(gamma), _ptr_array(dz_skip), b, s, h, t, float(p), cu, n_seqs,
            NORMS[norm], _ptr_array(dresidual), _ptr_array(dgathered), len(dgathered),
            _ptr(dgamma), _ptr(dbeta) if ln else None, _ptr(dbias), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(st), _stream(dev))
    _check(code)


def sp_rs_norm_bwd(dy_partials, z, mask, mean, rstd, gamma, dz_skip=None, *, p,
                   cu_seqlens=None, norm="layernorm", dresidual, dgathered, dgamma=None,
                   dbeta=None, dbias=None, workspace, status=None):
    """Backward entered through g: reduce-scatter of the t partial gradients of
    the gathered input, fused into the norm / dropout backward."""
    _rs_norm_bwd_call("sp_rs_norm_bwd", 1, dy_partials, z, mask, mean, rstd, gamma, dz_skip, p,
                      cu_seqlens, norm, dresidual, dgathered, dgamma, dbeta, dbias, workspace,
                      status)


def sp_rs_norm_bwd_bitmask(dy_partials, z, mask_bits, mean, rstd, gamma, dz_skip=None, *, p,
                           cu_seqlens=None, norm="layernorm", dresidual, dgathered,
                           dgamma=None, dbeta=None, dbias=None, workspace, status=None):
    """sp_rs_norm_bwd reading the mask stored one bit per element
    (mask_bits[k]: (b, s_k, h / 8) uint8, bit e of byte j = channel 8j + e)."""
    _rs_norm_bwd_call("sp_rs_norm_bwd_bitmask", 8, dy_partials, z, mask_bits, mean, rstd, gamma,
                      dz_skip, p, cu_seqlens, norm, dresidual, dgathered, dgamma, dbeta, dbias,
                      workspace, status)


def _rs_norm_bwd_call(entry, mask_div, dy_partials, z, mask, mean, rstd, gamma, dz_skip, p,
                      cu_seqlens, norm, dresidual, dgathered, dgamma, dbeta, dbias, workspace,
                      status):
    lib = load()
    t = len(dy_partials)
    b, s, h = dy_partials[0].shape
    dev = dy_partials[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    ln = norm == "layernorm"
    for r in range(t):
        _need(dy_partials[r], (b, s, h), bf, dev, f"dy_partials[{r}]")
    for k in range(t):
        _need(z[k], (b, sizes[k], h), bf, dev, f"z[{k}]")
        _need(mask[k], (b, sizes[k], h // mask_div), torch.uint8, dev, f"mask[{k}]")
        _need(rstd[k], (b, sizes[k]), torch.float32, dev, f"rstd[{k}]")
        if ln:
            _need(mean[k], (b, sizes[k]), torch.float32, dev, f"mean[{k}]")
        if dz_skip is not None:
            _need(dz_skip[k], (b, sizes[k], h), bf, dev, f"dz_skip[{k}]")
        _need(dresidual[k], (b, sizes[k], h), bf, dev, f"dresidual[{k}]")
    for j, g in enumerate(dgathered):
        _need(g, (b, s, h), bf, dev, f"dgathered[{j}]")
    _need(gamma, (h,), bf, dev, "gamma")
    for name, v in (("dgamma", dgamma), ("dbeta", dbeta), ("dbias", dbias)):
        if v is not None:
            _need(v, (h,), torch.float32, dev, name)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        _check(getattr(lib, entry)(
            _ptr_array(dy_partials), _ptr_array(z), _ptr_array(mask),
            _ptr_array(mean) if ln else None, _ptr_array(rstd), _ptr(gamma), _ptr_array(dz_skip),
            b, s, h, t, float(p), cu, n_seqs, NORMS[norm], _ptr_array(dresidual),
            _ptr_array(dgathered), len(dgathered), _ptr(dgamma), _ptr(dbeta) if ln else None,
            _ptr(dbias), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(st),
            _stream(dev)))


def sp_norm_bwd_philox(dy, z, mean, rstd, gamma, dz_skip=None, *, s, p, seed, offset=0,
                       cu_seqlens=None, norm="layernorm", dresidual, dgathered, dgamma=None,
                       dbeta=None, dbias=None, workspace, status=None):
    """Mask-free backward: the dropout mask is drawn again from (seed, offset, p)."""
    lib = load()
    t = len(dy)
    b, _, h = dy[0].shape
    dev = dy[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    ln = norm == "layernorm"
    for k in range(t):
        _need(dy[k], (b, sizes[k], h), bf, dev, f"dy[{k}]")
        _need(z[k], (b, sizes[k], h), bf, dev, f"z[{k}]")
        _need(rstd[k], (b, sizes[k]), torch.float32, dev, f"rstd[{k}]")
        if ln:
            _need(mean[k], (b, sizes[k]), torch.float32, dev, f"mean[{k}]")
        if dz_skip is not None:
            _need(dz_skip[k], (b, sizes[k], h), bf, dev, f"dz_skip[{k}]")
        _need(dresidual[k], (b, sizes[k], h), bf, dev, f"dresidual[{k}]")
    for j, g in enumerate(dgathered):
        _need(g, (b, s, h), bf, dev, f"dgathered[{j}]")
    _need(gamma, (h,), bf, dev, "gamma")
    for name, v in (("dgamma", dgamma), ("dbeta", dbeta), ("dbias", dbias)):
        if v is not None:
            _need(v, (h,), torch.float32, dev, name)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        _check(lib.sp_norm_bwd_philox(
            _ptr_array(dy), _ptr_array(z), _ptr_array(mean) if ln else None, _ptr_array(rstd),
            _ptr(gamma), _ptr_array(dz_skip), b, s, h, t, float(p), int(seed), int(offset), cu,
            n_seqs, NORMS[norm], _ptr_array(dresidual), _ptr_array(dgathered), len(dgathered),
            _ptr(dgamma), _ptr(dbeta) if ln else None, _ptr(dbias), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(st), _stream(dev)))


NOALLOC_WORKSPACE_BYTES = 16 << 20


def sp_norm_bwd_noalloc(dy, z, mask, mean, rstd, gamma, dz_skip=None, *, s, p, cu_seqlens=None,
                        norm="layernorm", dresidual, dgathered, dgamma=None, dbeta=None,
                        dbias=None, status=None):
    """sp_norm_bwd for callers that cannot allocate: no workspace argument.

    The library keeps the parameter-gradient partials in a fixed array of its
    own device memory (16 MiB per GPU, for the life of the process), so a
    caller that has no allocator to draw scratch from can still run the
    backward.  Calls on one device share that array: do not let two of them
    run concurrently on different streams.  The first call on a device looks
    up the array's address; make it before any stream capture.
    """
    lib = load()
    t = len(dy)
    b, _, h = dy[0].shape
    dev = dy[0].device
    bf = torch.bfloat16
    sizes = shard_sizes(s, t)
    ln = norm == "layernorm"
    for k in range(t):
        _need(dy[k], (b, sizes[k], h), bf, dev, f"dy[{k}]")
        _need(z[k], (b, sizes[k], h), bf, dev, f"z[{k}]")
        _need(mask[k], (b, sizes[k], h), torch.uint8, dev, f"mask[{k}]")
        _need(rstd[k], (b, sizes[k]), torch.float32, dev, f"rstd[{k}]")
        if ln:
            _need(mean[k], (b, sizes[k]), torch.float32, dev, f"mean[{k}]")
        if dz_skip is not None:
            _need(dz_skip[k], (b, sizes[k], h), bf, dev, f"dz_skip[{k}]")
        _need(dresidual[k], (b, sizes[k], h), bf, dev, f"dresidual[{k}]")
    for j, g in enumerate(dgathered):
        _need(g, (b, s, h), bf, dev, f"dgathered[{j}]")
    _need(gamma, (h,), bf, dev, "gamma")
    for name, v in (("dgamma", dgamma), ("dbeta", dbeta), ("dbias", dbias)):
        if v is not None:
            _need(v, (h,), torch.float32, dev, name)
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = device_status(dev) if status is None else status
    with _on_device(dev):
        code = lib.sp_norm_bwd_noalloc(
            _ptr_array(dy), _ptr_array(z), _ptr_array(mask), _ptr_array(mean) if ln else None,
            _ptr_array(rstd), _ptr(gamma), _ptr_array(dz_skip), b, s, h, t, float(p), cu, n_seqs,
            NORMS[norm], _ptr_array(dresidual), _ptr_array(dgathered), len(dgathered),
            _ptr(dgamma), _ptr(dbeta) if ln else None, _ptr(dbias), _ptr(st), _stream(dev))
    _check(code)


# ------------------------------------------------ between g and the next g* --
# Tensors there are lists of t rank buffers of one shape.  Rows may be slices
# of a wider buffer: the last dimension is contiguous, and the leading ones
# follow each other with one stride between rows, the same for every rank.

def _dense(shape, strides):
    """Whether strides are those of a contiguous tensor."""
    step = 1
    for n, stride in zip(reversed(shape), reversed(strides)):
        if n != 1 and stride != step:
            return 0 in shape
        step *= n
    return True


def _row_stride(shape, strides, what):
    """Elements between the rows (every dimension but the last)."""
    if _dense(shape, strides):
        return shape[-1]
    if shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    ld, span = None, 1
    for n, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != ld * span:
            raise ValueError(f"{what}: rows of strides {tuple(strides)} do not follow each other "
                             "evenly")
        span *= n
    return shape[-1] if ld is None else ld


_module = None


def _quick():
    """The compiled short way: calls an entry point whose arguments are exactly right
    (its status), or gives None."""
    global _module
    if _module is None:
        lib = load()
        if not os.path.exists(_build.MODULE_PATH):
            raise RuntimeError(f"{_build.MODULE_PATH} is missing: build the library first")
        spec = importlib.util.spec_from_file_location("_sptensors", _build.MODULE_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        if hasattr(torch._C, "_cuda_getCurrentRawStream"):
            entries = (lib.sp_rope_fwd, lib.sp_rope_bwd, lib.sp_gated_scan_fwd,
                       lib.sp_gated_scan_bwd, lib.sp_group_norm_fwd, lib.sp_group_norm_bwd)
            module.setup(tuple(ctypes.cast(e, _vp).value for e in entries),
                         torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        _module = module
    return _module


def _pointers(xs):
    return (_vp * len(xs))(*[x.data_ptr() for x in xs])


def _rank_buffers(xs, x0, t, what):
    """Checks that xs are t buffers of x0's shape, type and device, one by one."""
    if len(xs) != t:
        raise ValueError(f"{what}: {len(xs)} ranks, expected {t}")
    for i, x in enumerate(xs):
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{what}[{i}] must be a torch.Tensor")
        if x.shape != x0.shape:
            raise ValueError(f"{what}[{i}]: shape {tuple(x.shape)} != {tuple(x0.shape)}")
        if x.dtype is not x0.dtype:
            raise ValueError(f"{what}[{i}]: dtype {x.dtype} != {x0.dtype}")
        if x.device != x0.device:
            raise ValueError(f"{what}[{i}]: on {x.device}, expected {x0.device}")


def _rank_rows(x0, t, **lists):
    """Pointer array and row stride of each list of t rank buffers, which are of x0's
    shape, type and device."""
    out = []
    for what, xs in lists.items():
        _rank_buffers(xs, x0, t, what)
        lds = [_row_stride(x.shape, x.stride(), what) for x in xs]
        if any(ld != lds[0] for ld in lds):
            raise ValueError(f"{what}: every rank needs the same row stride")
        out += [_pointers(xs), lds[0]]
    return out


def _rank_floats(x0, t, shape, **lists):
    """Pointer array of each list of t dense float32 rank buffers (None: no array)."""
    out = []
    for what, xs in lists.items():
        if xs is None:
            out.append(None)
            continue
        if len(xs) != t:
            raise ValueError(f"{what}: {len(xs)} ranks, expected {t}")
        for i, x in enumerate(xs):
            _need(x, shape, torch.float32, x0.device, f"{what}[{i}]")
        out.append(_pointers(xs))
    return out


def _params(x0, n, **vectors):
    """Address of each contiguous vector of n elements of x0's type (None: none)."""
    for what, v in vectors.items():
        if v is not None:
            _need(v, (n,), x0.dtype, x0.device, what)
    return [_ptr(v) for v in vectors.values()]


def _first(xs, dims, what):
    """Ranks, dtype code and device of a list of rank buffers."""
    t = len(xs)
    if not 1 <= t <= MAX_RANKS:
        raise ValueError("1 <= t <= 16")
    x = xs[0]
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what}[0] must be a torch.Tensor")
    if x.dim() != dims:
        raise ValueError(f"{what}[0]: {x.dim()} dimensions, expected {dims}")
    if x.dtype not in DTYPES:
        raise ValueError(f"{what}[0]: dtype {x.dtype} is not bfloat16, float16 or float32")
    return t, x, DTYPES[x.dtype]


def _status_word(dev, status):
    """Address of the caller's status word, or of the binding's own of the device."""
    if status is not None:
        if status.device != dev or status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError(f"status must be an int32 tensor on {dev}")
        return status.data_ptr()
    st = device_status(dev)
    if dev.type == "cuda":
        _quick().status(dev.index, st.data_ptr())     # the short way knows it from now on
    return st.data_ptr()


def _call(dev, fn, *args):
    """The call on the tensors' device and its current stream (the last argument)."""
    if dev.type != "cuda":
        raise ValueError(f"tensors on {dev}: the kernels need a CUDA device")
    stream = torch._C._cuda_getCurrentRawStream(dev.index)   # the current stream's handle
    if torch._C._cuda_getDevice() == dev.index:
        _check(fn(*args, stream))
    else:
        with _on_device(dev):
            _check(fn(*args, stream))


def _choice(table, key, what):
    if key not in table:
        raise ValueError(f"{what}: {key!r} is not one of {sorted(table)}")
    return table[key]


def sp_rope_table(rot_dim, *, base=10000.0, scaling="none", factor=1.0, original_len=0,
                  low_turns=1.0, high_turns=32.0, mscale=1.0):
    """Frequencies of rotary positions for heads of which rot_dim elements turn
    (kept by the caller, one per model).  scaling: "none", "linear" (positions
    divided by factor), "base" (base * factor^(rot_dim / (rot_dim - 2))) or
    "parts" (pairs that turn at most low_turns times over original_len positions
    are slowed by factor, those of high_turns or more are not, linear between);
    mscale multiplies cosine and sine."""
    out = RopeTable()
    _check(load().sp_rope_table(int(rot_dim), float(base),
                                _choice(ROPE_SCALINGS, scaling, "scaling"), float(factor),
                                int(original_len), float(low_turns), float(high_turns),
                                float(mscale), ctypes.byref(out)))
    return out


def _head_strides(x, what):
    """Token stride and head stride of a (b, s, heads, d) buffer."""
    b, s, heads, d = x.shape
    if _dense(x.shape, x.stride()):
        return heads * d, d
    s0, s1, s2, s3 = x.stride()
    if d > 1 and s3 != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if heads == 1:
        s2 = d
    if s > 1:
        if b > 1 and s0 != s * s1:
            raise ValueError(f"{what}: batch rows must follow each other")
        return s1, s2
    return (s0 if b > 1 else max(s1, heads * s2)), s2


def _rank_heads(x0, t, **lists):
    """Pointer array, token stride and head stride of each list of t (b, s, heads, d)
    rank buffers, which are of x0's shape, type and device."""
    out = []
    for what, xs in lists.items():
        _rank_buffers(xs, x0, t, what)
        strides = [_head_strides(x, what) for x in xs]
        if any(st != strides[0] for st in strides):
            raise ValueError(f"{what}: every rank needs the same strides")
        out += [_pointers(xs), *strides[0]]
    return out


def _rope_call(entry, x, table, layout, positions, first_position, cu_seqlens, y, status):
    if type(table) is RopeTable:
        code = _quick().rope(entry == "sp_rope_bwd", x, ctypes.addressof(table),
                             ROPE_LAYOUTS.get(layout), positions, first_position, cu_seqlens, y,
                             status)
        if code is not None:
            return _check(code)
    lib = load()
    t, x0, dt = _first(x, 4, "x")
    b, s, heads, d = x0.shape
    dev = x0.device
    if not isinstance(table, RopeTable):
        raise TypeError("table must come from sp_rope_table")
    xa, x_ld, x_head, ya, y_ld, y_head = _rank_heads(x0, t, x=x, y=y)
    if positions is not None:
        _need(positions, (b, s), torch.int64, dev, "positions")
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    st = _status_word(dev, status)
    _call(dev, getattr(lib, entry), xa, x_ld, x_head, b, s, heads, d, t, dt, ctypes.byref(table),
          _choice(ROPE_LAYOUTS, layout, "layout"), _ptr(positions), int(first_position), cu,
          n_seqs, ya, y_ld, y_head, st)


def sp_rope_fwd(x, table, *, layout="half", positions=None, first_position=0, cu_seqlens=None, y,
                status=None):
    """Rotary positions: turns the pairs of every head of the (b, s, heads, d) rank
    buffers x into y (y may be x: in place).  A token's heads may lie apart, and tokens
    too, but heads between tokens: the stride from token to token spans a token's heads
    (a heads-first tensor seen as (b, s, heads, d) is refused), and batch rows follow
    each other.  A token's position: positions (int64 (b, s)), else first_position plus its
    index in its batch row, or with cu_seqlens in its packed sequence."""
    _rope_call("sp_rope_fwd", x, table, layout, positions, first_position, cu_seqlens, y, status)


def sp_rope_bwd(dy, table, *, layout="half", positions=None, first_position=0, cu_seqlens=None,
                dx, status=None):
    """Gradient of sp_rope_fwd (dx may be dy)."""
    _rope_call("sp_rope_bwd", dy, table, layout, positions, first_position, cu_seqlens, dx, status)


def sp_gated_scan_states_shape(b, s, c):
    """Shape of one rank's float32 states buffer of sp_gated_scan_fwd."""
    return (b, (s + SCAN_RUN - 1) // SCAN_RUN, c)


def sp_gated_scan_fwd(gate, value, *, h0=None, tied=True, cu_seqlens=None, y, hT=None, states=None,
                      status=None):
    """Gated linear recurrence along s of (b, s, c) rank buffers:
    h = sigmoid(gate) h + (sigmoid(-gate) value if tied else value), y = h.
    h0, hT: float32 (sequences, c) states before and after each sequence (hT may be
    h0); states: sp_gated_scan_states_shape buffers that sp_gated_scan_bwd needs."""
    code = _quick().scan_fwd(gate, value, h0, tied, cu_seqlens, y, hT, states, status)
    if code is not None:
        return _check(code)
    lib = load()
    t, x0, dt = _first(gate, 3, "gate")
    b, s, c = x0.shape
    dev = x0.device
    ga, g_ld, va, v_ld, ya, y_ld = _rank_rows(x0, t, gate=gate, value=value, y=y)
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    n = b if cu is None else n_seqs
    ha, ta = _rank_floats(x0, t, (n, c), h0=h0, hT=hT)
    sa = None
    if states is not None:
        sa, = _rank_floats(x0, t, sp_gated_scan_states_shape(b, s, c), states=states)
    st = _status_word(dev, status)
    _call(dev, lib.sp_gated_scan_fwd, ga, g_ld, va, v_ld, ha, b, s, c, t, dt, int(bool(tied)), cu,
          n_seqs, ya, y_ld, ta, sa, st)


def sp_gated_scan_bwd(gate, value, states, dy, *, h0=None, dhT=None, tied=True, cu_seqlens=None,
                      dgate, dvalue, dh0=None, status=None):
    """Gradients of sp_gated_scan_fwd (same gate, value, h0, tied, cu_seqlens) from
    the states it saved; dhT: gradient of hT, dh0: gradient of h0."""
    code = _quick().scan_bwd(gate, value, h0, tied, cu_seqlens, states, dy, dhT, dgate, dvalue, dh0,
                             status)
    if code is not None:
        return _check(code)
    lib = load()
    t, x0, dt = _first(gate, 3, "gate")
    b, s, c = x0.shape
    dev = x0.device
    ga, g_ld, va, v_ld, da, d_ld, dga, dg_ld, dva, dv_ld = _rank_rows(
        x0, t, gate=gate, value=value, dy=dy, dgate=dgate, dvalue=dvalue)
    cu, n_seqs = _seq_meta(cu_seqlens, b, dev)
    n = b if cu is None else n_seqs
    ha, ta, oa = _rank_floats(x0, t, (n, c), h0=h0, dhT=dhT, dh0=dh0)
    sa, = _rank_floats(x0, t, sp_gated_scan_states_shape(b, s, c), states=states)
    st = _status_word(dev, status)
    _call(dev, lib.sp_gated_scan_bwd, ga, g_ld, va, v_ld, ha, sa, da, d_ld, ta, b, s, c, t, dt,
          int(bool(tied)), cu, n_seqs, dga, dg_ld, dva, dv_ld, oa, st)


def sp_group_norm_fwd(x, gamma, beta=None, *, groups, eps, norm="layernorm", act="none", y,
                      mean=None, rstd):
    """Group norm with an activation ("none" or "silu") of (n, l, c) rank buffers,
    channels last; the statistics of each of the `groups` groups of a rank span the l
    rows of a sample (l = 1: per token).  gamma, beta: (t * c).  mean (LayerNorm) and
    rstd: float32 (n, groups) per rank, written for the backward."""
    code = _quick().norm_fwd(x, gamma, beta, groups, eps, NORMS.get(norm), ACTS.get(act), y, mean,
                             rstd)
    if code is not None:
        return _check(code)
    lib = load()
    t, x0, dt = _first(x, 3, "x")
    n, l, c = x0.shape
    dev = x0.device
    ln = norm == "layernorm"
    xa, x_ld, ya, y_ld = _rank_rows(x0, t, x=x, y=y)
    if gamma is None or ln and beta is None:
        raise TypeError("gamma (and beta for layernorm) must be a torch.Tensor")
    gp, bp = _params(x0, t * c, gamma=gamma, beta=beta if ln else None)
    if ln and mean is None:
        raise ValueError("mean is required for layernorm")
    ma, ra = _rank_floats(x0, t, (n, groups), mean=mean if ln else None, rstd=rstd)
    _call(dev, lib.sp_group_norm_fwd, xa, x_ld, gp, bp, n, l, c, groups, t, dt, float(eps),
          _choice(NORMS, norm, "norm"), _choice(ACTS, act, "act"), ya, y_ld, ma, ra)


def sp_group_norm_bwd_workspace_bytes(n, l, c, groups, t, dtype=torch.bfloat16):
    """Bytes of sp_group_norm_bwd's workspace on the current device."""
    return int(load().sp_group_norm_bwd_workspace_bytes(n, l, c, groups, t, DTYPES[dtype]))


def sp_group_norm_bwd(dy, x, mean, rstd, gamma, beta=None, *, groups, norm="layernorm",
                      act="none", dx, dgamma=None, dbeta=None, workspace=None):
    """Gradients of sp_group_norm_fwd from its input and saved statistics: dx, and
    where given the float32 (t * c) dgamma and dbeta (these need the workspace of
    sp_group_norm_bwd_workspace_bytes, one per call that may run at the same time)."""
    code = _quick().norm_bwd(dy, x, mean, rstd, gamma, beta, groups, NORMS.get(norm), ACTS.get(act),
                             dx, dgamma, dbeta, workspace)
    if code is not None:
        return _check(code)
    lib = load()
    t, x0, dt = _first(x, 3, "x")
    n, l, c = x0.shape
    dev = x0.device
    ln = norm == "layernorm"
    da, d_ld, xa, x_ld, oa, o_ld = _rank_rows(x0, t, dy=dy, x=x, dx=dx)
    if gamma is None or ln and beta is None:
        raise TypeError("gamma (and beta for layernorm) must be a torch.Tensor")
    gp, bp = _params(x0, t * c, gamma=gamma, beta=beta if ln else None)
    if ln and mean is None:
        raise ValueError("mean is required for layernorm")
    ma, ra = _rank_floats(x0, t, (n, groups), mean=mean if ln else None, rstd=rstd)
    for name, v in (("dgamma", dgamma), ("dbeta", dbeta)):
        if v is not None:
            _need(v, (t * c,), torch.float32, dev, name)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(dev, lib.sp_group_norm_bwd, da, d_ld, xa, x_ld, ma, ra, gp, bp, n, l, c, groups, t, dt,
          _choice(NORMS, norm, "norm"), _choice(ACTS, act, "act"), oa, o_ld,
          dgamma.data_ptr() if dgamma is not None else None,
          dbeta.data_ptr() if dbeta is not None and ln else None,
          workspace.data_ptr() if workspace is not None else None, size)


def sp_debug_inject(code):
    load().sp_debug_inject(int(code))


def sp_debug_scan_withhold(step):
    _check(load().sp_debug_scan_withhold(int(step)))


def sp_debug_tune(kernel, stages=0, blocks_per_sm=0, threads=0, chunks=0):
    _check(load().sp_debug_tune(int(kernel), int(stages), int(blocks_per_sm), int(threads),
                                int(chunks)))


def sp_debug_last_shape(kernel):
    """Launch shape of this thread's last forward (0) or backward (1) call:
    dict(threads, chunks, stages, grid, cluster, smem)."""
    out = (ctypes.c_int32 * 6)()
    _check(load().sp_debug_last_shape(int(kernel), ctypes.cast(out, _vp)))
    return dict(zip(("threads", "chunks", "stages", "grid", "cluster", "smem"), list(out)))


def sp_debug_group_norm_shape(n, l, c, groups, t, dtype=torch.bfloat16, backward=False):
    """How a group norm call is split on the current device."""
    out = (ctypes.c_int64 * 8)()
    _check(load().sp_debug_group_norm_shape(n, l, c, groups, t, DTYPES[dtype], int(backward), out))
    return dict(zip(("form", "threads", "cluster", "cols", "slabs", "rows", "parts", "smem"),
                    list(out)))


def sp_debug_philox(ctr_key):
    """Device Philox4x32-10 of an (n, 6) uint32 tensor of (c0..c3, k0, k1)."""
    if ctr_key.dtype != torch.int32 or ctr_key.dim() != 2 or ctr_key.shape[1] != 6:
        raise ValueError("ctr_key must be an (n, 6) int32 tensor (uint32 bits)")
    out = torch.empty((ctr_key.shape[0], 4), dtype=torch.int32, device=ctr_key.device)
    _check(load().sp_debug_philox(_ptr(ctr_key.contiguous()), _ptr(out), ctr_key.shape[0],
                                  _stream(ctr_key.device)))
    return out


def sp_abi_version():
    return int(load().sp_abi_version())
