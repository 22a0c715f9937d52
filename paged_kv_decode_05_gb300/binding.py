"""Thin ctypes binding over ``libpkv.so`` (argument marshalling only).

Each function has the name of the C entry point it calls (``include/pkv.h``),
takes torch CUDA tensors, passes their device pointers, sizes and the current
CUDA stream, and raises :class:`PkvError` on a non-OK status. All arithmetic
runs in the library's kernels; there is no other code path. If the library
has not been built, loading it raises.
"""

from __future__ import annotations

import array
import ctypes
import os

from .build import LIB, up_to_date

PKV_F16, PKV_BF16, PKV_I8 = 0, 1, 2
STATUS = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED",
          3: "PKV_ERR_WORKSPACE", 4: "PKV_ERR_CUDA"}
DEV_BAD_BLOCK, DEV_BAD_LENGTH, DEV_BAD_SLOT, DEV_TIMEOUT, DEV_BAD_INDEX = 1, 2, 4, 8, 16
BLOCK_SIZE = 16


class PkvError(RuntimeError):
    def __init__(self, func, code, msg):
        super().__init__(f"{func}: {msg}")
        self.code = code


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int)]


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_DESC = ctypes.POINTER(CacheDesc)

_SIGS = {
    "pkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "pkv_append_workspace_size": (_SZ, [_DESC]),
    "pkv_append": (ctypes.c_int, [_P, _P, ctypes.c_int, _I32, _P, _P, _P, _P, _P, _DESC, _P, _SZ,
                                  _P, _P]),
    "pkv_decode_default_parts": (_I32, [_I32, _I32, _I32, _DESC]),
    "pkv_decode_workspace_size": (_SZ, [_I32, _I32, _DESC, _I32]),
    "pkv_decode_attn": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32, _P,
                                       _I32, _I32, ctypes.c_float, _P, _P, _SZ, _I32, _P, _P]),
    "pkv_decode_split": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32, _P,
                                        _I32, _I32, ctypes.c_float, _P, _P, _SZ, _I32, _P, _P]),
    "pkv_decode_combine": (ctypes.c_int, [_DESC, _I32, _I32, ctypes.c_int, _P, _P, _SZ, _I32, _P]),
    "pkv_decode_step": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _P, _P, _DESC, _P, _I32,
                                       _P, _I32, _I32, ctypes.c_float, _P, _P, _SZ, _I32, _I32,
                                       _P, _P]),
    "pkv_copy_blocks": (ctypes.c_int, [_P, _P, _P, _P, _DESC, _P, _P, _I32, _P, _P]),
    "pkv_multiquery_workspace_size": (_SZ, [_I32, _I32, _I32, _DESC, _I32]),
    "pkv_multiquery_attn": (ctypes.c_int, [_P, ctypes.c_int, _P, _I32, _P, _P, _P, _P, _DESC, _P,
                                           _I32, _P, _I32, _I32, ctypes.c_float, _P, _P, _SZ,
                                           _I32, _P, _P]),
    "pkv_decode_attn_noalloc": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32,
                                               _P, _I32, _I32, ctypes.c_float, _P, _I32, _P, _P]),
    "pkv_merge_states": (ctypes.c_int, [_P, _P, _P, ctypes.c_int64, _P, _I32, _I32, _I32,
                                        ctypes.c_int, _P, _P, _P, _P, _P]),
    "pkv_qk_norm_rope": (ctypes.c_int, [_P, _I64, _P, _I64, ctypes.c_int, _I32, _I32, _I32, _I32,
                                        _P, _P, ctypes.c_float, _P, _I32, _I32, _I32, _P, _I32,
                                        _P, _P, _P, _P, _P]),
    "pkv_qk_norm_rope_append": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, ctypes.c_int, _I32,
                                               _I32, _P, _P, ctypes.c_float, _P, _I32, _I32,
                                               _I32, _P, _I32, _P, _P, _P, _P, _P, _DESC, _P,
                                               _P]),
    "pkv_block_bounds": (ctypes.c_int, [_P, _DESC, _P, _I32, _P, _P, _I32, _I32, _P, _P, _P]),
    "pkv_block_scores": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _DESC, _P, _I32, _P, _I32, _I32,
                                        _P, _P, _P]),
    "pkv_block_select": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _I32, _I32, _I32, _P, _P, _P,
                                        _P]),
    "pkv_sparse_decode_workspace_size": (_SZ, [_I32, _I32, _DESC, _I32]),
    "pkv_sparse_decode_attn": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32,
                                              _P, _P, _I32, _P, _I32, _I32, ctypes.c_float, _P,
                                              _P, _SZ, _I32, _P, _P]),
    "pkv_decode_mass_workspace_size": (_SZ, [_I32, _I32, _I32, _DESC, _I32]),
    "pkv_decode_attn_mass": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32, _P,
                                            _I32, _I32, ctypes.c_float, _P, _P, _P, _P, _SZ, _I32,
                                            _P, _P]),
    "pkv_evict_tokens": (ctypes.c_int, [_P, _P, _P, _P, _DESC, _P, _I32, _P, _P, _I32, _I32, _I32,
                                        _I32, _P, _I32, _P, _P, _P, _P, _P]),
    # test hooks (include/pkv_testing.h)
    "pkv_testing_decode_attn_stall": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P,
                                                     _I32, _P, _I32, _I32, ctypes.c_float, _P, _P,
                                                     _SZ, _I32, ctypes.c_uint64, _I32,
                                                     _P, _P]),
    "pkv_testing_sparse_decode_attn_stall": (ctypes.c_int, [
        _P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32, _P, _P, _I32, _P, _I32, _I32,
        ctypes.c_float, _P, _P, _SZ, _I32, ctypes.c_uint64, _I32, _P, _P]),
    "pkv_testing_decode_attn_mass_stall": (ctypes.c_int, [
        _P, ctypes.c_int, _P, _P, _P, _P, _DESC, _P, _I32, _P, _I32, _I32, ctypes.c_float, _P, _P,
        _P, _P, _SZ, _I32, ctypes.c_uint64, _I32, _P, _P]),
    "pkv_testing_multiquery_kernel": (ctypes.c_int, [_I32, _I32, _I32, _DESC, ctypes.c_int, _I32,
                                                     _P, _P]),
    "pkv_testing_multiquery_attn_stall": (ctypes.c_int, [_P, ctypes.c_int, _P, _I32, _P, _P, _P,
                                                         _P, _DESC, _P, _I32, _P, _I32, _I32,
                                                         ctypes.c_float, _P, _P, _SZ, _I32,
                                                         ctypes.c_uint64, _I32, _P, _P]),
}


def lib() -> ctypes.CDLL:
    """Load ``libpkv.so`` once; raise if it is missing or older than its sources."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is not built: run paged_kv_decode_05_gb300.build.build()")
        if not up_to_date():
            raise RuntimeError(f"{LIB} is older than its sources: rebuild it")
        L = ctypes.CDLL(LIB)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _check(func, code):
    if code != 0:
        raise PkvError(func, code, lib().pkv_status_string(code).decode())


_torch = None          # torch, imported by the first call that takes a tensor
_DTYPES = {}


def _tt():
    global _torch
    if _torch is None:
        import torch
        _DTYPES.update({torch.float16: PKV_F16, torch.bfloat16: PKV_BF16, torch.int8: PKV_I8})
        _torch = torch
    return _torch


def _dtype_code(t):
    _tt()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    torch = _torch or _tt()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def cache_desc(k_cache) -> CacheDesc:
    """Describe a ``[num_blocks, num_kv_heads, 16, head_dim]`` cache tensor."""
    NB, H, bs, D = k_cache.shape
    return CacheDesc(NB, bs, H, D, _dtype_code(k_cache))


def pkv_status_string(code: int) -> str:
    return lib().pkv_status_string(code).decode()


def pkv_append_workspace_size(k_cache) -> int:
    return int(lib().pkv_append_workspace_size(ctypes.byref(cache_desc(k_cache))))


def pkv_append(k_new, v_new, slot_mapping, k_cache, v_cache, k_scales=None, v_scales=None,
               workspace=None, dev_status=None, stream=None):
    """Write ``k_new/v_new [N, Hkv, D]`` to the cache at ``slot_mapping [N] int64``."""
    desc = cache_desc(k_cache)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib().pkv_append(_ptr(k_new), _ptr(v_new), _dtype_code(k_new), int(k_new.shape[0]),
                            _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                            _ptr(v_scales), ctypes.byref(desc), _ptr(workspace), ws_bytes,
                            _ptr(dev_status), _stream(stream))
    _check("pkv_append", code)


def pkv_decode_default_parts(batch, num_q_heads, k_cache, device=None) -> int:
    import torch
    dev = torch.cuda.current_device() if device is None else device
    return int(lib().pkv_decode_default_parts(dev, batch, num_q_heads,
                                              ctypes.byref(cache_desc(k_cache))))


def pkv_decode_workspace_size(batch, num_q_heads, k_cache, num_parts=0) -> int:
    return int(lib().pkv_decode_workspace_size(batch, num_q_heads,
                                               ctypes.byref(cache_desc(k_cache)), num_parts))


def _decode(name, q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
            workspace, k_scales, v_scales, num_parts, dev_status, stream):
    desc = cache_desc(k_cache)
    B, Hq, D = q.shape
    code = getattr(lib(), name)(
        _ptr(q), _dtype_code(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
        ctypes.byref(desc), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
        B, Hq, float(softmax_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(num_parts), _ptr(dev_status),
        _stream(stream))
    _check(name, code)


def pkv_decode_attn(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                    workspace, k_scales=None, v_scales=None, num_parts=0, dev_status=None,
                    stream=None):
    """``out [B, Hq, D] = softmax(scale q K^T) V`` over each sequence's paged KV."""
    _decode("pkv_decode_attn", q, k_cache, v_cache, block_tables, context_lens, softmax_scale,
            out, workspace, k_scales, v_scales, num_parts, dev_status, stream)


def pkv_decode_split(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                     workspace, k_scales=None, v_scales=None, num_parts=0, dev_status=None,
                     stream=None):
    _decode("pkv_decode_split", q, k_cache, v_cache, block_tables, context_lens, softmax_scale,
            out, workspace, k_scales, v_scales, num_parts, dev_status, stream)


def pkv_decode_step(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, softmax_scale,
                    out, workspace, num_parts=0, dev_status=None, stream=None, run_combine=True,
                    k_scales=None, v_scales=None):
    """Write ``k_new/v_new [B, Hkv, D]`` at each sequence's last position, then attend
    (``run_combine=False``: split phase only; :func:`pkv_decode_combine` must follow).
    INT8 caches take their ``k_scales/v_scales``."""
    desc = cache_desc(k_cache)
    B, Hq, D = q.shape
    code = lib().pkv_decode_step(
        _ptr(q), _dtype_code(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(k_scales), _ptr(v_scales),
        ctypes.byref(desc), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
        B, Hq, float(softmax_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(num_parts), int(bool(run_combine)),
        _ptr(dev_status), _stream(stream))
    _check("pkv_decode_step", code)


def pkv_decode_combine(out, k_cache, workspace, num_parts=0, stream=None):
    """Merge the partial states a preceding :func:`pkv_decode_split` left in ``workspace``."""
    desc = cache_desc(k_cache)
    B, Hq, D = out.shape
    code = lib().pkv_decode_combine(ctypes.byref(desc), B, Hq, _dtype_code(out), _ptr(out),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    int(num_parts), _stream(stream))
    _check("pkv_decode_combine", code)


def pkv_copy_blocks(k_cache, v_cache, src_blocks, dst_blocks, k_scales=None, v_scales=None,
                    dev_status=None, stream=None):
    """Copy whole blocks ``src_blocks[i] -> dst_blocks[i]`` (int32 device tensors)."""
    desc = cache_desc(k_cache)
    code = lib().pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                                 ctypes.byref(desc), _ptr(src_blocks), _ptr(dst_blocks),
                                 int(src_blocks.numel()), _ptr(dev_status), _stream(stream))
    _check("pkv_copy_blocks", code)


def pkv_multiquery_workspace_size(batch, num_q_heads, max_q_len, k_cache, num_parts=0) -> int:
    return int(lib().pkv_multiquery_workspace_size(batch, num_q_heads, max_q_len,
                                                   ctypes.byref(cache_desc(k_cache)), num_parts))


def pkv_multiquery_attn(q, cu_q, max_q_len, k_cache, v_cache, block_tables, context_lens,
                        softmax_scale, out, workspace, num_parts=0, dev_status=None, stream=None,
                        k_scales=None, v_scales=None):
    """Causal attention of ``cu_q``-delimited new queries ``q [total_q, Hq, D]``
    (``k_scales``, ``v_scales``: INT8 caches only)."""
    desc = cache_desc(k_cache)
    code = lib().pkv_multiquery_attn(
        _ptr(q), _dtype_code(q), _ptr(cu_q), int(max_q_len), _ptr(k_cache), _ptr(v_cache),
        _ptr(k_scales), _ptr(v_scales), ctypes.byref(desc), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens),
        int(cu_q.numel() - 1), int(q.shape[1]), float(softmax_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(num_parts), _ptr(dev_status),
        _stream(stream))
    _check("pkv_multiquery_attn", code)


def pkv_decode_attn_noalloc(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                            k_scales=None, v_scales=None, num_parts=0, dev_status=None,
                            stream=None):
    """:func:`pkv_decode_attn` using the library's built-in scratch array.

    For callers that cannot allocate device memory: no workspace is passed and
    nothing is allocated. Raises PkvError(PKV_ERR_WORKSPACE) when the sizes
    need more scratch than the built-in array holds.
    """
    desc = cache_desc(k_cache)
    B, Hq, D = q.shape
    code = lib().pkv_decode_attn_noalloc(
        _ptr(q), _dtype_code(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
        ctypes.byref(desc), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
        B, Hq, float(softmax_scale), _ptr(out), int(num_parts), _ptr(dev_status),
        _stream(stream))
    _check("pkv_decode_attn_noalloc", code)


def pkv_merge_states(part_m, part_l, part_o, row_ptr, out, out_m=None, out_l=None,
                     dev_status=None, stream=None):
    """Merge partial states ``(m, l, o)`` (``[S, H]``, ``[S, H]``, ``[S, H, D]`` fp32):
    row ``r`` of ``out [R, H, D]`` merges states ``row_ptr[r] .. row_ptr[r+1]-1``."""
    S, H, D = part_o.shape
    R = int(row_ptr.numel()) - 1
    code = lib().pkv_merge_states(_ptr(part_m), _ptr(part_l), _ptr(part_o), int(S),
                                  _ptr(row_ptr), R, int(H), int(D), _dtype_code(out), _ptr(out),
                                  _ptr(out_m), _ptr(out_l), _ptr(dev_status), _stream(stream))
    _check("pkv_merge_states", code)


def _refuse(t, dtype, shape, dev, name):
    """Say what is wrong with an argument that :func:`_arg` turned away."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.get_device() != dev:
        raise ValueError(f"{name} must live on the current CUDA device ({dev})")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of this type and shape on the current device."""
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, dtype, shape, dev, name)
    return t.data_ptr()


def _opt(t, dtype, shape, dev, name):
    return None if t is None else _arg(t, dtype, shape, dev, name)


def _rows_arg(t, dtype, shape, dev, name):
    """(pointer, token stride) of ``[N, heads, D]`` whose head rows are contiguous: a tensor of
    its own or a part of a projection's rows."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, dtype, shape, dev, name)
    row, head, one = t.stride()
    if (one != 1 and shape[2] > 1) or (head != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must have contiguous head rows")
    return t.data_ptr(), (row if shape[0] > 1 else shape[1] * shape[2])


def _device(t, name):
    """The current device; a first argument that is on no CUDA device is refused at once."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    return (_torch or _tt())._C._cuda_getDevice()


def _stream_on(stream, dev):
    """Handle of ``stream`` (None: the current one), which must be the device's."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError("stream must belong to the current CUDA device")
    return stream.cuda_stream


def _status_arg(t, dev):
    if t is None:
        return None
    if t.get_device() != dev or t.element_size() != 4 or t.numel() < 1:
        raise ValueError("dev_status must be one int32 on the current CUDA device")
    return t.data_ptr()


def _workspace_arg(t, dev):
    """(pointer, bytes) of a workspace; None is passed on, for the library to refuse."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be contiguous and live on the current CUDA device")
    return t.data_ptr(), t.numel() * t.element_size()


def _rope_args(q, k, positions, cos_sin, q_weight, k_weight, pair_axis):
    """The checked arguments that both norm-and-rotation calls share."""
    torch = _tt()
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    dev, dt = _device(q, "q"), q.dtype
    qp, qs = _rows_arg(q, dt, (N, Hq, D), dev, "q")
    kp, ks = _rows_arg(k, dt, (N, Hkv, D), dev, "k")
    table = pos = axis = None
    rows = rot = axes = 0
    if cos_sin is not None:
        rows, rot = cos_sin.shape
        table = _arg(cos_sin, torch.float32, (rows, rot), dev, "cos_sin")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        pos = _arg(positions, torch.int32, (N,) if positions.dim() == 1 else (axes, N), dev,
                   "positions")
    if pair_axis is not None:
        if len(pair_axis) != rot // 2:
            raise ValueError("pair_axis must name one axis per rotated pair")
        axis = array.array("i", pair_axis).tobytes()   # int32, read during the call
    return (N, Hq, Hkv, D, dev, dt, qp, qs, kp, ks, _opt(q_weight, dt, (D,), dev, "q_weight"),
            _opt(k_weight, dt, (D,), dev, "k_weight"), table, rows, rot, pos, axes, axis)


def pkv_qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight=None, k_weight=None,
                     eps=1e-6, pair_axis=None, interleaved=False, dev_status=None, stream=None):
    """Per-head norms (where a weight is given) and position rotation of ``q [N, Hq, D]`` and
    ``k [N, Hkv, D]`` into ``q_out``, ``k_out``. ``positions``: int32 ``[N]`` or ``[axes, N]``;
    ``cos_sin``: fp32 ``[max_position, rot_dim]`` (None: norms only); ``pair_axis``: the axis of
    each of the ``rot_dim / 2`` pairs (a sequence of ints)."""
    (N, Hq, Hkv, D, dev, dt, qp, qs, kp, ks, qw, kw, table, rows, rot, pos, axes,
     axis) = _rope_args(q, k, positions, cos_sin, q_weight, k_weight, pair_axis)
    code = lib().pkv_qk_norm_rope(
        qp, qs, kp, ks, _dtype_code(q), N, Hq, Hkv, D, qw, kw, eps, table, rows, rot,
        1 if interleaved else 0, pos, axes, axis, _arg(q_out, dt, (N, Hq, D), dev, "q_out"),
        _arg(k_out, dt, (N, Hkv, D), dev, "k_out"), _status_arg(dev_status, dev),
        _stream_on(stream, dev))
    if code:
        _check("pkv_qk_norm_rope", code)


def pkv_qk_norm_rope_append(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out,
                            q_weight=None, k_weight=None, eps=1e-6, pair_axis=None,
                            interleaved=False, dev_status=None, stream=None):
    """:func:`pkv_qk_norm_rope` that writes K, and ``v [N, Hkv, D]`` as it is, to
    ``slot_mapping [N] int64`` of a 16-bit cache."""
    (N, Hq, Hkv, D, dev, dt, qp, qs, kp, ks, qw, kw, table, rows, rot, pos, axes,
     axis) = _rope_args(q, k, positions, cos_sin, q_weight, k_weight, pair_axis)
    desc, shape, kvt = cache_desc(k_cache), k_cache.shape, k_cache.dtype
    if shape[1] != Hkv or shape[3] != D:
        raise ValueError("k must match the cache's heads and head_dim")
    vp, vs = _rows_arg(v, dt, (N, Hkv, D), dev, "v")
    code = lib().pkv_qk_norm_rope_append(
        qp, qs, kp, ks, vp, vs, _dtype_code(q), N, Hq, qw, kw, eps, table, rows, rot,
        1 if interleaved else 0, pos, axes, axis, _arg(q_out, dt, (N, Hq, D), dev, "q_out"),
        _arg(slot_mapping, _tt().int64, (N,), dev, "slot_mapping"),
        _arg(k_cache, kvt, shape, dev, "k_cache"), _arg(v_cache, kvt, shape, dev, "v_cache"),
        desc, _status_arg(dev_status, dev), _stream_on(stream, dev))
    if code:
        _check("pkv_qk_norm_rope_append", code)


def pkv_block_bounds(k_cache, block_tables, context_lens, bounds, num_new=None, max_new=1,
                     dev_status=None, stream=None):
    """Channel-wise min and max of the keys, ``bounds [num_blocks, Hkv, 2, D]`` in the cache's
    type, of the blocks that hold each sequence's last ``num_new [B] int32`` tokens (None: 1)."""
    i32, dev = _tt().int32, _device(k_cache, "k_cache")
    desc, kvt = cache_desc(k_cache), k_cache.dtype
    NB, H, bs, D = k_cache.shape
    B, mb = block_tables.shape
    code = lib().pkv_block_bounds(
        _arg(k_cache, kvt, (NB, H, bs, D), dev, "k_cache"), desc,
        _arg(block_tables, i32, (B, mb), dev, "block_tables"), mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"),
        _opt(num_new, i32, (B,), dev, "num_new"), max_new, B,
        _arg(bounds, kvt, (NB, H, 2, D), dev, "bounds"), _status_arg(dev_status, dev),
        _stream_on(stream, dev))
    if code:
        _check("pkv_block_bounds", code)


def pkv_block_scores(q, bounds, k_cache, block_tables, context_lens, scores, k_scales=None,
                     dev_status=None, stream=None):
    """Upper bounds of every block's ``<q, k>``: ``scores [B, Hkv, blocks] fp32`` (the cache is
    named for its sizes and type; only ``bounds`` is read)."""
    torch, dev = _tt(), _device(q, "q")
    i32, f32 = torch.int32, torch.float32
    desc = cache_desc(k_cache)
    NB, H, _, D = k_cache.shape
    B, mb = block_tables.shape
    Hq = q.shape[1]
    code = lib().pkv_block_scores(
        _arg(q, q.dtype, (B, Hq, D), dev, "q"), _dtype_code(q),
        _arg(bounds, k_cache.dtype, (NB, H, 2, D), dev, "bounds"),
        _opt(k_scales, f32, (NB, H), dev, "k_scales"), desc,
        _arg(block_tables, i32, (B, mb), dev, "block_tables"), mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"), B, Hq,
        _arg(scores, f32, (B, H, mb), dev, "scores"), _status_arg(dev_status, dev),
        _stream_on(stream, dev))
    if code:
        _check("pkv_block_scores", code)


def pkv_block_select(scores, context_lens, keep_first, keep_last, block_lists, list_lens,
                     dev_status=None, stream=None):
    """The best blocks of ``scores [B, Hkv, blocks]``: ``block_lists [B, Hkv, budget] int32``,
    ascending, and ``list_lens [B] int32``."""
    torch, dev = _tt(), _device(scores, "scores")
    i32 = torch.int32
    B, H, mb = scores.shape
    budget = block_lists.shape[2]
    code = lib().pkv_block_select(
        _arg(scores, torch.float32, (B, H, mb), dev, "scores"), B, H, mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"), keep_first, keep_last, budget,
        _arg(block_lists, i32, (B, H, budget), dev, "block_lists"),
        _arg(list_lens, i32, (B,), dev, "list_lens"), _status_arg(dev_status, dev),
        _stream_on(stream, dev))
    if code:
        _check("pkv_block_select", code)


def pkv_sparse_decode_workspace_size(batch, num_q_heads, k_cache, num_parts=0) -> int:
    return int(lib().pkv_sparse_decode_workspace_size(batch, num_q_heads, cache_desc(k_cache),
                                                      num_parts))


def _sparse_args(q, k_cache, v_cache, block_tables, context_lens, block_lists, list_lens,
                 softmax_scale, out, workspace, k_scales, v_scales, num_parts):
    torch, dev = _tt(), _device(q, "q")
    i32, f32 = torch.int32, torch.float32
    desc, shape, kvt = cache_desc(k_cache), k_cache.shape, k_cache.dtype
    H, D = shape[1], shape[3]
    B, mb = block_tables.shape
    Hq = q.shape[1]
    n = block_lists.shape[2]
    ws, ws_bytes = _workspace_arg(workspace, dev)
    return dev, (
        _arg(q, q.dtype, (B, Hq, D), dev, "q"), _dtype_code(q),
        _arg(k_cache, kvt, shape, dev, "k_cache"), _arg(v_cache, kvt, shape, dev, "v_cache"),
        _opt(k_scales, f32, shape[:2], dev, "k_scales"),
        _opt(v_scales, f32, shape[:2], dev, "v_scales"), desc,
        _arg(block_tables, i32, (B, mb), dev, "block_tables"), mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"),
        _arg(block_lists, i32, (B, H, n), dev, "block_lists"), n,
        _arg(list_lens, i32, (B,), dev, "list_lens"), B, Hq, softmax_scale,
        _arg(out, q.dtype, (B, Hq, D), dev, "out"), ws, ws_bytes, num_parts)


def pkv_sparse_decode_attn(q, k_cache, v_cache, block_tables, context_lens, block_lists,
                           list_lens, softmax_scale, out, workspace, k_scales=None, v_scales=None,
                           num_parts=0, dev_status=None, stream=None):
    """:func:`pkv_decode_attn` over the blocks of ``block_lists [B, Hkv, n] int32`` (the first
    ``list_lens[b]`` of each, indices into the sequence's blocks)."""
    dev, args = _sparse_args(q, k_cache, v_cache, block_tables, context_lens, block_lists,
                             list_lens, softmax_scale, out, workspace, k_scales, v_scales,
                             num_parts)
    code = lib().pkv_sparse_decode_attn(*args, _status_arg(dev_status, dev),
                                        _stream_on(stream, dev))
    if code:
        _check("pkv_sparse_decode_attn", code)


def pkv_decode_mass_workspace_size(batch, num_q_heads, max_blocks, k_cache, num_parts=0) -> int:
    return int(lib().pkv_decode_mass_workspace_size(batch, num_q_heads, max_blocks,
                                                    cache_desc(k_cache), num_parts))


def _mass_args(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out, mass_in,
               mass_out, workspace, k_scales, v_scales, num_parts):
    torch, dev = _tt(), _device(q, "q")
    i32, f32 = torch.int32, torch.float32
    desc, shape, kvt = cache_desc(k_cache), k_cache.shape, k_cache.dtype
    H, D = shape[1], shape[3]
    B, mb = block_tables.shape
    Hq = q.shape[1]
    tokens = (B, H, mb * BLOCK_SIZE)
    ws, ws_bytes = _workspace_arg(workspace, dev)
    return dev, (
        _arg(q, q.dtype, (B, Hq, D), dev, "q"), _dtype_code(q),
        _arg(k_cache, kvt, shape, dev, "k_cache"), _arg(v_cache, kvt, shape, dev, "v_cache"),
        _opt(k_scales, f32, shape[:2], dev, "k_scales"),
        _opt(v_scales, f32, shape[:2], dev, "v_scales"), desc,
        _arg(block_tables, i32, (B, mb), dev, "block_tables"), mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"), B, Hq, softmax_scale,
        _arg(out, q.dtype, (B, Hq, D), dev, "out"), _opt(mass_in, f32, tokens, dev, "mass_in"),
        _arg(mass_out, f32, tokens, dev, "mass_out"), ws, ws_bytes, num_parts)


def pkv_decode_attn_mass(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                         mass_in, mass_out, workspace, k_scales=None, v_scales=None, num_parts=0,
                         dev_status=None, stream=None):
    """:func:`pkv_decode_attn` that also writes ``mass_out = mass_in + `` each token's weights,
    fp32 ``[B, Hkv, blocks * 16]`` (``mass_in`` may be None, or ``mass_out`` itself)."""
    dev, args = _mass_args(q, k_cache, v_cache, block_tables, context_lens, softmax_scale, out,
                           mass_in, mass_out, workspace, k_scales, v_scales, num_parts)
    code = lib().pkv_decode_attn_mass(*args, _status_arg(dev_status, dev),
                                      _stream_on(stream, dev))
    if code:
        _check("pkv_decode_attn_mass", code)


def pkv_evict_tokens(k_cache, v_cache, block_tables, context_lens, mass, keep_first, keep_last,
                     new_tables, new_lens, new_mass, kept, k_scales=None, v_scales=None,
                     dev_status=None, stream=None):
    """Cut every (sequence, kv head) to ``budget = kept.shape[2]`` tokens by ``mass [B, Hkv,
    blocks * 16]`` and compact them into ``new_tables [B, new_blocks] int32`` (``block_tables``
    itself, a copy, or of its first columns: in place). Writes ``kept [B, Hkv, budget] int32``, ``new_lens [B] int32`` and
    ``new_mass [B, Hkv, new_blocks * 16]``, which stand for ``context_lens`` and ``mass`` from
    then on. Every block's bounds are stale afterwards: call ``pkv_block_bounds(k_cache, new_tables,
    new_lens, bounds, new_lens, budget)``."""
    torch, dev = _tt(), _device(k_cache, "k_cache")
    i32, f32 = torch.int32, torch.float32
    desc, shape, kvt = cache_desc(k_cache), k_cache.shape, k_cache.dtype
    H = shape[1]
    B, mb = block_tables.shape
    new_mb = new_tables.shape[1]
    budget = kept.shape[2]
    code = lib().pkv_evict_tokens(
        _arg(k_cache, kvt, shape, dev, "k_cache"), _arg(v_cache, kvt, shape, dev, "v_cache"),
        _opt(k_scales, f32, shape[:2], dev, "k_scales"),
        _opt(v_scales, f32, shape[:2], dev, "v_scales"), desc,
        _arg(block_tables, i32, (B, mb), dev, "block_tables"), mb,
        _arg(context_lens, i32, (B,), dev, "context_lens"),
        _arg(mass, f32, (B, H, mb * BLOCK_SIZE), dev, "mass"), B, budget, keep_first, keep_last,
        _arg(new_tables, i32, (B, new_mb), dev, "new_tables"), new_mb,
        _arg(new_lens, i32, (B,), dev, "new_lens"),
        _arg(new_mass, f32, (B, H, new_mb * BLOCK_SIZE), dev, "new_mass"),
        _arg(kept, i32, (B, H, budget), dev, "kept"), _status_arg(dev_status, dev),
        _stream_on(stream, dev))
    if code:
        _check("pkv_evict_tokens", code)


def pkv_testing_decode_attn_stall(q, k_cache, v_cache, block_tables, context_lens, softmax_scale,
                                  out, workspace, wait_limit_ns, stall_worker, k_scales=None,
                                  v_scales=None, num_parts=0, dev_status=None, stream=None):
    """Test hook: :func:`pkv_decode_attn` whose worker ``stall_worker`` never completes
    the wait for its first unit (bounded by ``wait_limit_ns``); see ``include/pkv_testing.h``."""
    desc = cache_desc(k_cache)
    B, Hq, D = q.shape
    code = lib().pkv_testing_decode_attn_stall(
        _ptr(q), _dtype_code(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
        ctypes.byref(desc), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
        B, Hq, float(softmax_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(num_parts), int(wait_limit_ns),
        int(stall_worker), _ptr(dev_status), _stream(stream))
    _check("pkv_testing_decode_attn_stall", code)


def pkv_testing_multiquery_attn_stall(q, cu_q, max_q_len, k_cache, v_cache, block_tables,
                                      context_lens, softmax_scale, out, workspace, wait_limit_ns,
                                      stall_cta, num_parts=0, dev_status=None, stream=None,
                                      k_scales=None, v_scales=None):
    """Test hook: :func:`pkv_multiquery_attn` whose CTA ``stall_cta`` stalls."""
    desc = cache_desc(k_cache)
    code = lib().pkv_testing_multiquery_attn_stall(
        _ptr(q), _dtype_code(q), _ptr(cu_q), int(max_q_len), _ptr(k_cache), _ptr(v_cache),
        _ptr(k_scales), _ptr(v_scales), ctypes.byref(desc), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens),
        int(cu_q.numel() - 1), int(q.shape[1]), float(softmax_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), int(num_parts), int(wait_limit_ns),
        int(stall_cta), _ptr(dev_status), _stream(stream))
    _check("pkv_testing_multiquery_attn_stall", code)


MQ_KERNELS = {0: "mq_tc_kernel", 1: "mqt_split_kernel", 2: "mqt_i8_split_kernel",
              3: "mq_split_kernel"}


def pkv_testing_multiquery_kernel(batch, num_q_heads, max_q_len, desc, q_dtype, num_parts=16):
    """Test hook: (kernel name, rows per tile) that pkv_multiquery_attn runs for
    these sizes, from the library's own planner (no GPU needed)."""
    kernel, rt = ctypes.c_int32(-1), ctypes.c_int32(0)
    code = lib().pkv_testing_multiquery_kernel(int(batch), int(num_q_heads), int(max_q_len),
                                               ctypes.byref(desc), int(q_dtype), int(num_parts),
                                               ctypes.byref(kernel), ctypes.byref(rt))
    _check("pkv_testing_multiquery_kernel", code)
    return MQ_KERNELS[kernel.value], rt.value


def pkv_testing_sparse_decode_attn_stall(*args, wait_limit_ns, stall_worker, num_parts=0,
                                         k_scales=None, v_scales=None, dev_status=None,
                                         stream=None):
    """Test hook: :func:`pkv_sparse_decode_attn` (its positional arguments) whose worker
    ``stall_worker`` stalls."""
    dev, args = _sparse_args(*args, k_scales, v_scales, num_parts)
    _check("pkv_testing_sparse_decode_attn_stall", lib().pkv_testing_sparse_decode_attn_stall(
        *args, wait_limit_ns, stall_worker, _status_arg(dev_status, dev),
        _stream_on(stream, dev)))


def pkv_testing_decode_attn_mass_stall(*args, wait_limit_ns, stall_worker, num_parts=0,
                                       k_scales=None, v_scales=None, dev_status=None,
                                       stream=None):
    """Test hook: :func:`pkv_decode_attn_mass` (its positional arguments) whose worker
    ``stall_worker`` stalls."""
    dev, args = _mass_args(*args, k_scales, v_scales, num_parts)
    _check("pkv_testing_decode_attn_mass_stall", lib().pkv_testing_decode_attn_mass_stall(
        *args, wait_limit_ns, stall_worker, _status_arg(dev_status, dev),
        _stream_on(stream, dev)))
