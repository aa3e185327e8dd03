"""B200-native multi-scale deformable attention (MSDA) and BEVFormer Spatial
Cross-Attention (SCA).

The compute lives in ``libmsda.so`` (hand-written sm_100a CUDA kernels behind
the C ABI of ``include/msda.h``).  This module only marshals arguments: it
reads shapes and device pointers from torch tensors, allocates outputs with
torch, passes the current CUDA stream and raises ``MsdaError`` on a non-zero
status.  There is no fallback: without the built library every call raises.

Functions (same names as the C ABI): ``msda_forward``, ``msda_forward_fused``,
``msda_backward``, ``sca_compact``, ``sca_rebatched_forward``,
``sca_camera_average``, ``sca_camera_average_linear``, ``sca_forward``,
``sca_forward_query_major``, ``sca_rebatched_backward``, ``sca_backward``
and ``msda_backward`` (``deterministic=True``: the fixed-point variants),
``sca_backward_full``,
``sca_backward_inputs``, ``tsa_reference_points``, ``tsa_forward``,
``tsa_backward``, ``msda_linear`` (with dropout), ``sca_module_forward``,
``msda_group_norm``, ``msda_group_norm_backward``, ``msda_query_attention``,
``msda_query_attention_backward``, ``msda_clip_grad_norm``,
``msda_workspace_size``, ``sca_compact_workspace_size``; the remaining C
entry points (workspace sizes, status strings, the no-alloc compaction, the
GEMM's timeout counter and test switch) are reached through ``lib()``.
"""
import array
import contextlib
import ctypes
import operator
import os

import numpy as np

HEAD_DIM = 32
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsda.so")

MSDA_F32, MSDA_BF16 = 0, 1


class MsdaError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Ncam", "Nq", "Nv", "H", "L", "P", "R")]


_vp = ctypes.c_void_p


class ScaModuleParams(ctypes.Structure):
    _fields_ = [("query", _vp), ("query_pos", _vp), ("features", _vp), ("w_value", _vp),
                ("b_value", _vp), ("w_offsets", _vp), ("b_offsets", _vp), ("w_weights", _vp),
                ("b_weights", _vp), ("w_output", _vp), ("b_output", _vp),
                ("reference_points_cam", _vp), ("bev_mask", _vp), ("value_dtype", ctypes.c_int),
                ("dropout_p", ctypes.c_float), ("dropout_seed", ctypes.c_uint64),
                ("camera_embeds", _vp), ("level_embeds", _vp)]


class NormDims(ctypes.Structure):
    """msda_norm_dims_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Nv", "C", "L", "G")]


class Attention(ctypes.Structure):
    """msda_attention_t: the inputs of msda_query_attention."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("q_points", _vp),
                ("k_points", _vp), ("tau", _vp), ("q_group", _vp), ("k_group", _vp),
                ("scale", ctypes.c_float), ("B", ctypes.c_int32), ("Nq", ctypes.c_int32),
                ("Nk", ctypes.c_int32), ("H", ctypes.c_int32)]


class Grad(ctypes.Structure):
    """msda_grad_t: one gradient tensor of msda_clip_grad_norm."""
    _fields_ = [("grad", _vp), ("out", _vp), ("numel", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


_lib = None
_i64p = ctypes.POINTER(ctypes.c_int64)


def lib():
    """The loaded libmsda.so (raises MsdaError when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MsdaError(f"{LIB_PATH} is missing: build it with "
                            "`python -m scale_deformable_attention_03_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        st = ctypes.c_int
        L.msda_forward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, Dims, _vp, _vp]
        L.msda_forward_fused.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, Dims, _vp, _vp]
        L.msda_backward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, Dims, _vp, _vp, _vp, _vp]
        L.msda_backward_deterministic.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, Dims,
                                                  _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]
        L.msda_backward_deterministic.restype = ctypes.c_int
        L.msda_backward_deterministic_workspace_size.argtypes = [Dims]
        L.msda_backward_deterministic_workspace_size.restype = ctypes.c_size_t
        L.sca_backward_deterministic.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, _vp,
                                                 Dims, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]
        L.sca_backward_deterministic.restype = ctypes.c_int
        L.sca_backward_deterministic_workspace_size.argtypes = [Dims]
        L.sca_backward_deterministic_workspace_size.restype = ctypes.c_size_t
        L.msda_workspace_size.argtypes = [Dims]
        L.msda_workspace_size.restype = ctypes.c_size_t
        L.sca_compact_workspace_size.argtypes = [Dims]
        L.sca_compact_workspace_size.restype = ctypes.c_size_t
        L.sca_compact.argtypes = [_vp, Dims, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp]
        L.sca_forward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, Dims, _vp,
                                  ctypes.c_size_t, _vp, _vp]
        L.sca_backward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, _vp, Dims, _vp,
                                   ctypes.c_size_t, _vp, _vp, _vp, _vp]
        L.sca_rebatched_forward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, _vp, Dims,
                                            _vp, _vp]
        L.sca_camera_average.argtypes = [_vp, _vp, _vp, Dims, _vp, _vp]
        L.sca_rebatched_backward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _vp, Dims, _vp, _vp, _vp, _vp]
        for f in ("msda_forward", "msda_forward_fused", "msda_backward", "sca_compact",
                  "sca_forward", "sca_backward", "sca_rebatched_forward", "sca_camera_average",
                  "sca_rebatched_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.msda_linear.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_int32, st, _vp, _vp]
        L.msda_linear.restype = ctypes.c_int
        L.msda_linear_dropout.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32,
                                          ctypes.c_int32, st, _vp, ctypes.c_float,
                                          ctypes.c_uint64, _vp]
        L.msda_linear_dropout.restype = ctypes.c_int
        L.sca_camera_average_linear.argtypes = [_vp, _vp, _vp, Dims, _vp, _vp, _vp,
                                                ctypes.c_int32, st, _vp, ctypes.c_float,
                                                ctypes.c_uint64, _vp]
        L.sca_camera_average_linear.restype = ctypes.c_int
        L.msda_linear_timeouts.restype = ctypes.c_uint32
        L.msda_linear_test_withhold_load.restype = ctypes.c_int
        L.sca_module_workspace_size.argtypes = [Dims, ctypes.c_int]
        L.sca_module_workspace_size.restype = ctypes.c_size_t
        L.sca_module_forward.argtypes = [ctypes.POINTER(ScaModuleParams), _i64p, _i64p, Dims, _vp,
                                         ctypes.c_size_t, _vp, _vp]
        L.sca_module_forward.restype = ctypes.c_int
        L.sca_backward_inputs.argtypes = [_i64p, _i64p, _vp, _vp, _vp, _vp, Dims, _vp, _vp, _vp,
                                          _vp]
        L.sca_backward_inputs.restype = ctypes.c_int
        L.sca_backward_full_workspace_size.argtypes = [Dims]
        L.sca_backward_full_workspace_size.restype = ctypes.c_size_t
        L.sca_backward_full.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, _vp, Dims,
                                        _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp]
        L.sca_backward_full.restype = ctypes.c_int
        i32, f64 = ctypes.c_int32, ctypes.c_double
        L.tsa_reference_points.argtypes = [_vp, i32, i32, i32, i32, f64, f64, _vp, _vp]
        L.tsa_reference_points.restype = ctypes.c_int
        L.tsa_forward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, i32, Dims, _vp, _vp]
        L.tsa_forward.restype = ctypes.c_int
        L.tsa_backward_workspace_size.argtypes = [Dims, i32]
        L.tsa_backward_workspace_size.restype = ctypes.c_size_t
        L.tsa_backward.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, i32, _vp, Dims, _vp,
                                   ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp]
        L.tsa_backward.restype = ctypes.c_int
        L.sca_forward_query_major.argtypes = [_vp, st, _i64p, _i64p, _vp, _vp, _vp, _vp, Dims,
                                              _vp, _vp]
        L.sca_forward_query_major.restype = ctypes.c_int
        L.msda_group_norm_workspace_size.argtypes = [NormDims]
        L.msda_group_norm_workspace_size.restype = ctypes.c_size_t
        L.msda_group_norm.argtypes = [_vp, st, _vp, _vp, NormDims, _vp, _vp, ctypes.c_float,
                                      st, st, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.msda_group_norm.restype = ctypes.c_int
        L.msda_group_norm_backward_workspace_size.argtypes = [NormDims]
        L.msda_group_norm_backward_workspace_size.restype = ctypes.c_size_t
        L.msda_group_norm_backward.argtypes = [_vp, st, _vp, _vp, NormDims, _vp, _vp, _vp,
                                               _vp, st, _vp, st, st, _vp, _vp, _vp, _vp,
                                               ctypes.c_size_t, _vp]
        L.msda_group_norm_backward.restype = ctypes.c_int
        ap = ctypes.POINTER(Attention)
        L.msda_query_attention.argtypes = [ap, _vp, _vp, _vp]
        L.msda_query_attention.restype = ctypes.c_int
        L.msda_query_attention_backward_workspace_size.argtypes = [ap]
        L.msda_query_attention_backward_workspace_size.restype = ctypes.c_size_t
        L.msda_query_attention_backward.argtypes = [ap, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                    ctypes.c_size_t, _vp]
        L.msda_query_attention_backward.restype = ctypes.c_int
        L.msda_clip_grad_norm_workspace_size.argtypes = [i32]
        L.msda_clip_grad_norm_workspace_size.restype = ctypes.c_size_t
        L.msda_clip_grad_norm.argtypes = [_vp, i32, ctypes.c_float, ctypes.c_float,
                                          ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]
        L.msda_clip_grad_norm.restype = ctypes.c_int
        L.msda_status_string.argtypes = [ctypes.c_int]
        L.msda_status_string.restype = ctypes.c_char_p
        L.msda_last_error.restype = ctypes.c_char_p
        L.msda_version.restype = ctypes.c_int32
        _lib = L
    return _lib


def _check(status, name):
    if status != 0:
        L = lib()
        raise MsdaError(f"{name}: {L.msda_status_string(status).decode()}: "
                        f"{L.msda_last_error().decode()}")


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _levels(spatial_shapes, level_start_index):
    """Host int64 copies of the level tables (kept alive by the caller)."""
    torch = _torch()

    def host(a):
        if isinstance(a, torch.Tensor):
            a = a.detach().cpu().numpy()
        return np.ascontiguousarray(np.asarray(a, dtype=np.int64))
    shapes = host(spatial_shapes).reshape(-1, 2)
    if level_start_index is None:
        sizes = shapes[:, 0] * shapes[:, 1]
        level_start_index = np.concatenate([[0], np.cumsum(sizes)[:-1]])
    starts = host(level_start_index).reshape(-1)
    return shapes, starts


def _vdt(value):
    torch = _torch()
    if value.dtype == torch.float32:
        return MSDA_F32
    if value.dtype == torch.bfloat16:
        return MSDA_BF16
    raise MsdaError(f"value dtype {value.dtype} is not float32 or bfloat16")


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise MsdaError("tensors must be contiguous")


_HERE_ALREADY = contextlib.nullcontext()


def _scope(torch, name, stream, first, *others):
    """The context of a call on the tensors' device: that device current and
    `stream` (of that device), when given, the current stream, so that what is
    allocated inside belongs to the stream that the kernels run on."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            index = -1
    if index < 0:
        raise MsdaError(f"{name}: the tensors must be on one CUDA device")
    if stream is not None:
        if stream.device.index != index:
            raise MsdaError(f"{name}: the stream is on {stream.device}, the tensors on "
                            f"{first.device}")
        return torch.cuda.stream(stream)
    return _HERE_ALREADY if torch.cuda.current_device() == index else torch.cuda.device(index)


def _raw_stream(torch, tensor):
    """The handle of the tensor's device's current stream (as an integer)."""
    return torch._C._cuda_getCurrentRawStream(tensor.get_device())


def _address(t):
    return None if t is None else t.data_ptr()


def msda_forward(value, spatial_shapes, level_start_index, sampling_locations,
                 attention_weights, out=None, stream=None):
    """value [B, Nv, H, 32] (f32/bf16); locations [B, Nq, H, L, P, 2];
    weights [B, Nq, H, L, P] -> out [B, Nq, H*32] fp32."""
    torch = _torch()
    _contig(value, sampling_locations, attention_weights, out)
    B, Nv, H, _ = value.shape
    _, Nq, _, L, P, _ = sampling_locations.shape
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((B, Nq, H * HEAD_DIM), device=value.device, dtype=torch.float32)
    d = Dims(B, 1, Nq, Nv, H, L, P, 1)
    _check(lib().msda_forward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                              starts.ctypes.data_as(_i64p), _ptr(sampling_locations),
                              _ptr(attention_weights), d, _ptr(out), _stream(stream)),
           "msda_forward")
    return out


def msda_forward_fused(value, spatial_shapes, level_start_index, reference_points,
                       sampling_offsets, attention_logits, out=None, stream=None):
    """reference_points [B, Nq, R, 2]; offsets [B, Nq, H, L, P, 2] (level
    pixels); logits [B, Nq, H, L, P] -> out [B, Nq, H*32] fp32."""
    torch = _torch()
    _contig(value, reference_points, sampling_offsets, attention_logits, out)
    B, Nv, H, _ = value.shape
    _, Nq, _, L, P, _ = sampling_offsets.shape
    R = reference_points.shape[2]
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((B, Nq, H * HEAD_DIM), device=value.device, dtype=torch.float32)
    d = Dims(B, 1, Nq, Nv, H, L, P, R)
    _check(lib().msda_forward_fused(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                                    starts.ctypes.data_as(_i64p), _ptr(reference_points),
                                    _ptr(sampling_offsets), _ptr(attention_logits), d, _ptr(out),
                                    _stream(stream)),
           "msda_forward_fused")
    return out


def tsa_reference_points(ego_motion, bev_h, bev_w, grid_length=(0.512, 0.512), out=None,
                         stream=None):
    """ego_motion [B, T, 3] fp32 (dx m, dy m, yaw degrees) on the device ->
    reference points [B, T, bev_h * bev_w, 2] fp32; grid_length = (gy, gx)."""
    torch = _torch()
    _contig(ego_motion, out)
    B, T, _ = ego_motion.shape
    if out is None:
        out = torch.empty((B, T, bev_h * bev_w, 2), device=ego_motion.device,
                          dtype=torch.float32)
    gy, gx = grid_length
    _check(lib().tsa_reference_points(_ptr(ego_motion), B, T, bev_h, bev_w, float(gy), float(gx),
                                      _ptr(out), _stream(stream)),
           "tsa_reference_points")
    return out


def tsa_forward(value, spatial_shapes, level_start_index, reference_points, sampling_offsets,
                attention_logits, num_queues, out=None, stream=None):
    """value [B*T, Nv, H, 32] (item b*T + t = queue t of sample b);
    reference_points [B*T, Nq, R, 2]; offsets [B*T, Nq, H, L, P, 2];
    logits [B*T, Nq, H, L, P] -> out [B, Nq, H*32] fp32, the mean over the
    T = num_queues queues of the fused MSDA."""
    torch = _torch()
    _contig(value, reference_points, sampling_offsets, attention_logits, out)
    BT, Nv, H, _ = value.shape
    T = int(num_queues)
    if T < 1 or BT % T:
        raise MsdaError("tsa_forward: the value batch is not a multiple of num_queues")
    _, Nq, _, L, P, _ = sampling_offsets.shape
    R = reference_points.shape[2]
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((BT // T, Nq, H * HEAD_DIM), device=value.device, dtype=torch.float32)
    d = Dims(BT // T, 1, Nq, Nv, H, L, P, R)
    _check(lib().tsa_forward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                             starts.ctypes.data_as(_i64p), _ptr(reference_points),
                             _ptr(sampling_offsets), _ptr(attention_logits), T, d, _ptr(out),
                             _stream(stream)),
           "tsa_forward")
    return out


def tsa_backward(value, spatial_shapes, level_start_index, reference_points, sampling_offsets,
                 attention_logits, num_queues, grad_out, workspace=None, stream=None, out=None):
    """-> (grad_value [B*T, Nv, H, 32], grad_sampling_offsets [B*T, Nq, H, L, P, 2],
    grad_attention_logits [B*T, Nq, H, L, P], grad_reference_points [B*T, Nq, R, 2])."""
    torch = _torch()
    _contig(value, reference_points, sampling_offsets, attention_logits, grad_out)
    BT, Nv, H, _ = value.shape
    T = int(num_queues)
    if T < 1 or BT % T:
        raise MsdaError("tsa_backward: the value batch is not a multiple of num_queues")
    _, Nq, _, L, P, _ = sampling_offsets.shape
    R = reference_points.shape[2]
    shapes, starts = _levels(spatial_shapes, level_start_index)
    d = Dims(BT // T, 1, Nq, Nv, H, L, P, R)
    dev = value.device
    if out is not None:
        gv, g_off, g_lg, g_ref = out
        _contig(gv, g_off, g_lg, g_ref)
    else:
        gv = torch.empty(value.shape, device=dev, dtype=torch.float32)
        g_off = torch.empty(sampling_offsets.shape, device=dev, dtype=torch.float32)
        g_lg = torch.empty(attention_logits.shape, device=dev, dtype=torch.float32)
        g_ref = torch.empty(reference_points.shape, device=dev, dtype=torch.float32)
    workspace = _workspace(int(lib().tsa_backward_workspace_size(d, T)), dev, workspace)
    _check(lib().tsa_backward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                              starts.ctypes.data_as(_i64p), _ptr(reference_points),
                              _ptr(sampling_offsets), _ptr(attention_logits), T, _ptr(grad_out),
                              d, _ptr(workspace), workspace.numel(), _ptr(gv), _ptr(g_off),
                              _ptr(g_lg), _ptr(g_ref), _stream(stream)),
           "tsa_backward")
    return gv, g_off, g_lg, g_ref


def msda_backward(value, spatial_shapes, level_start_index, sampling_locations,
                  attention_weights, grad_out, grad_value=None, grad_sampling_locations=None,
                  grad_attention_weights=None, stream=None, deterministic=False, workspace=None):
    """-> (grad_value [B, Nv, H, 32] fp32, grad_sampling_locations,
    grad_attention_weights).  deterministic=True accumulates grad_value in
    fixed point (bitwise reproducible; needs a workspace, allocated here when
    not given)."""
    torch = _torch()
    _contig(value, sampling_locations, attention_weights, grad_out)
    B, Nv, H, _ = value.shape
    _, Nq, _, L, P, _ = sampling_locations.shape
    shapes, starts = _levels(spatial_shapes, level_start_index)
    dev = value.device
    if grad_value is None:
        grad_value = torch.empty(value.shape, device=dev, dtype=torch.float32)
    if grad_sampling_locations is None:
        grad_sampling_locations = torch.empty(sampling_locations.shape, device=dev,
                                              dtype=torch.float32)
    if grad_attention_weights is None:
        grad_attention_weights = torch.empty(attention_weights.shape, device=dev,
                                             dtype=torch.float32)
    d = Dims(B, 1, Nq, Nv, H, L, P, 1)
    args = (_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p), starts.ctypes.data_as(_i64p),
            _ptr(sampling_locations), _ptr(attention_weights), _ptr(grad_out), d)
    outs = (_ptr(grad_value), _ptr(grad_sampling_locations), _ptr(grad_attention_weights),
            _stream(stream))
    if deterministic:
        workspace = _workspace(int(lib().msda_backward_deterministic_workspace_size(d)), dev,
                               workspace)
        _check(lib().msda_backward_deterministic(*args, _ptr(workspace), workspace.numel(),
                                                 *outs), "msda_backward_deterministic")
    else:
        _check(lib().msda_backward(*args, *outs), "msda_backward")
    return grad_value, grad_sampling_locations, grad_attention_weights


def _sca_dims(value, sampling_offsets, reference_points_cam):
    B, Ncam, Nv, H, _ = value.shape
    _, Nq, _, L, P, _ = sampling_offsets.shape
    R = reference_points_cam.shape[3]
    return Dims(B, Ncam, Nq, Nv, H, L, P, R)


def msda_workspace_size(dims):
    return int(lib().msda_workspace_size(dims))


def sca_compact_workspace_size(dims):
    return int(lib().sca_compact_workspace_size(dims))


def _workspace(nbytes, device, workspace):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    return workspace


def sca_compact(bev_mask, workspace=None, stream=None, out=None):
    """bev_mask [Ncam, B, Nq, R] (uint8 / bool) -> (idx [B, Ncam, Nq],
    count [B, Ncam], pos [B, Ncam, Nq], hits [B, Nq]), int32; `out` may
    supply the four tensors."""
    torch = _torch()
    _contig(bev_mask)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    Ncam, B, Nq, R = bev_mask.shape
    dev = bev_mask.device
    if out is not None:
        idx, count, pos, hits = out
        _contig(idx, count, pos, hits)
    else:
        idx = torch.empty((B, Ncam, Nq), dtype=torch.int32, device=dev)
        count = torch.empty((B, Ncam), dtype=torch.int32, device=dev)
        pos = torch.empty((B, Ncam, Nq), dtype=torch.int32, device=dev)
        hits = torch.empty((B, Nq), dtype=torch.int32, device=dev)
    d = Dims(B, Ncam, Nq, 1, 1, 1, 1, R)
    nbytes = sca_compact_workspace_size(d)
    workspace = _workspace(nbytes, dev, workspace)
    _check(lib().sca_compact(_ptr(bev_mask), d, _ptr(workspace), workspace.numel(), _ptr(idx),
                             _ptr(count), _ptr(pos), _ptr(hits), _stream(stream)),
           "sca_compact")
    return idx, count, pos, hits


def sca_forward(value, spatial_shapes, level_start_index, reference_points_cam, bev_mask,
                sampling_offsets, attention_logits, out=None, workspace=None, stream=None):
    """value [B, Ncam, Nv, H, 32]; reference_points_cam [Ncam, B, Nq, R, 2];
    bev_mask [Ncam, B, Nq, R]; offsets [B, Nq, H, L, P, 2]; logits
    [B, Nq, H, L, P] -> out [B, Nq, H*32] fp32."""
    torch = _torch()
    _contig(value, reference_points_cam, bev_mask, sampling_offsets, attention_logits, out)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((d.B, d.Nq, d.H * HEAD_DIM), device=value.device, dtype=torch.float32)
    workspace = _workspace(msda_workspace_size(d), value.device, workspace)
    _check(lib().sca_forward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                             starts.ctypes.data_as(_i64p), _ptr(reference_points_cam),
                             _ptr(bev_mask), _ptr(sampling_offsets), _ptr(attention_logits), d,
                             _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)),
           "sca_forward")
    return out


def sca_forward_query_major(value, spatial_shapes, level_start_index, reference_points_cam,
                            bev_mask, sampling_offsets, attention_logits, out=None, stream=None):
    """sca_forward's result from one query-major kernel, without workspace."""
    torch = _torch()
    _contig(value, reference_points_cam, bev_mask, sampling_offsets, attention_logits, out)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((d.B, d.Nq, d.H * HEAD_DIM), device=value.device, dtype=torch.float32)
    _check(lib().sca_forward_query_major(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                                         starts.ctypes.data_as(_i64p), _ptr(reference_points_cam),
                                         _ptr(bev_mask), _ptr(sampling_offsets),
                                         _ptr(attention_logits), d, _ptr(out), _stream(stream)),
           "sca_forward_query_major")
    return out


def sca_backward(value, spatial_shapes, level_start_index, reference_points_cam, bev_mask,
                 sampling_offsets, attention_logits, grad_out, grad_value=None,
                 grad_sampling_locations_rb=None, grad_attention_weights_rb=None,
                 workspace=None, stream=None, deterministic=False):
    """-> (grad_value [B, Ncam, Nv, H, 32], grad_sampling_locations_rb
    [B, Ncam, Nq, H, L, P, 2], grad_attention_weights_rb [B, Ncam, Nq, H, L, P]).
    deterministic=True accumulates grad_value in fixed point (bitwise
    reproducible; the workspace then also holds the fixed-point copy)."""
    torch = _torch()
    _contig(value, reference_points_cam, bev_mask, sampling_offsets, attention_logits, grad_out)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    dev = value.device
    if grad_value is None:
        grad_value = torch.empty(value.shape, device=dev, dtype=torch.float32)
    if grad_sampling_locations_rb is None:
        grad_sampling_locations_rb = torch.empty((d.B, d.Ncam, d.Nq, d.H, d.L, d.P, 2),
                                                 device=dev, dtype=torch.float32)
    if grad_attention_weights_rb is None:
        grad_attention_weights_rb = torch.empty((d.B, d.Ncam, d.Nq, d.H, d.L, d.P), device=dev,
                                                dtype=torch.float32)
    fn = lib().sca_backward_deterministic if deterministic else lib().sca_backward
    need = (int(lib().sca_backward_deterministic_workspace_size(d)) if deterministic
            else msda_workspace_size(d))
    workspace = _workspace(need, dev, workspace)
    _check(fn(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
              starts.ctypes.data_as(_i64p), _ptr(reference_points_cam), _ptr(bev_mask),
              _ptr(sampling_offsets), _ptr(attention_logits), _ptr(grad_out), d, _ptr(workspace),
              workspace.numel(), _ptr(grad_value), _ptr(grad_sampling_locations_rb),
              _ptr(grad_attention_weights_rb), _stream(stream)),
           "sca_backward_deterministic" if deterministic else "sca_backward")
    return grad_value, grad_sampling_locations_rb, grad_attention_weights_rb


def sca_backward_full(value, spatial_shapes, level_start_index, reference_points_cam, bev_mask,
                      sampling_offsets, attention_logits, grad_out, out=None, workspace=None,
                      stream=None):
    """The SCA backward down to its inputs -> (grad_value [B, Ncam, Nv, H, 32],
    grad_sampling_offsets [B, Nq, H, L, P, 2], grad_attention_logits
    [B, Nq, H, L, P], grad_reference_points_cam [Ncam, B, Nq, R, 2]); `out`
    may supply the four tensors."""
    torch = _torch()
    _contig(value, reference_points_cam, bev_mask, sampling_offsets, attention_logits, grad_out)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    dev = value.device
    if out is not None:
        gv, g_off, g_lg, g_ref = out
        _contig(gv, g_off, g_lg, g_ref)
    else:
        gv = torch.empty(value.shape, device=dev, dtype=torch.float32)
        g_off = torch.empty(sampling_offsets.shape, device=dev, dtype=torch.float32)
        g_lg = torch.empty(attention_logits.shape, device=dev, dtype=torch.float32)
        g_ref = torch.empty(reference_points_cam.shape, device=dev, dtype=torch.float32)
    workspace = _workspace(int(lib().sca_backward_full_workspace_size(d)), dev, workspace)
    _check(lib().sca_backward_full(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                                   starts.ctypes.data_as(_i64p), _ptr(reference_points_cam),
                                   _ptr(bev_mask), _ptr(sampling_offsets), _ptr(attention_logits),
                                   _ptr(grad_out), d, _ptr(workspace), workspace.numel(),
                                   _ptr(gv), _ptr(g_off), _ptr(g_lg), _ptr(g_ref),
                                   _stream(stream)),
           "sca_backward_full")
    return gv, g_off, g_lg, g_ref


def sca_rebatched_forward(value, spatial_shapes, level_start_index, reference_points_cam,
                          sampling_offsets, attention_logits, idx, count, out_rb=None,
                          stream=None):
    """Fused MSDA of every camera's seeing queries (idx, count from
    sca_compact) -> out_rb [B, Ncam, Nq, H*32]; rows >= count untouched."""
    torch = _torch()
    _contig(value, reference_points_cam, sampling_offsets, attention_logits, idx, count, out_rb)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out_rb is None:
        out_rb = torch.empty((d.B, d.Ncam, d.Nq, d.H * HEAD_DIM), device=value.device,
                             dtype=torch.float32)
    _check(lib().sca_rebatched_forward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                                       starts.ctypes.data_as(_i64p), _ptr(reference_points_cam),
                                       _ptr(sampling_offsets), _ptr(attention_logits), _ptr(idx),
                                       _ptr(count), d, _ptr(out_rb), _stream(stream)),
           "sca_rebatched_forward")
    return out_rb


def sca_camera_average(out_rb, pos, hits, out=None, stream=None):
    """out[b, q] = sum over seeing cameras of out_rb rows / max(1, hits)."""
    torch = _torch()
    _contig(out_rb, pos, hits, out)
    B, Ncam, Nq, C = out_rb.shape
    if out is None:
        out = torch.empty((B, Nq, C), device=out_rb.device, dtype=torch.float32)
    d = Dims(B, Ncam, Nq, 1, C // HEAD_DIM, 1, 1, 1)
    _check(lib().sca_camera_average(_ptr(out_rb), _ptr(pos), _ptr(hits), d, _ptr(out),
                                    _stream(stream)),
           "sca_camera_average")
    return out


def sca_camera_average_linear(out_rb, pos, hits, w, bias=None, residual=None, out=None,
                              out_dtype=None, stream=None, dropout_p=0.0, dropout_seed=0):
    """y = residual + dropout(bf16(camera average of out_rb) w^T + bias), the
    average formed inside the tensor-core projection.  out_rb [B, Ncam, Nq, C]
    fp32; pos, hits from sca_compact; w [N, C] bf16; bias [N] fp32; residual
    [B * Nq, N] fp32 -> y [B * Nq, N] (fp32, or bf16 when out_dtype / out is
    bfloat16)."""
    torch = _torch()
    _contig(out_rb, pos, hits, w, bias, residual, out)
    if w.dtype != torch.bfloat16:
        raise MsdaError("sca_camera_average_linear takes a bfloat16 w")
    B, Ncam, Nq, C = out_rb.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((B * Nq, N), device=out_rb.device, dtype=out_dtype or torch.float32)
    ydt = MSDA_BF16 if out.dtype == torch.bfloat16 else MSDA_F32
    d = Dims(B, Ncam, Nq, 1, C // HEAD_DIM, 1, 1, 1)
    _check(lib().sca_camera_average_linear(_ptr(out_rb), _ptr(pos), _ptr(hits), d, _ptr(w),
                                           _ptr(bias), _ptr(residual), N, ydt, _ptr(out),
                                           float(dropout_p), int(dropout_seed), _stream(stream)),
           "sca_camera_average_linear")
    return out


def sca_rebatched_backward(value, spatial_shapes, level_start_index, reference_points_cam,
                           sampling_offsets, attention_logits, grad_out, idx, count, hits,
                           grad_value=None, grad_sampling_locations_rb=None,
                           grad_attention_weights_rb=None, stream=None):
    """Backward of sca_rebatched_forward + sca_camera_average on a given
    compaction -> (grad_value, grad_sampling_locations_rb, grad_attention_weights_rb)."""
    torch = _torch()
    _contig(value, reference_points_cam, sampling_offsets, attention_logits, grad_out, idx, count,
            hits)
    d = _sca_dims(value, sampling_offsets, reference_points_cam)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    dev = value.device
    if grad_value is None:
        grad_value = torch.empty(value.shape, device=dev, dtype=torch.float32)
    if grad_sampling_locations_rb is None:
        grad_sampling_locations_rb = torch.empty((d.B, d.Ncam, d.Nq, d.H, d.L, d.P, 2),
                                                 device=dev, dtype=torch.float32)
    if grad_attention_weights_rb is None:
        grad_attention_weights_rb = torch.empty((d.B, d.Ncam, d.Nq, d.H, d.L, d.P), device=dev,
                                                dtype=torch.float32)
    _check(lib().sca_rebatched_backward(_ptr(value), _vdt(value), shapes.ctypes.data_as(_i64p),
                                        starts.ctypes.data_as(_i64p), _ptr(reference_points_cam),
                                        _ptr(sampling_offsets), _ptr(attention_logits),
                                        _ptr(grad_out), _ptr(idx), _ptr(count), _ptr(hits), d,
                                        _ptr(grad_value), _ptr(grad_sampling_locations_rb),
                                        _ptr(grad_attention_weights_rb), _stream(stream)),
           "sca_rebatched_backward")
    return grad_value, grad_sampling_locations_rb, grad_attention_weights_rb


def msda_linear(x, w, bias=None, residual=None, out=None, out_dtype=None, stream=None,
                dropout_p=0.0, dropout_seed=0):
    """y = x w^T (+ bias) (+ residual) on the tensor cores.  x [M, K] bf16,
    w [N, K] bf16, bias [N] fp32, residual [M, N] fp32 -> y [M, N] (fp32, or
    bf16 when out_dtype / out is bfloat16).  dropout_p > 0 applies
    training-time dropout to x w^T + bias before the residual."""
    torch = _torch()
    _contig(x, w, bias, residual, out)
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise MsdaError("msda_linear takes bfloat16 x and w")
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), device=x.device, dtype=out_dtype or torch.float32)
    ydt = MSDA_BF16 if out.dtype == torch.bfloat16 else MSDA_F32
    _check(lib().msda_linear_dropout(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), M, N, K,
                                     ydt, _ptr(out), float(dropout_p), int(dropout_seed),
                                     _stream(stream)),
           "msda_linear")
    return out


def sca_module_forward(query, query_pos, features, w_value, b_value, w_offsets, b_offsets,
                       w_weights, b_weights, w_output, b_output, reference_points_cam, bev_mask,
                       spatial_shapes, level_start_index, num_levels, num_points,
                       value_dtype=None, out=None, workspace=None, stream=None, dropout_p=0.0,
                       dropout_seed=0, camera_embeds=None, level_embeds=None):
    """The SCA module forward: q_hat = q + output_proj(SCA(value_proj(F~),
    offsets(q + pos), weights(q + pos))).  query, query_pos [B, Nq, C] fp32;
    features [B, Ncam, Nv, C] bf16; weights bf16 [out, in]; biases fp32;
    reference_points_cam [Ncam, B, Nq, R, 2]; bev_mask [Ncam, B, Nq, R]
    -> q_hat [B, Nq, C] fp32."""
    torch = _torch()
    _contig(query, query_pos, features, w_value, w_offsets, w_weights, w_output,
            reference_points_cam, bev_mask, camera_embeds, level_embeds)
    if bev_mask.dtype == torch.bool:
        bev_mask = bev_mask.view(torch.uint8)
    B, Nq, C = query.shape
    _, Ncam, Nv, _ = features.shape
    H = C // HEAD_DIM
    R = reference_points_cam.shape[3]
    vdt = MSDA_BF16 if value_dtype == torch.bfloat16 else MSDA_F32
    d = Dims(B, Ncam, Nq, Nv, H, num_levels, num_points, R)
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if out is None:
        out = torch.empty((B, Nq, C), device=query.device, dtype=torch.float32)
    nbytes = int(lib().sca_module_workspace_size(d, vdt))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=query.device)
    prm = ScaModuleParams(*[_ptr(t) for t in (query, query_pos, features, w_value, b_value,
                                              w_offsets, b_offsets, w_weights, b_weights,
                                              w_output, b_output, reference_points_cam,
                                              bev_mask)], vdt, float(dropout_p),
                           int(dropout_seed), _ptr(camera_embeds), _ptr(level_embeds))
    _check(lib().sca_module_forward(ctypes.byref(prm), shapes.ctypes.data_as(_i64p),
                                    starts.ctypes.data_as(_i64p), d, _ptr(workspace),
                                    workspace.numel(), _ptr(out), _stream(stream)),
           "sca_module_forward")
    return out


def sca_backward_inputs(spatial_shapes, level_start_index, attention_logits, pos,
                        grad_sampling_locations_rb, grad_attention_weights_rb, num_cameras,
                        num_anchors, out=None, stream=None):
    """-> (grad_sampling_offsets [B, Nq, H, L, P, 2], grad_attention_logits
    [B, Nq, H, L, P], grad_reference_points_cam [Ncam, B, Nq, R, 2]); `out`
    may supply the three tensors."""
    torch = _torch()
    _contig(attention_logits, pos, grad_sampling_locations_rb, grad_attention_weights_rb)
    B, Nq, H, L, P = attention_logits.shape
    Ncam, R = num_cameras, num_anchors
    shapes, starts = _levels(spatial_shapes, level_start_index)
    nv = int(np.max(starts + shapes[:, 0] * shapes[:, 1]))  # value rows the levels span
    d = Dims(B, Ncam, Nq, nv, H, L, P, R)
    dev = attention_logits.device
    if out is not None:
        g_off, g_lg, g_ref = out
        _contig(g_off, g_lg, g_ref)
    else:
        g_off = torch.empty((B, Nq, H, L, P, 2), device=dev, dtype=torch.float32)
        g_lg = torch.empty((B, Nq, H, L, P), device=dev, dtype=torch.float32)
        g_ref = torch.empty((Ncam, B, Nq, R, 2), device=dev, dtype=torch.float32)
    _check(lib().sca_backward_inputs(shapes.ctypes.data_as(_i64p), starts.ctypes.data_as(_i64p),
                                     _ptr(attention_logits), _ptr(pos),
                                     _ptr(grad_sampling_locations_rb),
                                     _ptr(grad_attention_weights_rb), d, _ptr(g_off), _ptr(g_lg),
                                     _ptr(g_ref), _stream(stream)),
           "sca_backward_inputs")
    return g_off, g_lg, g_ref


def _same_dense_layout(a, b):
    """Whether a and b hold one value per element in the same order, without gaps."""
    if 0 in a.shape:
        return True
    # (of a dimension of size 1 the stride says nothing)
    order = sorted((sa, n, sb) for n, sa, sb in zip(a.shape, a.stride(), b.stride()) if n != 1)
    at = 1
    for sa, n, sb in order:
        if sa != at or sb != at:
            return False
        at *= n
    return True


def msda_clip_grad_norm(grads, max_norm, eps=1e-6, grad_scale=1.0, out=None, total_norm=None,
                        workspace=None, stream=None):
    """The gradients (a list of fp32 or bf16 tensors) scaled by grad_scale and
    clipped to the global norm max_norm, in place or into `out` (a list of the
    same shapes, fp32 or bf16) -> total_norm [1] fp32, the norm before the
    clipping.  Tensors hold their values without gaps, in any order of their
    dimensions that their outputs share."""
    torch = _torch()
    grads = list(grads)
    n = len(grads)
    outs = grads if out is None else list(out)
    if len(outs) != n:
        raise MsdaError(f"msda_clip_grad_norm: {n} gradients and {len(outs)} outputs")
    if n == 0 and total_norm is None:
        raise MsdaError("msda_clip_grad_norm: no gradients, and no total_norm to write")
    # one pass over the list per attribute, each a C-level map: of a list of
    # hundreds these lines are most of the call's host time
    every = grads if out is None else grads + outs
    Tensor, dtype_of = torch.Tensor, operator.attrgetter("dtype")
    first = every[0] if n else total_norm
    try:
        devices = set(map(Tensor.get_device, every or [first]))
    except TypeError:
        raise MsdaError("msda_clip_grad_norm: the list holds something that is no tensor (the "
                        "gradient of a parameter that has none?)") from None
    if len(devices) > 1 or devices.pop() < 0:
        raise MsdaError("msda_clip_grad_norm: the tensors must be on one CUDA device")
    codes = {torch.float32: MSDA_F32, torch.bfloat16: MSDA_BF16}
    kinds = [set(map(dtype_of, grads)), set(map(dtype_of, outs))]
    if not codes.keys() >= kinds[0] | kinds[1]:
        raise MsdaError("msda_clip_grad_norm: a tensor is neither float32 nor bfloat16")
    sizes = list(map(Tensor.numel, grads))
    if not all(map(Tensor.is_contiguous, every)):
        if not all(g.shape == o.shape and _same_dense_layout(g, o) for g, o in zip(grads, outs)):
            raise MsdaError("msda_clip_grad_norm: a tensor is not dense, or an output is not "
                            "laid out as its gradient")
    elif out is not None and sizes != list(map(Tensor.numel, outs)):
        raise MsdaError("msda_clip_grad_norm: an output has another size than its gradient")
    # msda_grad_t as four 64-bit words, the two dtypes in the last
    words = [0] * (4 * n)
    words[0::4] = map(Tensor.data_ptr, grads)
    words[1::4] = words[0::4] if out is None else map(Tensor.data_ptr, outs)
    words[2::4] = sizes
    if len(kinds[0]) < 2 and len(kinds[1]) < 2:
        words[3::4] = [codes[dtype_of(grads[0])] | codes[dtype_of(outs[0])] << 32] * n if n else []
    else:
        words[3::4] = [codes[g.dtype] | codes[o.dtype] << 32 for g, o in zip(grads, outs)]
    table = array.array("Q", words)
    with _scope(torch, "msda_clip_grad_norm", stream, first, total_norm, workspace):
        if total_norm is None:
            total_norm = torch.empty(1, device=first.device, dtype=torch.float32)
        elif total_norm.dtype != torch.float32 or total_norm.numel() != 1:
            raise MsdaError("msda_clip_grad_norm: total_norm must be one float32 value")
        workspace = _workspace(int(lib().msda_clip_grad_norm_workspace_size(n)), first.device,
                               workspace)
        _check(lib().msda_clip_grad_norm(table.buffer_info()[0], n, max_norm, eps,
                                         grad_scale, _address(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _address(total_norm), _raw_stream(torch, first)),
               "msda_clip_grad_norm")
    return total_norm


_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2}


def _arg(name, t, shape, dtypes, what):
    """An argument's shape, dtype and layout; None passes."""
    if t is None:
        return
    if t.shape != shape:
        raise MsdaError(f"{name}: {what} has the shape {list(t.shape)}, not {list(shape)}")
    if t.dtype not in dtypes:
        raise MsdaError(f"{name}: {what} is {t.dtype}")
    if not t.is_contiguous():
        raise MsdaError(f"{name}: {what} must be contiguous")


def _out(name, t, shape, dtypes, what, like):
    """An output: the given tensor, checked, or a new one of dtypes[0] beside `like`."""
    if t is None:
        return like.new_empty(shape, dtype=dtypes[0])
    _arg(name, t, shape, dtypes, what)
    return t


def _norm_args(name, x, spatial_shapes, level_start_index, num_groups, gamma, beta, activation):
    torch = _torch()
    f32, data = (torch.float32,), (torch.float32, torch.bfloat16)
    if x.dim() < 2:
        raise MsdaError(f"{name}: x must be [..., Nv, C]")
    _arg(name, x, x.shape, data, "x")
    if activation not in _ACTIVATIONS:
        raise MsdaError(f"{name}: activation {activation!r} is not none, relu or silu")
    shapes, starts = _levels(spatial_shapes, level_start_index)
    if len(starts) != len(shapes):
        raise MsdaError(f"{name}: {len(shapes)} levels and {len(starts)} starts")
    Nv, C, L, G = x.shape[-2], x.shape[-1], len(shapes), int(num_groups)
    _arg(name, gamma, (L, C), f32, "gamma")
    _arg(name, beta, (L, C), f32, "beta")
    B = 1
    for s in x.shape[:-2]:
        B *= s
    return shapes, starts, NormDims(B, Nv, C, L, G)


def msda_group_norm(x, spatial_shapes, level_start_index, num_groups, gamma=None, beta=None,
                    eps=1e-5, activation="none", out_dtype=None, out=None, mean=None, rstd=None,
                    workspace=None, stream=None):
    """Group norm and activation (none, relu, silu) of every level of the
    channels-last rows x [..., Nv, C] (fp32 or bf16), gamma and beta [L, C]
    fp32 -> (y [..., Nv, C] of out_dtype, by default x's; mean and rstd
    [..., L, num_groups] fp32, for the backward).  Rows of no level get 0."""
    torch = _torch()
    name = "msda_group_norm"
    shapes, starts, d = _norm_args(name, x, spatial_shapes, level_start_index, num_groups, gamma,
                                   beta, activation)
    f32, data = (torch.float32,), (torch.float32, torch.bfloat16)
    small = tuple(x.shape[:-2]) + (d.L, d.G)
    with _scope(torch, name, stream, x, gamma, beta, out, mean, rstd, workspace):
        y = _out(name, out, x.shape, data if out is not None else (out_dtype or x.dtype,), "out",
                 x)
        if out_dtype is not None and y.dtype != out_dtype:
            raise MsdaError(f"{name}: out is {y.dtype}, not {out_dtype}")
        mean = _out(name, mean, small, f32, "mean", x)
        rstd = _out(name, rstd, small, f32, "rstd", x)
        workspace = _workspace(int(lib().msda_group_norm_workspace_size(d)), x.device, workspace)
        _check(lib().msda_group_norm(_address(x), _vdt(x), shapes.ctypes.data,
                                     starts.ctypes.data, d, _address(gamma), _address(beta),
                                     eps, _ACTIVATIONS[activation], _vdt(y), _address(y), _address(mean),
                                     _address(rstd), _address(workspace), workspace.numel(),
                                     _raw_stream(torch, x)), name)
    return y, mean, rstd


def msda_group_norm_backward(x, spatial_shapes, level_start_index, num_groups, mean, rstd,
                             grad_out, gamma=None, beta=None, activation="none", out_dtype=None,
                             out=None, workspace=None, stream=None):
    """-> (grad_x [..., Nv, C] of out_dtype, by default x's; grad_gamma and
    grad_beta [L, C] fp32); `out` may supply the three tensors.  mean and rstd
    come from msda_group_norm."""
    torch = _torch()
    name = "msda_group_norm_backward"
    shapes, starts, d = _norm_args(name, x, spatial_shapes, level_start_index, num_groups, gamma,
                                   beta, activation)
    f32, data = (torch.float32,), (torch.float32, torch.bfloat16)
    small = tuple(x.shape[:-2]) + (d.L, d.G)
    _arg(name, mean, small, f32, "mean")
    _arg(name, rstd, small, f32, "rstd")
    _arg(name, grad_out, x.shape, data, "grad_out")
    gx, gg, gb = out if out is not None else (None, None, None)
    with _scope(torch, name, stream, x, gamma, beta, mean, rstd, grad_out, gx, gg, gb, workspace):
        gx = _out(name, gx, x.shape, data if gx is not None else (out_dtype or x.dtype,), "grad_x",
                  x)
        if out_dtype is not None and gx.dtype != out_dtype:
            raise MsdaError(f"{name}: grad_x is {gx.dtype}, not {out_dtype}")
        gg = _out(name, gg, (d.L, d.C), f32, "grad_gamma", x)
        gb = _out(name, gb, (d.L, d.C), f32, "grad_beta", x)
        workspace = _workspace(int(lib().msda_group_norm_backward_workspace_size(d)), x.device,
                               workspace)
        _check(lib().msda_group_norm_backward(
            _address(x), _vdt(x), shapes.ctypes.data, starts.ctypes.data, d,
            _address(gamma), _address(beta), _address(mean), _address(rstd), _ACTIVATIONS[activation],
            _address(grad_out), _vdt(grad_out), _vdt(gx), _address(gx), _address(gg), _address(gb),
            _address(workspace), workspace.numel(), _raw_stream(torch, x)), name)
    return gx, gg, gb


def _rows_stride(name, t, what):
    """Values between the rows of a [B, N, H, 32] tensor whose rows are dense
    and whose items follow one another, such as a slice of a joint projection."""
    torch = _torch()
    if t.dim() != 4 or t.shape[3] != HEAD_DIM:
        raise MsdaError(f"{name}: {what} must be [B, N, H, {HEAD_DIM}]")
    if t.dtype != torch.bfloat16:
        raise MsdaError(f"{name}: {what} is {t.dtype}, not bfloat16")
    B, N, H, _ = t.shape
    sb, sn, sh, sd = t.stride()
    row = sn if N > 1 else sb if B > 1 else H * HEAD_DIM
    if t.numel() and (sd != 1 or (H > 1 and sh != HEAD_DIM) or (B > 1 and sb != N * row)):
        raise MsdaError(f"{name}: the rows of {what} must be dense and evenly spaced")
    return row


def _attention_args(name, q, k, v, q_points, k_points, tau, q_group, k_group, scale):
    torch = _torch()
    strides = [_rows_stride(name, t, w) for t, w in ((q, "q"), (k, "k"), (v, "v"))]
    (B, Nq, H, _), Nk = q.shape, k.shape[1]
    if k.shape != (B, Nk, H, HEAD_DIM) or v.shape != k.shape:
        raise MsdaError(f"{name}: q, k and v are {list(q.shape)}, {list(k.shape)}, {list(v.shape)}")
    f32, i32 = (torch.float32,), (torch.int32,)
    _arg(name, q_points, (B, Nq, 2), f32, "q_points")
    _arg(name, k_points, (B, Nk, 2), f32, "k_points")
    _arg(name, tau, (B, Nq, H), f32, "tau")
    _arg(name, q_group, (B, Nq), i32, "q_group")
    _arg(name, k_group, (B, Nk), i32, "k_group")
    if len({t is None for t in (q_points, k_points, tau)}) > 1:
        raise MsdaError(f"{name}: q_points, k_points and tau go together")
    if (q_group is None) != (k_group is None):
        raise MsdaError(f"{name}: q_group and k_group go together")
    return Attention(_address(q), _address(k), _address(v), *strides, _address(q_points), _address(k_points),
                     _address(tau), _address(q_group), _address(k_group),
                     HEAD_DIM ** -0.5 if scale is None else scale, B, Nq, Nk, H)


def msda_query_attention(q, k, v, q_points=None, k_points=None, tau=None, q_group=None,
                         k_group=None, scale=None, out=None, lse=None, stream=None):
    """Attention of the queries q [B, Nq, H, 32] to k and v [B, Nk, H, 32]
    (bf16; rows may be slices of a wider projection), the scores lowered by
    tau [B, Nq, H] times the distance of q_points [B, Nq, 2] and k_points
    [B, Nk, 2] (fp32), a query seeing the keys of its own group and of group 0
    (q_group [B, Nq], k_group [B, Nk] int32; negative: padding); scale is
    32^-1/2 by default -> (out [B, Nq, H * 32] bf16, lse [B, H, Nq] fp32)."""
    torch = _torch()
    name = "msda_query_attention"
    p = _attention_args(name, q, k, v, q_points, k_points, tau, q_group, k_group, scale)
    with _scope(torch, name, stream, q, k, v, q_points, k_points, tau, q_group, k_group, out, lse):
        out = _out(name, out, (p.B, p.Nq, p.H * HEAD_DIM), (torch.bfloat16,), "out", q)
        lse = _out(name, lse, (p.B, p.H, p.Nq), (torch.float32,), "lse", q)
        _check(lib().msda_query_attention(p, _address(out), _address(lse), _raw_stream(torch, q)),
               name)
    return out, lse


def msda_query_attention_backward(q, k, v, lse, grad_out, q_points=None, k_points=None, tau=None,
                                  q_group=None, k_group=None, scale=None, out=None,
                                  workspace=None, stream=None):
    """-> (grad_q [B, Nq, H, 32], grad_k and grad_v [B, Nk, H, 32] bf16,
    grad_tau [B, Nq, H] fp32 or None without tau); lse comes from the forward
    of the same inputs, grad_out [B, Nq, H * 32] is bf16, `out` may supply the
    gradients.  The points get none."""
    torch = _torch()
    name = "msda_query_attention_backward"
    p = _attention_args(name, q, k, v, q_points, k_points, tau, q_group, k_group, scale)
    b16, f32 = (torch.bfloat16,), (torch.float32,)
    _arg(name, lse, (p.B, p.H, p.Nq), f32, "lse")
    _arg(name, grad_out, (p.B, p.Nq, p.H * HEAD_DIM), b16, "grad_out")
    gq, gk, gv, gt = out if out is not None else (None,) * 4
    with _scope(torch, name, stream, q, k, v, q_points, k_points, tau, q_group, k_group, lse, grad_out,
                gq, gk, gv, gt, workspace):
        gq = _out(name, gq, q.shape, b16, "grad_q", q)
        gk = _out(name, gk, k.shape, b16, "grad_k", q)
        gv = _out(name, gv, v.shape, b16, "grad_v", q)
        gt = _out(name, gt, tau.shape, f32, "grad_tau", q) if tau is not None else None
        need = int(lib().msda_query_attention_backward_workspace_size(p))
        workspace = _workspace(need, q.device, workspace)
        _check(lib().msda_query_attention_backward(
            p, _address(lse), _address(grad_out), _address(gq), _address(gk), _address(gv), _address(gt),
            _address(workspace), workspace.numel(), _raw_stream(torch, q)), name)
    return gq, gk, gv, gt
