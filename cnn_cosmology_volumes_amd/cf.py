"""ctypes binding of libcf.so (include/cf.h), one Python function per C entry
point with the same name.  Argument marshalling only: shapes are read from
torch tensors, outputs and workspaces are allocated with torch on the
tensors' device, the call goes to the library on torch's current stream, and
a non-zero status raises CfError.  Every step of the computation runs in the
library's HIP kernels; there is no other code path.

cf_groupnorm_fwd / _bwd, cf_linear_fwd / _bwd, cf_resnorm_fwd / _bwd,
cf_grad_clip, cf_newton_schulz and cf_muon check that tensors are on the current
GPU.  With stream=s they make their outputs in s's memory; order s
after what wrote the inputs, and the current stream after s before it reads the
outputs (wait_stream).
"""
import array
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcf.so")

CF_OK, CF_ERR_INVALID, CF_ERR_UNSUPPORTED, CF_ERR_WORKSPACE, CF_ERR_HIP = 0, -1, -2, -3, -4
CF_F32, CF_BF16 = 0, 1
CF_CONV_FWD, CF_CONV_BWD_DATA, CF_CONV_BWD_WEIGHT, CF_CONV_POOL_FWD, CF_POOL_CONV_BWD_WEIGHT = 0, 1, 2, 3, 4
CF_MAX_BLOCKS = 8
CF_MAX_OPT_TENSORS = 32


class CfError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s (status %d): %s" % (_status_name(status), status, msg))
        self.status = status


class cf_dims(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("d", ctypes.c_int64), ("h", ctypes.c_int64),
                ("w", ctypes.c_int64), ("c", ctypes.c_int64)]


class cf_conv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("stride", ctypes.c_int32), ("pad", ctypes.c_int32)]


class cf_model_desc(ctypes.Structure):
    _fields_ = [("nblocks", ctypes.c_int32), ("cin", ctypes.c_int32), ("d", ctypes.c_int32),
                ("h", ctypes.c_int32), ("w", ctypes.c_int32),
                ("filters", ctypes.c_int32 * CF_MAX_BLOCKS), ("dense", ctypes.c_int32 * 3),
                ("slope", ctypes.c_float)]


class cf_step_aux(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("fork", ctypes.c_void_p * CF_MAX_BLOCKS), ("join", ctypes.c_void_p)]


class cf_adam_larc_params(ctypes.Structure):
    _fields_ = [("lr0", ctypes.c_float), ("lr_end", ctypes.c_float), ("decay_steps", ctypes.c_int64),
                ("power", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("trust", ctypes.c_float)]


CF_MAX_DENSE = 4
CF_POOL_MAX, CF_POOL_AVG, CF_POOL_NONE = 0, 1, 2
CF_OPT_SGD, CF_OPT_ADAM_LARC = 0, 1
CF_ACT_LRELU, CF_ACT_SILU = 0, 1
CF_MUON_SCALE_ASPECT, CF_MUON_SCALE_RMS = 0, 1
CF_NORM_RMS, CF_NORM_LAYER = 0, 1
CF_MAX_CLIP_TENSORS = 1024


class cf_net_desc(ctypes.Structure):
    _fields_ = [("nlayers", ctypes.c_int32), ("cin", ctypes.c_int32), ("d", ctypes.c_int32), ("h", ctypes.c_int32),
                ("w", ctypes.c_int32), ("filters", ctypes.c_int32 * CF_MAX_BLOCKS),
                ("stride", ctypes.c_int32 * CF_MAX_BLOCKS), ("pool", ctypes.c_int32 * CF_MAX_BLOCKS),
                ("batch_norm", ctypes.c_int32), ("bn_eps", ctypes.c_float), ("ndense", ctypes.c_int32),
                ("dense", ctypes.c_int32 * CF_MAX_DENSE), ("dense_bias", ctypes.c_int32), ("slope", ctypes.c_float)]


class cf_optimizer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("lr", ctypes.c_float), ("adam", cf_adam_larc_params),
                ("t", ctypes.c_int64)]


class cf_newton_schulz_params(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("eps", ctypes.c_float)]


class cf_muon_params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_int32), ("ns", cf_newton_schulz_params)]


class cf_resnorm_params(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
                ("gpre", ctypes.c_void_p), ("bpre", ctypes.c_void_p), ("gpost", ctypes.c_void_p),
                ("bpost", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_n", ctypes.c_int32)]


_P = ctypes.c_void_p
_PI64 = ctypes.POINTER(ctypes.c_int64)
_SIG = {
    "cf_abi_version": ([], ctypes.c_int32),
    "cf_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "cf_last_error": ([], ctypes.c_char_p),
    "cf_conv3d_workspace_size": ([ctypes.c_int, cf_dims, ctypes.c_int32, cf_conv, ctypes.c_int], ctypes.c_size_t),
    "cf_conv3d_fwd": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, cf_conv, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_conv3d_bwd_data": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, cf_conv, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_conv3d_bwd_weight": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, cf_conv, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_conv3d_bwd_weight_noalloc": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, cf_conv, _P, _P], ctypes.c_int),
    "cf_conv3d_pool_fwd": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, cf_conv, ctypes.c_float, _P, _P, _P,
                            ctypes.c_size_t, _P], ctypes.c_int),
    "cf_pool_conv3d_bwd_weight": ([ctypes.c_int, cf_dims, _P, _P, _P, _P, ctypes.c_int32, cf_conv, ctypes.c_float, _P,
                                   _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_pool3d_fwd": ([ctypes.c_int, cf_dims, _P, ctypes.c_float, _P, _P, _P], ctypes.c_int),
    "cf_pool3d_bwd": ([ctypes.c_int, cf_dims, _P, _P, _P, ctypes.c_float, _P, _P], ctypes.c_int),
    "cf_avgpool3d_fwd": ([ctypes.c_int, cf_dims, _P, ctypes.c_float, _P, _P], ctypes.c_int),
    "cf_avgpool3d_bwd": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_float, _P, _P], ctypes.c_int),
    "cf_lrelu": ([ctypes.c_int, ctypes.c_int64, _P, _P, ctypes.c_float, _P, _P], ctypes.c_int),
    "cf_dense_workspace_size": ([ctypes.c_int32] * 3, ctypes.c_size_t),
    "cf_dense_fwd": ([ctypes.c_int32] * 3 + [_P, _P, _P, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_dense_bwd": ([ctypes.c_int32] * 3 + [_P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P], ctypes.c_int),
    "cf_mse": ([ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _P], ctypes.c_int),
    "cf_sgd": ([ctypes.c_int64, ctypes.c_float, _P, _P, _P], ctypes.c_int),
    "cf_adam_larc_workspace_size": ([ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)], ctypes.c_size_t),
    "cf_adam_larc": ([ctypes.POINTER(cf_adam_larc_params), ctypes.c_int64, ctypes.c_int32,
                      ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P),
                      ctypes.POINTER(_P), _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_batchnorm_workspace_size": ([ctypes.c_int, cf_dims], ctypes.c_size_t),
    "cf_batchnorm_fwd": ([ctypes.c_int, cf_dims, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P],
                         ctypes.c_int),
    "cf_batchnorm_bwd": ([ctypes.c_int, cf_dims, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
                         ctypes.c_int),
    "cf_groupnorm_workspace_size": ([ctypes.c_int, cf_dims, ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
    "cf_groupnorm_fwd": ([ctypes.c_int, cf_dims, _P, ctypes.c_int32, _P, _P, ctypes.c_float, ctypes.c_int,
                          ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_groupnorm_bwd": ([ctypes.c_int, cf_dims, _P, _P, ctypes.c_int32, _P, _P, _P, _P, ctypes.c_int,
                          ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_newton_schulz_workspace_size": ([ctypes.c_int, ctypes.c_int32, _PI64, _PI64], ctypes.c_size_t),
    "cf_newton_schulz": ([ctypes.POINTER(cf_newton_schulz_params), ctypes.c_int, ctypes.c_int32, _PI64, _PI64,
                          ctypes.POINTER(_P), ctypes.POINTER(_P), _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_muon_workspace_size": ([ctypes.POINTER(cf_muon_params), ctypes.c_int32, _PI64, _PI64], ctypes.c_size_t),
    "cf_muon": ([ctypes.POINTER(cf_muon_params), ctypes.c_int32, _PI64, _PI64, ctypes.POINTER(_P),
                 ctypes.POINTER(_P), ctypes.POINTER(_P), _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_linear_workspace_size": ([ctypes.c_int, ctypes.c_int64] + [ctypes.c_int32] * 3, ctypes.c_size_t),
    "cf_linear_fwd": ([ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, ctypes.c_int,
                       ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_linear_bwd": ([ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, ctypes.c_int,
                       ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "cf_resnorm_workspace_size": ([ctypes.c_int, cf_dims, ctypes.c_int32], ctypes.c_size_t),
    "cf_resnorm_fwd": ([ctypes.c_int, cf_dims, ctypes.POINTER(cf_resnorm_params), _P, _P, _P, _P, _P], ctypes.c_int),
    "cf_resnorm_bwd": ([ctypes.c_int, cf_dims, ctypes.POINTER(cf_resnorm_params)] + [_P] * 12 + [ctypes.c_size_t, _P],
                       ctypes.c_int),
    "cf_grad_clip_workspace_size": ([ctypes.c_int, ctypes.c_int32, _P], ctypes.c_size_t),
    "cf_grad_clip": ([ctypes.c_int, ctypes.c_int32, _P, _P, _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P],
                     ctypes.c_int),
    "cf_net_param_count": ([ctypes.POINTER(cf_net_desc), ctypes.POINTER(ctypes.c_int64)], ctypes.c_int32),
    "cf_net_train_step_workspace_size": ([ctypes.POINTER(cf_net_desc), ctypes.c_int, ctypes.c_int32], ctypes.c_size_t),
    "cf_net_train_step": ([ctypes.POINTER(cf_net_desc), ctypes.c_int, ctypes.c_int32, _P, _P, ctypes.POINTER(_P),
                           ctypes.POINTER(cf_optimizer), ctypes.POINTER(_P), ctypes.POINTER(_P), _P, _P, _P,
                           ctypes.c_size_t, _P], ctypes.c_int),
    "cf_train_step_workspace_size": ([ctypes.POINTER(cf_model_desc), ctypes.c_int, ctypes.c_int32], ctypes.c_size_t),
    "cf_step_aux_create": ([ctypes.POINTER(cf_step_aux)], ctypes.c_int),
    "cf_step_aux_destroy": ([ctypes.POINTER(cf_step_aux)], ctypes.c_int),
    "cf_train_step": ([ctypes.POINTER(cf_model_desc), ctypes.c_int, ctypes.c_int32, _P, _P, ctypes.POINTER(_P),
                       ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P, ctypes.POINTER(cf_step_aux)], ctypes.c_int),
}

_lib = None


def lib():
    """The loaded libcf.so.  Raises if it has not been built: there is no
    fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libcf.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIG.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _status_name(s):
    return {0: "CF_OK", -1: "CF_ERR_INVALID", -2: "CF_ERR_UNSUPPORTED", -3: "CF_ERR_WORKSPACE",
            -4: "CF_ERR_HIP"}.get(s, "?")


def check(status):
    if status != CF_OK:
        raise CfError(status, lib().cf_last_error().decode())


def dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return CF_F32
    if t == torch.bfloat16:
        return CF_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t)


def _ptr(t):
    return None if t is None else t.data_ptr()


# (torch.cuda.current_stream builds a Stream object, which takes longer than a small kernel's launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def dims(shape) -> cf_dims:
    n, d, h, w, c = (int(v) for v in shape)
    return cf_dims(n, d, h, w, c)


CONV3 = cf_conv(3, 1, 1)


def conv_geometry(stride, size):
    """cf_conv for a 3^3 convolution of the given stride with "same" padding
    on a volume whose sizes have the parity of `size`."""
    if stride == 1:
        return CONV3
    return cf_conv(3, 2, int(size) & 1)


def out_shape(shape, cout, stride):
    n, d, h, w, _ = (int(v) for v in shape)
    if stride == 1:
        return (n, d, h, w, cout)
    return (n, (d + 1) // 2, (h + 1) // 2, (w + 1) // 2, cout)


def _ws(nbytes, device, ws=None):
    if nbytes == 0:
        return ws
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _wsbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# --------------------------------------------------------------------- conv
def cf_conv3d_workspace_size(dtype, xshape, cout, pass_, stride=1):
    geom = conv_geometry(stride, xshape[1])
    return int(lib().cf_conv3d_workspace_size(dtype, dims(xshape), int(cout), geom, int(pass_)))


def cf_conv3d_fwd(X, W, Y=None, ws=None, stream=None, stride=1):
    """X [N,D,H,W,Cin], W [3,3,3,Cin,Cout] (same dtype) -> Y [N,D,H,W,Cout]
    (stride 2: "same" padding, output ceil(D/2) etc.)."""
    dt = dtype_code(X.dtype)
    cout = int(W.shape[4])
    if Y is None:
        Y = torch.empty(out_shape(X.shape, cout, stride), dtype=X.dtype, device=X.device)
    ws = _ws(cf_conv3d_workspace_size(dt, X.shape, cout, CF_CONV_FWD, stride), X.device, ws)
    check(lib().cf_conv3d_fwd(dt, dims(X.shape), _ptr(X), _ptr(W), cout, conv_geometry(stride, X.shape[1]), _ptr(Y),
                              _ptr(ws), _wsbytes(ws), _stream(stream)))
    return Y


def cf_conv3d_bwd_data(dY, W, dX=None, ws=None, stream=None, xshape=None, stride=1):
    """dY [N,D,H,W,Cout], W [3,3,3,Cin,Cout] -> dX [N,D,H,W,Cin]; with
    stride 2, xshape is the forward input's shape."""
    dt = dtype_code(dY.dtype)
    cin, cout = int(W.shape[3]), int(W.shape[4])
    if xshape is None:
        xshape = tuple(dY.shape[:4]) + (cin,)
    xshape = tuple(int(v) for v in xshape)
    if dX is None:
        dX = torch.empty(xshape, dtype=dY.dtype, device=dY.device)
    ws = _ws(cf_conv3d_workspace_size(dt, xshape, cout, CF_CONV_BWD_DATA, stride), dY.device, ws)
    check(lib().cf_conv3d_bwd_data(dt, dims(xshape), _ptr(dY), _ptr(W), cout, conv_geometry(stride, xshape[1]),
                                   _ptr(dX), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return dX


def cf_conv3d_bwd_weight(X, dY, dW=None, ws=None, stream=None, stride=1):
    """X [N,D,H,W,Cin], dY [N,Do,Ho,Wo,Cout] -> dW [3,3,3,Cin,Cout] fp32."""
    dt = dtype_code(X.dtype)
    cout = int(dY.shape[4])
    if dW is None:
        dW = torch.empty((3, 3, 3, int(X.shape[4]), cout), dtype=torch.float32, device=X.device)
    ws = _ws(cf_conv3d_workspace_size(dt, X.shape, cout, CF_CONV_BWD_WEIGHT, stride), X.device, ws)
    check(lib().cf_conv3d_bwd_weight(dt, dims(X.shape), _ptr(X), _ptr(dY), cout, conv_geometry(stride, X.shape[1]),
                                     _ptr(dW), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return dW


def cf_conv3d_bwd_weight_noalloc(X, dY, dW, stream=None):
    """As cf_conv3d_bwd_weight, with no workspace: the library's static
    per-device scratch holds the partial sums.  dW must be given (the call
    allocates nothing)."""
    dt = dtype_code(X.dtype)
    cout = int(dY.shape[4])
    check(lib().cf_conv3d_bwd_weight_noalloc(dt, dims(X.shape), _ptr(X), _ptr(dY), cout, CONV3, _ptr(dW),
                                             _stream(stream)))
    return dW


def cf_conv3d_pool_fwd(X, W, slope, P=None, idx=None, ws=None, stream=None):
    """Fused block forward: pool(lrelu(conv(X, W))) -> (P, idx)."""
    dt = dtype_code(X.dtype)
    cout = int(W.shape[4])
    N, D, H, Wd = (int(v) for v in X.shape[:4])
    pshape = (N, D // 2, H // 2, Wd // 2, cout)
    if P is None:
        P = torch.empty(pshape, dtype=X.dtype, device=X.device)
    if idx is None:
        idx = torch.empty(pshape, dtype=torch.uint8, device=X.device)
    ws = _ws(cf_conv3d_workspace_size(dt, X.shape, cout, CF_CONV_POOL_FWD), X.device, ws)
    check(lib().cf_conv3d_pool_fwd(dt, dims(X.shape), _ptr(X), _ptr(W), cout, CONV3, float(slope), _ptr(P), _ptr(idx),
                                   _ptr(ws), _wsbytes(ws), _stream(stream)))
    return P, idx


def cf_pool_conv3d_bwd_weight(X, dP, P, idx, slope, dW=None, ws=None, stream=None):
    """Fused block weight gradient: wgrad(X, pool_bwd(dP, P, idx)) -> dW fp32."""
    dt = dtype_code(X.dtype)
    cout = int(dP.shape[4])
    if dW is None:
        dW = torch.empty((3, 3, 3, int(X.shape[4]), cout), dtype=torch.float32, device=X.device)
    ws = _ws(cf_conv3d_workspace_size(dt, X.shape, cout, CF_POOL_CONV_BWD_WEIGHT), X.device, ws)
    check(lib().cf_pool_conv3d_bwd_weight(dt, dims(X.shape), _ptr(X), _ptr(dP), _ptr(P), _ptr(idx), cout, CONV3,
                                          float(slope), _ptr(dW), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return dW


# --------------------------------------------------------------------- pool
def cf_pool3d_fwd(Z, slope, P=None, idx=None, stream=None):
    """Z [N,D,H,W,C] -> (P [N,D/2,H/2,W/2,C], idx uint8)."""
    dt = dtype_code(Z.dtype)
    N, D, H, W, C = (int(v) for v in Z.shape)
    pshape = (N, D // 2, H // 2, W // 2, C)
    if P is None:
        P = torch.empty(pshape, dtype=Z.dtype, device=Z.device)
    if idx is None:
        idx = torch.empty(pshape, dtype=torch.uint8, device=Z.device)
    check(lib().cf_pool3d_fwd(dt, dims(Z.shape), _ptr(Z), float(slope), _ptr(P), _ptr(idx), _stream(stream)))
    return P, idx


def cf_pool3d_bwd(dP, P, idx, slope, dZ=None, stream=None):
    dt = dtype_code(dP.dtype)
    N, Dp, Hp, Wp, C = (int(v) for v in dP.shape)
    zshape = (N, 2 * Dp, 2 * Hp, 2 * Wp, C)
    if dZ is None:
        dZ = torch.empty(zshape, dtype=dP.dtype, device=dP.device)
    check(lib().cf_pool3d_bwd(dt, dims(zshape), _ptr(dP), _ptr(P), _ptr(idx), float(slope), _ptr(dZ),
                              _stream(stream)))
    return dZ


def cf_avgpool3d_fwd(Z, slope, P=None, stream=None):
    """Z [N,D,H,W,C] -> P [N,D/2,H/2,W/2,C] = mean over 2^3 of lrelu(Z)."""
    dt = dtype_code(Z.dtype)
    N, D, H, W, C = (int(v) for v in Z.shape)
    if P is None:
        P = torch.empty((N, D // 2, H // 2, W // 2, C), dtype=Z.dtype, device=Z.device)
    check(lib().cf_avgpool3d_fwd(dt, dims(Z.shape), _ptr(Z), float(slope), _ptr(P), _stream(stream)))
    return P


def cf_avgpool3d_bwd(dP, Z, slope, dZ=None, stream=None):
    dt = dtype_code(Z.dtype)
    if dZ is None:
        dZ = torch.empty_like(Z)
    check(lib().cf_avgpool3d_bwd(dt, dims(Z.shape), _ptr(dP), _ptr(Z), float(slope), _ptr(dZ), _stream(stream)))
    return dZ


def cf_lrelu(x, slope, dy=None, out=None, stream=None):
    dt = dtype_code(x.dtype)
    if out is None:
        out = torch.empty_like(x)
    check(lib().cf_lrelu(dt, x.numel(), _ptr(x), _ptr(dy), float(slope), _ptr(out), _stream(stream)))
    return out


# -------------------------------------------------------------------- dense
def cf_dense_fwd(X, W, b, slope, pre=None, Y=None, ws=None, stream=None):
    """X [B,in] fp32, W [in,out], b [out] or None -> (pre, Y)."""
    B, fin = (int(v) for v in X.shape)
    fout = int(W.shape[1])
    if pre is None:
        pre = torch.empty((B, fout), dtype=torch.float32, device=X.device)
    if Y is None:
        Y = torch.empty((B, fout), dtype=torch.float32, device=X.device)
    ws = _ws(int(lib().cf_dense_workspace_size(B, fin, fout)), X.device, ws)
    check(lib().cf_dense_fwd(B, fin, fout, _ptr(X), _ptr(W), _ptr(b), float(slope), _ptr(pre), _ptr(Y), _ptr(ws),
                             _wsbytes(ws), _stream(stream)))
    return pre, Y


def cf_dense_bwd(X, W, pre, dY, slope, need_dx=True, stream=None):
    B, fin = (int(v) for v in X.shape)
    fout = int(W.shape[1])
    dX = torch.empty((B, fin), dtype=torch.float32, device=X.device) if need_dx else None
    dW = torch.empty((fin, fout), dtype=torch.float32, device=X.device)
    db = torch.empty((fout,), dtype=torch.float32, device=X.device)
    check(lib().cf_dense_bwd(B, fin, fout, _ptr(X), _ptr(W), _ptr(pre), _ptr(dY), float(slope), _ptr(dX), _ptr(dW),
                             _ptr(db), _stream(stream)))
    return dX, dW, db


def cf_mse(yhat, t, stream=None):
    """-> (loss [1] device tensor, dyhat)."""
    B, K = (int(v) for v in yhat.shape)
    loss = torch.empty((1,), dtype=torch.float32, device=yhat.device)
    dy = torch.empty_like(yhat)
    check(lib().cf_mse(B, K, _ptr(yhat), _ptr(t), _ptr(loss), _ptr(dy), _stream(stream)))
    return loss, dy


def cf_sgd(W, dW, lr, stream=None):
    """In place: W -= lr * dW (fp32)."""
    check(lib().cf_sgd(W.numel(), float(lr), _ptr(W), _ptr(dW), _stream(stream)))
    return W


# -------------------------------------------------------------- train step
def model_desc(in_channels, size, filters, dense=(128, 64, 3), slope=0.3):
    """cf_model_desc for a cubic input (or size = (d, h, w))."""
    m = cf_model_desc()
    d, h, w = (size, size, size) if isinstance(size, int) else size
    m.nblocks, m.cin, m.d, m.h, m.w = len(filters), in_channels, d, h, w
    for i, f in enumerate(filters):
        m.filters[i] = f
    for i, f in enumerate(dense):
        m.dense[i] = f
    m.slope = slope
    return m


def cf_train_step_workspace_size(m, dtype, B):
    return int(lib().cf_train_step_workspace_size(ctypes.byref(m), dtype, int(B)))


class StepAux:
    """A cf_step_aux (second stream and events for cf_train_step) created on
    the current device; destroyed with the object or by close()."""

    def __init__(self):
        self.aux = cf_step_aux()
        check(lib().cf_step_aux_create(ctypes.byref(self.aux)))

    def close(self):
        if self.aux is not None:
            torch.cuda.synchronize()
            check(lib().cf_step_aux_destroy(ctypes.byref(self.aux)))
            self.aux = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def cf_train_step(m, X, targets, params, lr, ws=None, loss=None, pred=None, stream=None, aux=None):
    """One training step; `params` (fp32 masters: conv W per block, then W1,
    b1, W2, b2, W3, b3) are updated in place.  `aux`: a StepAux whose stream
    runs the weight gradients beside the rest of the backward pass, or None
    (everything on one stream).  Returns (loss, pred)."""
    dt = dtype_code(X.dtype)
    B = int(X.shape[0])
    ws = _ws(cf_train_step_workspace_size(m, dt, B), X.device, ws)
    if loss is None:
        loss = torch.empty((1,), dtype=torch.float32, device=X.device)
    arr = (_P * len(params))(*[p.data_ptr() for p in params])
    auxp = None if aux is None else ctypes.byref(aux.aux)
    check(lib().cf_train_step(ctypes.byref(m), dt, B, _ptr(X), _ptr(targets), arr, float(lr), _ptr(loss), _ptr(pred),
                              _ptr(ws), _wsbytes(ws), _stream(stream), auxp))
    return loss, pred


# ---------------------------------------------------------------- optimizer
def adam_larc_params(lr0, lr_end=None, decay_steps=1, power=1.0, beta1=0.9, beta2=0.999, eps=1e-8, trust=0.0):
    """cf_adam_larc_params; lr_end defaults to lr0 (no decay)."""
    return cf_adam_larc_params(float(lr0), float(lr0 if lr_end is None else lr_end), int(decay_steps), float(power),
                               float(beta1), float(beta2), float(eps), float(trust))


def cf_adam_larc(hp, t, params, grads, m, v, lr_out=None, ws=None, stream=None):
    """Update t (1-based) of the fp32 tensors `params` in place from `grads`,
    with Adam moments m, v (same shapes, updated in place)."""
    k = len(params)
    n = (ctypes.c_int64 * k)(*[p.numel() for p in params])
    arr = lambda ts: (_P * k)(*[q.data_ptr() for q in ts])
    ws = _ws(int(lib().cf_adam_larc_workspace_size(k, n)), params[0].device, ws)
    check(lib().cf_adam_larc(ctypes.byref(hp), int(t), k, n, arr(params), arr(grads), arr(m), arr(v), _ptr(lr_out),
                             _ptr(ws), _wsbytes(ws), _stream(stream)))


def cf_grad_clip(grads, max_norm, out=None, stats=None, ws=None, stream=None):
    """Scales gradients (all fp32 or all bf16, at most CF_MAX_CLIP_TENSORS), in
    place or into the tensors of `out` (each of its gradient's shape), to a global
    norm of at most max_norm (an fp32 value; math.inf: measures only) -> [norm,
    factor], two floats on the GPU."""
    k = len(grads)
    if not k or (out is not None and len(out) != k):
        raise ValueError("grads must not be empty, and out be as long")
    if stream is not None:
        return _on_stream(stream, cf_grad_clip, (*grads, *(out or ()), stats, ws), grads, max_norm, out, stats, ws)
    # (lists at a time: hundreds of tensors take longer here than on the GPU if each is looked at by itself)
    first = grads[0]
    dt, kind = dtype_code(first.dtype), first.dtype
    every = grads if out is None else [*grads, *out]
    if {t.dtype for t in every} != {kind} or not all(map(torch.Tensor.is_contiguous, every)) or (
            out is not None and not all(map(torch.Tensor.is_same_size, grads, out))):
        for i, t in enumerate(grads):
            _packed("gradient %d" % i, t, kind)
            if out is not None:
                _packed("output %d" % i, out[i], kind, t.shape)
    if stats is not None:
        _packed("stats", stats, torch.float32, (2,))
    at = first.get_device()
    s = _on_gpu(ws, first, stats, *[t for t in every if t.get_device() != at][:1])
    counts, pointers = array.array("q", map(torch.Tensor.numel, grads)), array.array("Q", map(torch.Tensor.data_ptr, every))
    n, p = counts.buffer_info()[0], pointers.buffer_info()[0]
    stats = first.new_empty(2, dtype=torch.float32) if stats is None else stats
    L = lib()
    ws = _ws(L.cf_grad_clip_workspace_size(dt, k, n), first.device, ws)
    check(L.cf_grad_clip(dt, k, n, p, None if out is None else p + 8 * k, float(max_norm), _ptr(stats), _ptr(ws),
                         _wsbytes(ws), s))
    return stats


# ------------------------------------------------- Newton-Schulz and Muon
def newton_schulz_params(steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7):
    return cf_newton_schulz_params(int(steps), float(a), float(b), float(c), float(eps))


def muon_params(lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=CF_MUON_SCALE_ASPECT, ns=None):
    return cf_muon_params(float(lr), float(momentum), int(bool(nesterov)), float(weight_decay), int(scale),
                          newton_schulz_params() if ns is None else ns)


def _mat_sizes(mats):
    """(rows, cols) arrays of weights taken as matrices: all but the last
    dimension are rows (a conv weight [3,3,3,cin,cout] is [27 cin, cout])."""
    k = len(mats)
    rows, cols = (ctypes.c_int64 * k)(), (ctypes.c_int64 * k)()
    for i, t in enumerate(mats):
        if t.dim() < 2:
            raise ValueError("matrix %d has fewer than two dimensions" % i)
        cols[i] = t.shape[-1]
        rows[i] = t.numel() // max(1, t.shape[-1])
    return rows, cols


def _pointers(ts):
    return (_P * len(ts))(*[t.data_ptr() for t in ts])


def cf_newton_schulz(ns, mats, out=None, ws=None, stream=None):
    """The nearly orthogonal factor of each matrix (all fp32 or all bf16, two
    dimensions or more, the last one the columns) -> list of tensors like
    them.  `out` may not overlap `mats`."""
    if not mats:
        raise ValueError("no matrices")
    if stream is not None:
        return _on_stream(stream, cf_newton_schulz, (*mats, *(out or ()), ws), ns, mats, out, ws)
    dt = dtype_code(mats[0].dtype)
    out = [torch.empty_like(t) for t in mats] if out is None else out
    if len(out) != len(mats):
        raise ValueError("%d outputs for %d matrices" % (len(out), len(mats)))
    for i, (t, o) in enumerate(zip(mats, out)):
        _packed("matrix %d" % i, t, mats[0].dtype)
        _packed("output %d" % i, o, t.dtype, t.shape)
    rows, cols = _mat_sizes(mats)
    s = _on_gpu(ws, *mats, *out)
    ws = _ws(int(lib().cf_newton_schulz_workspace_size(dt, len(mats), rows, cols)), mats[0].device, ws)
    check(lib().cf_newton_schulz(ctypes.byref(ns), dt, len(mats), rows, cols, _pointers(mats), _pointers(out),
                                 _ptr(ws), _wsbytes(ws), s))
    return out


def cf_muon(hp, params, grads, m, ws=None, stream=None):
    """One Muon update of the fp32 weights `params` (two dimensions or more)
    in place from `grads`, with momenta m (same shapes, updated in place)."""
    k = len(params)
    if not k or len(grads) != k or len(m) != k:
        raise ValueError("params, grads and m must be lists of one length, not empty")
    if stream is not None:
        return _on_stream(stream, cf_muon, (*params, *grads, *m, ws), hp, params, grads, m, ws)
    for i in range(k):
        _packed("param %d" % i, params[i], torch.float32)
        _packed("gradient %d" % i, grads[i], torch.float32, params[i].shape)
        _packed("momentum %d" % i, m[i], torch.float32, params[i].shape)
    rows, cols = _mat_sizes(params)
    s = _on_gpu(ws, *params, *grads, *m)
    ws = _ws(int(lib().cf_muon_workspace_size(ctypes.byref(hp), k, rows, cols)), params[0].device, ws)
    check(lib().cf_muon(ctypes.byref(hp), k, rows, cols, _pointers(params), _pointers(grads), _pointers(m), _ptr(ws),
                        _wsbytes(ws), s))


# --------------------------------------------------------------- batch norm
def cf_batchnorm_fwd(X, gamma, beta, eps, Y=None, mean=None, invstd=None, ws=None, stream=None):
    """Training-mode batch norm of NDHWC X per channel -> (Y, mean, invstd)."""
    dt = dtype_code(X.dtype)
    C = int(X.shape[4])
    Y = torch.empty_like(X) if Y is None else Y
    mean = torch.empty((C,), dtype=torch.float32, device=X.device) if mean is None else mean
    invstd = torch.empty((C,), dtype=torch.float32, device=X.device) if invstd is None else invstd
    ws = _ws(int(lib().cf_batchnorm_workspace_size(dt, dims(X.shape))), X.device, ws)
    check(lib().cf_batchnorm_fwd(dt, dims(X.shape), _ptr(X), _ptr(gamma), _ptr(beta), float(eps), _ptr(Y), _ptr(mean),
                                 _ptr(invstd), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return Y, mean, invstd


def cf_batchnorm_bwd(X, dY, gamma, mean, invstd, dX=None, ws=None, stream=None):
    """-> (dX, dgamma, dbeta)."""
    dt = dtype_code(X.dtype)
    C = int(X.shape[4])
    dX = torch.empty_like(X) if dX is None else dX
    dgamma = torch.empty((C,), dtype=torch.float32, device=X.device)
    dbeta = torch.empty((C,), dtype=torch.float32, device=X.device)
    ws = _ws(int(lib().cf_batchnorm_workspace_size(dt, dims(X.shape))), X.device, ws)
    check(lib().cf_batchnorm_bwd(dt, dims(X.shape), _ptr(X), _ptr(dY), _ptr(gamma), _ptr(mean), _ptr(invstd),
                                 _ptr(dX), _ptr(dgamma), _ptr(dbeta), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return dX, dgamma, dbeta


def _packed(name, t, dtype=None, shape=None):
    """Raises where a tensor is not what the library will take it for."""
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))


def _on_gpu(ws, first, *others):
    """The current stream, where all tensors (or None) are on its GPU, on which
    the kernels take bare addresses, and the workspace has no gaps; else raises."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError("tensors must be on one GPU: %s and %s" % (first.device, t.device))
    if ws is not None:
        _packed("ws", ws)
        if ws.get_device() != at:
            raise ValueError("ws must be on the tensors' GPU: %s and %s" % (ws.device, first.device))
    if at < 0:
        raise ValueError("tensors must be on a GPU")
    if _current_device() != at:
        raise ValueError("tensors and stream must be on the current GPU: %d and %d" % (at, _current_device()))
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(at)


def _on_stream(stream, call, given, *args):
    """call(*args) on another stream than the current one.  What the call makes
    is made in that stream's memory: the current stream's may still be in use
    there.  Nothing has its memory reused before both streams are done with it;
    for the values of the `given` tensors and of the outputs the caller orders
    the streams (wait_stream)."""
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in given:
        if t is not None:
            t.record_stream(stream)
    for t in (out,) if isinstance(out, torch.Tensor) else out or ():
        if t is not None:
            t.record_stream(here)
    return out


# --------------------------------------------------------------- group norm
def cf_groupnorm_workspace_size(dtype, xshape, groups, backward):
    return int(lib().cf_groupnorm_workspace_size(dtype, dims(xshape), int(groups), int(bool(backward))))


def cf_groupnorm_fwd(X, groups, gamma, beta, eps, act=CF_ACT_LRELU, slope=1.0, Y=None, mean=None, rstd=None, ws=None,
                     stream=None):
    """Group norm of NDHWC X, then the activation -> (Y, mean [N, groups],
    rstd [N, groups])."""
    if stream is not None:
        return _on_stream(stream, cf_groupnorm_fwd, (X, gamma, beta, Y, mean, rstd, ws), X, groups, gamma, beta, eps, act,
                          slope, Y, mean, rstd, ws)
    dt, d, groups = dtype_code(X.dtype), cf_dims(*X.shape), int(groups)
    _packed("X", X)
    _packed("gamma", gamma, torch.float32, (d.c,))
    _packed("beta", beta, torch.float32, (d.c,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _packed(name, t, torch.float32, (d.n, groups))
    if Y is not None:
        _packed("Y", Y, X.dtype, X.shape)
    s = _on_gpu(ws, X, gamma, beta, Y, mean, rstd)
    Y = torch.empty_like(X) if Y is None else Y
    mean = gamma.new_empty((d.n, groups)) if mean is None else mean
    rstd = torch.empty_like(mean) if rstd is None else rstd
    ws = _ws(int(lib().cf_groupnorm_workspace_size(dt, d, groups, 0)), X.device, ws)
    check(lib().cf_groupnorm_fwd(dt, d, _ptr(X), groups, _ptr(gamma), _ptr(beta), float(eps), int(act), float(slope),
                                 _ptr(Y), _ptr(mean), _ptr(rstd), _ptr(ws), _wsbytes(ws), s))
    return Y, mean, rstd


def cf_groupnorm_bwd(X, dY, groups, gamma, beta, mean, rstd, act=CF_ACT_LRELU, slope=1.0, dX=None, ws=None,
                     stream=None):
    """-> (dX, dgamma, dbeta) from the forward's mean and rstd."""
    if stream is not None:
        return _on_stream(stream, cf_groupnorm_bwd, (X, dY, gamma, beta, mean, rstd, dX, ws), X, dY, groups, gamma, beta,
                          mean, rstd, act, slope, dX, ws)
    dt, d, groups = dtype_code(X.dtype), cf_dims(*X.shape), int(groups)
    _packed("X", X)
    _packed("dY", dY, X.dtype, X.shape)
    _packed("gamma", gamma, torch.float32, (d.c,))
    _packed("beta", beta, torch.float32, (d.c,))
    _packed("mean", mean, torch.float32, (d.n, groups))
    _packed("rstd", rstd, torch.float32, (d.n, groups))
    if dX is not None:
        _packed("dX", dX, X.dtype, X.shape)
    s = _on_gpu(ws, X, dY, gamma, beta, mean, rstd, dX)
    dX = torch.empty_like(X) if dX is None else dX
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = _ws(int(lib().cf_groupnorm_workspace_size(dt, d, groups, 1)), X.device, ws)
    check(lib().cf_groupnorm_bwd(dt, d, _ptr(X), _ptr(dY), groups, _ptr(gamma), _ptr(beta), _ptr(mean), _ptr(rstd),
                                 int(act), float(slope), _ptr(dX), _ptr(dgamma), _ptr(dbeta), _ptr(ws), _wsbytes(ws), s))
    return dX, dgamma, dbeta


# ------------------------------------------------------------- linear layers
def cf_linear_workspace_size(dtype, rows, fin, fout, backward):
    return int(lib().cf_linear_workspace_size(dtype, int(rows), int(fin), int(fout), int(bool(backward))))


def _linear_sizes(X, W):
    """(rows, in, out) of X [..., in] and W [in, out]."""
    if W.dim() != 2 or X.dim() < 1 or X.shape[-1] != W.shape[0]:
        raise ValueError("X must be [..., in] and W [in, out], not %s and %s" % (tuple(X.shape), tuple(W.shape)))
    if W.dtype != X.dtype or not (X.is_contiguous() and W.is_contiguous()):
        _packed("X", X)
        _packed("W", W, X.dtype)
    fin, fout = W.shape
    if max(fin, fout) >> 31:      # (the library's sizes are 32 bits: they would wrap)
        raise ValueError("in or out too large: %s" % (tuple(W.shape),))
    return X.numel() // max(1, fin), fin, fout


def cf_linear_fwd(X, W, bias=None, act=CF_ACT_LRELU, slope=1.0, R=None, need_pre=True, pre=None, Y=None, ws=None,
                  stream=None):
    """act(X W + bias) + R -> (pre, Y).  X [..., in] (an NDHWC tensor: a 1^3
    convolution), W [in, out] of X's type, bias [out] fp32 or None, R [..., out]
    or None.  need_pre=False (serving): pre is neither made nor written, and
    None is returned for it unless it is given."""
    if stream is not None:
        return _on_stream(stream, cf_linear_fwd, (X, W, bias, R, pre, Y, ws), X, W, bias, act, slope, R, need_pre, pre,
                          Y, ws)
    dt = dtype_code(X.dtype)
    rows, fin, fout = _linear_sizes(X, W)
    shape = X.shape[:-1] + (fout,)
    if bias is not None:
        _packed("bias", bias, torch.float32, (fout,))
    if R is not None:
        _packed("R", R, X.dtype, shape)
    if pre is not None:
        _packed("pre", pre, X.dtype, shape)
    if Y is not None:
        _packed("Y", Y, X.dtype, shape)
    s = _on_gpu(ws, X, W, bias, R, pre, Y)
    Y = X.new_empty(shape) if Y is None else Y
    pre = X.new_empty(shape) if pre is None and need_pre else pre
    L = lib()
    ws = _ws(L.cf_linear_workspace_size(dt, rows, fin, fout, 0), X.device, ws)
    check(L.cf_linear_fwd(dt, rows, fin, fout, _ptr(X), _ptr(W), _ptr(bias), int(act), float(slope), _ptr(R), _ptr(pre),
                          _ptr(Y), _ptr(ws), _wsbytes(ws), s))
    return pre, Y


def cf_linear_bwd(X, W, pre, dY, act=CF_ACT_LRELU, slope=1.0, need_dx=True, dX=None, dW=None, db=None, ws=None,
                  stream=None):
    """-> (dX, dW, db), dW and db fp32, dX None unless need_dx or given; pre may
    be None without an activation (CF_ACT_LRELU with slope 1).  The gradient of
    the forward's R is dY."""
    if stream is not None:
        return _on_stream(stream, cf_linear_bwd, (X, W, pre, dY, dX, dW, db, ws), X, W, pre, dY, act, slope, need_dx, dX,
                          dW, db, ws)
    dt = dtype_code(X.dtype)
    rows, fin, fout = _linear_sizes(X, W)
    shape = X.shape[:-1] + (fout,)
    _packed("dY", dY, X.dtype, shape)
    if pre is not None:
        _packed("pre", pre, X.dtype, shape)
    if dX is not None:
        _packed("dX", dX, X.dtype, X.shape)
    if dW is not None:
        _packed("dW", dW, torch.float32, W.shape)
    if db is not None:
        _packed("db", db, torch.float32, (fout,))
    s = _on_gpu(ws, X, W, pre, dY, dX, dW, db)
    dX = torch.empty_like(X) if dX is None and need_dx else dX
    dW = X.new_empty((fin, fout), dtype=torch.float32) if dW is None else dW
    db = X.new_empty((fout,), dtype=torch.float32) if db is None else db
    L = lib()
    ws = _ws(L.cf_linear_workspace_size(dt, rows, fin, fout, 1), X.device, ws)
    check(L.cf_linear_bwd(dt, rows, fin, fout, _ptr(X), _ptr(W), _ptr(pre), _ptr(dY), int(act), float(slope), _ptr(dX),
                          _ptr(dW), _ptr(db), _ptr(ws), _wsbytes(ws), s))
    return dX, dW, db


# ------------------------------------------------ norms around a residual join
def cf_resnorm_workspace_size(dtype, xshape, gate_n):
    return int(lib().cf_resnorm_workspace_size(dtype, dims(xshape), int(gate_n)))


def _resnorm_dims(X):
    if X.dim() != 5 or max(X.shape) > 1 << 30:      # (the library's limit, before memory is made for the outputs)
        raise ValueError("X and F must be NDHWC tensors, 2^30 at most along a dimension, not %s" % (tuple(X.shape),))
    return cf_dims(*X.shape)


def _resnorm_params(d, kind, eps, gpre, bpre, gpost, bpost, gate, alpha):
    if gpre is not None:
        _packed("gpre", gpre, torch.float32, (d.c,))
    if bpre is not None:
        _packed("bpre", bpre, torch.float32, (d.c,))
    if gpost is not None:
        _packed("gpost", gpost, torch.float32, (d.c,))
    if bpost is not None:
        _packed("bpost", bpost, torch.float32, (d.c,))
    gate_n = 0
    if gate is not None:
        gate_n = gate.shape[0] if gate.dim() == 2 else 1
        _packed("gate", gate, torch.float32, (gate_n, d.c) if gate.dim() == 2 else (d.c,))
    return cf_resnorm_params(kind, eps, alpha, _ptr(gpre), _ptr(bpre), _ptr(gpost), _ptr(bpost), _ptr(gate), gate_n)


def cf_resnorm_fwd(X, F, kind, eps, gpre=None, bpre=None, gpost=None, bpost=None, gate=None, alpha=1.0, need_y=True,
                   R=None, Y=None, stream=None):
    """The join of a residual block, over the channels of NDHWC tensors:
    R = alpha X + gate post(F), Y = pre(R) -> (R, Y).  kind: CF_NORM_RMS or
    CF_NORM_LAYER; gpost None: no norm of F; gate [C], [1, C] or, one for each
    sample, [N, C].  need_y=False: no further norm, None for Y unless it is given."""
    if stream is not None:
        return _on_stream(stream, cf_resnorm_fwd, (X, F, gpre, bpre, gpost, bpost, gate, R, Y), X, F, kind, eps, gpre,
                          bpre, gpost, bpost, gate, alpha, need_y, R, Y)
    dt, d = dtype_code(X.dtype), _resnorm_dims(X)
    _packed("X", X)
    _packed("F", F, X.dtype, X.shape)
    if R is not None:
        _packed("R", R, X.dtype, X.shape)
    if Y is not None:
        _packed("Y", Y, X.dtype, X.shape)
    p = _resnorm_params(d, kind, eps, gpre, bpre, gpost, bpost, gate, alpha)
    s = _on_gpu(None, X, F, gpre, bpre, gpost, bpost, gate, R, Y)
    R = torch.empty_like(X) if R is None else R
    Y = torch.empty_like(X) if Y is None and need_y else Y
    check(lib().cf_resnorm_fwd(dt, d, ctypes.byref(p), _ptr(X), _ptr(F), _ptr(R), _ptr(Y), s))
    return R, Y


def cf_resnorm_bwd(F, R, dR, dY, kind, eps, gpre=None, bpre=None, gpost=None, bpost=None, gate=None, alpha=1.0, dX=None,
                   dF=None, ws=None, stream=None):
    """-> (dX, dF, dgpre, dbpre, dgpost, dbpost, dgate) from the forward's F and
    R; dR or dY may be None (not both).  None is returned for the gradients of
    vectors that are None, and for dgpre and dbpre without dY."""
    if stream is not None:
        return _on_stream(stream, cf_resnorm_bwd, (F, R, dR, dY, gpre, bpre, gpost, bpost, gate, dX, dF, ws), F, R, dR,
                          dY, kind, eps, gpre, bpre, gpost, bpost, gate, alpha, dX, dF, ws)
    dt, d = dtype_code(F.dtype), _resnorm_dims(F)
    _packed("F", F)
    for name, t in (("R", R), ("dR", dR), ("dY", dY), ("dX", dX), ("dF", dF)):
        if t is not None:
            _packed(name, t, F.dtype, F.shape)
    p = _resnorm_params(d, kind, eps, gpre, bpre, gpost, bpost, gate, alpha)
    s = _on_gpu(ws, F, R, dR, dY, gpre, bpre, gpost, bpost, gate, dX, dF)
    dX = torch.empty_like(F) if dX is None else dX
    dF = torch.empty_like(F) if dF is None else dF
    like = lambda t, wanted=True: torch.empty_like(t) if t is not None and wanted else None
    g = [like(gpre, dY is not None), like(bpre, dY is not None), like(gpost), like(bpost), like(gate)]
    L = lib()
    ws = _ws(L.cf_resnorm_workspace_size(dt, d, p.gate_n), F.device, ws)
    check(L.cf_resnorm_bwd(dt, d, ctypes.byref(p), _ptr(F), _ptr(R), _ptr(dR), _ptr(dY), _ptr(dX), _ptr(dF),
                           *[_ptr(t) for t in g], _ptr(ws), _wsbytes(ws), s))
    return (dX, dF, *g)


# ------------------------------------------------------ general network step
def net_desc(in_channels, size, filters, strides=None, pools=None, dense=(128, 64, 3), dense_bias=True,
             batch_norm=False, bn_eps=1e-5, slope=0.3):
    """cf_net_desc for a cubic input (or size = (d, h, w)); pools are
    CF_POOL_* values (default max after every layer)."""
    m = cf_net_desc()
    d, h, w = (size, size, size) if isinstance(size, int) else size
    m.nlayers, m.cin, m.d, m.h, m.w = len(filters), in_channels, d, h, w
    strides = strides or [1] * len(filters)
    pools = pools if pools is not None else [CF_POOL_MAX] * len(filters)
    for i, f in enumerate(filters):
        m.filters[i], m.stride[i], m.pool[i] = f, strides[i], pools[i]
    m.batch_norm, m.bn_eps = int(bool(batch_norm)), bn_eps
    m.ndense = len(dense)
    for i, f in enumerate(dense):
        m.dense[i] = f
    m.dense_bias, m.slope = int(bool(dense_bias)), slope
    return m


def cf_net_param_count(m):
    n = (ctypes.c_int64 * CF_MAX_OPT_TENSORS)()
    k = int(lib().cf_net_param_count(ctypes.byref(m), n))
    if k < 0:
        raise CfError(CF_ERR_INVALID, lib().cf_last_error().decode())
    return [int(n[i]) for i in range(k)]


def sgd_optimizer(lr):
    o = cf_optimizer()
    o.kind, o.lr = CF_OPT_SGD, float(lr)
    return o


def adam_optimizer(hp, t):
    o = cf_optimizer()
    o.kind, o.adam, o.t = CF_OPT_ADAM_LARC, hp, int(t)
    return o


def cf_net_train_step(m, X, targets, params, opt, moments=None, ws=None, loss=None, pred=None, stream=None):
    """One step of the general network; params (and Adam moments (m, v)) in
    cf_net_param_count's order, updated in place.  Returns (loss, pred)."""
    dt = dtype_code(X.dtype)
    B = int(X.shape[0])
    ws = _ws(int(lib().cf_net_train_step_workspace_size(ctypes.byref(m), dt, B)), X.device, ws)
    if loss is None:
        loss = torch.empty((1,), dtype=torch.float32, device=X.device)
    k = len(params)
    arr = lambda ts: (_P * k)(*[q.data_ptr() for q in ts])
    mp = vp = None
    if moments is not None:
        mp, vp = arr(moments[0]), arr(moments[1])
    check(lib().cf_net_train_step(ctypes.byref(m), dt, B, _ptr(X), _ptr(targets), arr(params), ctypes.byref(opt), mp,
                                  vp, _ptr(loss), _ptr(pred), _ptr(ws), _wsbytes(ws), _stream(stream)))
    return loss, pred
