"""ctypes binding of libbitnet.so: the C entry points under the same names.

Argument marshalling only: every function takes torch tensors that already
live on the GPU, checks that dtypes, shapes and contiguity match what the C
ABI documents, and passes raw device pointers and the current HIP stream.
All computation happens in the library's kernels. Outputs are preallocated
by the caller, as in the C ABI. If the library is not built this module
raises; there is no other compute path.
"""

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbitnet.so")

BITNET_OK = 0
BITNET_BF16 = 0
BITNET_F32 = 1
BITNET_SIGN1 = 2

_lib = None


def _hip_runtimes_mapped():
    """Paths of the libamdhip64 copies mapped into this process."""
    paths = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    paths.add(os.path.realpath(line.split()[-1]))
    except OSError:
        pass
    return paths


def lib():
    """Load libbitnet.so (after torch, so that both share torch's HIP
    runtime) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m ternary_weight_quantization_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    i64, sz, vp, st = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    L.bitnet_status_string.argtypes = [st]
    L.bitnet_status_string.restype = ctypes.c_char_p
    L.bitnet_k_pad.argtypes = [i64]
    L.bitnet_k_pad.restype = i64
    L.bitnet_ternarize_workspace_bytes.argtypes = [i64, i64]
    L.bitnet_ternarize_workspace_bytes.restype = sz
    L.bitlinear_fwd_workspace_bytes.argtypes = [i64, i64, i64]
    L.bitlinear_fwd_workspace_bytes.restype = sz
    L.bitlinear_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    L.bitlinear_bwd_workspace_bytes.restype = sz
    L.bitnet_ternarize_pack.argtypes = [vp, st, i64, i64, vp, vp, vp, sz, vp]
    L.bitnet_ternarize_pack.restype = st
    L.bitnet_quantize.argtypes = [vp, st, i64, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.bitnet_quantize.restype = st
    L.bitnet_quantize2.argtypes = [vp, vp, st, i64, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.bitnet_quantize2.restype = st
    L.bitnet_quantize_static.argtypes = [vp, st, i64, i64, vp, i64, vp, vp, vp, vp, vp]
    L.bitnet_quantize_static.restype = st
    L.bitnet_code_counts.argtypes = [vp, i64, i64, vp, vp]
    L.bitnet_code_counts.restype = st
    L.bitnet_act_quant.argtypes = [vp, i64, i64, vp, vp, vp]
    L.bitnet_act_quant.restype = st
    L.bitlinear_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.bitlinear_fwd.restype = st
    L.bitlinear_fwd_bias.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.bitlinear_fwd_bias.restype = st
    L.bitlinear_bias_grad.argtypes = [vp, i64, i64, vp, st, vp]
    L.bitlinear_bias_grad.restype = st
    L.bitlinear_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, st, vp, sz, vp]
    L.bitlinear_bwd.restype = st
    L.ttq_workspace_bytes.argtypes = [i64, i64, i64]
    L.ttq_workspace_bytes.restype = sz
    L.ttq_init.argtypes = [vp, st, i64, i64, vp, vp, sz, vp]
    L.ttq_init.restype = st
    L.ttq_quantize.argtypes = [vp, st, i64, i64, vp, vp, vp, vp]
    L.ttq_quantize.restype = st
    L.ttq_fwd.argtypes = [vp, vp, i64, i64, i64, vp, vp, sz, vp]
    L.ttq_fwd.restype = st
    L.ttq_bwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, st, vp, vp, sz, vp]
    L.ttq_bwd.restype = st
    L.ttq_fwd_codes_workspace_bytes.argtypes = [i64, i64, i64]
    L.ttq_fwd_codes_workspace_bytes.restype = sz
    L.ttq_fwd_codes.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, sz, vp]
    L.ttq_fwd_codes.restype = st
    f32 = ctypes.c_float
    L.bitnet_layernorm_workspace_bytes.argtypes = [i64, i64]
    L.bitnet_layernorm_workspace_bytes.restype = sz
    L.bitnet_layernorm_fwd.argtypes = [vp, st, vp, vp, st, i64, i64, f32, vp, st, vp, vp, vp, vp, vp]
    L.bitnet_layernorm_fwd.restype = st
    L.bitnet_layernorm_bwd.argtypes = [vp, st, vp, st, vp, vp, vp, st, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp]
    L.bitnet_layernorm_bwd.restype = st
    L.bitnet_ckpt_pad.argtypes = [i64]
    L.bitnet_ckpt_pad.restype = i64
    L.bitnet_ckpt_pack.argtypes = [vp, st, i64, i64, vp, vp, vp]
    L.bitnet_ckpt_pack.restype = st
    L.bitnet_ckpt_unpack.argtypes = [vp, vp, i64, i64, vp, st, vp]
    L.bitnet_ckpt_unpack.restype = st
    L.bitnet_gate_fwd.argtypes = [st, vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    L.bitnet_gate_fwd.restype = st
    L.bitnet_gate_bwd.argtypes = [st, vp, vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, i64, vp]
    L.bitnet_gate_bwd.restype = st
    L.ttq_fwd_ckpt_workspace_bytes.argtypes = [i64, i64, i64]
    L.ttq_fwd_ckpt_workspace_bytes.restype = sz
    L.ttq_fwd_ckpt.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    L.ttq_fwd_ckpt.restype = st
    L.ttq_bwd_ckpt_workspace_bytes.argtypes = [i64, i64, i64]
    L.ttq_bwd_ckpt_workspace_bytes.restype = sz
    L.ttq_bwd_ckpt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, st, vp, vp, sz, vp]
    L.ttq_bwd_ckpt.restype = st
    L.bitnet_xent_fwd_workspace_bytes.argtypes = [i64, i64, i64]
    L.bitnet_xent_fwd_workspace_bytes.restype = sz
    L.bitnet_xent_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    L.bitnet_xent_bwd_workspace_bytes.restype = sz
    L.bitnet_xent_fwd.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, st, vp, sz, vp]
    L.bitnet_xent_fwd.restype = st
    L.bitnet_xent_bwd.argtypes = [vp, vp, vp, i64, vp, vp, st, i64, i64, i64, vp, vp, st, vp, sz, vp]
    L.bitnet_xent_bwd.restype = st
    for name in ("bitnet_gated_fwd", "bitnet_gated_bwd", "bitnet_int8_fwd", "bitnet_int8_bwd"):
        f = getattr(L, name + "_workspace_bytes")
        f.argtypes, f.restype = [i64, i64, i64], sz
    L.bitnet_gated_slopes_bytes.argtypes = [i64, i64]
    L.bitnet_gated_slopes_bytes.restype = sz
    L.bitnet_rmsnorm_workspace_bytes.argtypes = [i64, i64]
    L.bitnet_rmsnorm_workspace_bytes.restype = sz
    L.bitnet_rmsnorm_fwd.argtypes = [vp, st, vp, st, vp, st, i64, i64, f32, vp, vp, st, vp, vp, vp, vp]
    L.bitnet_rmsnorm_fwd.restype = st
    L.bitnet_rmsnorm_bwd.argtypes = [vp, st, vp, vp, st, vp, st, vp, i64, i64, vp, vp, vp, vp, sz, vp]
    L.bitnet_rmsnorm_bwd.restype = st
    L.bitnet_rows_quant.argtypes = [vp, st, i64, i64, vp, vp, vp]
    L.bitnet_rows_quant.restype = st
    L.bitnet_rows_quant2.argtypes = [vp, i64, vp, vp, vp, st, i64, vp, vp, i64, vp]
    L.bitnet_rows_quant2.restype = st
    L.bitnet_rows_unpack.argtypes = [vp, vp, i64, i64, vp, vp]
    L.bitnet_rows_unpack.restype = st
    L.bitnet_gated_fwd.argtypes = [st, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.bitnet_rows_direct.argtypes = [i64]
    L.bitnet_rows_direct.restype = ctypes.c_int
    L.bitnet_gated_fwd.restype = st
    L.bitnet_gated_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, st, vp, sz, vp]
    L.bitnet_gated_bwd.restype = st
    L.bitnet_int8_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, sz, vp]
    L.bitnet_int8_fwd.restype = st
    L.bitnet_int8_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, st, vp, st, vp, sz, vp]
    L.bitnet_int8_bwd.restype = st
    i32, u32 = ctypes.c_int32, ctypes.c_uint32
    L.bitnet_set_test_knobs.argtypes = [st, st, st, u32]
    L.bitnet_set_test_knobs.restype = None
    L.bitnet_default_spin_limit.argtypes = []
    L.bitnet_default_spin_limit.restype = u32
    L.bitnet_split_timeouts.argtypes = [vp]
    L.bitnet_split_timeouts.restype = st
    L.bitnet_quantize_recomputes.argtypes = [vp]
    L.bitnet_quantize_recomputes.restype = st
    L.bitnet_debug_split_pieces.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, i64]
    L.bitnet_debug_split_pieces.restype = i64
    L.bitnet_debug_partial_slots.argtypes = [i64, i32]
    L.bitnet_debug_partial_slots.restype = i32
    L.bitnet_debug_mfma_probe.argtypes = [i32, i32, vp, vp, vp]
    L.bitnet_debug_mfma_probe.restype = st
    L.bitnet_debug_cta_order.argtypes = [i32, vp]
    L.bitnet_debug_cta_order.restype = None
    if len(_hip_runtimes_mapped()) > 1:
        raise RuntimeError("more than one libamdhip64 is mapped into this process: "
                           f"{sorted(_hip_runtimes_mapped())}")
    _lib = L
    return _lib


_ops = None


def ops():
    """The torch autograd functions over the library (csrc/host/torch_ops.cpp)."""
    global _ops
    if _ops is None:
        lib()
        if not os.path.exists(os.path.join(HERE, "_bitnet_ops.so")):
            raise RuntimeError("_bitnet_ops.so is not built; run `python -m ternary_weight_quantization_amd.build`")
        from . import _bitnet_ops

        _ops = _bitnet_ops
    return _ops


def _check(code):
    if code != BITNET_OK:
        msg = lib().bitnet_status_string(code).decode()
        raise RuntimeError(f"libbitnet: {msg}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")


def _value_dtype(t, name):
    if t.dtype == torch.bfloat16:
        return BITNET_BF16
    if t.dtype == torch.float32:
        return BITNET_F32
    raise TypeError(f"{name}: expected bfloat16 or float32, got {t.dtype}")


def _same_device(like, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise ValueError(f"{name}: on {t.device}, expected {like.device}")


# the current stream's handle on a device, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(fn, index, *args):
    """fn(*args, stream) with device `index` current, on its current stream.
    No checks but the library's own: for callers that have made theirs."""
    if index == torch.cuda.current_device():
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        _check(code)


def _run(fn, like, stream, *args):
    """_launch on like's device, on `stream` if one is given."""
    if stream is None:
        _launch(fn, like.device.index, *args)
    else:
        with torch.cuda.device(like.device):
            _check(fn(*args, stream.cuda_stream))


# --- size queries ----------------------------------------------------------

def bitnet_k_pad(K):
    return int(lib().bitnet_k_pad(int(K)))


def bitnet_ternarize_workspace_bytes(N, K):
    return int(lib().bitnet_ternarize_workspace_bytes(int(N), int(K)))


def bitlinear_fwd_workspace_bytes(M, N, K):
    return int(lib().bitlinear_fwd_workspace_bytes(int(M), int(N), int(K)))


def bitlinear_bwd_workspace_bytes(M, N, K):
    return int(lib().bitlinear_bwd_workspace_bytes(int(M), int(N), int(K)))


# --- GEMM workspace ----------------------------------------------------------

_workspaces = {}


def _workspace(nbytes, like, stream):
    """A cached device buffer of at least nbytes for the GEMM calls, one per
    (device, stream): calls on one stream run in order and may share it.
    The library needs no particular contents."""
    if nbytes == 0:
        return None
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    key = (like.device.index, stream.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=like.device)
        _workspaces[key] = ws
    return ws


# --- entry points ----------------------------------------------------------

def bitnet_ternarize_pack(W, w_packed, gamma, workspace, stream=None):
    """W [N, K] bf16 or float32 -> w_packed uint8 [N, Kp/4], gamma float32 [1]."""
    N, K = W.shape
    Kp = bitnet_k_pad(K)
    if W.dtype == torch.bfloat16:
        wd = BITNET_BF16
    elif W.dtype == torch.float32:
        wd = BITNET_F32
    else:
        raise TypeError(f"W: expected bfloat16 or float32, got {W.dtype}")
    _need(W, W.dtype, (N, K), "W")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().bitnet_ternarize_pack(_ptr(W), wd, N, K, _ptr(w_packed), _ptr(gamma),
                                       _ptr(workspace), ws_bytes, _stream(stream)))


def bitnet_quantize(W, x, w_packed, gamma, x_q, s_x, workspace, stream=None):
    """bitnet_ternarize_pack(W, ...) and bitnet_act_quant(x, ...) in one call
    (W [N, K] bf16 or float32, x [M, K] bf16)."""
    N, K = W.shape
    M = x.shape[0]
    Kp = bitnet_k_pad(K)
    if W.dtype == torch.bfloat16:
        wd = BITNET_BF16
    elif W.dtype == torch.float32:
        wd = BITNET_F32
    else:
        raise TypeError(f"W: expected bfloat16 or float32, got {W.dtype}")
    _need(W, W.dtype, (N, K), "W")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _need(x_q, torch.int8, (M, Kp), "x_q")
    _need(s_x, torch.float32, (M,), "s_x")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().bitnet_quantize(_ptr(W), wd, N, K, _ptr(x), M, _ptr(w_packed), _ptr(gamma), _ptr(x_q), _ptr(s_x),
                                 _ptr(workspace), ws_bytes, _stream(stream)))


def bitnet_quantize2(W0, W1, x, w_packed, gamma, x_q, s_x, workspace, stream=None):
    """bitnet_ternarize_pack of W0 and W1 [N, K] (one dtype) -> w_packed uint8
    [2 N, Kp/4], gamma float32 [2]; x bf16 [M, K] or None -> x_q, s_x as
    bitnet_rows_quant makes them."""
    N, K = W0.shape
    Kp = bitnet_k_pad(K)
    if W0.dtype == torch.bfloat16:
        wd = BITNET_BF16
    elif W0.dtype == torch.float32:
        wd = BITNET_F32
    else:
        raise TypeError(f"W0: expected bfloat16 or float32, got {W0.dtype}")
    _need(W0, W0.dtype, (N, K), "W0")
    _need(W1, W0.dtype, (N, K), "W1")
    _need(w_packed, torch.uint8, (2 * N, Kp // 4), "w_packed")
    _need(gamma, torch.float32, (2,), "gamma")
    M = 0
    if x is not None:
        M = x.shape[0]
        _need(x, torch.bfloat16, (M, K), "x")
        _need(x_q, torch.int8, (M, Kp), "x_q")
        _need(s_x, torch.float32, (M,), "s_x")
    _same_device(W0, W1=W1, x=x, w_packed=w_packed, gamma=gamma, x_q=None if x is None else x_q,
                 s_x=None if x is None else s_x, workspace=workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _run(lib().bitnet_quantize2, W0, stream, _ptr(W0), _ptr(W1), wd, N, K, _ptr(x), M, _ptr(w_packed), _ptr(gamma),
         _ptr(x_q), _ptr(s_x), _ptr(workspace), ws_bytes)


def bitnet_quantize_static(W, x, w_packed, gamma, x_q, s_x, stream=None):
    """bitnet_quantize with the library's own scratch array: no workspace,
    nothing allocated."""
    N, K = W.shape
    M = x.shape[0]
    Kp = bitnet_k_pad(K)
    if W.dtype == torch.bfloat16:
        wd = BITNET_BF16
    elif W.dtype == torch.float32:
        wd = BITNET_F32
    else:
        raise TypeError(f"W: expected bfloat16 or float32, got {W.dtype}")
    _need(W, W.dtype, (N, K), "W")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _need(x_q, torch.int8, (M, Kp), "x_q")
    _need(s_x, torch.float32, (M,), "s_x")
    _check(lib().bitnet_quantize_static(_ptr(W), wd, N, K, _ptr(x), M, _ptr(w_packed), _ptr(gamma), _ptr(x_q),
                                        _ptr(s_x), _stream(stream)))


def bitnet_code_counts(w_packed, K, counts, stream=None):
    """counts int64 [2] = (number of -1 codes, number of +1 codes) in
    w_packed uint8 [N, Kp/4] over the true N x K weights."""
    N = w_packed.shape[0]
    _need(w_packed, torch.uint8, (N, bitnet_k_pad(K) // 4), "w_packed")
    _need(counts, torch.int64, (2,), "counts")
    _check(lib().bitnet_code_counts(_ptr(w_packed), N, int(K), _ptr(counts), _stream(stream)))


def bitnet_act_quant(x, x_q, s_x, stream=None):
    """x [M, K] bf16 -> x_q int8 [M, Kp], s_x float32 [M]."""
    M, K = x.shape
    _need(x, torch.bfloat16, (M, K), "x")
    _need(x_q, torch.int8, (M, bitnet_k_pad(K)), "x_q")
    _need(s_x, torch.float32, (M,), "s_x")
    _check(lib().bitnet_act_quant(_ptr(x), M, K, _ptr(x_q), _ptr(s_x), _stream(stream)))


def bitlinear_fwd(x_q, s_x, w_packed, gamma, K, y, acc_out=None, workspace=None, stream=None, bias=None):
    """INT8 forward: y [M, N] bf16 (and optionally acc_out int32 [M, N]);
    with `bias` (bf16 [N]) the bias is added before the rounding
    (bitlinear_fwd_bias)."""
    M, Kp = x_q.shape
    N = w_packed.shape[0]
    if Kp != bitnet_k_pad(K):
        raise ValueError("x_q: second dimension must be bitnet_k_pad(K)")
    _need(x_q, torch.int8, (M, Kp), "x_q")
    _need(s_x, torch.float32, (M,), "s_x")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _need(y, torch.bfloat16, (M, N), "y")
    if acc_out is not None:
        _need(acc_out, torch.int32, (M, N), "acc_out")
    if bias is not None:
        _need(bias, torch.bfloat16, (N,), "bias")
    if workspace is None:
        workspace = _workspace(bitlinear_fwd_workspace_bytes(M, N, K), y, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if bias is None:
        _check(lib().bitlinear_fwd(_ptr(x_q), _ptr(s_x), _ptr(w_packed), _ptr(gamma), M, N, int(K),
                                   _ptr(y), _ptr(acc_out), _ptr(workspace), ws_bytes, _stream(stream)))
    else:
        _check(lib().bitlinear_fwd_bias(_ptr(x_q), _ptr(s_x), _ptr(w_packed), _ptr(gamma), _ptr(bias), M, N,
                                        int(K), _ptr(y), _ptr(acc_out), _ptr(workspace), ws_bytes,
                                        _stream(stream)))


def bitlinear_bias_grad(dY, db, stream=None):
    """db [N] (float32 or bf16) = the token sum of dY [M, N] bf16."""
    M, N = dY.shape
    _need(dY, torch.bfloat16, (M, N), "dY")
    if db.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("db: expected float32 or bfloat16")
    _need(db, db.dtype, (N,), "db")
    dt = BITNET_F32 if db.dtype == torch.float32 else BITNET_BF16
    _check(lib().bitlinear_bias_grad(_ptr(dY), M, N, _ptr(db), dt, _stream(stream)))


def bitlinear_bwd(dY, x_q, s_x, w_packed, gamma, K, dX=None, dW=None, workspace=None, stream=None):
    """STE backward: dX [M, K] bf16 and/or dW [N, K] (bf16 or float32), or
    dW as 1-bit signs (uint8 [N, Kp/8]; bit j of byte b of row n set iff
    dW[n, 8b + j] < 0)."""
    M, N = dY.shape
    Kp = bitnet_k_pad(K)
    _need(dY, torch.bfloat16, (M, N), "dY")
    if dX is not None:
        _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
        _need(gamma, torch.float32, (1,), "gamma")
        _need(dX, torch.bfloat16, (M, int(K)), "dX")
    dw_dtype = BITNET_BF16
    if dW is not None:
        _need(x_q, torch.int8, (M, Kp), "x_q")
        _need(s_x, torch.float32, (M,), "s_x")
        if dW.dtype == torch.uint8:
            dw_dtype = BITNET_SIGN1
            _need(dW, torch.uint8, (N, Kp // 8), "dW")
        else:
            if dW.dtype == torch.float32:
                dw_dtype = BITNET_F32
            _need(dW, dW.dtype, (N, int(K)), "dW")
            if dW.dtype not in (torch.bfloat16, torch.float32):
                raise TypeError("dW: expected bfloat16, float32 or uint8 (1-bit signs)")
    if workspace is None:
        workspace = _workspace(bitlinear_bwd_workspace_bytes(M, N, K), dY, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().bitlinear_bwd(_ptr(dY), _ptr(x_q), _ptr(s_x), _ptr(w_packed), _ptr(gamma),
                               M, N, int(K), _ptr(dX), _ptr(dW), dw_dtype, _ptr(workspace), ws_bytes,
                               _stream(stream)))


# --- TTQ ---------------------------------------------------------------------

def ttq_workspace_bytes(M, N, K):
    return int(lib().ttq_workspace_bytes(int(M), int(N), int(K)))


def _w_dtype(W):
    if W.dtype == torch.bfloat16:
        return BITNET_BF16
    if W.dtype == torch.float32:
        return BITNET_F32
    raise TypeError(f"W: expected bfloat16 or float32, got {W.dtype}")


def ttq_init(W, params, workspace, stream=None):
    """W [N, K] bf16 or float32 -> params float32 [3] = (delta, Wp, Wn)."""
    N, K = W.shape
    wd = _w_dtype(W)
    _need(W, W.dtype, (N, K), "W")
    _need(params, torch.float32, (3,), "params")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().ttq_init(_ptr(W), wd, N, K, _ptr(params), _ptr(workspace), ws_bytes, _stream(stream)))


def ttq_quantize(W, params, w_packed, wt, stream=None):
    """W [N, K], params (delta, Wp, Wn) -> codes uint8 [N, Kp/4] and bf16
    values wt [N, Kp]."""
    N, K = W.shape
    Kp = bitnet_k_pad(K)
    wd = _w_dtype(W)
    _need(W, W.dtype, (N, K), "W")
    _need(params, torch.float32, (3,), "params")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(wt, torch.bfloat16, (N, Kp), "wt")
    _check(lib().ttq_quantize(_ptr(W), wd, N, K, _ptr(params), _ptr(w_packed), _ptr(wt), _stream(stream)))


def ttq_fwd(x, wt, y, workspace=None, stream=None):
    """y [M, N] bf16 = x [M, K] bf16 @ wt[:, :K]^T."""
    M, K = x.shape
    N, Kp = wt.shape
    if Kp != bitnet_k_pad(K):
        raise ValueError("wt: second dimension must be bitnet_k_pad(K)")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(wt, torch.bfloat16, (N, Kp), "wt")
    _need(y, torch.bfloat16, (M, N), "y")
    if workspace is None:
        workspace = _workspace(ttq_workspace_bytes(M, N, K), y, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ttq_fwd(_ptr(x), _ptr(wt), M, N, K, _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)))


def ttq_fwd_codes_workspace_bytes(M, N, K):
    return int(lib().ttq_fwd_codes_workspace_bytes(int(M), int(N), int(K)))


def ttq_fwd_codes(x, w_packed, params, y, workspace=None, stream=None):
    """y [M, N] bf16 from x [M, K] bf16, the codes uint8 [N, Kp/4] and params
    float32 [3] = (delta, Wp, Wn)."""
    M, K = x.shape
    N = w_packed.shape[0]
    Kp = bitnet_k_pad(K)
    _need(x, torch.bfloat16, (M, K), "x")
    _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    _need(params, torch.float32, (3,), "params")
    _need(y, torch.bfloat16, (M, N), "y")
    if workspace is None:
        workspace = _workspace(ttq_fwd_codes_workspace_bytes(M, N, K), y, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ttq_fwd_codes(_ptr(x), _ptr(w_packed), _ptr(params), M, N, K, _ptr(y), _ptr(workspace), ws_bytes,
                               _stream(stream)))


def ttq_bwd(dY, x, wt, w_packed, K, dX=None, dW=None, grads=None, workspace=None, stream=None):
    """dX [M, K] bf16, dW [N, K] (bf16 or float32) and grads float32 [2] =
    (dL/dWp, dL/dWn), each optional (grads needs dW)."""
    M, N = dY.shape
    Kp = bitnet_k_pad(K)
    _need(dY, torch.bfloat16, (M, N), "dY")
    if dX is not None:
        _need(wt, torch.bfloat16, (N, Kp), "wt")
        _need(dX, torch.bfloat16, (M, int(K)), "dX")
    dw_dtype = BITNET_BF16
    if dW is not None:
        _need(x, torch.bfloat16, (M, int(K)), "x")
        if dW.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dW: expected bfloat16 or float32")
        _need(dW, dW.dtype, (N, int(K)), "dW")
        dw_dtype = BITNET_F32 if dW.dtype == torch.float32 else BITNET_BF16
    if grads is not None:
        _need(grads, torch.float32, (2,), "grads")
        _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    if workspace is None:
        workspace = _workspace(ttq_workspace_bytes(M, N, K), dY, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ttq_bwd(_ptr(dY), _ptr(x), _ptr(wt), _ptr(w_packed), M, N, int(K), _ptr(dX), _ptr(dW),
                         dw_dtype, _ptr(grads), _ptr(workspace), ws_bytes, _stream(stream)))


def ttq_fwd_ckpt_workspace_bytes(M, N, K):
    return int(lib().ttq_fwd_ckpt_workspace_bytes(int(M), int(N), int(K)))


def ttq_fwd_ckpt(x, wt, y, codes=None, scales=None, workspace=None, stream=None):
    """ttq_fwd that also writes the 8-bit checkpoint of x: codes int8
    [M, Kc], scales float32 [M, Kc/128]."""
    M, K = x.shape
    N, Kp = wt.shape
    if Kp != bitnet_k_pad(K):
        raise ValueError("wt: second dimension must be bitnet_k_pad(K)")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(wt, torch.bfloat16, (N, Kp), "wt")
    _need(y, torch.bfloat16, (M, N), "y")
    if codes is not None:
        _need_codes(codes, scales, M, K)
    _same_device(x, wt=wt, y=y, codes=codes, scales=scales, workspace=workspace)
    if workspace is None:
        workspace = _workspace(ttq_fwd_ckpt_workspace_bytes(M, N, K), x, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().ttq_fwd_ckpt, x, stream, _ptr(x), _ptr(wt), M, N, K, _ptr(y), _ptr(codes), _ptr(scales),
         _ptr(workspace), ws_bytes)


def ttq_bwd_ckpt_workspace_bytes(M, N, K):
    return int(lib().ttq_bwd_ckpt_workspace_bytes(int(M), int(N), int(K)))


def ttq_bwd_ckpt(dY, codes, scales, wt, w_packed, K, dX=None, dW=None, grads=None, workspace=None, stream=None):
    """ttq_bwd with x as its 8-bit checkpoint: codes int8 [M, Kc], scales
    float32 [M, Kc/128] (bitnet_ckpt_pack)."""
    M, N = dY.shape
    K = int(K)
    Kp = bitnet_k_pad(K)
    _need(dY, torch.bfloat16, (M, N), "dY")
    _same_device(dY, codes=codes, scales=scales, wt=wt, w_packed=w_packed, dX=dX, dW=dW, grads=grads,
                 workspace=workspace)
    if dX is not None:
        _need(wt, torch.bfloat16, (N, Kp), "wt")
        _need(dX, torch.bfloat16, (M, K), "dX")
    dw_dtype = BITNET_BF16
    if dW is not None:
        _need_codes(codes, scales, M, K)
        dw_dtype = _value_dtype(dW, "dW")
        _need(dW, dW.dtype, (N, K), "dW")
    if grads is not None:
        _need(grads, torch.float32, (2,), "grads")
        _need(w_packed, torch.uint8, (N, Kp // 4), "w_packed")
    if workspace is None:
        workspace = _workspace(ttq_bwd_ckpt_workspace_bytes(M, N, K), dY, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().ttq_bwd_ckpt, dY, stream, _ptr(dY), _ptr(codes), _ptr(scales), _ptr(wt), _ptr(w_packed), M, N, K,
         _ptr(dX), _ptr(dW), dw_dtype, _ptr(grads), _ptr(workspace), ws_bytes)


# --- layer norm ----------------------------------------------------------------

def bitnet_layernorm_workspace_bytes(M, K):
    return int(lib().bitnet_layernorm_workspace_bytes(int(M), int(K)))


def _norm_params(w, b, K, like):
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _value_dtype(t, name)
            _need(t, t.dtype, (K,), name)
    if w is not None and b is not None and w.dtype != b.dtype:
        raise TypeError(f"w and b: one dtype expected, got {w.dtype} and {b.dtype}")
    _same_device(like, w=w, b=b)
    p = w if w is not None else b
    return BITNET_F32 if p is None else _value_dtype(p, "w")


def bitnet_layernorm_fwd(x, w, b, eps, y, mean=None, rstd=None, codes=None, scales=None, stream=None):
    """y [M, K] (bf16 or float32) = the layer norm of x [M, K] (bf16 or
    float32) with w, b [K] or None. Optional outputs: mean, rstd float32 [M];
    codes int8 [M, Kc] and scales float32 [M, Kc/128], the 8-bit checkpoint
    of x."""
    M, K = x.shape
    xd, yd = _value_dtype(x, "x"), _value_dtype(y, "y")
    _need(x, x.dtype, (M, K), "x")
    _need(y, y.dtype, (M, K), "y")
    pd = _norm_params(w, b, K, x)
    if mean is not None:
        _need(mean, torch.float32, (M,), "mean")
    if rstd is not None:
        _need(rstd, torch.float32, (M,), "rstd")
    if codes is not None:
        _need_codes(codes, scales, M, K)
    _same_device(x, y=y, mean=mean, rstd=rstd, codes=codes, scales=scales)
    _run(lib().bitnet_layernorm_fwd, x, stream, _ptr(x), xd, _ptr(w), _ptr(b), pd, M, K, float(eps), _ptr(y), yd,
         _ptr(mean), _ptr(rstd), _ptr(codes), _ptr(scales))


def bitnet_layernorm_bwd(dY, x, w, mean, rstd, dX=None, dw=None, db=None, codes=None, scales=None, x_dtype=None,
                         workspace=None, stream=None):
    """dX [M, K], dw and db [K] (each optional) of the layer norm, from dY
    [M, K], mean and rstd, and x or its 8-bit checkpoint (x None, codes and
    scales given; x_dtype names dX's dtype when dX is None too)."""
    M, K = dY.shape
    yd = _value_dtype(dY, "dY")
    _need(dY, dY.dtype, (M, K), "dY")
    if codes is not None:
        _need_codes(codes, scales, M, K)
        xt = dX.dtype if dX is not None else (x_dtype or torch.bfloat16)
    else:
        if x is None:
            raise ValueError("x: needed without codes")
        _value_dtype(x, "x")
        _need(x, x.dtype, (M, K), "x")
        xt = x.dtype
    if dX is not None:
        _value_dtype(dX, "dX")
        _need(dX, xt, (M, K), "dX")
    _need(mean, torch.float32, (M,), "mean")
    _need(rstd, torch.float32, (M,), "rstd")
    pd = _norm_params(w, None, K, dY)
    for name, t in (("dw", dw), ("db", db)):
        if t is not None:
            if w is None:
                pd = _value_dtype(t, name)
            _need(t, torch.float32 if pd == BITNET_F32 else torch.bfloat16, (K,), name)
    _same_device(dY, x=x, mean=mean, rstd=rstd, codes=codes, scales=scales, dX=dX, dw=dw, db=db, workspace=workspace)
    if workspace is None and (dw is not None or db is not None):
        workspace = _workspace(bitnet_layernorm_workspace_bytes(M, K), dY, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().bitnet_layernorm_bwd, dY, stream, _ptr(dY), yd, _ptr(x), BITNET_F32 if xt == torch.float32 else BITNET_BF16,
         _ptr(codes), _ptr(scales), _ptr(w), pd, _ptr(mean), _ptr(rstd), M, K, _ptr(dX), _ptr(dw), _ptr(db),
         _ptr(workspace), ws_bytes)


# --- 8-bit checkpoints, the gated activation ------------------------------------

BITNET_ACT_SILU = 0
BITNET_ACT_RELU2 = 1


def bitnet_ckpt_pad(K):
    return int(lib().bitnet_ckpt_pad(int(K)))


def _need_codes(codes, scales, M, K, name=""):
    Kc = (int(K) + 127) // 128 * 128
    if codes is None or scales is None:
        raise ValueError(f"{name}codes and scales: both needed")
    _need(codes, torch.int8, (M, Kc), name + "codes")
    _need(scales, torch.float32, (M, Kc // 128), name + "scales")


def bitnet_ckpt_pack(x, codes, scales, stream=None):
    """x [M, K] (bf16 or float32) -> codes int8 [M, Kc], scales float32
    [M, Kc/128], Kc = bitnet_ckpt_pad(K)."""
    M, K = x.shape
    xd = _value_dtype(x, "x")
    _need(x, x.dtype, (M, K), "x")
    _need_codes(codes, scales, M, K)
    _same_device(x, codes=codes, scales=scales)
    _run(lib().bitnet_ckpt_pack, x, stream, _ptr(x), xd, M, K, _ptr(codes), _ptr(scales))


def bitnet_ckpt_unpack(codes, scales, x, stream=None):
    """x [M, K] (bf16 or float32) = the values of codes and scales."""
    M, K = x.shape
    xd = _value_dtype(x, "x")
    _need(x, x.dtype, (M, K), "x")
    _need_codes(codes, scales, M, K)
    _same_device(x, codes=codes, scales=scales)
    _run(lib().bitnet_ckpt_unpack, x, stream, _ptr(codes), _ptr(scales), M, K, _ptr(x), xd)


def _need_rows(t, M, K, name):
    """bf16 rows [M, K] with unit column stride; returns their stride."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if tuple(t.shape) != (M, K):
        raise ValueError(f"{name}: expected shape {(M, K)}, got {tuple(t.shape)}")
    if K > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be contiguous")
    if M > 1 and t.stride(0) < K:
        raise ValueError(f"{name}: rows must not overlap")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    return t.stride(0) if M > 1 else K


def bitnet_gate_fwd(act, gate, up, y, gate_codes=None, gate_scales=None, up_codes=None, up_scales=None, stream=None):
    """y [M, K] = act(gate) * up (up None: act(gate)); gate and up are bf16
    rows of any stride. With gate_codes the 8-bit checkpoints of both are
    written too."""
    M, K = gate.shape
    ldg = _need_rows(gate, M, K, "gate")
    ldu = K if up is None else _need_rows(up, M, K, "up")
    _need(y, torch.bfloat16, (M, K), "y")
    if gate_codes is not None:
        _need_codes(gate_codes, gate_scales, M, K, "gate_")
        if up is not None:
            _need_codes(up_codes, up_scales, M, K, "up_")
    _same_device(gate, up=up, y=y, gate_codes=gate_codes, gate_scales=gate_scales, up_codes=up_codes,
                 up_scales=up_scales)
    _run(lib().bitnet_gate_fwd, gate, stream, int(act), _ptr(gate), ldg, _ptr(up), ldu, M, K, _ptr(y),
         _ptr(gate_codes), _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales))


def bitnet_gate_bwd(act, dY, dgate, dup=None, gate=None, up=None, gate_codes=None, gate_scales=None, up_codes=None,
                    up_scales=None, stream=None):
    """dgate and (with up) dup, bf16 rows of any stride, from dY [M, K] and
    gate, up or their 8-bit checkpoints."""
    M, K = dY.shape
    _need(dY, torch.bfloat16, (M, K), "dY")
    lddg = _need_rows(dgate, M, K, "dgate")
    lddu = K if dup is None else _need_rows(dup, M, K, "dup")
    ldg = ldu = K
    if gate_codes is not None:
        _need_codes(gate_codes, gate_scales, M, K, "gate_")
        if dup is not None:
            _need_codes(up_codes, up_scales, M, K, "up_")
    else:
        if gate is None:
            raise ValueError("gate: needed without codes")
        ldg = _need_rows(gate, M, K, "gate")
        if up is not None:
            ldu = _need_rows(up, M, K, "up")
    _same_device(dY, dgate=dgate, dup=dup, gate=gate, up=up, gate_codes=gate_codes, gate_scales=gate_scales,
                 up_codes=up_codes, up_scales=up_scales)
    _run(lib().bitnet_gate_bwd, dY, stream, int(act), _ptr(dY), _ptr(gate), ldg, _ptr(up), ldu, _ptr(gate_codes),
         _ptr(gate_scales), _ptr(up_codes), _ptr(up_scales), M, K, _ptr(dgate), lddg, _ptr(dup), lddu)


# --- root-mean-square norm, 8-bit rows -------------------------------------------

def bitnet_rmsnorm_workspace_bytes(M, K):
    return int(lib().bitnet_rmsnorm_workspace_bytes(int(M), int(K)))


def _need_rows8(q, s, M, K, name):
    _need(q, torch.int8, (M, bitnet_k_pad(K)), name + "_q")
    _need(s, torch.float32, (M,), "s_" + name)


def bitnet_rmsnorm_fwd(x, w, eps, res=None, h=None, y=None, x_q=None, s_x=None, rstd=None, stream=None):
    """The RMS norm of x [M, K], or of h = res + x (written to h, of res' dtype), with
    w [K] or None: y [M, K] (bf16 or float32), or 8-bit rows x_q int8 [M, Kp], s_x
    float32 [M]. Optional: rstd float32 [M]."""
    M, K = x.shape
    xd = _value_dtype(x, "x")
    _need(x, x.dtype, (M, K), "x")
    hd = xd
    if res is not None:
        hd = _value_dtype(res, "res")
        _need(res, res.dtype, (M, K), "res")
        if h is None:
            raise ValueError("h: needed with res")
        _need(h, res.dtype, (M, K), "h")
    pd = _norm_params(w, None, K, x)
    yd = BITNET_BF16
    if y is not None:
        yd = _value_dtype(y, "y")
        _need(y, y.dtype, (M, K), "y")
    if x_q is not None:
        if s_x is None:
            raise ValueError("s_x: needed with x_q")
        _need_rows8(x_q, s_x, M, K, "x")
    if rstd is not None:
        _need(rstd, torch.float32, (M,), "rstd")
    _same_device(x, res=res, h=h, y=y, x_q=x_q, s_x=s_x, rstd=rstd)
    _run(lib().bitnet_rmsnorm_fwd, x, stream, _ptr(x), xd, _ptr(res), hd, _ptr(w), pd, M, K, float(eps), _ptr(h), _ptr(y),
         yd, _ptr(x_q), _ptr(s_x), _ptr(rstd))


def bitnet_rmsnorm_bwd(dY, h, w, rstd, dH=None, dh=None, dx=None, dw=None, workspace=None, stream=None):
    """dh [M, K] in h's dtype, dx its bf16 copy (h float32) and dw [K] (each
    optional) of the RMS norm, from dY [M, K], the normed rows h, rstd and dH [M, K],
    the gradient of h itself, or None."""
    M, K = dY.shape
    yd, hd = _value_dtype(dY, "dY"), _value_dtype(h, "h")
    _need(dY, dY.dtype, (M, K), "dY")
    _need(h, h.dtype, (M, K), "h")
    _need(rstd, torch.float32, (M,), "rstd")
    for name, t, dt in (("dH", dH, h.dtype), ("dh", dh, h.dtype), ("dx", dx, torch.bfloat16)):
        if t is not None:
            _need(t, dt, (M, K), name)
    pd = _norm_params(w, None, K, dY)
    if dw is not None:
        if w is None:
            pd = _value_dtype(dw, "dw")
        _need(dw, torch.float32 if pd == BITNET_F32 else torch.bfloat16, (K,), "dw")
    _same_device(dY, h=h, rstd=rstd, dH=dH, dh=dh, dx=dx, dw=dw, workspace=workspace)
    if workspace is None and dw is not None:
        workspace = _workspace(bitnet_rmsnorm_workspace_bytes(M, K), dY, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().bitnet_rmsnorm_bwd, dY, stream, _ptr(dY), yd, _ptr(dH), _ptr(h), hd, _ptr(w), pd, _ptr(rstd), M, K,
         _ptr(dh), _ptr(dx), _ptr(dw), _ptr(workspace), ws_bytes)


def bitnet_rows_quant(x, x_q, s_x, stream=None):
    """x [M, K] (bf16 or float32) -> x_q int8 [M, Kp], s_x float32 [M]."""
    M, K = x.shape
    xd = _value_dtype(x, "x")
    _need(x, x.dtype, (M, K), "x")
    _need_rows8(x_q, s_x, M, K, "x")
    _same_device(x, x_q=x_q, s_x=s_x)
    _run(lib().bitnet_rows_quant, x, stream, _ptr(x), xd, M, K, _ptr(x_q), _ptr(s_x))


def bitnet_rows_quant2(x, x_q, s_x, w, w_q, s_w, stream=None):
    """bitnet_rows_quant of x [M, K] bf16 and of w [N, K] (bf16 or float32) in one
    launch."""
    (M, K), N = x.shape, w.shape[0]
    wd = _value_dtype(w, "w")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(w, w.dtype, (N, K), "w")
    _need_rows8(x_q, s_x, M, K, "x")
    _need_rows8(w_q, s_w, N, K, "w")
    _same_device(x, x_q=x_q, s_x=s_x, w=w, w_q=w_q, s_w=s_w)
    _run(lib().bitnet_rows_quant2, x, stream, _ptr(x), M, _ptr(x_q), _ptr(s_x), _ptr(w), wd, N, _ptr(w_q), _ptr(s_w), K)


def bitnet_rows_unpack(x_q, s_x, x, stream=None):
    """x [M, K] bf16 = the values of x_q and s_x."""
    M, K = x.shape
    _need(x, torch.bfloat16, (M, K), "x")
    _need_rows8(x_q, s_x, M, K, "x")
    _same_device(x, x_q=x_q, s_x=s_x)
    _run(lib().bitnet_rows_unpack, x, stream, _ptr(x_q), _ptr(s_x), M, K, _ptr(x))


# --- the gated pair of ternary projections ---------------------------------------

def bitnet_gated_slopes_bytes(M, N):
    return int(lib().bitnet_gated_slopes_bytes(int(M), int(N)))


def bitnet_gated_fwd_workspace_bytes(M, N, K):
    return int(lib().bitnet_gated_fwd_workspace_bytes(int(M), int(N), int(K)))


def bitnet_gated_bwd_workspace_bytes(M, N, K):
    return int(lib().bitnet_gated_bwd_workspace_bytes(int(M), int(N), int(K)))


def _ws_args(workspace, need, like, stream):
    if workspace is None:
        workspace = _workspace(need, like, stream)
    return _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size()


def bitnet_rows_direct(K):
    return int(lib().bitnet_rows_direct(int(K)))


def bitnet_gated_fwd(act, x_q, s_x, w_packed, gamma, K, y, slopes=None, workspace=None, stream=None, x=None):
    """y [M, N] bf16 = act(gate) * up of 8-bit rows x_q, s_x (or of x bf16 [M, K], M <=
    bitnet_rows_direct(K)) and the codes w_packed uint8 [2N, Kp/4] with gamma float32 [2];
    slopes uint8 [bitnet_gated_slopes_bytes(M, N)] is written too if given."""
    M, N = y.shape
    _need(y, torch.bfloat16, (M, N), "y")
    if x is None:
        _need_rows8(x_q, s_x, M, K, "x")
    else:
        _need(x, torch.bfloat16, (M, K), "x")
    _need(w_packed, torch.uint8, (2 * N, bitnet_k_pad(K) // 4), "w_packed")
    _need(gamma, torch.float32, (2,), "gamma")
    if slopes is not None:
        _need(slopes, torch.uint8, (bitnet_gated_slopes_bytes(M, N),), "slopes")
    _same_device(y, x=x, x_q=x_q, s_x=s_x, w_packed=w_packed, gamma=gamma, slopes=slopes, workspace=workspace)
    ws, n = _ws_args(workspace, bitnet_gated_fwd_workspace_bytes(M, N, K), y, stream)
    _run(lib().bitnet_gated_fwd, y, stream, int(act), _ptr(x), _ptr(x_q), _ptr(s_x), _ptr(w_packed), _ptr(gamma), M, N,
         int(K), _ptr(y), _ptr(slopes), ws, n)


def bitnet_gated_bwd(dY, slopes, x_q, s_x, w_packed, gamma, K, dX=None, dW_gate=None, dW_up=None, workspace=None,
                     stream=None):
    """dX [M, K] bf16 and/or dW_gate and dW_up [N, K] (bf16 or float32) from dY [M, N]
    and what bitnet_gated_fwd read and wrote (x_q, s_x may be None without the
    weights' gradients, w_packed without dX)."""
    M, N = dY.shape
    Kp = bitnet_k_pad(K)
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(slopes, torch.uint8, (bitnet_gated_slopes_bytes(M, N),), "slopes")
    _need(gamma, torch.float32, (2,), "gamma")
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
        _need(w_packed, torch.uint8, (2 * N, Kp // 4), "w_packed")
    dd = BITNET_BF16
    if dW_gate is not None:
        dd = _value_dtype(dW_gate, "dW_gate")
        for name, t in (("dW_gate", dW_gate), ("dW_up", dW_up)):
            if t is None:
                raise ValueError("dW_gate and dW_up: both or neither")
            _need(t, dW_gate.dtype, (N, K), name)
        _need_rows8(x_q, s_x, M, K, "x")
    _same_device(dY, slopes=slopes, x_q=x_q, s_x=s_x, w_packed=w_packed, gamma=gamma, dX=dX, dW_gate=dW_gate,
                 dW_up=dW_up, workspace=workspace)
    ws, n = _ws_args(workspace, bitnet_gated_bwd_workspace_bytes(M, N, K), dY, stream)
    _run(lib().bitnet_gated_bwd, dY, stream, _ptr(dY), _ptr(slopes), _ptr(x_q), _ptr(s_x), _ptr(w_packed),
         _ptr(gamma), M, N, int(K), _ptr(dX), _ptr(dW_gate), _ptr(dW_up), dd, ws, n)


# --- linear layer in 8-bit integers -----------------------------------------------

def bitnet_int8_fwd_workspace_bytes(M, N, K):
    return int(lib().bitnet_int8_fwd_workspace_bytes(int(M), int(N), int(K)))


def bitnet_int8_bwd_workspace_bytes(M, N, K):
    return int(lib().bitnet_int8_bwd_workspace_bytes(int(M), int(N), int(K)))


def bitnet_int8_fwd(x_q, s_x, w_q, s_w, K, y, bias=None, workspace=None, stream=None, x=None):
    """y [M, N] bf16 of 8-bit rows x_q, s_x (tokens; or of x bf16 [M, K], M <=
    bitnet_rows_direct(K)) and w_q, s_w (channels), with an optional bf16 bias [N]."""
    M, N = y.shape
    _need(y, torch.bfloat16, (M, N), "y")
    if x is None:
        _need_rows8(x_q, s_x, M, K, "x")
    else:
        _need(x, torch.bfloat16, (M, K), "x")
    _need_rows8(w_q, s_w, N, K, "w")
    if bias is not None:
        _need(bias, torch.bfloat16, (N,), "bias")
    _same_device(y, x=x, x_q=x_q, s_x=s_x, w_q=w_q, s_w=s_w, bias=bias, workspace=workspace)
    ws, n = _ws_args(workspace, bitnet_int8_fwd_workspace_bytes(M, N, K), y, stream)
    _run(lib().bitnet_int8_fwd, y, stream, _ptr(x), _ptr(x_q), _ptr(s_x), _ptr(w_q), _ptr(s_w), _ptr(bias), M, N, int(K),
         _ptr(y), ws, n)


def bitnet_int8_bwd(dY, x_q, s_x, w_q, s_w, K, dX=None, dW=None, db=None, workspace=None, stream=None):
    """dX [M, K] bf16, dW [N, K] and db [N] (bf16 or float32), each optional, from dY [M, N]
    (w_q, s_w may be None without dX, x_q, s_x without dW)."""
    M, N = dY.shape
    _need(dY, torch.bfloat16, (M, N), "dY")
    dd = bd = BITNET_BF16
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
        _need_rows8(w_q, s_w, N, K, "w")
    if dW is not None:
        dd = _value_dtype(dW, "dW")
        _need(dW, dW.dtype, (N, K), "dW")
        _need_rows8(x_q, s_x, M, K, "x")
    if db is not None:
        bd = _value_dtype(db, "db")
        _need(db, db.dtype, (N,), "db")
    _same_device(dY, x_q=x_q, s_x=s_x, w_q=w_q, s_w=s_w, dX=dX, dW=dW, db=db, workspace=workspace)
    ws, n = _ws_args(workspace, bitnet_int8_bwd_workspace_bytes(M, N, K), dY, stream)
    _run(lib().bitnet_int8_bwd, dY, stream, _ptr(dY), _ptr(x_q), _ptr(s_x), _ptr(w_q), _ptr(s_w), M, N, int(K), _ptr(dX),
         _ptr(dW), dd, _ptr(db), bd, ws, n)


# --- linear layer with softmax cross entropy -------------------------------------

BITNET_REDUCE_NONE = 0
BITNET_REDUCE_SUM = 1
BITNET_REDUCE_MEAN = 2


def bitnet_xent_fwd_workspace_bytes(T, V, D):
    return int(lib().bitnet_xent_fwd_workspace_bytes(int(T), int(V), int(D)))


def bitnet_xent_bwd_workspace_bytes(T, V, D):
    return int(lib().bitnet_xent_bwd_workspace_bytes(int(T), int(V), int(D)))


def _need_xent(h, w, targets):
    T, D = h.shape
    V = w.shape[0]
    _need(h, torch.bfloat16, (T, D), "h")
    _need(w, torch.bfloat16, (V, D), "w")
    _need(targets, torch.int64, (T,), "targets")
    return T, V, D


def bitnet_xent_fwd(h, w, targets, ignore_index, loss, lse, total=None, reduce=BITNET_REDUCE_NONE, workspace=None,
                    stream=None):
    """loss, lse float32 [T] of the logits h [T, D] bf16 @ w [V, D]^T bf16
    with int64 targets [T], and total float32 [1], their sum or mean."""
    T, V, D = _need_xent(h, w, targets)
    _need(loss, torch.float32, (T,), "loss")
    _need(lse, torch.float32, (T,), "lse")
    if total is not None:
        _need(total, torch.float32, (1,), "total")
    _same_device(h, w=w, targets=targets, loss=loss, lse=lse, total=total, workspace=workspace)
    if workspace is None:
        workspace = _workspace(bitnet_xent_fwd_workspace_bytes(T, V, D), h, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().bitnet_xent_fwd, h, stream, _ptr(h), _ptr(w), _ptr(targets), int(ignore_index), T, V, D, _ptr(loss),
         _ptr(lse), _ptr(total), int(reduce), _ptr(workspace), ws_bytes)


def bitnet_xent_bwd(h, w, targets, ignore_index, lse, dloss, dh=None, dw=None, reduce=BITNET_REDUCE_NONE,
                    workspace=None, stream=None):
    """dh [T, D] bf16 and/or dw [V, D] (bf16 or float32) from lse and dloss
    (float32 [T], or [1] with a sum or mean)."""
    T, V, D = _need_xent(h, w, targets)
    _need(lse, torch.float32, (T,), "lse")
    _need(dloss, torch.float32, (T,) if int(reduce) == BITNET_REDUCE_NONE else (1,), "dloss")
    if dh is not None:
        _need(dh, torch.bfloat16, (T, D), "dh")
    dd = BITNET_BF16
    if dw is not None:
        dd = _value_dtype(dw, "dw")
        _need(dw, dw.dtype, (V, D), "dw")
    _same_device(h, w=w, targets=targets, lse=lse, dloss=dloss, dh=dh, dw=dw, workspace=workspace)
    if workspace is None:
        workspace = _workspace(bitnet_xent_bwd_workspace_bytes(T, V, D), h, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run(lib().bitnet_xent_bwd, h, stream, _ptr(h), _ptr(w), _ptr(targets), int(ignore_index), _ptr(lse), _ptr(dloss),
         int(reduce), T, V, D, _ptr(dh), _ptr(dw), dd, _ptr(workspace), ws_bytes)


# --- test hooks --------------------------------------------------------------

def bitnet_set_test_knobs(split_ctas=0, pair_cols=0, no_skinny=0, spin_limit=None):
    """Process-wide launch knobs (see the header); no arguments restores the
    defaults (cost models, default spin limit)."""
    L = lib()
    if spin_limit is None:
        spin_limit = int(L.bitnet_default_spin_limit())
    L.bitnet_set_test_knobs(int(split_ctas), int(pair_cols), int(no_skinny), int(spin_limit))


def bitnet_split_timeouts():
    """Waits for partial tiles that gave up since the last call (synchronizes
    the device)."""
    c = ctypes.c_uint32(0)
    _check(lib().bitnet_split_timeouts(ctypes.byref(c)))
    return int(c.value)


def bitnet_quantize_recomputes():
    """Partial sums one-pass quantize launches computed themselves after
    their wait gave up, since the last call (synchronizes the device)."""
    c = ctypes.c_uint32(0)
    _check(lib().bitnet_quantize_recomputes(ctypes.byref(c)))
    return int(c.value)


def bitnet_debug_split_pieces(tiles, stages, grid):
    """The pieces of a split launch, as numpy arrays keyed v, t, s0, s1,
    slot, va, n (host-side computation; no GPU needed)."""
    import numpy as np

    L = lib()
    cap = int(grid) + int(tiles) + 1
    arrs = {k: np.zeros(cap, dtype=np.int32) for k in ("v", "t", "s0", "s1", "va", "n")}
    arrs["slot"] = np.zeros(cap, dtype=np.int64)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    n = int(L.bitnet_debug_split_pieces(int(tiles), int(stages), int(grid), ptr(arrs["v"]), ptr(arrs["t"]),
                                        ptr(arrs["s0"]), ptr(arrs["s1"]), ptr(arrs["slot"]), ptr(arrs["va"]),
                                        ptr(arrs["n"]), cap))
    if n < 0 or n > cap:
        raise ValueError(f"bitnet_debug_split_pieces({tiles}, {stages}, {grid}) returned {n}")
    return {k: a[:n] for k, a in arrs.items()}


def bitnet_debug_partial_slots(tiles, grid):
    return int(lib().bitnet_debug_partial_slots(int(tiles), int(grid)))


def bitnet_debug_cta_order(grid):
    import numpy as np

    out = np.zeros(int(grid), dtype=np.int32)
    lib().bitnet_debug_cta_order(int(grid), out.ctypes.data_as(ctypes.c_void_p))
    return out


def bitnet_debug_mfma_probe(int8, iters, sink, stream=None):
    """Enqueue the MFMA rate probe; returns the operations it performs.
    sink: float32 [2048] on the GPU."""
    _need(sink, torch.float32, (2048,), "sink")
    ops = ctypes.c_double(0.0)
    _check(lib().bitnet_debug_mfma_probe(1 if int8 else 0, int(iters), _ptr(sink), ctypes.byref(ops), _stream(stream)))
    return float(ops.value)
