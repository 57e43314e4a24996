"""Python binding of libsvdq (include/svdq.h): argument marshalling only.

Every function keeps the C name and forwards raw pointers and the current CUDA
stream of PyTorch; PyTorch only provides device memory and streams.  There is
no fallback: if the library is missing the import fails, and on a device that
is not sm_100 the calls raise.
"""

import ctypes
import functools
import operator
import os

import numpy as np
import torch

from .build import LIB_PATH

RANK = 32

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "device is not sm_100 (B200)",
           4: "CUDA error", 5: "kernel wait timed out", 6: "device-side scale product out of range (clamped)"}


class SvdqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, 'unknown')} (status {status})")


class LoraPlanStruct(ctypes.Structure):
    """svdq_lora_plan of the header: the sizes of a packed plan."""
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "requests", "slots", "adapters", "tiles", "copy_tiles", "groups",
                                              "copy_groups")] + [("bytes", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libsvdq.so not built at {LIB_PATH}; run `python bit_diffusion_transformer_act_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    sig = {
        "svdq_status_string": ([i], ctypes.c_char_p),
        "svdq_abi_version": ([], i),
        "svdq_packed_weight_bytes": ([i, i, i], sz),
        "svdq_pack_weights": ([vp, vp, vp, vp, vp, i, i, i, vp, sz, ctypes.POINTER(ctypes.c_float)], i),
        "svdq_act_scale_bytes": ([i, i], sz),
        "svdq_quantize_act_lowrank_down": ([vp, vp, vp, i, i, i, f, vp, vp, vp, vp], i),
        "svdq_w4a4_nvfp4_linear": ([vp, vp, vp, f, vp, f, i, i, i, i, vp, vp], i),
        "svdq_w4a4_nvfp4_linear_qkv": ([vp, vp, vp, f, vp, f, i, i, i, i, i, i, vp, vp, f, vp, vp, vp, vp], i),
        "svdq_gelu_quant_workspace_bytes": ([i, i], sz),
        "svdq_gelu_table_bytes": ([], sz),
        "svdq_int4_packed_weight_bytes": ([i, i, i], sz),
        "svdq_int4_pack_weights": ([vp, vp, vp, vp, vp, i, i, i, vp, sz], i),
        "svdq_int4_quantize_act_lowrank_down": ([vp, vp, vp, i, i, i, vp, vp, vp, vp], i),
        "svdq_w4a4_int4_linear": ([vp, vp, vp, vp, i, i, i, i, vp, vp], i),
        "svdq_gelu_table_fill": ([vp, vp], i),
        "svdq_w4a4_nvfp4_linear_gelu_quant": ([vp, vp, vp, f, vp, f, i, i, i, i, vp, vp, f, vp, vp, vp, vp, sz, vp, vp,
                                               vp], i),
        "awq_w4a16_linear": ([vp, vp, vp, vp, vp, i, i, i, vp, vp], i),
        "svdq_act_amax": ([vp, vp, i, i, vp, vp], i),
        "svdq_act_amax_noalloc": ([vp, vp, i, i, vp, vp], i),
        "svdq_quantize_act_lowrank_down_dyn": ([vp, vp, vp, i, i, i, vp, vp, vp, vp, vp], i),
        "svdq_w4a4_nvfp4_linear_dyn": ([vp, vp, vp, vp, vp, f, i, i, i, i, vp, vp], i),
        "svdq_unswizzle_scales": ([vp, i, i, vp], i),
        "svdq_swizzle_scales": ([vp, i, i, vp], i),
        "svdq_device_status": ([i], i),
        "svdq_selftest_wait_timeout": ([vp], i),
        "svdq_lora_plan_bytes": ([i, i, i], sz),
        "svdq_lora_plan_pack": ([vp, vp, vp, i, i, i, i, vp, sz, vp], i),
        "svdq_lora_workspace_bytes": ([vp, i, i], sz),
        "svdq_lora_add": ([vp, i64, vp, i64, vp, vp, vp, vp, sz, i, i, i, i, vp, sz, vp, i64, vp], i),
        "svdq_qk_norm_rope": ([vp, i64, i64, i, vp, i64, i64, i, i, i, vp, vp, f, vp, i, i, i, vp, vp, i, vp, i64, i64,
                               vp, i64, i64, vp], i),
        "svdq_rope_axes_tables": ([vp, i, i, i, vp, vp, i, i, vp, vp, vp], i),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


LIB = _load()
EXPORTED = ("svdq_status_string", "svdq_abi_version", "svdq_packed_weight_bytes", "svdq_pack_weights",
            "svdq_act_scale_bytes", "svdq_quantize_act_lowrank_down", "svdq_w4a4_nvfp4_linear",
            "awq_w4a16_linear", "svdq_unswizzle_scales", "svdq_swizzle_scales", "svdq_device_status",
            "svdq_act_amax", "svdq_quantize_act_lowrank_down_dyn", "svdq_w4a4_nvfp4_linear_dyn",
            "svdq_act_amax_noalloc", "svdq_w4a4_nvfp4_linear_qkv", "svdq_gelu_quant_workspace_bytes",
            "svdq_w4a4_nvfp4_linear_gelu_quant", "svdq_selftest_wait_timeout", "svdq_gelu_table_bytes",
            "svdq_gelu_table_fill", "svdq_int4_packed_weight_bytes", "svdq_int4_pack_weights",
            "svdq_int4_quantize_act_lowrank_down", "svdq_w4a4_int4_linear", "svdq_lora_plan_bytes",
            "svdq_lora_plan_pack", "svdq_lora_workspace_bytes", "svdq_lora_add", "svdq_qk_norm_rope",
            "svdq_rope_axes_tables")


def _check(fn, st):
    if st != 0:
        raise SvdqError(fn, st)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _np_ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p) if a is not None else None


def _on_device(t, name):
    """Device calls take raw pointers: a host tensor (or one on another GPU) would be read as
    device memory, so it is refused here, before the call."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _require(t, dtype, shape, name):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {dtype} tensor of shape {tuple(shape)}, got "
                         f"{getattr(t, 'dtype', type(t))} {tuple(getattr(t, 'shape', ()))}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on_device(t, name)


def _device_of(t):
    """The current device where `t` is a CUDA tensor, else -1 (the checks of the call's tensors refuse it)."""
    return torch._C._cuda_getDevice() if isinstance(t, torch.Tensor) and t.is_cuda else -1


def _addr(t, dtype, shape, name, dev):
    """The address of a tensor of that type and shape, contiguous and on device `dev` (the current one).
    One pass of cheap comparisons; what they reject, _require explains."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and
            t.get_device() == dev >= 0):
        _require(t, dtype, shape, name)
    return t.data_ptr()


def _writable(t, name):
    """Refuses an output tensor that the calling code differentiates: the call writes through its address, which
    its graph would not know of."""
    if torch.is_grad_enabled() and getattr(t, "requires_grad", False):
        raise ValueError(f"{name} carries gradients, which this call has none of: call it under torch.no_grad(), or on "
                         "a detached tensor")


def _written(*tensors):
    """Counts the call's writes to tensors of the caller's, so that a graph that saved one of them notices."""
    for t in tensors:
        torch.autograd.graph.increment_version(t)


def _l1_section_end(K, rank):
    """Bytes of the packed blob that the activation kernel reads: the 1 KB header and the
    low-rank down factor section that follows it (two bf16 [rank, K] parts, hi and lo).  The C
    call has no size argument, so this is the only guard against a blob that is too short
    (or packed for a smaller K)."""
    return 1024 + 4 * rank * K


def _require_blob(t, name, min_bytes=0):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < min_bytes:
        raise ValueError(f"{name}: expected a contiguous uint8 tensor of at least {min_bytes} bytes")
    _on_device(t, name)


# ---------------------------------------------------------------- host side

def svdq_packed_weight_bytes(N, K, rank=RANK):
    return int(LIB.svdq_packed_weight_bytes(N, K, rank))


def svdq_act_scale_bytes(M, K):
    return int(LIB.svdq_act_scale_bytes(M, K))


def svdq_pack_weights(R, L1_bits, L2_bits, bias_bits, smooth_bits):
    """R float32 [N, K]; L1 bf16 bits uint16 [K, r]; L2 bits [r, N]; bias bits [N] or None;
    smooth_inv bits [K] (the same vector later given to the activation kernel).

    Returns (blob uint8 numpy array, w_global_scale float)."""
    R = np.ascontiguousarray(R, dtype=np.float32)
    N, K = R.shape
    L1_bits = np.ascontiguousarray(L1_bits, dtype=np.uint16)
    L2_bits = np.ascontiguousarray(L2_bits, dtype=np.uint16)
    rank = L1_bits.shape[1]
    if L1_bits.shape != (K, rank) or L2_bits.shape != (rank, N):
        raise ValueError("L1 must be [K, r] and L2 [r, N]")
    if bias_bits is not None:
        bias_bits = np.ascontiguousarray(bias_bits, dtype=np.uint16)
        if bias_bits.shape != (N,):
            raise ValueError("bias must be [N]")
    smooth_bits = np.ascontiguousarray(smooth_bits, dtype=np.uint16)
    if smooth_bits.shape != (K,):
        raise ValueError("smooth_inv must be [K]")
    nbytes = svdq_packed_weight_bytes(N, K, rank)
    if nbytes == 0:
        _check("svdq_pack_weights", 2)
    out = np.empty(nbytes, dtype=np.uint8)
    g = ctypes.c_float(0.0)
    st = LIB.svdq_pack_weights(_np_ptr(R), _np_ptr(L1_bits), _np_ptr(L2_bits), _np_ptr(bias_bits),
                               _np_ptr(smooth_bits), N, K, rank, _np_ptr(out), nbytes, ctypes.byref(g))
    _check("svdq_pack_weights", st)
    return out, float(g.value)


def svdq_int4_pack_weights(R, L1_bits, L2_bits, bias_bits, smooth_bits):
    """The int4 / group-64 row's packed weights (numpy uint8 blob) of R float32 [N, K], L1 bits
    [K, r], L2 bits [r, N], bias bits [N] or None, smooth_inv bits [K]."""
    R = np.ascontiguousarray(R, dtype=np.float32)
    N, K = R.shape
    L1_bits = np.ascontiguousarray(L1_bits, dtype=np.uint16)
    L2_bits = np.ascontiguousarray(L2_bits, dtype=np.uint16)
    rank = L1_bits.shape[1]
    if L1_bits.shape != (K, rank) or L2_bits.shape != (rank, N):
        raise ValueError("L1 must be [K, r] and L2 [r, N]")
    if bias_bits is not None:
        bias_bits = np.ascontiguousarray(bias_bits, dtype=np.uint16)
        if bias_bits.shape != (N,):
            raise ValueError("bias must be [N]")
    smooth_bits = np.ascontiguousarray(smooth_bits, dtype=np.uint16)
    if smooth_bits.shape != (K,):
        raise ValueError("smooth_inv must be [K]")
    nbytes = int(LIB.svdq_int4_packed_weight_bytes(N, K, rank))
    if nbytes == 0:
        _check("svdq_int4_pack_weights", 2)
    out = np.empty(nbytes, dtype=np.uint8)
    _check("svdq_int4_pack_weights", LIB.svdq_int4_pack_weights(_np_ptr(R), _np_ptr(L1_bits), _np_ptr(L2_bits),
                                                                 _np_ptr(bias_bits), _np_ptr(smooth_bits), N, K,
                                                                 rank, _np_ptr(out), nbytes))
    return out


def svdq_unswizzle_scales(swizzled, rows, K):
    """Swizzled scale bytes (numpy uint8 or a torch tensor) -> numpy uint8 [rows, K/16]."""
    if isinstance(swizzled, torch.Tensor):
        swizzled = swizzled.detach().cpu().numpy()
    sw = np.ascontiguousarray(swizzled, dtype=np.uint8)
    out = np.empty((rows, K // 16), dtype=np.uint8)
    _check("svdq_unswizzle_scales", LIB.svdq_unswizzle_scales(_np_ptr(sw), rows, K, _np_ptr(out)))
    return out


def svdq_swizzle_scales(plain, rows, K):
    plain = np.ascontiguousarray(plain, dtype=np.uint8)
    out = np.empty(svdq_act_scale_bytes(rows, K), dtype=np.uint8)
    _check("svdq_swizzle_scales", LIB.svdq_swizzle_scales(_np_ptr(plain), rows, K, _np_ptr(out)))
    return out


def svdq_device_status(clear=True):
    """Synchronizes the device and returns the library's status word (0 or 5)."""
    return int(LIB.svdq_device_status(1 if clear else 0))


# ---------------------------------------------------------------- device side

def svdq_quantize_act_lowrank_down(X, smooth_inv, packed_w, act_global_scale, rank=RANK,
                                   act_codes=None, act_scales=None, lowrank_act=None):
    """X bf16 [M, K] cuda; smooth_inv bf16 [K]; packed_w uint8 cuda (the blob).

    Returns (act_codes uint8 [M, K/2], act_scales uint8 [svdq_act_scale_bytes],
    lowrank_act bf16 [M, 2r] holding U / g_a as a high part then a low part)."""
    M, K = X.shape
    dev = X.device
    _require_blob(packed_w, "packed_w", _l1_section_end(K, rank))
    _require(X, torch.bfloat16, (M, K), "X")
    _require(smooth_inv, torch.bfloat16, (K,), "smooth_inv")
    if act_codes is None:
        act_codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if act_scales is None:
        act_scales = torch.empty((svdq_act_scale_bytes(M, K),), dtype=torch.uint8, device=dev)
    if lowrank_act is None:
        lowrank_act = torch.empty((M, 2 * rank), dtype=torch.bfloat16, device=dev)
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    st = LIB.svdq_quantize_act_lowrank_down(_ptr(X), _ptr(smooth_inv), _ptr(packed_w), M, K, rank,
                                            float(act_global_scale), _ptr(act_codes), _ptr(act_scales),
                                            _ptr(lowrank_act), _stream())
    _check("svdq_quantize_act_lowrank_down", st)
    return act_codes, act_scales, lowrank_act


def svdq_w4a4_nvfp4_linear(act_codes, act_scales, lowrank_act, act_global_scale, packed_w, w_global_scale,
                           M, N, K, rank=RANK, Y=None):
    """Returns Y bf16 [M, N] = bf16(g_a g_w Q(X_hat) Q(R)^T + lowrank_act L2 + b)."""
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    _require_blob(packed_w, "packed_w", svdq_packed_weight_bytes(N, K, rank))
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=act_codes.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    st = LIB.svdq_w4a4_nvfp4_linear(_ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act),
                                    float(act_global_scale), _ptr(packed_w), float(w_global_scale),
                                    M, N, K, rank, _ptr(Y), _stream())
    _check("svdq_w4a4_nvfp4_linear", st)
    return Y


def svdq_w4a4_nvfp4_linear_qkv(act_codes, act_scales, lowrank_act, act_global_scale, packed_w, w_global_scale,
                               M, N, K, heads, norm_wq, norm_wk, eps, rope_cos, rope_sin, rank=RANK, Y=None):
    """The fused Q/K/V projection: Y bf16 [M, N = 3 heads 128] holding q, k (RMS-normalised per
    head with norm_wq / norm_wk bf16 [128], then rotated by rope_cos / rope_sin float32 [64, M],
    pair-major) and v."""
    D = 128
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    _require_blob(packed_w, "packed_w", svdq_packed_weight_bytes(N, K, rank))
    _require(norm_wq, torch.bfloat16, (D,), "norm_wq")
    _require(norm_wk, torch.bfloat16, (D,), "norm_wk")
    _require(rope_cos, torch.float32, (D // 2, M), "rope_cos")
    _require(rope_sin, torch.float32, (D // 2, M), "rope_sin")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=act_codes.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    st = LIB.svdq_w4a4_nvfp4_linear_qkv(_ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act),
                                        float(act_global_scale), _ptr(packed_w), float(w_global_scale),
                                        M, N, K, rank, heads, D, _ptr(norm_wq), _ptr(norm_wk), float(eps),
                                        _ptr(rope_cos), _ptr(rope_sin), _ptr(Y), _stream())
    _check("svdq_w4a4_nvfp4_linear_qkv", st)
    return Y


def svdq_gelu_quant_workspace_bytes(M, N):
    return int(LIB.svdq_gelu_quant_workspace_bytes(M, N))


def svdq_gelu_table_fill(table=None, device=None):
    """The GELU table (uint8 [svdq_gelu_table_bytes()] CUDA tensor) filled by the library."""
    if table is None:
        table = torch.empty((int(LIB.svdq_gelu_table_bytes()),), dtype=torch.uint8,
                            device=device if device is not None else torch.device("cuda", torch.cuda.current_device()))
    _require_blob(table, "gelu_table", int(LIB.svdq_gelu_table_bytes()))
    _check("svdq_gelu_table_fill", LIB.svdq_gelu_table_fill(_ptr(table), _stream()))
    return table


_GELU_TABLES = {}


def _gelu_table(device):
    """A filled GELU table per device, made on first use (on the current stream)."""
    key = device.index if device.index is not None else torch.cuda.current_device()
    if key not in _GELU_TABLES:
        _GELU_TABLES[key] = svdq_gelu_table_fill(device=torch.device("cuda", key))
    return _GELU_TABLES[key]


def svdq_w4a4_nvfp4_linear_gelu_quant(act_codes, act_scales, lowrank_act, act_global_scale, packed_w, w_global_scale,
                                      M, N, K, down_smooth_inv, down_packed_w, down_act_global_scale, rank=RANK,
                                      out_codes=None, out_scales=None, out_lowrank_act=None, workspace=None,
                                      h_out=None, gelu_table=None):
    """The MLP up projection with GELU and the down projection's activation pass fused: returns the
    down projection's (act_codes uint8 [M, N/2], act_scales, lowrank_act bf16 [M, 2r]) for its
    smooth_inv (bf16 [N]), packed weights (its low-rank section is used) and g_a.  h_out (bf16
    [M, N]), if given, also receives the hidden state."""
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    _require_blob(packed_w, "packed_w", svdq_packed_weight_bytes(N, K, rank))
    _require(down_smooth_inv, torch.bfloat16, (N,), "down_smooth_inv")
    _require_blob(down_packed_w, "down_packed_w", _l1_section_end(N, rank))
    dev = act_codes.device
    if out_codes is None:
        out_codes = torch.empty((M, N // 2), dtype=torch.uint8, device=dev)
    if out_scales is None:
        out_scales = torch.empty((svdq_act_scale_bytes(M, N),), dtype=torch.uint8, device=dev)
    if out_lowrank_act is None:
        out_lowrank_act = torch.empty((M, 2 * rank), dtype=torch.bfloat16, device=dev)
    ws_bytes = svdq_gelu_quant_workspace_bytes(M, N)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, device=dev)
    _require(out_codes, torch.uint8, (M, N // 2), "out_codes")
    _require(out_scales, torch.uint8, (svdq_act_scale_bytes(M, N),), "out_scales")
    _require(out_lowrank_act, torch.bfloat16, (M, 2 * rank), "out_lowrank_act")
    _require_blob(workspace, "workspace", ws_bytes)
    if gelu_table is None:
        gelu_table = _gelu_table(dev)
    _require_blob(gelu_table, "gelu_table", int(LIB.svdq_gelu_table_bytes()))
    if h_out is not None:
        _require(h_out, torch.bfloat16, (M, N), "h_out")
    st = LIB.svdq_w4a4_nvfp4_linear_gelu_quant(_ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act),
                                               float(act_global_scale), _ptr(packed_w), float(w_global_scale),
                                               M, N, K, rank, _ptr(down_smooth_inv), _ptr(down_packed_w),
                                               float(down_act_global_scale), _ptr(out_codes), _ptr(out_scales),
                                               _ptr(out_lowrank_act), _ptr(workspace), workspace.numel(),
                                               _ptr(gelu_table), _ptr(h_out), _stream())
    _check("svdq_w4a4_nvfp4_linear_gelu_quant", st)
    return out_codes, out_scales, out_lowrank_act


def int4_padded_rows(M):
    """Rows of the int4 row's activation-scale array: M rounded up to a multiple of 128."""
    return (M + 127) // 128 * 128


def svdq_int4_quantize_act_lowrank_down(X, smooth_inv, packed_w, rank=RANK, act_codes=None, act_scales=None,
                                        lowrank_act=None):
    """The int4 row's activation pass: (act_codes uint8 [M, K] (E4M3 bytes of the int4 codes),
    act_scales bf16 [K/64, Mp] (group-major, rows padded to Mp = a multiple of 128 with zero
    scales), lowrank_act bf16 [M, 2r] (U as hi then lo))."""
    M, K = X.shape
    Mp = int4_padded_rows(M)
    dev = X.device
    _require_blob(packed_w, "packed_w", _l1_section_end(K, rank))
    _require(X, torch.bfloat16, (M, K), "X")
    _require(smooth_inv, torch.bfloat16, (K,), "smooth_inv")
    if act_codes is None:
        act_codes = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if act_scales is None:
        act_scales = torch.empty((K // 64, Mp), dtype=torch.bfloat16, device=dev)
    if lowrank_act is None:
        lowrank_act = torch.empty((M, 2 * rank), dtype=torch.bfloat16, device=dev)
    _require(act_codes, torch.uint8, (M, K), "act_codes")
    _require(act_scales, torch.bfloat16, (K // 64, Mp), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    st = LIB.svdq_int4_quantize_act_lowrank_down(_ptr(X), _ptr(smooth_inv), _ptr(packed_w), M, K, rank,
                                                 _ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act), _stream())
    _check("svdq_int4_quantize_act_lowrank_down", st)
    return act_codes, act_scales, lowrank_act


def svdq_w4a4_int4_linear(act_codes, act_scales, lowrank_act, packed_w, M, N, K, rank=RANK, Y=None):
    """Y bf16 [M, N] of the int4 / group-64 row."""
    _require(act_codes, torch.uint8, (M, K), "act_codes")
    _require(act_scales, torch.bfloat16, (K // 64, int4_padded_rows(M)), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    _require_blob(packed_w, "packed_w", int(LIB.svdq_int4_packed_weight_bytes(N, K, rank)))
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=act_codes.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    st = LIB.svdq_w4a4_int4_linear(_ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act), _ptr(packed_w), M, N, K,
                                   rank, _ptr(Y), _stream())
    _check("svdq_w4a4_int4_linear", st)
    return Y


def svdq_act_amax(X, smooth_inv, act_amax=None):
    """Returns the 16-byte device buffer (int32 [4]) whose word 0 holds the bits of
    max |X smooth_inv| (the dynamic scale's input); a buffer passed in must have been
    zero-filled once (the call leaves words 1-3 zero)."""
    M, K = X.shape
    _require(X, torch.bfloat16, (M, K), "X")
    _require(smooth_inv, torch.bfloat16, (K,), "smooth_inv")
    if act_amax is None:
        act_amax = torch.zeros((4,), dtype=torch.int32, device=X.device)
    _require(act_amax, torch.int32, (4,), "act_amax")
    st = LIB.svdq_act_amax(_ptr(X), _ptr(smooth_inv), M, K, _ptr(act_amax), _stream())
    _check("svdq_act_amax", st)
    return act_amax


def svdq_act_amax_noalloc(X, smooth_inv, amax):
    """max |X smooth_inv| into `amax` (a float32 [1] CUDA tensor), through the C call that
    allocates nothing (its scratch is the library's own static array; calls must not overlap
    on the GPU)."""
    M, K = X.shape
    _require(X, torch.bfloat16, (M, K), "X")
    _require(smooth_inv, torch.bfloat16, (K,), "smooth_inv")
    _require(amax, torch.float32, (1,), "amax")
    st = LIB.svdq_act_amax_noalloc(_ptr(X), _ptr(smooth_inv), M, K, _ptr(amax), _stream())
    _check("svdq_act_amax_noalloc", st)
    return amax


def svdq_quantize_act_lowrank_down_dyn(X, smooth_inv, packed_w, act_amax, rank=RANK,
                                       act_codes=None, act_scales=None, lowrank_act=None):
    """As svdq_quantize_act_lowrank_down with g_a formed on the device from act_amax."""
    M, K = X.shape
    dev = X.device
    _require_blob(packed_w, "packed_w", _l1_section_end(K, rank))
    _require(X, torch.bfloat16, (M, K), "X")
    _require(smooth_inv, torch.bfloat16, (K,), "smooth_inv")
    _require(act_amax, torch.int32, (4,), "act_amax")
    if act_codes is None:
        act_codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if act_scales is None:
        act_scales = torch.empty((svdq_act_scale_bytes(M, K),), dtype=torch.uint8, device=dev)
    if lowrank_act is None:
        lowrank_act = torch.empty((M, 2 * rank), dtype=torch.bfloat16, device=dev)
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    st = LIB.svdq_quantize_act_lowrank_down_dyn(_ptr(X), _ptr(smooth_inv), _ptr(packed_w), M, K, rank,
                                                _ptr(act_amax), _ptr(act_codes), _ptr(act_scales),
                                                _ptr(lowrank_act), _stream())
    _check("svdq_quantize_act_lowrank_down_dyn", st)
    return act_codes, act_scales, lowrank_act


def svdq_w4a4_nvfp4_linear_dyn(act_codes, act_scales, lowrank_act, act_amax, packed_w, w_global_scale,
                               M, N, K, rank=RANK, Y=None):
    """As svdq_w4a4_nvfp4_linear with g_a formed on the device from act_amax."""
    _require(act_codes, torch.uint8, (M, K // 2), "act_codes")
    _require(act_scales, torch.uint8, (svdq_act_scale_bytes(M, K),), "act_scales")
    _require(lowrank_act, torch.bfloat16, (M, 2 * rank), "lowrank_act")
    _require(act_amax, torch.int32, (4,), "act_amax")
    _require_blob(packed_w, "packed_w", svdq_packed_weight_bytes(N, K, rank))
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=act_codes.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    st = LIB.svdq_w4a4_nvfp4_linear_dyn(_ptr(act_codes), _ptr(act_scales), _ptr(lowrank_act), _ptr(act_amax),
                                        _ptr(packed_w), float(w_global_scale), M, N, K, rank, _ptr(Y), _stream())
    _check("svdq_w4a4_nvfp4_linear_dyn", st)
    return Y


def awq_w4a16_linear(X, qweight, scales, zeros, bias=None, Y=None):
    """X bf16 [M, K]; qweight uint8 [N, K/2]; scales, zeros bf16 [N, K/64]; bias bf16 [N] or None.

    With K % 512 == 0, K <= 4096 and scales / zeros 16-byte aligned (tensors of their own are)
    the kernels stage the scale and zero rows in shared memory: the faster path, with results
    bit-identical to those of any other alignment."""
    M, K = X.shape
    N = qweight.shape[0]
    _require(X, torch.bfloat16, (M, K), "X")
    _require(qweight, torch.uint8, (N, K // 2), "qweight")
    _require(scales, torch.bfloat16, (N, K // 64), "scales")
    _require(zeros, torch.bfloat16, (N, K // 64), "zeros")
    if bias is not None:
        _require(bias, torch.bfloat16, (N,), "bias")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _require(Y, torch.bfloat16, (M, N), "Y")
    st = LIB.awq_w4a16_linear(_ptr(X), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(bias), M, N, K,
                              _ptr(Y), _stream())
    _check("awq_w4a16_linear", st)
    return Y


def _int32_array(v, name):
    a = np.asarray(v)
    if a.size and (a.dtype.kind not in "iu" or a.min() < -(2 ** 31) or a.max() >= 2 ** 31):
        raise ValueError(f"{name}: 32-bit integers expected")
    return np.ascontiguousarray(a, dtype=np.int32)


LORA_MAX_RANK = 128                     # of slots * rank


class LoraPlan:
    """The plan of a batch whose requests carry low-rank adapters (svdq_lora_plan_pack): which rows belong
    to which request, which adapters each has, and how strongly.  One plan serves every layer and
    step of the batch.

    row_offsets [requests + 1] (host integers): request s owns rows row_offsets[s] .. row_offsets[s + 1] - 1
    of the `rows` rows; adapter_ids [requests, slots] (or [requests]), -1 for none; weights the same shape;
    adapters: how many the pool holds.  The plan is on the device when the constructor returns; keep it until the
    calls that use it, on whatever stream, and the graphs that hold such calls are done."""

    def __init__(self, row_offsets, adapter_ids, weights, rows, adapters, device="cuda"):
        off = _int32_array(row_offsets, "row_offsets").reshape(-1)
        ids = _int32_array(adapter_ids, "adapter_ids")
        w = np.ascontiguousarray(weights, dtype=np.float32)
        if ids.ndim == 1:
            ids, w = ids[:, None], w.reshape(-1, 1)
        if ids.ndim != 2 or ids.shape != w.shape or off.shape[0] != ids.shape[0] + 1:
            raise ValueError("row_offsets must be [requests + 1], adapter_ids and weights [requests, slots]")
        self.rows, self.adapters = int(rows), int(adapters)
        self.requests, self.slots = ids.shape
        self.struct = LoraPlanStruct()
        nbytes = int(LIB.svdq_lora_plan_bytes(self.rows, self.requests, self.slots))
        if nbytes == 0:
            _check("svdq_lora_plan_pack", 2)
        host = np.zeros(nbytes, dtype=np.uint8)
        _check("svdq_lora_plan_pack",
               LIB.svdq_lora_plan_pack(_np_ptr(off), _np_ptr(ids), _np_ptr(w), self.requests, self.slots, self.rows,
                                       self.adapters, _np_ptr(host), nbytes, ctypes.byref(self.struct)))
        self._keep(torch.from_numpy(host[: self.struct.bytes]).to(device))

    @classmethod
    def from_parts(cls, words, sizes):
        """The plan of a packed blob on the device and its struct's fields (`sizes()`)."""
        self = cls.__new__(cls)
        self.struct = LoraPlanStruct(*sizes)
        self.rows, self.requests = self.struct.M, self.struct.requests
        self.slots, self.adapters = self.struct.slots, self.struct.adapters
        _require_blob(words, "plan", self.struct.bytes)
        self._keep(words)
        return self

    def _keep(self, words):
        self.words = words
        self.nbytes = self.struct.bytes
        self.struct_ref = ctypes.byref(self.struct)
        self._workspace = {}

    def workspace_bytes(self, K, rank, dev):
        """svdq_lora_workspace_bytes on the current device `dev` (a number that follows from the sizes)."""
        n = self._workspace.get((K, rank, dev))
        if n is None:
            n = self._workspace[(K, rank, dev)] = svdq_lora_workspace_bytes(self, K, rank)
        return n

    def sizes(self):
        return [getattr(self.struct, n) for n, _ in LoraPlanStruct._fields_]


def _row_strided(t, rows, cols, name, dev):
    """A bf16 [rows, cols] tensor on device `dev` (the current one) whose rows may be apart (a column window
    of a wider one): (address, row stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != (rows, cols):
        raise ValueError(f"{name}: expected a torch.bfloat16 tensor of shape {(rows, cols)}, got "
                         f"{getattr(t, 'dtype', type(t))} {tuple(getattr(t, 'shape', ()))}")
    ld, inner = t.stride()
    if rows <= 1:
        ld = cols
    if (cols > 1 and inner != 1) or ld < cols:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    if not t.get_device() == dev >= 0:
        _on_device(t, name)
    return t.data_ptr(), ld


def svdq_lora_workspace_bytes(plan, K, rank):
    return int(LIB.svdq_lora_workspace_bytes(ctypes.byref(plan.struct), K, rank))


def svdq_lora_add(X, Y, A, B, plan, out=None, workspace=None):
    """Y + the adapters of each request: out[m] = Y[m] + sum_j w[s, j] B[id] (A[id] X[m]) for the rows m of
    request s of `plan` (a LoraPlan); rows without an adapter keep Y.

    X bf16 [M, K], Y bf16 [M, N] (a projection's output for X), rows possibly strided; A bf16
    [adapters, rank, K], B bf16 [adapters, N, rank].  out: Y itself for in place, a [M, N] tensor that
    overlaps neither, or None for a new one.  Returns out, which is no part of an autograd graph."""
    if not isinstance(plan, LoraPlan):
        raise ValueError("plan must be a LoraPlan")
    _writable(out, "out")
    M, K = X.shape
    adapters, rank, _ = A.shape
    N = Y.shape[1]
    if M != plan.rows or adapters != plan.adapters:
        raise ValueError(f"the plan is for {plan.rows} rows and {plan.adapters} adapters, got {M} and {adapters}")
    bf16 = torch.bfloat16
    dev = _device_of(X)
    xp, ldx = _row_strided(X, M, K, "X", dev)
    yp, ldyin = _row_strided(Y, M, N, "Y", dev)
    ap = _addr(A, bf16, (adapters, rank, K), "A", dev)
    bp = _addr(B, bf16, (adapters, N, rank), "B", dev)
    words = plan.words
    if words.get_device() != dev:
        _require_blob(words, "plan", plan.struct.bytes)
    given = out is not None
    if given:
        op, ldy = _row_strided(out, M, N, "out", dev)
    else:
        out = Y.new_empty(M, N)
        op, ldy = out.data_ptr(), N
    ws_bytes = plan.workspace_bytes(K, rank, dev)
    if workspace is None:
        workspace = words.new_empty(ws_bytes)
    else:
        _require_blob(workspace, "workspace", ws_bytes)
    st = LIB.svdq_lora_add(xp, ldx, yp, ldyin, ap, bp, plan.struct_ref, words.data_ptr(), plan.nbytes, M, N, K, rank,
                           workspace.data_ptr(), workspace.numel(), op, ldy, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check("svdq_lora_add", st)
    if given:
        _written(out)
    return out


@functools.lru_cache(maxsize=64)
def _axes_arrays(dims, theta):
    """The ctypes arrays of axes of these widths (a tuple) and thetas (one, or a tuple)."""
    thetas = theta if isinstance(theta, tuple) else (theta,) * len(dims)
    if len(thetas) != len(dims):
        raise ValueError(f"{len(dims)} axes need one theta or {len(dims)}")
    return (ctypes.c_int32 * len(dims))(*dims), (ctypes.c_double * len(dims))(*thetas)


def _rope_axes(positions, axes_dims, theta):
    """Checked positions and the ctypes arrays of the axes: (device, P, axes, is_float, dims, thetas)."""
    is_float = isinstance(positions, torch.Tensor) and positions.dtype is torch.float32
    if not isinstance(positions, torch.Tensor) or not (is_float or positions.dtype is torch.int32) or \
            positions.dim() != 2 or not positions.is_contiguous():
        raise ValueError("positions: expected a contiguous int32 or float32 tensor [P, axes]")
    dev = _device_of(positions)
    if positions.get_device() != dev or dev < 0:
        _on_device(positions, "positions")
    P, axes = positions.shape
    if len(axes_dims) != axes:
        raise ValueError(f"{axes} axes need {axes} widths, got {len(axes_dims)}")
    # plain numbers: the cache must not go by the identity of something that may change
    dims, thetas = _axes_arrays(tuple(map(operator.index, axes_dims)),
                                tuple(map(float, theta)) if isinstance(theta, (list, tuple)) else float(theta))
    return dev, P, axes, int(is_float), dims, thetas


_PAIRINGS = {"interleaved": 0, "half": 1}


def _heads(t, M, D, name, dev):
    """A bf16 [M, heads, D] tensor on device `dev` (the current one) with any strides over tokens and heads:
    (address, token stride, head stride, heads)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise ValueError(f"{name}: expected a torch.bfloat16 tensor [{M}, heads, {D}], got "
                         f"{getattr(t, 'dtype', type(t))} {tuple(getattr(t, 'shape', ()))}")
    rows, heads, width = t.shape
    row, head, inner = t.stride()
    if rows != M or width != D:
        raise ValueError(f"{name}: expected a torch.bfloat16 tensor [{M}, heads, {D}], got {tuple(t.shape)}")
    if inner != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if not t.get_device() == dev >= 0:
        _on_device(t, name)
    return t.data_ptr(), row, head, heads


def _heads_in_out(t, out, w, M, D, name, dev):
    """(address, token stride, head stride, heads) of q or k, its output and that one's address and strides, the
    address of its norm weights; a missing t has none of them."""
    if t is None:
        if out is not None or w is not None:
            raise ValueError(f"out_{name} and norm_w{name} need {name}")
        return None, 0, 0, 0, None, None, 0, 0, None
    tp, row, head, heads = _heads(t, M, D, name, dev)
    if out is None:
        out = t.new_empty(M, heads, D)
        op, orow, ohead = out.data_ptr(), heads * D, D
    else:
        op, orow, ohead, oheads = _heads(out, M, D, "out_" + name, dev)
        if oheads != heads:
            raise ValueError(f"out_{name} must have {heads} heads, got {oheads}")
    wp = _addr(w, torch.bfloat16, (D,), "norm_w" + name, dev) if w is not None else None
    return tp, row, head, heads, out, op, orow, ohead, wp


def svdq_qk_norm_rope(q, k, norm_wq, norm_wk, eps, positions, axes_dims, theta, pairing="interleaved", out_q=None,
                      out_k=None):
    """Per-head RMSNorm and rotary positions with several axes: q bf16 [M, q_heads, D] and k bf16
    [M, k_heads, D] (or None), with any strides over tokens and heads (views of a packed projection),
    norm_wq / norm_wk bf16 [D] or None for no normalisation, positions int32 or float32 [P, axes]
    (token m has position m % P), axes_dims the rotated columns of each axis, theta one value or one per axis,
    pairing "interleaved" or "half".  out_q / out_k: q / k themselves for in place, tensors of their
    shape, or None for new ones.  Returns (out_q, out_k), which are no part of an autograd graph."""
    if q is None and k is None:
        raise ValueError("q or k is needed")
    _writable(out_q, "out_q")
    _writable(out_k, "out_k")
    given = [t for t in (out_q, out_k) if t is not None]
    M, _, D = (q if q is not None else k).shape
    dev, P, axes, is_float, dims, thetas = _rope_axes(positions, axes_dims, theta)
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing: one of {sorted(_PAIRINGS)}, got {pairing!r}")
    qp, qr, qh, nq, out_q, oqp, oqr, oqh, wq = _heads_in_out(q, out_q, norm_wq, M, D, "q", dev)
    kp, kr, kh, nk, out_k, okp, okr, okh, wk = _heads_in_out(k, out_k, norm_wk, M, D, "k", dev)
    st = LIB.svdq_qk_norm_rope(qp, qr, qh, nq, kp, kr, kh, nk, M, D, wq, wk, eps, positions.data_ptr(), is_float, P,
                               axes, dims, thetas, _PAIRINGS[pairing], oqp, oqr, oqh, okp, okr, okh,
                               torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check("svdq_qk_norm_rope", st)
    _written(*given)
    return out_q, out_k


def svdq_rope_axes_tables(positions, axes_dims, theta, head_dim, rows=None, rope_cos=None, rope_sin=None):
    """The (cos, sin) tables, float32 [head_dim / 2, rows], of positions with several axes, in the layout
    of svdq_w4a4_nvfp4_linear_qkv; arguments as svdq_qk_norm_rope (rows: a multiple of P, by default P)."""
    dev, P, axes, is_float, dims, thetas = _rope_axes(positions, axes_dims, theta)
    M = P if rows is None else rows
    shape = (head_dim // 2, M)
    tables, given = [], []
    for t, name in ((rope_cos, "rope_cos"), (rope_sin, "rope_sin")):
        if t is None:
            t = positions.new_empty(*shape, dtype=torch.float32)
            tables.append((t, t.data_ptr()))
        else:
            _writable(t, name)
            given.append(t)
            tables.append((t, _addr(t, torch.float32, shape, name, dev)))
    (rope_cos, cp), (rope_sin, sp) = tables
    st = LIB.svdq_rope_axes_tables(positions.data_ptr(), is_float, P, axes, dims, thetas, M, head_dim, cp, sp,
                                   torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check("svdq_rope_axes_tables", st)
    _written(*given)
    return rope_cos, rope_sin


# ---------------------------------------------------------------- layers

class SvdqW4A4Linear:
    """An SVDQuant W4A4 NVFP4 linear layer held on one GPU.

    Built from the exporter's parameters: residual R [N, K] (float32), L1 [K, r],
    L2 [r, N], bias [N] (bf16 bit patterns as uint16, or None), smooth_inv [K]
    (bf16 bits) and the static activation scale g_a (a power of two)."""

    def __init__(self, R, L1_bits, L2_bits, bias_bits, smooth_inv_bits, act_global_scale, device="cuda"):
        blob, g_w = svdq_pack_weights(R, L1_bits, L2_bits, bias_bits, smooth_inv_bits)
        self.N, self.K = R.shape
        self.rank = L1_bits.shape[1]
        self.packed = torch.from_numpy(blob).to(device)
        self.w_global_scale = g_w
        self.act_global_scale = float(act_global_scale)
        self.smooth_inv = torch.from_numpy(np.ascontiguousarray(smooth_inv_bits, np.uint16).view(np.int16)) \
            .view(torch.bfloat16).to(device)

    def __call__(self, X, Y=None):
        M = X.shape[0]
        codes, scales, U = svdq_quantize_act_lowrank_down(X, self.smooth_inv, self.packed, self.act_global_scale,
                                                          self.rank)
        return svdq_w4a4_nvfp4_linear(codes, scales, U, self.act_global_scale, self.packed, self.w_global_scale,
                                      M, self.N, self.K, self.rank, Y)


class AwqW4A16Linear:
    """An AWQ-style W4A16 int4 (group 64) linear layer held on one GPU."""

    def __init__(self, qweight, scales, zeros, bias=None):
        self.qweight, self.scales, self.zeros, self.bias = qweight, scales, zeros, bias

    def __call__(self, X, Y=None):
        return awq_w4a16_linear(X, self.qweight, self.scales, self.zeros, self.bias, Y)
