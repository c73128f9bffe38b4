"""Python binding of libkimodo.so, the B200 two-stage DDIM denoiser.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the shared library is missing or cannot
be loaded, every entry point raises.  Tensors may be torch tensors (CUDA or CPU)
or numpy arrays; the library detects host versus device memory itself.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

__all__ = ["KimodoError", "load_library", "Kimodo", "N_PARAMS", "FP32", "BF16", "NET_ROOT", "NET_BODY"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkimodo.so")

N_PARAMS = 281_963_799
FP32, BF16 = 0, 1
NET_ROOT, NET_BODY = 0, 1
TEXT_DIM, MOTION_DIM, ROOT_DIM, BODY_DIM = 4096, 279, 5, 274
STATUS = {0: "OK", -1: "EINVAL", -2: "ENOMEM", -3: "ECUDA", -4: "EUNSUPPORTED", -5: "ETIMEOUT"}

# (name, restype, argtypes) for every symbol declared in include/kimodo.h
_P, _I, _F, _SZ, _LL, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_void_p
SIGNATURES = [
    ("kimodo_load_weights", _I, [ctypes.POINTER(_P), _P, _SZ, _I, _I]),
    ("kimodo_denoiser_forward", _I, [_P, _I, _P, _P, _I, _P, _I, _I, _P, _P]),
    ("kimodo_denoiser_forward_noalloc", _I, [_P, _I, _P, _P, _I, _P, _I, _I, _P, _P]),
    ("kimodo_ddim_step", _I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _F, _P, _P]),
    ("kimodo_ddim_sample", _I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _P, _P]),
    ("kimodo_ddim_step_ex", _I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _F, _P, _P, _P]),
    ("kimodo_ddim_sample_ex", _I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _P, _P, _P]),
    ("kimodo_sync_status", _I, [_P, _P]),
    ("kimodo_wait_selftest", _I, [_P, _I, _P]),
    ("kimodo_profile_enable", _I, [_P, _I]),
    ("kimodo_profile_read", _I, [_P, _I, _P, _P, _P, _P]),
    ("kimodo_last_launch_count", _LL, [_P]),
    ("kimodo_free", None, [_P]),
    ("kimodo_last_error", ctypes.c_char_p, []),
    # include/kimodo_kernels.h
    ("kimodo_gemm_bf16", _I, [_P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    ("kimodo_gemm_bf16_pair", _I, [_P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    ("kimodo_gemm_f32", _I, [_P, _I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    ("kimodo_attention_bf16", _I, [_P, _P, _P, _I, _I, _P]),
    ("kimodo_attention_f32", _I, [_P, _P, _P, _I, _I, _P]),
    ("kimodo_layernorm", _I, [_P, _P, _I, _P, _P, _I, _P]),
    ("kimodo_global_to_local_root", _I, [_P, _P, _P, _I, _I, _P, _P]),
    ("kimodo_quantize_int8", _I, [_P, _LL, _I, _P, _LL, _P, _I, _I, _P]),
    ("kimodo_rms_norm_int8", _I, [_P, _LL, _I, _P, _LL, _P, _LL, _I, _P, _F, _P, _LL, _P, _I, _I, _P]),
    ("kimodo_gemm_int8", _I, [_P, _LL, _P, _P, _LL, _P, _P, _P, _LL, _P, _LL, _I, _I, _I, _I, _I, _P]),
    ("kimodo_attention_scored_workspace", _I, [_P, _P]),
    ("kimodo_attention_scored", _I, [_P, _P, _SZ, _P]),
    ("kimodo_kernel_status", _I, [_P]),
]
EPI_BIAS, EPI_BIAS_GELU, EPI_BIAS_SILU, EPI_BIAS_RESID = 0, 1, 2, 3


SCHEDULES = {"linear": 0, "cosine": 1}


class SamplerOptions(ctypes.Structure):
    """struct kimodo_sampler of include/kimodo.h."""
    _fields_ = [("schedule", ctypes.c_int), ("eta", ctypes.c_float), ("step_noise", ctypes.c_void_p),
                ("text_batch", ctypes.c_int)]


class ScoredAttention(ctypes.Structure):
    """struct kimodo_scored_attention of include/kimodo_kernels.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "slopes", "prefix", "q_documents", "kv_documents",
                                                "kv_lengths", "q_start")]
                + [(n, ctypes.c_longlong * 3) for n in ("q_strides", "k_strides", "v_strides", "out_strides")]
                + [(n, ctypes.c_int) for n in ("batch", "q_len", "kv_len", "q_heads", "kv_heads", "head_dim", "dtype",
                                               "causal")]
                + [("scale", ctypes.c_float), ("cap", ctypes.c_float)])


class KimodoError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"kimodo {STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libkimodo.so and declare its C signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m transformer_denoiser_b200.build`")
    lib = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise KimodoError(status, _lib.kimodo_last_error().decode())


def _ptr(a):
    """Data pointer of a contiguous torch tensor or numpy array."""
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        if not a.flags.c_contiguous:
            raise ValueError("numpy arrays must be C-contiguous")
        return a.ctypes.data
    if not a.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return a.data_ptr()


def _ptr_rows(a):
    """Data pointer of a row-major 2-D tensor whose rows may be padded (stride(1) == 1)."""
    if a is None:
        return None
    if a.dim() != 2 or a.stride(1) != 1:
        raise ValueError("need a 2-D tensor with unit column stride")
    return a.data_ptr()


def _is_cuda(a):
    return hasattr(a, "is_cuda") and a.is_cuda


def _stream(stream, *tensors):
    if stream is not None:
        return stream
    if any(_is_cuda(t) for t in tensors):
        import torch
        return torch.cuda.current_stream().cuda_stream
    return None


def _like(ref, shape, dtype_np=np.float32):
    if _is_cuda(ref):
        import torch
        return torch.empty(shape, dtype=torch.float32, device=ref.device)
    return np.empty(shape, dtype=dtype_np)


def _f32(a):
    if isinstance(a, np.ndarray):
        return np.ascontiguousarray(a, dtype=np.float32)
    return a.contiguous()


def _i32(a):
    if isinstance(a, np.ndarray) or isinstance(a, (list, tuple)):
        return np.ascontiguousarray(np.asarray(a), dtype=np.int32)
    return a.contiguous()


def _cur_stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------ kernel-level calls (torch CUDA tensors)

def gemm_bf16(A, W, bias, epilogue=EPI_BIAS, out_f32=False, resid=None, out=None, K=None, tile_n=0, pair=False):
    """out = epilogue(A[:, :K] W[:, :K]^T + bias) on the tcgen05 GEMM (A, W bf16 CUDA tensors);
    pair=True runs the CTA-pair kernel (256-row tiles)."""
    import torch
    lib = load_library()
    M, N = A.shape[0], W.shape[0]
    K = A.shape[1] if K is None else K
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32 if out_f32 else torch.bfloat16, device=A.device)
    args = [_ptr_rows(A), A.stride(0), _ptr_rows(W), W.stride(0), _ptr(bias), _ptr_rows(resid),
            0 if resid is None else resid.stride(0), _ptr_rows(out), out.stride(0), M, N, K,
            int(epilogue), int(bool(out_f32))]
    fn = lib.kimodo_gemm_bf16_pair if pair else lib.kimodo_gemm_bf16
    _check(fn(*args, int(tile_n), _cur_stream()))
    return out


def gemm_f32(A, W, bias, epilogue=EPI_BIAS, resid=None, out=None, K=None):
    import torch
    lib = load_library()
    M, N = A.shape[0], W.shape[0]
    K = A.shape[1] if K is None else K
    out = torch.empty((M, N), dtype=torch.float32, device=A.device) if out is None else out
    _check(lib.kimodo_gemm_f32(_ptr(A), A.stride(0), _ptr(W), W.stride(0), _ptr(bias), _ptr(resid),
                               0 if resid is None else resid.stride(0), _ptr(out), out.stride(0), M, N, K,
                               int(epilogue), _cur_stream()))
    return out


def attention(qkv, lengths, nseq, S):
    """Masked attention over qkv [nseq*S, 3072] (CUDA tensor): bf16 runs the tcgen05
    kernel, fp32 the fp32 one."""
    import torch
    lib = load_library()
    out = torch.empty((nseq * S, 1024), dtype=qkv.dtype, device=qkv.device)
    fn = lib.kimodo_attention_bf16 if qkv.dtype == torch.bfloat16 else lib.kimodo_attention_f32
    _check(fn(_ptr(qkv), _ptr(out), _ptr(lengths), nseq, S, _cur_stream()))
    return out


def layernorm(y, gamma, beta, out_bf16=True):
    import torch
    lib = load_library()
    out = torch.empty(y.shape, dtype=torch.bfloat16 if out_bf16 else torch.float32, device=y.device)
    _check(lib.kimodo_layernorm(_ptr(y), _ptr(out), int(bool(out_bf16)), _ptr(gamma), _ptr(beta), y.shape[0],
                                _cur_stream()))
    return out


def global_to_local_root(root, x, lengths):
    """[x[..., 5:] | globalRootToLocalRoot(root)] (fp32 CUDA tensors root [B, T, 5],
    x [B, T, 279], int32 lengths [B])."""
    import torch
    lib = load_library()
    B, T = x.shape[0], x.shape[1]
    out = torch.empty((B, T, MOTION_DIM), dtype=torch.float32, device=x.device)
    _check(lib.kimodo_global_to_local_root(_ptr(root), _ptr(x), _ptr(lengths), B, T, _ptr(out), _cur_stream()))
    return out


# ------------------------------------------------------------ 8-bit projections, scored attention
#
# These take CUDA tensors of one device, which need not be the current one; work is enqueued
# on that device's current stream and outputs are allocated there.  A call on a single token
# takes a few microseconds on the GPU, so the checks are written to cost little on the host.

_SCORED_PACK = struct.Struct("10Q12q8i2f").pack   # struct kimodo_scored_attention
_T = None            # torch, once it is needed
_raw_stream = None   # device index -> cudaStream_t of its current stream
_current_device = None


def _use_torch():
    global _T, _raw_stream, _current_device
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _T = torch
    return torch


def _device_of(t, what):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    return dev


def _also_on(dev, **tensors):
    """Raises unless every given tensor is on CUDA device `dev`."""
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev} with the other tensors (it is on {t.device})")


def _float_flag(t, what):
    """1 for bf16, 0 for fp32."""
    dt = t.dtype
    if dt is _T.bfloat16:
        return 1
    if dt is _T.float32:
        return 0
    raise ValueError(f"{what} must be bf16 or fp32 (got {dt})")


def _rows_of(t, what):
    """(rows, columns, row stride) of a 2-D tensor with consecutive columns."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor (got {t.dim()} dimensions)")
    rows, cols = t.shape
    ld, sc = t.stride()
    if sc != 1 and cols > 1:
        raise ValueError(f"{what} must have a unit column stride")
    return rows, cols, ld if rows > 1 else cols   # the stride of a single row is never used


def _vector(t, what, n):
    """Data pointer of a contiguous fp32 [n] tensor."""
    if t.dtype is not _T.float32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous fp32 tensor of {n} values (got {t.dtype}, {tuple(t.shape)})")
    return t.data_ptr()


def _indices(t, what, shape):
    """Data pointer of a contiguous int32 tensor, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not _T.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {shape} (got {t.dtype}, {tuple(t.shape)})")
    return t.data_ptr()


def _launch(dev, fn, *args):
    """fn(*args, stream) on device `dev`'s current stream, with `dev` current."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with _T.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


def _int8_rows(x, rows, cols):
    """An int8 [rows, cols] tensor on x's device whose rows start on 16-byte boundaries, as gemm_int8 asks."""
    if cols % 16 == 0:
        return x.new_empty((rows, cols), dtype=_T.int8)
    return x.new_empty((rows, (cols + 15) // 16 * 16), dtype=_T.int8)[:, :cols]


def quantize_int8(x):
    """(q, scale) of the rows of x [rows, cols] (fp32 or bf16): int8 [rows, cols] with rows on
    16-byte boundaries and fp32 [rows], x ~ q * scale[:, None]."""
    lib = _lib or load_library()
    T = _T or _use_torch()
    dev = _device_of(x, "x")
    flag = _float_flag(x, "x")
    rows, cols, ldx = _rows_of(x, "x")
    q = _int8_rows(x, rows, cols)
    scale = x.new_empty(rows, dtype=T.float32)
    _launch(dev, lib.kimodo_quantize_int8, x.data_ptr(), ldx, flag, q.data_ptr(), (cols + 15) // 16 * 16,
            scale.data_ptr(), rows, cols)
    return q, scale


def rms_norm_int8(x, gamma, residual=None, eps=1e-6, residual_out=None):
    """(q, scale, residual_out): int8 rows and fp32 scales of the RMS norm of x + residual times
    gamma (fp32 [cols]), and the sum in the residual's type (None without a residual).
    x and residual [rows, cols], fp32 or bf16; residual_out may be residual itself, not x."""
    lib = _lib or load_library()
    T = _T or _use_torch()
    dev = _device_of(x, "x")
    flag = _float_flag(x, "x")
    rows, cols, ldx = _rows_of(x, "x")
    rp = rop = None
    ldr = ldro = rflag = 0
    if residual is not None:
        rflag = _float_flag(residual, "residual")
        rr, rc, ldr = _rows_of(residual, "residual")
        if rr != rows or rc != cols:
            raise ValueError("residual must have the shape of x")
        if residual_out is None:
            residual_out = x.new_empty((rows, cols), dtype=residual.dtype)
            ldro = cols
        else:
            rr, rc, ldro = _rows_of(residual_out, "residual_out")
            if rr != rows or rc != cols or residual_out.dtype is not residual.dtype:
                raise ValueError("residual_out must have the shape and type of residual")
        rp, rop = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    _also_on(dev, gamma=gamma, residual=residual, residual_out=residual_out)
    q = _int8_rows(x, rows, cols)
    scale = x.new_empty(rows, dtype=T.float32)
    _launch(dev, lib.kimodo_rms_norm_int8, x.data_ptr(), ldx, flag, rp, ldr, rop, ldro, rflag,
            _vector(gamma, "gamma", cols), eps, q.data_ptr(), (cols + 15) // 16 * 16, scale.data_ptr(), rows, cols)
    return q, scale, residual_out


def gemm_int8(a, a_scale, w, w_scale, bias=None, epilogue=EPI_BIAS, out_f32=False, resid=None, out=None):
    """out = epilogue(a_scale[:, None] * w_scale * (a w^T) + bias): int8 a [M, K], w [N, K] (rows on
    16-byte boundaries), fp32 scales [M], [N] and bias [N] or None; out bf16 or fp32 [M, N];
    resid fp32 [M, N] with EPI_BIAS_RESID (may be out, which overlaps no other input)."""
    lib = _lib or load_library()
    T = _T or _use_torch()
    dev = _device_of(a, "a")
    if a.dtype is not T.int8 or w.dtype is not T.int8:
        raise ValueError(f"a and w must be int8 (got {a.dtype}, {w.dtype})")
    M, K, lda = _rows_of(a, "a")
    N, K2, ldw = _rows_of(w, "w")
    if K != K2:
        raise ValueError(f"a has {K} columns, w {K2}")
    if M == 1:   # the stride of a single row is never used
        lda = (K + 15) // 16 * 16
    if N == 1:
        ldw = (K + 15) // 16 * 16
    dtype = T.float32 if out_f32 else T.bfloat16
    rp = None
    ldr = 0
    if resid is not None:
        rm, rn, ldr = _rows_of(resid, "resid")
        if resid.dtype is not T.float32 or rm != M or rn != N:
            raise ValueError(f"resid must be an fp32 tensor of shape {(M, N)}")
        rp = resid.data_ptr()
    if out is None:
        out = a.new_empty((M, N), dtype=dtype)
        ldo = N
    else:
        om, on, ldo = _rows_of(out, "out")
        if out.dtype is not dtype or om != M or on != N:
            raise ValueError(f"out must be a {dtype} tensor of shape {(M, N)}")
    _also_on(dev, a_scale=a_scale, w=w, w_scale=w_scale, bias=bias, resid=resid, out=out)
    _launch(dev, lib.kimodo_gemm_int8, a.data_ptr(), lda, _vector(a_scale, "a_scale", M), w.data_ptr(), ldw,
            _vector(w_scale, "w_scale", N), None if bias is None else _vector(bias, "bias", N), rp, ldr, out.data_ptr(),
            ldo, M, N, K, epilogue, 1 if out_f32 else 0)
    return out


def attention_scored(q, k, v, scale=None, cap=0.0, slopes=None, causal=False, prefix=None, q_documents=None,
                     kv_documents=None, kv_lengths=None, q_start=None, out=None):
    """Attention of q [B, Sq, Hq, D] over k, v [B, Sk, Hkv, D] (bf16 or fp32, D 64 or 128, last
    dimension consecutive, other strides free in multiples of 16 bytes); head h reads key
    head h // (Hq // Hkv).  scale: default D ** -0.5; cap > 0: cap * tanh(score / cap); slopes
    fp32 [Hq]: minus slope * |position distance|; causal, with prefix int32 [B] keys seen by
    all; documents int32 [B, Sq], [B, Sk]: only equal numbers >= 0 meet; kv_lengths int32
    [B]; q_start int32 [B]: position of the first query (default Sk - Sq).  A query that sees
    no key gets 0.  out must not overlap the inputs.  Returns [B, Sq, Hq, D]."""
    lib = _lib or load_library()
    T = _T or _use_torch()
    dev = _device_of(q, "q")
    bf = _float_flag(q, "q")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be 4-D [batch, tokens, heads, dims]")
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    if k.dtype is not q.dtype or v.dtype is not q.dtype or v.shape != k.shape or Bk != B or Dk != D:
        raise ValueError("q, k and v must agree in type, batch and dims, and k and v in shape")
    if out is None:
        out = q.new_empty((B, Sq, Hq, D))
    elif out.dtype is not q.dtype or out.shape != q.shape:
        raise ValueError("out must have the shape and type of q")
    q0, q1, q2, q3 = q.stride()
    k0, k1, k2, k3 = k.stride()
    v0, v1, v2, v3 = v.stride()
    o0, o1, o2, o3 = out.stride()
    if q3 != 1 or k3 != 1 or v3 != 1 or o3 != 1:
        raise ValueError("the last dimension of q, k, v and out must be consecutive")
    _also_on(dev, k=k, v=v, slopes=slopes, prefix=prefix, q_documents=q_documents, kv_documents=kv_documents,
             kv_lengths=kv_lengths, q_start=q_start, out=out)
    args = _SCORED_PACK(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 0 if slopes is None else _vector(slopes, "slopes", Hq),
        _indices(prefix, "prefix", (B,)), _indices(q_documents, "q_documents", (B, Sq)),
        _indices(kv_documents, "kv_documents", (B, Sk)), _indices(kv_lengths, "kv_lengths", (B,)),
        _indices(q_start, "q_start", (B,)), q0, q1, q2, k0, k1, k2, v0, v1, v2, o0, o1, o2, B, Sq, Sk, Hq, Hkv, D, bf,
        1 if causal else 0, D ** -0.5 if scale is None else scale, cap)
    size = ctypes.c_size_t()
    if dev == _current_device():
        status = lib.kimodo_attention_scored_workspace(args, ctypes.byref(size))
    else:
        with T.cuda.device(dev):
            status = lib.kimodo_attention_scored_workspace(args, ctypes.byref(size))
    if status:
        _check(status)
    n = size.value
    ws = q.new_empty(n, dtype=T.uint8) if n else None
    _launch(dev, lib.kimodo_attention_scored, args, ws.data_ptr() if n else None, n)
    return out


def kernel_status(device=None):
    """Synchronise the current stream and raise if a wait in a kernel-level call ran out."""
    import torch
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(lib.kimodo_kernel_status(torch.cuda.current_stream().cuda_stream))


class Kimodo:
    """A loaded denoiser pair on one GPU (wraps a kimodo_ctx)."""

    def __init__(self, blob, precision: int = BF16, device: int = 0):
        lib = load_library()
        self._lib = lib
        self._ctx = ctypes.c_void_p()
        blob = _f32(blob)
        n = int(blob.size if isinstance(blob, np.ndarray) else blob.numel())
        _check(lib.kimodo_load_weights(ctypes.byref(self._ctx), _ptr(blob), n, int(precision), int(device)))
        self.precision = precision
        self.device = device

    def close(self):
        if getattr(self, "_ctx", None) and self._ctx.value:
            self._lib.kimodo_free(self._ctx)
            self._ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- entry points
    def denoiser_forward(self, net, x, emb, t, lengths, out=None, stream=None):
        x, emb, lengths = _f32(x), _f32(emb), _i32(lengths)
        B, T = x.shape[0], x.shape[1]
        dout = ROOT_DIM if net == NET_ROOT else BODY_DIM
        out = _like(x, (B, T, dout)) if out is None else out
        _check(self._lib.kimodo_denoiser_forward(self._ctx, int(net), _ptr(x), _ptr(emb), int(t), _ptr(lengths),
                                                 B, T, _ptr(out), _stream(stream, x, out)))
        return out

    def denoiser_forward_noalloc(self, net, x, emb, t, lengths, out=None, stream=None):
        """kimodo_denoiser_forward_noalloc: same result, no device allocation (size limits apply)."""
        x, emb, lengths = _f32(x), _f32(emb), _i32(lengths)
        B, T = x.shape[0], x.shape[1]
        dout = ROOT_DIM if net == NET_ROOT else BODY_DIM
        out = _like(x, (B, T, dout)) if out is None else out
        _check(self._lib.kimodo_denoiser_forward_noalloc(self._ctx, int(net), _ptr(x), _ptr(emb), int(t),
                                                         _ptr(lengths), B, T, _ptr(out), _stream(stream, x, out)))
        return out

    @staticmethod
    def _options(schedule, eta, step_noise, text_batch=0):
        """kimodo_sampler for the _ex calls, or None for the defaults (linear, eta 0, one
        text row per sequence)."""
        if schedule == "linear" and float(eta) == 0.0 and not text_batch:
            return None, None
        z = None if step_noise is None else _f32(step_noise)
        return SamplerOptions(SCHEDULES[schedule], float(eta), _ptr(z), int(text_batch)), z

    def ddim_step(self, x_t, text_emb, null_emb, lengths, t, t_prev, cfg_scale, out=None, stream=None,
                  schedule="linear", eta=0.0, step_noise=None):
        x_t, text_emb, null_emb, lengths = _f32(x_t), _f32(text_emb), _f32(null_emb), _i32(lengths)
        B, T = x_t.shape[0], x_t.shape[1]
        nb = 1 if null_emb.ndim == 1 else null_emb.shape[0]
        out = _like(x_t, (B, T, MOTION_DIM)) if out is None else out
        opts, z = self._options(schedule, eta, step_noise, text_emb.shape[0] if text_emb.shape[0] != B else 0)
        if opts is None:
            _check(self._lib.kimodo_ddim_step(self._ctx, _ptr(x_t), _ptr(text_emb), _ptr(null_emb), nb,
                                              _ptr(lengths), B, T, int(t), int(t_prev), float(cfg_scale), _ptr(out),
                                              _stream(stream, x_t, out)))
        else:
            _check(self._lib.kimodo_ddim_step_ex(self._ctx, _ptr(x_t), _ptr(text_emb), _ptr(null_emb), nb,
                                                 _ptr(lengths), B, T, int(t), int(t_prev), float(cfg_scale),
                                                 ctypes.byref(opts), _ptr(out), _stream(stream, x_t, out)))
        return out

    def ddim_sample(self, text_emb, null_emb, noise, lengths, steps, cfg_scale, out=None, stream=None,
                    schedule="linear", eta=0.0, step_noise=None):
        """Full sampler; schedule "linear" or "cosine", eta in [0, 1] with step_noise
        [steps, B, T, 279] standard-normal draws when eta > 0.  text_emb may have fewer
        rows than the batch (a divisor of B): variations, row b // (B // rows) per sequence."""
        text_emb, null_emb, noise, lengths = _f32(text_emb), _f32(null_emb), _f32(noise), _i32(lengths)
        B, T = noise.shape[0], noise.shape[1]
        nb = 1 if null_emb.ndim == 1 else null_emb.shape[0]
        out = _like(noise, (B, T, MOTION_DIM)) if out is None else out
        opts, z = self._options(schedule, eta, step_noise, text_emb.shape[0] if text_emb.shape[0] != B else 0)
        if opts is None:
            _check(self._lib.kimodo_ddim_sample(self._ctx, _ptr(text_emb), _ptr(null_emb), nb, _ptr(noise),
                                                _ptr(lengths), B, T, int(steps), float(cfg_scale), _ptr(out),
                                                _stream(stream, noise, out)))
        else:
            _check(self._lib.kimodo_ddim_sample_ex(self._ctx, _ptr(text_emb), _ptr(null_emb), nb, _ptr(noise),
                                                   _ptr(lengths), B, T, int(steps), float(cfg_scale),
                                                   ctypes.byref(opts), _ptr(out), _stream(stream, noise, out)))
        return out

    def wait_selftest(self, limit_us: int, stream=None):
        """kimodo_wait_selftest: a kernel whose bounded wait runs out and records a timeout."""
        _check(self._lib.kimodo_wait_selftest(self._ctx, int(limit_us), stream))

    def sync_status(self, stream=None):
        _check(self._lib.kimodo_sync_status(self._ctx, stream))

    def profile_enable(self, on: bool = True):
        _check(self._lib.kimodo_profile_enable(self._ctx, int(bool(on))))

    def profile_read(self, n_classes: int = 6):
        ms = (ctypes.c_double * n_classes)()
        cnt = (ctypes.c_longlong * n_classes)()
        fl = (ctypes.c_double * n_classes)()
        by = (ctypes.c_double * n_classes)()
        _check(self._lib.kimodo_profile_read(self._ctx, n_classes, ms, cnt, fl, by))
        names = ["gemm_tc", "attention", "layernorm", "motion", "gemm_f32", "setup", "c6", "c7"]
        return {names[i]: dict(ms=ms[i], launches=cnt[i], flops=fl[i], bytes=by[i]) for i in range(n_classes)}

    def last_launch_count(self) -> int:
        return int(self._lib.kimodo_last_launch_count(self._ctx))
