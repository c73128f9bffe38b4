"""The 8-bit projections and attention with scored masks on the host: what they refuse, before a
GPU is touched, and how the binding lays out its arguments."""
import ctypes

import pytest
import torch

import transformer_denoiser_b200 as kb


@pytest.fixture(scope="module")
def lib():
    from transformer_denoiser_b200.build import build
    build()
    return kb.load_library()


P = 4096   # an aligned address that is never followed


def _refused(lib, rc, text):
    assert rc == -1, rc
    assert text in lib.kimodo_last_error(), lib.kimodo_last_error()


def test_quantize_int8_refusals(lib):
    def call(x=P, ldx=8, bf=0, q=P, ldq=8, scale=P, rows=1, cols=8):
        return lib.kimodo_quantize_int8(x, ldx, bf, q, ldq, scale, rows, cols, None)
    for name in ("x", "q", "scale"):
        _refused(lib, call(**{name: None}), b"NULL")
    _refused(lib, call(rows=0), b"rows must be")
    _refused(lib, call(cols=0), b"cols must be")
    _refused(lib, call(cols=32769, ldx=40000, ldq=40000), b"cols must be")
    _refused(lib, call(ldx=7), b"leading")
    _refused(lib, call(ldq=7), b"leading")
    _refused(lib, call(bf=2), b"x_bf16")
    _refused(lib, call(x=P + 2), b"aligned to its elements")
    _refused(lib, call(x=P + 1, bf=1), b"aligned to its elements")
    _refused(lib, call(scale=P + 2), b"aligned")


def test_rms_norm_int8_refusals(lib):
    def call(x=P, ldx=8, bf=0, r=P, ldr=8, ro=P, ldro=8, rbf=0, gamma=P, eps=1e-6, q=P, ldq=8, scale=P, rows=1, cols=8):
        return lib.kimodo_rms_norm_int8(x, ldx, bf, r, ldr, ro, ldro, rbf, gamma, eps, q, ldq, scale, rows, cols, None)
    _refused(lib, call(gamma=None), b"NULL")
    _refused(lib, call(r=None), b"come together")
    _refused(lib, call(ro=None), b"come together")
    _refused(lib, call(ldr=4), b"leading")
    _refused(lib, call(ldro=16), b"in place")
    _refused(lib, call(rbf=3), b"resid_bf16")
    _refused(lib, call(ro=P + 2), b"aligned")
    for eps in (-1e-6, float("nan"), float("inf")):
        _refused(lib, call(eps=eps), b"eps")
    _refused(lib, call(gamma=P + 1), b"aligned")


def test_gemm_int8_refusals(lib):
    def call(A=P, lda=64, sa=P, W=P, ldw=64, sw=P, bias=None, resid=None, ldr=0, out=P, ldo=8, M=1, N=8, K=64, epi=0, f32=0):
        return lib.kimodo_gemm_int8(A, lda, sa, W, ldw, sw, bias, resid, ldr, out, ldo, M, N, K, epi, f32, None)
    for name in ("A", "sa", "W", "sw", "out"):
        _refused(lib, call(**{name: None}), b"NULL")
    for name in ("M", "N", "K"):
        _refused(lib, call(**{name: 0}), b"must be >= 1")
    _refused(lib, call(K=131072, lda=131072, ldw=131072), b"at most 131071")
    _refused(lib, call(lda=48), b"leading")
    _refused(lib, call(ldo=7), b"leading")
    _refused(lib, call(epi=4), b"unknown epilogue")
    _refused(lib, call(epi=3, f32=1), b"needs resid")
    _refused(lib, call(epi=3, f32=0, resid=P, ldr=8), b"writes fp32")
    _refused(lib, call(epi=3, f32=1, resid=P, ldr=4), b"leading")
    _refused(lib, call(epi=3, f32=1, resid=P, ldr=16), b"in place")
    _refused(lib, call(epi=1, f32=1), b"write bf16")
    _refused(lib, call(epi=2, f32=1), b"write bf16")
    _refused(lib, call(lda=72), b"16-byte aligned rows")
    _refused(lib, call(W=P + 8), b"16-byte aligned rows")
    _refused(lib, call(out=P + 1), b"aligned to their elements")
    _refused(lib, call(bias=P + 2), b"aligned to their elements")


def test_outputs_that_start_on_an_input_are_refused(lib):
    word = b"must not overlap the inputs"
    _refused(lib, lib.kimodo_quantize_int8(P, 8, 0, P, 8, 2 * P, 1, 8, None), word)
    for x, r, ro, q in ((P, 2 * P, P, 3 * P), (P, 2 * P, 3 * P, P), (P, 2 * P, 3 * P, 2 * P), (P, 2 * P, 3 * P, 3 * P),
                        (P, 2 * P, 2 * P, 2 * P)):
        _refused(lib, lib.kimodo_rms_norm_int8(x, 8, 0, r, 8, ro, 8, 0, 4 * P, 1e-6, q, 8, 5 * P, 1, 8, None), word)
    for out in (P, 2 * P):
        _refused(lib, lib.kimodo_gemm_int8(P, 64, 3 * P, 2 * P, 64, 4 * P, None, None, 0, out, 8, 1, 8, 64, 0, 0, None),
                 word)
    for out in (P, 2 * P, 3 * P):
        a = _args(q=P, k=2 * P, v=3 * P, out=out)
        _refused(lib, lib.kimodo_attention_scored(ctypes.byref(a), None, 0, None), word)


def _args(**change):
    a = kb.ScoredAttention(P, P, P, P, None, None, None, None, None, None, (512, 64, 64), (512, 64, 64), (512, 64, 64),
                           (512, 64, 64), 2, 8, 8, 1, 1, 64, kb.BF16, 0, 0.125, 0.0)
    for name, v in change.items():
        setattr(a, name, (ctypes.c_longlong * 3)(*v) if isinstance(v, tuple) else v)
    return a


@pytest.mark.parametrize("change,text", [
    (dict(q=None), b"NULL"), (dict(k=None), b"NULL"), (dict(v=None), b"NULL"), (dict(out=None), b"NULL"),
    (dict(batch=0), b"batch >= 1"), (dict(q_len=0), b"q_len >= 1"), (dict(kv_len=-1), b"kv_len >= 0"),
    (dict(q_heads=3, kv_heads=2), b"multiple of kv_heads"), (dict(kv_heads=0), b"multiple of kv_heads"),
    (dict(head_dim=96), b"head_dim"), (dict(dtype=2), b"dtype"), (dict(kv_len=16777217), b"at most"),
    (dict(batch=1 << 20, q_len=1 << 20), b"too many"), (dict(scale=float("nan")), b"scale"),
    (dict(cap=-1.0), b"cap"), (dict(cap=float("inf")), b"cap"), (dict(prefix=P), b"prefix needs causal"),
    (dict(q_documents=P), b"come together"), (dict(kv_documents=P), b"come together"),
    (dict(q=P + 8), b"16-byte aligned"), (dict(k_strides=(512, 68, 64)), b"strides"),
    (dict(v_strides=(512, 0, 64)), b"strides"), (dict(q_strides=(0, 64, 64)), b"strides"),
    (dict(out_strides=(512, 32, 64)), b"strides"), (dict(k_strides=(-512, 64, 64)), b"strides"),
    (dict(kv_lengths=P + 2), b"aligned to their elements"), (dict(slopes=P + 1), b"aligned to their elements"),
])
def test_attention_scored_refusals(lib, change, text):
    a = _args(**change)
    _refused(lib, lib.kimodo_attention_scored(ctypes.byref(a), None, 0, None), text)
    n = ctypes.c_size_t(77)
    _refused(lib, lib.kimodo_attention_scored_workspace(ctypes.byref(a), ctypes.byref(n)), text)
    assert n.value == 0


def test_documents_without_keys_are_not_refused(lib):
    """A tensor of no elements has no address: with kv_len 0, kv_documents may be NULL."""
    a, n = _args(kv_len=0, k=None, v=None, q_documents=P), ctypes.c_size_t(77)
    rc = lib.kimodo_attention_scored_workspace(ctypes.byref(a), ctypes.byref(n))
    assert rc == (0 if torch.cuda.is_available() else -4), lib.kimodo_last_error()
    _refused(lib, lib.kimodo_attention_scored_workspace(ctypes.byref(_args(kv_len=0, kv_documents=P)), ctypes.byref(n)),
             b"come together")


def test_attention_scored_null_arguments(lib):
    _refused(lib, lib.kimodo_attention_scored(None, None, 0, None), b"arguments are NULL")
    _refused(lib, lib.kimodo_attention_scored_workspace(ctypes.byref(_args()), None), b"bytes is NULL")


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_device_is_reported(lib):
    for rc in (lib.kimodo_quantize_int8(P, 8, 0, P, 8, P, 1, 8, None),
               lib.kimodo_gemm_int8(P, 64, P, P, 64, P, None, None, 0, P, 8, 1, 8, 64, 0, 0, None),
               lib.kimodo_attention_scored(ctypes.byref(_args()), None, 0, None), lib.kimodo_kernel_status(None)):
        assert rc in (-1, -4) and lib.kimodo_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kb.quantize_int8(x)
    with pytest.raises(ValueError, match="CUDA"):
        kb.rms_norm_int8(x, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        kb.gemm_int8(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        kb.attention_scored(*[torch.zeros(1, 2, 1, 64)] * 3)


def test_binding_packs_the_arguments_as_the_c_structure():
    """The packed bytes of attention_scored are the C structure, field by field."""
    values = [16 * (i + 1) for i in range(10)] + list(range(100, 112)) + list(range(1, 9)) + [0.5, 30.0]
    raw = kb._SCORED_PACK(*values)
    assert len(raw) == ctypes.sizeof(kb.ScoredAttention)
    a = kb.ScoredAttention.from_buffer_copy(raw)
    flat = []
    for name, kind in kb.ScoredAttention._fields_:
        v = getattr(a, name)
        flat += list(v) if hasattr(v, "__len__") else [v]
    assert flat == values
