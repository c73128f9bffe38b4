"""The operators of an 8-bit transformer layer one after another, as they are used: norm with the
residual, QKV product, attention with masks, quantised attention output, output product
onto the residual, norm, FFN.  Each link is checked against 64 bits on the tensors that
the link before really produced, and the captured layer replays bit for bit."""
import pytest
import torch

import transformer_denoiser_b200 as kb
from gpu_fixtures import require_cuda
from operator_refs import BF16_HALF, check_attention, check_rows, gemm_ref

pytestmark = pytest.mark.gpu

D, H, DH, F = 1024, 8, 128, 2048


@pytest.fixture(autouse=True)
def _fp32_default():
    was = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(was)


def _weights():
    g = torch.Generator().manual_seed(1)
    w = {}
    for name, (n, k) in dict(qkv=(3 * D, D), out=(D, D), ff1=(F, D), ff2=(D, F)).items():
        w[name] = kb.quantize_int8((torch.randn(n, k, generator=g) * 0.03).cuda())
        w[name + "_b"] = (torch.randn(n, generator=g) * 0.02).cuda()
    for name in ("g1", "g2"):
        w[name] = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    return w


def _layer(w, x, y, lengths, slopes, trace):
    """x: sub-layer output bf16 [B*S, D]; y: fp32 residual stream [B*S, D]; returns the new pair."""
    B, T = lengths.shape[0], x.shape[0]
    S = T // B
    q, s, y1 = kb.rms_norm_int8(x, w["g1"], y)
    qkv = kb.gemm_int8(q, s, *w["qkv"], w["qkv_b"])
    qh, kh, vh = (t.unflatten(1, (H, DH)).unflatten(0, (B, S)) for t in qkv.split(D, 1))
    a = kb.attention_scored(qh, kh, vh, slopes=slopes, cap=30.0, kv_lengths=lengths)
    aq, as_ = kb.quantize_int8(a.view(T, D))
    y2 = kb.gemm_int8(aq, as_, *w["out"], w["out_b"], kb.EPI_BIAS_RESID, True, y1)
    zero = torch.zeros_like(x)
    q2, s2, y3 = kb.rms_norm_int8(zero, w["g2"], y2)
    u = kb.gemm_int8(q2, s2, *w["ff1"], w["ff1_b"], kb.EPI_BIAS_GELU)
    uq, us = kb.quantize_int8(u)
    f = kb.gemm_int8(uq, us, *w["ff2"], w["ff2_b"])
    if trace is not None:
        trace.update(q=q, s=s, y1=y1, qkv=qkv, heads=(qh, kh, vh), a=a, aq=aq, as_=as_, y2=y2, q2=q2, s2=s2, y3=y3, u=u,
                     uq=uq, us=us, f=f)
    return f, y3


def _check_product(out, a, sa, w, b, kind, resid, what):
    ref, err = gemm_ref(a, sa, w[0], w[1], b, kind, resid)
    tol = err if out.dtype == torch.float32 else err * 1.01 + BF16_HALF * ref.abs()
    assert ((out.double() - ref).abs() <= tol + 1e-30).all(), what


@pytest.mark.parametrize("B,S,lengths", [(2, 31, [31, 7]), (1, 1, [1]), (2, 151, [151, 60])])
def test_layer(B, S, lengths):
    require_cuda()
    g = torch.Generator().manual_seed(2)
    w = _weights()
    x, y = torch.randn(B * S, D, generator=g).bfloat16().cuda(), torch.randn(B * S, D, generator=g).cuda()
    L = torch.tensor(lengths, dtype=torch.int32).cuda()
    slopes = torch.exp2(-torch.arange(1, H + 1)).float().cuda()
    t = {}
    f, y3 = _layer(w, x, y, L, slopes, t)
    torch.cuda.synchronize()
    h = x.float() + y
    assert torch.equal(t["y1"], h)
    h = h.double()
    check_rows(t["q"], t["s"], h * w["g1"].double() / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6), "norm 1", 70)
    _check_product(t["qkv"], t["q"], t["s"], w["qkv"], w["qkv_b"], 0, None, "qkv")
    some = slice(0, S, 7)   # every seventh query: the reference takes one at a time
    qh, kh, vh = t["heads"]
    check_attention(t["a"][:, some][:, -1:], qh[:, some][:, -1:], kh, vh, slopes=slopes, cap=30.0, kv_lengths=L,
                    q_start=torch.full((B,), (S - 1) // 7 * 7))
    check_attention(t["a"][:, :1], qh[:, :1], kh, vh, slopes=slopes, cap=30.0, kv_lengths=L, q_start=torch.zeros(B))
    check_rows(t["aq"], t["as_"], t["a"].view(B * S, D).double(), "attention rows")
    _check_product(t["y2"], t["aq"], t["as_"], w["out"], w["out_b"], 3, t["y1"], "out")
    assert torch.equal(t["y3"], t["y2"])
    h = t["y2"].double()
    check_rows(t["q2"], t["s2"], h * w["g2"].double() / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6), "norm 2", 70)
    _check_product(t["u"], t["q2"], t["s2"], w["ff1"], w["ff1_b"], 1, None, "ff1")
    check_rows(t["uq"], t["us"], t["u"].double(), "ffn rows")
    _check_product(f, t["uq"], t["us"], w["ff2"], w["ff2_b"], 0, None, "ff2")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2, y4 = _layer(w, x, y, L, slopes, None)
    x2 = torch.randn(B * S, D, generator=g).bfloat16().cuda()
    want = _layer(w, x2, y, L, slopes, None)
    x.copy_(x2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f2, want[0]) and torch.equal(y4, want[1])
    kb.kernel_status()


def test_layer_keeps_the_floating_point_layer():
    """The 8-bit layer's attention and FFN outputs against the same layer in float64 on unquantised
    weights: each 8-bit operand is off by at most half a step of its row's largest value
    over 127, so the relative error of a product's output (a sum of independent parts) is
    about sqrt(2) * (1 / 127) * (max / rms) / sqrt(12) < 2 % per product for rows whose
    largest value is under 5 times their root mean square; four products and the
    non-linear parts between them stay below 10 %."""
    require_cuda()
    g = torch.Generator().manual_seed(5)
    B, S = 1, 64
    ws = {n: torch.randn(r, c, generator=g) * 0.03 for n, (r, c) in
          dict(qkv=(3 * D, D), out=(D, D), ff1=(F, D), ff2=(D, F)).items()}
    w = {n: kb.quantize_int8(v.cuda()) for n, v in ws.items()}
    for n, r in dict(qkv=3 * D, out=D, ff1=F, ff2=D).items():
        w[n + "_b"] = torch.zeros(r, device="cuda")
    w["g1"] = w["g2"] = torch.ones(D, device="cuda")
    x, y = torch.randn(S, D, generator=g).bfloat16(), torch.randn(S, D, generator=g)
    L = torch.tensor([S], dtype=torch.int32).cuda()
    f, y3 = _layer(w, x.cuda(), y.cuda(), L, torch.zeros(H, device="cuda"), None)

    def norm(h):
        return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    wd = {n: v.double() for n, v in ws.items()}
    y1 = x.double() + y.double()
    q, k, v = (t.view(S, H, DH) for t in (norm(y1) @ wd["qkv"].T).split(D, 1))
    sc = 30 * torch.tanh(torch.einsum("ihd,jhd->hij", q, k) / (DH ** 0.5) / 30)
    a = torch.einsum("hij,jhd->ihd", torch.softmax(sc, -1), v).reshape(S, D)
    y2 = y1 + a @ wd["out"].T
    u = norm(y2) @ wd["ff1"].T
    u = 0.5 * u * (1 + torch.erf(u / 2 ** 0.5))
    ref = u @ wd["ff2"].T
    assert (y3.cpu().double() - y2).norm() / (y2 - y1).norm() < 0.1
    assert (f.cpu().double() - ref).norm() / ref.norm() < 0.1
