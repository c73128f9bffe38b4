"""The 8-bit projections and the attention with scored masks in 64 bits (torch float64),
written from their definitions, and the bounds on how far a kernel may be from them."""
import math

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2     # 2^-8: half a step, relative
FP32_HALF = torch.finfo(torch.float32).eps / 2      # 2^-24


def rows_ref(t):
    """(127 t / max|t| unrounded, scale) of float64 rows; a zero row gives zeros."""
    top = t.abs().amax(1)
    safe = torch.where(top > 0, top, torch.ones_like(top))
    return t * 127 / safe[:, None], top / 127


def check_rows(q, scale, t, what, sum_terms=0, near=3.1e-5):
    """q and scale of a kernel against float64 rows t.

    The kernel's t (127 / max|t|) carries at most four fp32 roundings (the product with gamma,
    its maximum, the quotient, the product) before the one that makes it whole: 127 * 4 * 2^-24
    = 3.03e-5 of a step, so q may differ from the rounded float64 value only where that value
    is within 3.1e-5 of a tie.  scale: one rounding, and with a norm those of a sum of
    `sum_terms` squares added in order, halved by the root, and five more."""
    u, s = rows_ref(t.cpu())
    q, scale = q.cpu().double(), scale.cpu().double()
    tie = ((u - u.floor()) - 0.5).abs() < near
    wrong = (q != torch.round(u)) & ~tie
    assert not wrong.any(), (what, int(wrong.sum()), q[wrong][:4], u[wrong][:4])
    assert ((q - u).abs() <= 0.5 + near).all(), what
    assert ((scale - s).abs() <= (sum_terms / 2 + 6) * FP32_HALF * s + 1e-45).all(), what


def gemm_ref(a, sa, w, sw, bias, kind, resid):
    """(result, bound on the fp32 part of the error) in float64; kind as the EPI_* constants."""
    y = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()
    # the sum, the two scales' product and their product: three roundings; the bias' addition one
    err = 3 * FP32_HALF * y.abs()
    if bias is not None:
        y = y + bias.double()
    err = err + FP32_HALF * y.abs()
    if kind == 1:
        z = 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
        # |GELU'| <= 1.13; the epilogue's erf is within 8e-6 (its own error-bound test)
        return z, 1.13 * err + 0.5 * y.abs() * 8e-6
    if kind == 2:
        z = y * torch.sigmoid(y)
        # |SiLU'| <= 1.1; expf within 2 steps, a sum and a quotient: 4 steps of the result
        return z, 1.1 * err + 8 * FP32_HALF * z.abs()
    if kind == 3:
        y = y + resid.double()
        err = err + FP32_HALF * y.abs()
    return y, err


def attention_ref(q, k, v, scale=None, cap=0.0, slopes=None, causal=False, prefix=None, q_documents=None,
                  kv_documents=None, kv_lengths=None, q_start=None):
    """(output, sum of |weight value|, largest score error of the row) in float64, a query
    at a time over the keys it sees."""
    q, k, v = q.cpu().double(), k.cpu().double(), v.cpu().double()
    (B, Sq, Hq, D), (Sk, Hkv) = q.shape, k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, Sq, Hq, D, dtype=torch.float64)
    mass = torch.zeros_like(out)
    delta = torch.zeros(B, Sq, Hq, 1, dtype=torch.float64)
    j = torch.arange(Sk)
    for b in range(B):
        n = Sk if kv_lengths is None else min(max(int(kv_lengths[b]), 0), Sk)
        first = Sk - Sq if q_start is None else int(q_start[b])
        for i in range(Sq):
            p = first + i
            seen = j < n
            if causal:
                ahead = j > p
                if prefix is not None:
                    ahead &= j >= int(prefix[b])
                seen = seen & ~ahead
            if q_documents is not None:
                d = int(q_documents[b, i])
                seen = seen & (kv_documents[b].cpu() == d) & (d >= 0)
            at = torch.nonzero(seen).flatten()
            if not len(at):
                continue
            for h in range(Hq):
                kk, vv = k[b, at, h // (Hq // Hkv)], v[b, at, h // (Hq // Hkv)]
                x = scale * (kk @ q[b, i, h])
                # a sum of D products in any order, each addition one fp32 rounding (a truncation at most)
                delta[b, i, h] = 2 * D * FP32_HALF * abs(scale) * (kk.abs() @ q[b, i, h].abs()).max()
                if cap:
                    x = cap * torch.tanh(x / cap)
                if slopes is not None:
                    x = x - float(slopes[h]) * (p - at).abs()
                w = torch.softmax(x, 0)
                out[b, i, h] = w @ vv
                mass[b, i, h] = w @ vv.abs()
                # forming the score in log2 units, its cap and bias: 8 roundings of the largest part
                big = x.abs().max() + (cap or 0) + (float(slopes[h]) * (p - at).abs().max() if slopes is not None else 0)
                delta[b, i, h] += 8 * FP32_HALF * big + 8 * FP32_HALF
    return out, mass, delta


def check_attention(got, q, k, v, what="", **options):
    """A kernel's output against the definition.  Weights: an error d of a score moves a weight
    by a factor within e^d, and the normalised ones by twice that; bf16: each weight and the
    output are rounded to 8 bits; fp32: running sums of Sk terms."""
    ref, mass, delta = attention_ref(q, k, v, **options)
    if got.dtype == torch.bfloat16:
        tol = (BF16_HALF * 1.01 + 2 * delta) * mass + BF16_HALF * ref.abs() + 1e-30
    else:
        tol = (2 * delta + (k.shape[1] + 32) * FP32_HALF) * mass + 1e-30
    err = (got.cpu().double() - ref).abs()
    assert torch.isfinite(got).all(), what
    bad = err > tol
    assert not bad.any(), (what, int(bad.sum()), float((err / tol.clamp_min(1e-30)).max()),
                           [x.tolist() for x in torch.nonzero(bad)[:4]])
