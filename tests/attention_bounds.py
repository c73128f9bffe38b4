"""Attention with scored masks in 64 bits over whole matrices, and a bound on a kernel's error that
is weighted key by key: what a key's score may be off by counts with the key's weight in the
row, and neither the cap nor the distance of a row's farthest key widens it."""
import math

import torch

FP32_HALF = torch.finfo(torch.float32).eps / 2      # 2^-24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2     # 2^-8


def _row(q, k, v, x_opts, bf16):
    """(output, bound) of the rows of one head; q [R, D], k, v [S, D] float64, the rest per row."""
    scale, cap, slope, p, last, seen = x_opts
    S, D = k.shape
    x = scale * (q @ k.T)
    # a sum of D products in any order: an addition is one fp32 rounding (a truncation at most)
    delta = 2 * D * FP32_HALF * abs(scale) * (q.abs() @ k.abs().T)
    if cap:
        x = cap * torch.tanh(x / cap)
        # |d cap tanh(x / cap)| <= |dx|.  The polynomial is within 5.5e-7 of the value; beyond half of the
        # cap the other form, cap (1 - 2 / (1 + e^2z)), has an error of at most 9 roundings of
        # the quotient, which is below 1.17 |value|, and 4 of the value: 14.5 roundings,
        # below 5.5e-7 + 8 roundings (17.2).  tanhf (2 ulps) and five products are fewer.
        delta = delta + (5.5e-7 + 8 * FP32_HALF) * x.abs()
    else:
        delta = delta + 8 * FP32_HALF * x.abs()
    j = torch.arange(S, device=q.device)
    if slope:
        # softmax knows distances only up to a constant of the row: that of the nearest place the
        # row could see.  A bias is formed for 128 keys from the distance of their first.
        near = torch.minimum(p, last).clamp_min(0)
        far = (p[:, None] - j).abs() - (p - near).abs()[:, None]
        x = x - slope * far
        delta = delta + 6 * FP32_HALF * abs(slope) * (far.abs() + 128)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(1, keepdim=True)
    any_seen = top > -math.inf
    top = torch.where(any_seen, top, 0.0)
    p_ = torch.exp(x - top)
    total = p_.sum(1, keepdim=True)
    p_ = p_ / torch.where(total > 0, total, 1.0)
    # the difference from the row's reference in log2 units, the reference's moves (at most one a
    # key tile of 64: an exponential within 4 roundings and its argument's two) and the join of parts
    size = torch.where(seen, x.abs(), 0.0) + top.abs()
    delta = delta + 4 * FP32_HALF * size + (16 + 6 * ((S + 63) // 64)) * FP32_HALF
    eps = torch.expm1(torch.where(seen, delta, 0.0).clamp_max(1.0))
    out = p_ @ v
    sums = (S / 2 + 32 if bf16 else S + 32) * FP32_HALF   # running fp32 sums
    num = eps + sums + (BF16_HALF * 1.01 if bf16 else 0.0)
    moved = (p_ * (eps + sums)).sum(1, keepdim=True)      # of the weights' sum, which divides
    tol = ((p_ * num) @ v.abs() + out.abs() * moved) / (1 - moved).clamp_min(0.5)
    return out, tol + (BF16_HALF if bf16 else FP32_HALF) * out.abs() + 1e-30


def check(got, q, k, v, rows=None, heads=None, what="", scale=None, cap=0.0, slopes=None, causal=False, prefix=None,
          q_documents=None, kv_documents=None, kv_lengths=None, q_start=None):
    """Asserts that got [B, Sq, Hq, D] (only queries `rows` and `heads`, where given) is within the bound."""
    B, Sq, Hq, D = q.shape
    Sk, Hkv = k.shape[1:3]
    dev = q.device
    rows = torch.arange(Sq, device=dev) if rows is None else torch.as_tensor(rows, device=dev)
    scale = float(torch.tensor(D ** -0.5 if scale is None else scale, dtype=torch.float32))
    cap = float(torch.tensor(cap, dtype=torch.float32))
    bf16 = got.dtype == torch.bfloat16
    j = torch.arange(Sk, device=dev)
    worst = 0.0
    for b in range(B):
        n = Sk if kv_lengths is None else min(max(int(kv_lengths[b]), 0), Sk)
        p = (Sk - Sq if q_start is None else int(q_start[b])) + rows
        last = torch.full_like(p, n - 1)
        if causal:
            reach = p if prefix is None else p.clamp_min(int(prefix[b]) - 1)
            last = torch.minimum(last, reach)
        seen = j[None, :] <= last[:, None]
        if q_documents is not None:
            d = q_documents[b].to(dev)[rows]
            seen = seen & (d[:, None] == kv_documents[b].to(dev)[None, :]) & (d >= 0)[:, None]
        used = seen.any(0)[:, None]   # what no checked row sees may hold anything
        for h in range(Hq) if heads is None else heads:
            kk = torch.where(used, k[b, :, h // (Hq // Hkv)].double(), 0.0)
            vv = torch.where(used, v[b, :, h // (Hq // Hkv)].double(), 0.0)
            slope = 0.0 if slopes is None else float(slopes[h])
            ref, tol = _row(q[b, rows, h].double(), kk, vv, (scale, cap, slope, p, last, seen), bf16)
            y = got[b, rows, h].double()
            assert torch.isfinite(y).all(), (what, b, h)
            err = (y - ref).abs()
            worst = max(worst, float((err / tol).max()))
            bad = err > tol
            assert not bad.any(), (what, "sequence", b, "head", h, int(bad.sum()), "of", bad.numel(), "error / bound",
                                   float((err / tol).max()), "rows", rows[bad.any(1)][:5].tolist())
    return worst
