"""Outputs that share bytes with an input are refused wherever they start; parts of one buffer that
do not (columns of the same rows, heads of the same tokens) are not."""
import ctypes
import random

import pytest
import torch

import transformer_denoiser_b200 as kb

P = 1 << 30   # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    from transformer_denoiser_b200.build import build
    build()
    return kb.load_library()


def _overlap(lib, rc):
    assert rc != 0   # the addresses are not memory of a device
    return b"must not overlap the inputs" in lib.kimodo_last_error()


def _quantize(lib, x, ldx, q, ldq, rows, cols, bf=0):
    return _overlap(lib, lib.kimodo_quantize_int8(x, ldx, bf, q, ldq, 8 * P, rows, cols, None))


def test_quantize(lib):
    assert _quantize(lib, P, 64, P + 64 * 4 * 9 + 255, 64, 10, 64)       # the last byte of x
    assert not _quantize(lib, P, 64, P + 64 * 4 * 10, 64, 10, 64)        # behind it
    assert _quantize(lib, P + 639, 64, P, 64, 10, 64, 1) is False        # (not aligned: another refusal)
    assert _quantize(lib, P + 638, 64, P, 64, 10, 64, 1)                 # x starts on the last byte of q
    assert not _quantize(lib, P + 640, 64, P, 64, 10, 64, 1)
    # q in the spare columns of x's rows: 64 of 96 floats used, 128 spare bytes
    assert not _quantize(lib, P, 96, P + 256, 384, 10, 64)
    assert not _quantize(lib, P, 96, P + 320, 384, 10, 64)
    assert _quantize(lib, P, 96, P + 321, 384, 10, 64)
    assert _quantize(lib, P, 96, P + 255, 384, 10, 64)
    assert not _quantize(lib, P, 96, P + 384 * 9 + 256, 64, 1, 64)       # a row of its own behind the tenth
    # strides whose bytes leave 64 bits: x's rows are farther apart than q is wide
    assert not _quantize(lib, P, 2 ** 62 + 64, P + 256, 64, 2, 64)
    assert _quantize(lib, P, 2 ** 62 + 64, P + 252, 64, 2, 64)


def test_rms_norm(lib):
    def call(x, r, ro, q, rows=10, cols=64, ldr=64, ldro=64):
        return _overlap(lib, lib.kimodo_rms_norm_int8(x, 64, 1, r, ldr, ro, ldro, 0, 8 * P, 1e-6, q, 64, 9 * P, rows, cols,
                                                      None))
    assert not call(P, 2 * P, 2 * P, 3 * P)               # in place
    assert not call(P, 2 * P, 3 * P, 4 * P)
    assert call(P, 2 * P, 2 * P + 256, 4 * P)             # a row further
    assert call(P, 2 * P + 256, 2 * P, 4 * P)
    assert call(P, 2 * P, P + 1276, 4 * P)                # the end of x
    assert not call(P, 2 * P, P + 1280, 4 * P)
    assert call(P, 2 * P, 3 * P, 3 * P + 2559) and call(P, 2 * P, 3 * P, 2 * P - 639)
    assert not call(P, 2 * P, 3 * P, 3 * P + 2560) and not call(P, 2 * P, 3 * P, 2 * P - 640)
    assert not call(P, None, None, 3 * P)


def test_product(lib):
    def call(A=P, W=2 * P, out=3 * P, resid=4 * P, ldo=8, ldr=8, M=5, N=8, K=64, epi=3):
        return _overlap(lib, lib.kimodo_gemm_int8(A, 64, 8 * P, W, 64, 9 * P, None, resid, ldr, out, ldo, M, N, K, epi,
                                                  1 if epi == 3 else 0, None))
    assert not call() and not call(resid=3 * P)           # apart; in place
    assert call(resid=3 * P + 32) and call(resid=3 * P - 4 * 39)
    assert not call(resid=3 * P + 160) and not call(resid=3 * P + 32, epi=0)   # ignored without its epilogue
    assert call(out=P + 316) and not call(out=P + 320) and call(out=2 * P + 508) and not call(out=2 * P + 512)
    assert call(out=P - 156) and not call(out=P - 160)
    assert not call(resid=3 * P + 32, ldo=16, ldr=16) and call(resid=3 * P + 28, ldo=16, ldr=16)   # halves of one buffer's rows


def _attention(lib, **change):
    s = (512, 64, 64)
    v = dict(q=P, k=2 * P, v=3 * P, out=4 * P, qs=s, ks=s, vs=s, os=s, B=2, Sq=8, Sk=8, Hq=1, Hkv=1) | change
    a = kb.ScoredAttention(v["q"], v["k"], v["v"], v["out"], None, None, None, None, None, None,
                           *((ctypes.c_longlong * 3)(*v[n]) for n in ("qs", "ks", "vs", "os")), v["B"], v["Sq"], v["Sk"],
                           v["Hq"], v["Hkv"], 64, kb.BF16, 0, 0.125, 0.0)
    return _overlap(lib, lib.kimodo_attention_scored(ctypes.byref(a), None, 0, None))


def test_attention(lib):
    assert not _attention(lib)
    assert _attention(lib, out=P + 2032) and not _attention(lib, out=P + 2048)
    assert _attention(lib, out=2 * P - 2032) and not _attention(lib, out=2 * P - 2048)
    assert _attention(lib, out=3 * P + 16)
    assert not _attention(lib, k=None, v=None, Sk=0)
    # one buffer [batch 2, tokens 8, (q k v out) x 4 heads, 64]
    t = dict(qs=(8192, 1024, 64), ks=(8192, 1024, 64), vs=(8192, 1024, 64), os=(8192, 1024, 64), Hq=4, Hkv=4)
    assert not _attention(lib, q=P, k=P + 512, v=P + 1024, out=P + 1536, **t)
    assert _attention(lib, q=P, k=P + 512, v=P + 1024, out=P + 1520, **t)
    # heads before tokens: [batch 2, (q k v out) x 4 heads, tokens 8, 64]
    h = dict(qs=(8192, 64, 512), ks=(8192, 64, 512), vs=(8192, 64, 512), os=(8192, 64, 512), Hq=4, Hkv=4)
    assert not _attention(lib, q=P, k=P + 4096, v=P + 8192, out=P + 12288, **h)
    assert _attention(lib, q=P, k=P + 4096, v=P + 8192, out=P + 12272, **h)
    # the largest strides and extents: sums past 64 bits
    far = (1 << 36, 1 << 36, 1 << 36)
    assert _attention(lib, q=P, out=P + 16, qs=far, os=far, Sq=1 << 24, Hq=8, Hkv=8, B=2)


def test_no_shared_byte_is_missed(lib):
    """Random small layouts against the sets of their bytes: what is accepted shares none, and plain
    neighbours in one buffer are accepted."""
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        B, Sq, H = rng.choice([(1, 3, 2), (2, 2, 2), (2, 4, 1), (3, 1, 2), (1, 1, 1)])
        strides = [tuple(rng.choice([64, 72, 128, 136, 192, 256, 320, 512, 768]) for _ in range(3)) for _ in range(2)]
        if rng.random() < 0.5:
            strides[1] = strides[0]
        off = rng.randrange(-200, 200) * 16

        def places(base, st, s):
            return {base + 2 * (b * st[0] + i * st[1] + h * st[2]) + e for b in range(B) for i in range(s) for h in range(H)
                    for e in range(0, 128, 16)}
        shared = bool(places(P + off, strides[1], Sq) & places(P, strides[0], Sq))
        refused = _attention(lib, q=P, out=P + off, qs=strides[0], os=strides[1], k=5 * P, v=6 * P, B=B, Sq=Sq, Hq=H, Hkv=H)
        assert refused or not shared, (B, Sq, H, strides, off)
        seen[refused] += 1
    assert min(seen.values()) > 500, seen


@pytest.mark.gpu
def test_parts_of_one_buffer():
    """The attention's output in the fourth part of the projection's buffer; 8-bit rows in the spare
    columns of theirs."""
    from gpu_fixtures import require_cuda
    require_cuda()
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(2, 70, 4, 4, 64, generator=g, dtype=torch.float32).bfloat16().cuda()
    q, k, v, out = (buf[:, :, i] for i in range(4))
    want = kb.attention_scored(q, k, v, causal=True)
    before = buf.clone()
    kb.attention_scored(q, k, v, causal=True, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(buf[:, :, :3], before[:, :, :3])
    with pytest.raises(kb.KimodoError, match="overlap"):
        kb.attention_scored(q, k, v, out=buf.flatten(2, 3)[:, :, 1:5])
    y = torch.randn(40, 96, generator=g, dtype=torch.float32).cuda()
    a, w = (torch.randint(-127, 128, (n, 64), generator=g, dtype=torch.int8).cuda() for n in (40, 32))
    sa, sw = (torch.full((n,), 1 / 99, dtype=torch.float32, device="cuda") for n in (40, 32))
    kb.gemm_int8(a, sa, w, sw, None, kb.EPI_BIAS_RESID, True, y[:, :32], out=y[:, 32:64])
    assert torch.equal(y[:, 32:64], kb.gemm_int8(a, sa, w, sw, None, kb.EPI_BIAS_RESID, True, y[:, :32].clone()))
    with pytest.raises(kb.KimodoError, match="overlap"):
        kb.gemm_int8(a, sa, w, sw, None, kb.EPI_BIAS_RESID, True, y[:, :32], out=y[:, 31:63])
