"""Attention with scored masks under the bound that counts every key with its weight: the kernels for
few and for many rows over all options, and the form with two row tiles a CTA, which
takes calls with a cap and at least as many blocks of 256 rows as the GPU has SMs."""
import ctypes

import pytest
import torch

import transformer_denoiser_b200 as kb
from attention_bounds import check
from gpu_fixtures import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _fp32_default():
    """Tensors drawn here are fp32 whatever default another module has set."""
    was = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(was)

BF16, FP32 = torch.bfloat16, torch.float32


def _qkv(seed, B, Sq, Sk, Hq, Hkv, D, dtype):
    require_cuda()
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32)
    return tuple(t.to(dtype).cuda() for t in (1.5 * draw(B, Sq, Hq, D), draw(B, Sk, Hkv, D), draw(B, Sk, Hkv, D)))


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda().contiguous()


def _options(name, B, Sq, Sk, Hq, seed):
    g = torch.Generator().manual_seed(seed)
    slopes = torch.exp2(-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32) / Hq).cuda()
    lengths = _i32(torch.randint(0, Sk + 1, (B,), generator=g))
    # packed documents of up to 60 tokens, some tokens in none
    ends = torch.randint(1, 61, (B, max(Sq, Sk)), generator=g).cumsum(1)
    d = torch.searchsorted(ends, torch.arange(max(Sq, Sk)).expand(B, -1).contiguous(), right=True)
    d[:, 70:75] = -1
    docs = dict(q_documents=_i32(d[:, -Sq:]), kv_documents=_i32(d[:, -Sk:]))
    return {
        "full": {}, "causal": dict(causal=True), "slopes": dict(slopes=slopes), "lengths": dict(kv_lengths=lengths),
        "prefix": dict(causal=True, prefix=_i32(torch.randint(0, Sk + 1, (B,), generator=g))), "documents": docs,
        "causal slopes": dict(causal=True, slopes=slopes),
        "negative scale": dict(scale=-0.2, slopes=-slopes / 8), "no scale": dict(scale=0.0, causal=True),
        "all": dict(causal=True, prefix=_i32(torch.randint(0, 40, (B,), generator=g)), slopes=slopes, kv_lengths=lengths,
                    q_start=_i32(torch.randint(-Sq, Sk, (B,), generator=g)), scale=0.11, **docs),
    }[name]


NAMES = ["full", "causal", "slopes", "lengths", "prefix", "documents", "causal slopes", "negative scale", "no scale", "all"]


# 160 blocks of 256 rows; a second row tile with 44 rows, one row or none; grouped heads
TWO = [(10, 300, 300, 8, 8, 128), (10, 300, 333, 8, 8, 64), (19, 129, 200, 8, 8, 128), (38, 100, 130, 4, 4, 64),
       (13, 257, 257, 12, 6, 128), (5, 900, 1100, 8, 8, 64)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("shape", TWO)
@pytest.mark.parametrize("cap", [30.0, 4.0])
def test_two_row_tiles(cap, shape, name):
    B, Sq, Sk, Hq = shape[:4]
    kw = _options(name, B, Sq, Sk, Hq, Sq) | dict(cap=cap)
    q, k, v = _qkv(Sk, *shape, BF16)
    out = kb.attention_scored(q, k, v, **kw)
    torch.cuda.synchronize()
    check(out, q, k, v, rows=sorted({*range(0, Sq, 5), Sq - 1, min(127, Sq - 1), min(128, Sq - 1)}), what=name, **kw)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("shape", TWO[:2])
def test_two_row_tiles_unseen_keys_do_not_leak(shape, poison):
    """Behind the lengths (zeroed rows), and ahead of a causal query in its own tile (rows done again)."""
    B, Sq, Sk, Hq = shape[:4]
    q, k, v = _qkv(1, *shape, BF16)
    lengths = _i32([Sk - 1 - 17 * b for b in range(B)])
    for b in range(B):
        k[b, lengths[b]:], v[b, lengths[b]:] = poison, poison
    out = kb.attention_scored(q, k, v, kv_lengths=lengths, cap=20.0)
    check(out, q, k, v, rows=range(0, Sq, 9), kv_lengths=lengths, cap=20.0)
    q, k, v = _qkv(2, *shape, BF16)
    at = 201
    k[:, at], v[:, at] = poison, poison
    out = kb.attention_scored(q, k, v, causal=True, cap=20.0)
    check(out, q, k, v, rows=range(0, at - (Sk - Sq), 9), causal=True, cap=20.0)


def test_two_row_tiles_split_keys():
    """160 blocks over 8192 keys: the plan cuts the keys, and the parts are joined."""
    shape = (10, 300, 8192, 8, 8, 64)
    q, k, v = _qkv(3, *shape, BF16)
    slopes = torch.full((8,), 0.01, device="cuda")
    lib, out, n = kb.load_library(), torch.empty_like(q), ctypes.c_size_t()
    a = kb.ScoredAttention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), slopes.data_ptr(), None, None, None, None,
                           None, *(tuple(t.stride()[:3]) for t in (q, k, v, out)), 10, 300, 8192, 8, 8, 64, kb.BF16, 1, 0.125, 30.0)
    assert lib.kimodo_attention_scored_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
    for kw in (dict(cap=30.0, slopes=slopes, causal=True), dict(cap=30.0, kv_lengths=_i32([1 + 900 * b for b in range(10)]))):
        out = kb.attention_scored(q, k, v, **kw)
        check(out, q, k, v, rows=[0, 1, 127, 128, 255, 256, 299], heads=(0, 5), **kw)


def test_two_row_tiles_same_bits_captured_and_on_another_stream():
    q, k, v = _qkv(4, *TWO[0], BF16)
    kw = _options("all", 10, 300, 300, 8, 1) | dict(cap=30.0)
    want = kb.attention_scored(q, k, v, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kb.attention_scored(q, k, v, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = kb.attention_scored(q, k, v, **kw)
        for _ in range(5):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out) and torch.equal(want, other)
    kb.kernel_status()


# one and few rows in one part and in several, one row tile a CTA in one part and in several
ONE = [(2, 1, 130, 4, 2, 64), (3, 1, 2500, 8, 2, 128), (1, 5, 700, 6, 2, 128), (2, 16, 257, 1, 1, 64), (1, 31, 31, 8, 8, 128),
       (2, 129, 129, 2, 1, 64), (1, 151, 400, 7, 1, 128), (1, 300, 3000, 2, 2, 64)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("shape", ONE)
def test_every_option_key_by_key(shape, name, dtype):
    B, Sq, Sk, Hq = shape[:4]
    for cap in (0.0, 15.0):
        kw = _options(name, B, Sq, Sk, Hq, Sq + Sk) | dict(cap=cap)
        q, k, v = _qkv(Sq, *shape, dtype)
        check(kb.attention_scored(q, k, v, **kw), q, k, v, what=(name, cap), **kw)
