"""Caches that were allocated without being written: what lies behind the newest token may be
anything, and costs nothing."""
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


def _time(call):
    """Least of seven device times (ms)."""
    best = float("inf")
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Sq,Sk,at,Hq,Hkv,D,cap", [
    (2, 1, 32768, 30001, 8, 2, 128, 0.0),   # one new token each: the kernels for few rows
    (2, 3, 16384, 9000, 4, 2, 64, 30.0),
    (1, 130, 8192, 4000, 4, 2, 128, 0.0),   # a piece of a prompt: the kernels for many rows
    (10, 300, 2048, 1011, 8, 8, 64, 30.0),  # with enough rows for two row tiles a CTA
])
def test_what_lies_behind_the_newest_token(B, Sq, Sk, at, Hq, Hkv, D, cap, dtype):
    """Queries at positions at .. at + Sq - 1 under a causal mask, no lengths given: NaN behind them changes
    neither the result nor (by more than the noise of a short call) the time."""
    require_cuda()
    g = torch.Generator().manual_seed(1)

    def draw(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32).to(dtype).cuda()
    q, k, v = draw(B, Sq, Hq, D), draw(B, Sk, Hkv, D), draw(B, Sk, Hkv, D)
    kw = dict(causal=True, q_start=torch.full((B,), at, dtype=torch.int32).cuda(), cap=cap)
    clean = kb.attention_scored(q, k, v, **kw)
    plain = _time(lambda: kb.attention_scored(q, k, v, **kw))
    k[:, at + Sq:] = float("nan")
    v[:, at + Sq:] = float("nan")
    out = kb.attention_scored(q, k, v, **kw)
    assert torch.equal(out, clean)
    check(out, q, k, v, rows=sorted({0, Sq // 2, Sq - 1}), **kw)
    unwritten = _time(lambda: kb.attention_scored(q, k, v, **kw))
    # one row at a time over all its keys would take tens of times as long
    assert unwritten < 3 * plain + 0.05, (plain, unwritten)
