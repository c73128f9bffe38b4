"""Caps far above the scores, and scores on both sides of half of the cap, against 64 bits."""
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


# new tokens over a cache (at most 16 rows a key head), a prompt, enough rows for two row tiles a CTA
SHAPES = [(2, 1, 700, 8, 2, 128), (1, 3, 200, 4, 2, 64), (1, 200, 200, 2, 1, 128), (2, 130, 333, 2, 2, 64)]
LONG = [(10, 300, 300, 8, 8, 128), (10, 300, 300, 8, 8, 64)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cap", [5e3, 8.8e3, 1e4, 1e6, 1e7, 1e9, 1e16, 1e20, 1e30, 3e38])
def test_a_cap_far_above_the_scores_changes_nothing(cap, shape, dtype):
    q, k, v = _qkv(1, *shape, dtype)
    check(kb.attention_scored(q, k, v, cap=cap), q, k, v, cap=cap)
    # above 1e7, tanh differs from its argument by less than a rounding
    if cap >= 1e7:
        check(kb.attention_scored(q, k, v, cap=cap), q, k, v)


@pytest.mark.parametrize("shape", LONG)
@pytest.mark.parametrize("cap", [1e4, 1e6, 1e9, 1e30])
def test_large_caps_on_many_rows(cap, shape):
    q, k, v = _qkv(2, *shape, BF16)
    check(kb.attention_scored(q, k, v, cap=cap, causal=True), q, k, v, rows=range(0, 300, 7), cap=cap, causal=True)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cap", [3.0, 2e3, 1e5, 1e6])
def test_one_row_beyond_half_of_the_cap_leaves_the_others_alone(cap, shape, dtype):
    """Rows are independent: a query whose scores reach the cap does not coarsen its neighbours'."""
    q, k, v = _qkv(3, *shape, dtype)
    q[:, 0, 0] *= cap   # every query head shares its warp with others
    kw = dict(cap=cap, slopes=torch.full((shape[3],), 1e-3, device="cuda"))
    others = dict(rows=range(1, shape[1])) if shape[1] > 1 else dict(heads=range(1, shape[3]))
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **others, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scale,cap", [(1.0, 1e-6), (1e-9, 1e-5), (1e-9, 1e3), (3e3, 1e-2)])
def test_scales_and_caps_at_the_ends(scale, cap, dtype):
    """The smallest cap of a scale, and scales whose polynomial would leave the floats' range."""
    for shape in SHAPES[:3]:
        q, k, v = _qkv(4, *shape, dtype)
        q = q * (1.0 if scale >= 1e-3 else 1e6)
        check(kb.attention_scored(q, k, v, cap=cap, scale=scale), q, k, v, cap=cap, scale=scale)


def test_a_cap_below_a_millionth_of_the_scale_is_refused():
    """1e-9 in fp32 lies just below a millionth of 1e-3 in fp32."""
    q, k, v = _qkv(4, *SHAPES[0], BF16)
    with pytest.raises(kb.KimodoError, match="millionth"):
        kb.attention_scored(q, k, v, cap=1e-9, scale=1e-3)
