"""Distance bias of queries that lie far from every key they see: only the differences between the
keys' distances count, and they are not lost in the distance itself."""
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
# B, Sq, Sk, Hq, Hkv, D: new tokens over a cache in one part and in several, prompts in one part and in several
SHAPES = [(3, 1, 100, 8, 2, 128), (3, 2, 5000, 4, 1, 64), (3, 70, 300, 2, 1, 128), (3, 60, 2600, 2, 2, 128),
          (3, 300, 300, 2, 2, 64)]


def _qkv(seed, B, Sq, Sk, Hq, Hkv, D, dtype):
    require_cuda()
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32)
    return tuple(t.to(dtype).cuda() for t in (1.5 * draw(B, Sq, Hq, D), draw(B, Sk, Hkv, D), draw(B, Sk, Hkv, D)))


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _slopes(heads):
    return (0.5 / torch.arange(1, heads + 1, dtype=torch.float32)).cuda()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("far", [30000, 10 ** 6, 10 ** 9])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_queries_far_behind_and_far_ahead(far, shape, dtype, cap):
    q, k, v = _qkv(1, *shape, dtype)
    kw = dict(slopes=_slopes(shape[3]), q_start=_i32(shape[2] + far, -far - shape[1], 5), cap=cap)
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)
    kw |= dict(causal=True, prefix=_i32(0, shape[2] // 2, 1))
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_positions_at_the_ends_of_32_bits(shape, dtype):
    q, k, v = _qkv(2, *shape, dtype)
    kw = dict(slopes=_slopes(shape[3]), q_start=_i32(2 ** 31 - 1, -2 ** 31, 2 ** 31 - shape[1]))
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)
    out = kb.attention_scored(q, k, v, causal=True, **kw)
    check(out, q, k, v, causal=True, **kw)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Sq,Sk", [(1, 33000), (40, 33000), (700, 700)])
def test_lengths_far_short_of_the_positions(Sq, Sk, dtype):
    """Queries at the end of a padded batch whose keys end long before."""
    q, k, v = _qkv(3, 2, Sq, Sk, 4, 2, 64, dtype)
    kw = dict(slopes=_slopes(4), kv_lengths=_i32(90, 317))
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_computed_again_count_the_same_way(shape, dtype):
    """A NaN among the values of another document sends the rows through the one-row form."""
    B, Sq, Sk = shape[:3]
    q, k, v = _qkv(4, *shape, dtype)
    d = (torch.arange(Sk) >= Sk - 40).int().repeat(B, 1).cuda()
    v[:, Sk - 41] = float("nan")
    kw = dict(slopes=_slopes(shape[3]), q_start=_i32(Sk + 10 ** 6, -10 ** 6, 0), kv_documents=d,
              q_documents=torch.ones(B, Sq, dtype=torch.int32).cuda())
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Sq", [1, 40])
def test_a_document_far_from_its_query(Sq, dtype):
    """A bias is right to |slope| d 2^-20 at the distance d of the row's own document, no better."""
    Sk = 33000
    q, k, v = _qkv(5, 1, Sq, Sk, 4, 2, 64, dtype)
    d = torch.full((1, Sk), 7, dtype=torch.int32)
    d[0, 1000:1300] = 3
    kw = dict(slopes=_slopes(4), kv_documents=d.cuda(), q_documents=torch.full((1, Sq), 3, dtype=torch.int32).cuda())
    check(kb.attention_scored(q, k, v, **kw), q, k, v, **kw)
