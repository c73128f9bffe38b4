"""Attention with scored masks against its definition in 64 bits."""
import pytest
import torch

import transformer_denoiser_b200 as kb
from gpu_fixtures import require_cuda
from operator_refs import check_attention

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
    q = (1.5 * torch.randn(B, Sq, Hq, D, generator=g)).to(dtype)
    k = torch.randn(B, Sk, Hkv, D, generator=g).to(dtype)
    v = torch.randn(B, Sk, Hkv, D, generator=g).to(dtype)
    return q.cuda(), k.cuda(), v.cuda()


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _run(seed, shape, dtype, **options):
    q, k, v = _qkv(seed, *shape, dtype)
    out = kb.attention_scored(q, k, v, **options)
    torch.cuda.synchronize()
    check_attention(out, q, k, v, what=(shape, dtype, sorted(options)), **options)
    return q, k, v, out


SHAPES = [
    # B, Sq, Sk, Hq, Hkv, D
    (1, 1, 1, 1, 1, 128), (2, 1, 130, 4, 2, 64), (1, 3, 127, 7, 1, 128), (2, 31, 31, 8, 8, 128), (1, 128, 128, 2, 2, 64),
    (1, 129, 129, 1, 1, 128), (1, 151, 151, 2, 1, 128), (1, 257, 300, 3, 1, 64), (1, 65, 513, 4, 2, 128), (3, 2, 700, 8, 2, 128),
    (1, 300, 300, 2, 2, 64), (1, 100, 1500, 2, 2, 128), (1, 16, 257, 2, 1, 64), (2, 20, 600, 3, 3, 128), (1, 130, 1100, 2, 1, 128),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_full(shape, dtype):
    _run(sum(shape), shape, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_all_options(shape, dtype):
    """Cap, distance bias, causal with a prefix, ragged lengths and a start, together."""
    B, Sq, Sk, Hq = shape[:4]
    lengths = _i32(*[max(1, Sk - 13 * b) for b in range(B)])
    _run(sum(shape) + 1, shape, dtype, cap=5.0, slopes=torch.exp2(-torch.arange(1, Hq + 1.0)).cuda(), causal=True,
         prefix=_i32(*[Sk // 3 + b for b in range(B)]), kv_lengths=lengths, q_start=lengths - Sq, scale=0.11)


@pytest.mark.parametrize("option", [dict(cap=50.0), dict(cap=0.7), dict(causal=True),
                                    dict(slopes=torch.tensor([0.0, 0.5, 2.0, 0.01], dtype=torch.float32)), dict(scale=0.0), dict(scale=-0.3), dict(scale=-0.3, cap=4.0), dict(scale=0.0, cap=4.0),
                                    dict(cap=30.0, slopes=torch.tensor([0.3, -0.02, 0.0, 0.004], dtype=torch.float32))])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Sq,Sk", [(200, 200), (5, 400), (140, 1200)])
def test_one_option(Sq, Sk, dtype, option):
    option = {n: v.cuda() if torch.is_tensor(v) else v for n, v in option.items()}
    _run(Sq + Sk, (2, Sq, Sk, 4, 2, 128), dtype, **option)


def _documents(B, S, sizes):
    d = torch.cat([torch.full((n,), i) for i, n in enumerate(sizes)])
    d = torch.cat([d, torch.full((max(0, S - len(d)),), -1)])[:S]
    return d.to(torch.int32).repeat(B, 1).cuda()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("sizes", [(400,), (1,) * 50, (60, 200, 7, 133), (128, 128, 128), (5, 0, 300, 40)])
@pytest.mark.parametrize("causal", [False, True])
def test_documents(sizes, causal, dtype):
    """Packed documents; tokens past the last one are in none (their queries see nothing)."""
    S = 400
    d = _documents(2, S, sizes)
    _, _, _, out = _run(len(sizes), (2, S, S, 2, 1, 64), dtype, q_documents=d, kv_documents=d, causal=causal)
    assert (out[d < 0] == 0).all()


def test_documents_in_any_order():
    g = torch.Generator().manual_seed(4)
    d = torch.randint(-1, 5, (2, 333), generator=g, dtype=torch.int32).cuda()
    _run(8, (2, 333, 333, 2, 2, 128), BF16, q_documents=d, kv_documents=d,
         slopes=torch.tensor([0.1, 0.2]).cuda())
    qd = d[:, :3].contiguous()
    _run(9, (2, 3, 333, 4, 2, 128), BF16, q_documents=qd, kv_documents=d)


@pytest.mark.parametrize("shape", [(3, 1300, 1300, 2, 1, 64), (1, 40, 5003, 2, 2, 128), (5, 1025, 1025, 8, 8, 64),
                                   (1, 17, 1024, 1, 1, 64), (2, 300, 897, 2, 2, 128)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_documents_over_many_key_tiles(shape, cap):
    """From 8 key tiles on a kernel of its own summarises their documents: odd batches, tokens in no
    document, numbers up to the largest, lengths that end inside a tile, split keys, two row tiles."""
    B, Sq, Sk = shape[:3]
    g = torch.Generator().manual_seed(sum(shape))
    d = torch.repeat_interleave(torch.arange(Sk), torch.randint(1, 400, (Sk,), generator=g))[:B * Sk].reshape(B, Sk)
    d = (d - d[:, :1]).to(torch.int32)
    d[:, 100:131] = -7
    d[:, Sk - 200:Sk - 150] = 2 ** 31 - 1
    qd = d[:, Sk - Sq:].contiguous()
    lengths = torch.tensor([Sk - 37 * b for b in range(B)], dtype=torch.int32)
    _run(sum(shape), shape, BF16, q_documents=qd.cuda(), kv_documents=d.cuda(), cap=cap, kv_lengths=lengths.cuda())


@pytest.mark.parametrize("shape", [(9, 75, 140, 16, 8, 64), (20, 129, 33, 4, 4, 128)])
@pytest.mark.parametrize("options", ["lengths", "documents", "all", "poison"])
def test_fp32_rows_left_behind_whole_tiles(shape, options):
    """Heads whose last CTA has few rows (22 that share tokens with the one before, 1): warps without rows."""
    B, Sq, Sk, Hq = shape[:4]
    g = torch.Generator().manual_seed(Sq)
    lengths = torch.randint(0, Sk + 1, (B,), generator=g, dtype=torch.int32)
    if options == "poison":
        q, k, v = _qkv(Sk, *shape, FP32)
        for b in range(B):
            k[b, lengths[b]:] = float("nan")
            v[b, lengths[b]:] = float("inf")
        check_attention(kb.attention_scored(q, k, v, kv_lengths=lengths.cuda()), q, k, v, kv_lengths=lengths.cuda())
        return
    kw = {}
    if options != "documents":
        kw |= dict(kv_lengths=lengths.cuda(), slopes=(torch.arange(Hq) / 37).cuda())
    if options != "lengths":
        d = torch.randint(-1, 3, (B, max(Sq, Sk)), generator=g, dtype=torch.int32).cuda()
        kw |= dict(q_documents=d[:, :Sq].contiguous(), kv_documents=d[:, :Sk].contiguous())
    if options == "all":
        kw |= dict(causal=True, cap=20.0, prefix=torch.randint(0, 9, (B,), generator=g, dtype=torch.int32).cuda())
    _run(Sq, shape, FP32, **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Sq,Sk", [(40, 300), (1, 300), (300, 300)])
def test_rows_that_see_nothing(Sq, Sk, dtype):
    """Lengths of zero, and causal queries before the first key."""
    q, k, v, out = _run(1, (3, Sq, Sk, 2, 1, 64), dtype, kv_lengths=_i32(0, 1, Sk + 5))
    assert (out[0] == 0).all()
    _, _, _, out = _run(2, (2, Sq, Sk, 2, 1, 64), dtype, causal=True, q_start=_i32(-Sq - 3, -1))
    assert (out[0] == 0).all() and (out[1, 0] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_no_keys(dtype):
    q, k, v = _qkv(1, 2, 5, 0, 4, 2, 64, dtype)
    assert (kb.attention_scored(q, k, v) == 0).all()
    d = torch.zeros(2, 5, dtype=torch.int32).cuda()
    assert (kb.attention_scored(q, k, v, q_documents=d, kv_documents=d[:, :0].contiguous(), causal=True) == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Sq,Sk", [(150, 150), (1, 150), (1, 1100), (300, 300)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_unseen_keys_do_not_leak(Sq, Sk, dtype, poison):
    """NaN and infinities in keys and values behind a length, ahead of a causal query, and in other
    documents change nothing: every output is the definition's over the seen keys."""
    q, k, v = _qkv(7, 2, Sq, Sk, 4, 2, 128, dtype)
    n = Sk - 17
    opts = dict(kv_lengths=_i32(n, Sk - 1))
    k[0, n:], v[0, n:], k[1, Sk - 1:], v[1, Sk - 1:] = poison, poison, poison, poison
    check_attention(kb.attention_scored(q, k, v, **opts), q, k, v, **opts)
    at = Sk - min(Sq, 9)          # causal: queries before position `at` do not see it
    q, k, v = _qkv(8, 1, Sq, Sk, 4, 2, 128, dtype)
    k[0, at], v[0, at] = poison, poison
    out = kb.attention_scored(q, k, v, causal=True)
    first = at - (Sk - Sq)        # first query that sees it
    if first > 0:
        check_attention(out[:, :first], q[:, :first], k, v, causal=True, q_start=_i32(Sk - Sq))
    d = torch.zeros(1, Sk, dtype=torch.int32)
    d[0, Sk // 2:] = 1
    d = d.cuda()
    q, k, v = _qkv(9, 1, Sq, Sk, 4, 2, 128, dtype)
    k[0, 3], v[0, 5] = poison, poison
    qd = torch.ones(1, Sq, dtype=torch.int32).cuda()
    check_attention(kb.attention_scored(q, k, v, q_documents=qd, kv_documents=d), q, k, v, q_documents=qd, kv_documents=d)


def test_seen_nonfinite_values_are_seen():
    q, k, v = _qkv(3, 1, 140, 140, 2, 2, 64, BF16)
    v[0, 50, 0, 3] = float("nan")
    out = kb.attention_scored(q, k, v, causal=True)
    assert torch.isfinite(out[0, :50]).all() and torch.isnan(out[0, 50:, 0, 3]).all()
    assert torch.isfinite(out[0, :, 1]).all() and torch.isfinite(out[0, :, 0, :3]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides(dtype):
    """Views into a fused projection, heads before tokens, and an output inside a larger buffer."""
    require_cuda()
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(2, 70, 3 * 4 * 64, generator=g).to(dtype).cuda()
    q, k, v = (x.unflatten(2, (4, 64)) for x in qkv.split(256, 2))
    check_attention(kb.attention_scored(q, k, v, causal=True), q, k, v, causal=True)
    qh, kh, vh = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v))
    buf = torch.full((2, 80, 6, 64), 3.0, dtype=dtype, device="cuda")
    out = kb.attention_scored(qh, kh, vh, out=buf[:, 5:75, 1:5])
    check_attention(out, q, k, v)
    buf[:, 5:75, 1:5] = 3.0
    assert (buf == 3.0).all()


def test_scores_that_grow_along_the_keys():
    """The running maximum moves far in every tile, so every tile rescales what came before."""
    q, k, v = _qkv(5, 1, 200, 900, 2, 1, 128, BF16)
    k = (k.float() * torch.linspace(0.1, 6, 900, device="cuda")[None, :, None, None]).to(BF16)
    check_attention(kb.attention_scored(q, k, v), q, k, v)
    check_attention(kb.attention_scored(q[:, :2].contiguous(), k, v), q[:, :2], k, v)
    big = (q.float() * 30).to(BF16)
    check_attention(kb.attention_scored(big, k, v), big, k, v)


def test_same_bits_again_and_on_another_stream():
    q, k, v = _qkv(6, 3, 2, 1500, 8, 2, 128, BF16)
    L = _i32(1500, 700, 3)
    want = kb.attention_scored(q, k, v, kv_lengths=L, cap=30.0)
    assert torch.equal(want, kb.attention_scored(q, k, v, kv_lengths=L, cap=30.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = kb.attention_scored(q, k, v, kv_lengths=L, cap=30.0)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, other)


def test_two_captured_graphs():
    """Two captured calls, each with its own workspace, replayed at the same time on two streams."""
    sets = [_qkv(s, 2, 1, 3001, 8, 2, 128, BF16) for s in (1, 2)]
    want = [kb.attention_scored(*s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kb.attention_scored(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)
    kb.kernel_status()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_past_32_bits(dtype):
    """A batch stride of 2^31 elements in the cache, the queries and the output."""
    require_cuda()
    g = torch.Generator().manual_seed(12)
    far = 1 << 31
    buf = torch.empty(far + 4 * 40000, dtype=dtype, device="cuda")

    def view(at, tokens, heads):
        v = buf.as_strided((2, tokens, heads, 64), (far, heads * 64, 64, 1), at)
        v.copy_(torch.randn(2, tokens, heads, 64, generator=g).to(dtype))
        return v

    for Sq in (3, 150):
        k, v, q, out = view(0, 200, 1), view(40000, 200, 1), view(80000, Sq, 2), view(120000, Sq, 2)
        check_attention(kb.attention_scored(q, k, v, causal=True, out=out), q, k, v, causal=True)
    del buf, k, v, q, out


def test_more_key_tiles_than_the_document_list_holds():
    """Over 4096 key tiles of documents: every tile is gone through with its mask."""
    Sk = 4096 * 128 + 300
    q, k, v = _qkv(15, 1, 70, Sk, 1, 1, 64, BF16)
    kd = (torch.arange(Sk, dtype=torch.int32) // 200000)[None].cuda().contiguous()
    qd = (torch.arange(70, dtype=torch.int32) % 4 - 1)[None].cuda().contiguous()
    out = kb.attention_scored(q, k, v, q_documents=qd, kv_documents=kd)
    at = [0, 1, 2, 3, 33, 69]
    check_attention(out[:, at], q[:, at], k, v, q_documents=qd[:, at], kv_documents=kd)


def test_documents_split_over_ctas():
    """Few CTAs, so that the keys are split: lists of parts, empty parts, and their join."""
    d = (torch.arange(3000, dtype=torch.int32) // 170)[None].cuda().contiguous()
    qd = d[:, 1400:1570].contiguous()
    q, k, v = _qkv(16, 1, 170, 3000, 1, 1, 128, BF16)
    check_attention(kb.attention_scored(q, k, v, q_documents=qd, kv_documents=d, slopes=torch.tensor([0.05]).cuda()), q, k, v,
                    q_documents=qd, kv_documents=d, slopes=torch.tensor([0.05]))


def test_a_workspace_that_is_missing_or_short_is_refused():
    import ctypes
    q, k, v = _qkv(17, 1, 1, 3000, 8, 2, 128, BF16)
    out = torch.empty_like(q)
    lib = kb.load_library()
    s = [tuple(t.stride()[:3]) for t in (q, k, v, out)]
    a = kb.ScoredAttention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None, None, None, None, None, None, *s,
                           1, 1, 3000, 8, 2, 128, kb.BF16, 0, 0.1, 0.0)
    n = ctypes.c_size_t()
    assert lib.kimodo_attention_scored_workspace(ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.kimodo_attention_scored(ctypes.byref(a), None, 0, None) == -1
    assert b"workspace" in lib.kimodo_last_error()
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    assert lib.kimodo_attention_scored(ctypes.byref(a), ws.data_ptr(), n.value - 1, None) == -1
    host = torch.empty(16, dtype=torch.int32)
    a.kv_lengths = host.data_ptr()
    assert lib.kimodo_attention_scored(ctypes.byref(a), ws.data_ptr(), n.value, None) == -1   # host memory


def test_binding_checks():
    q, k, v = _qkv(18, 2, 4, 9, 4, 2, 64, BF16)
    for bad, text in ((dict(q=q.half()), "bf16 or fp32"), (dict(k=k.float()), "agree"), (dict(v=v[:, :8]), "agree"),
                      (dict(q=q[0]), "4-D"), (dict(q=q.transpose(2, 3)), "agree"), (dict(k=k.cpu(), v=v), "must be on cuda")):
        t = dict(q=q, k=k, v=v) | bad
        with pytest.raises(ValueError, match=text):
            kb.attention_scored(t["q"], t["k"], t["v"])
    for bad, text in ((dict(slopes=torch.ones(3).cuda()), "slopes"), (dict(prefix=_i32(1), causal=True), "prefix"),
                      (dict(kv_lengths=torch.ones(2, dtype=torch.int64).cuda()), "kv_lengths"), (dict(q_start=torch.zeros(2, dtype=torch.int32)), "q_start"),
                      (dict(out=torch.empty(1).cuda()), "out")):
        with pytest.raises(ValueError, match=text):
            kb.attention_scored(q, k, v, **bad)
    for bad, text in ((dict(prefix=_i32(1, 1)), "prefix needs causal"), (dict(q_documents=torch.zeros(2, 4, dtype=torch.int32).cuda()), "together"),
                      (dict(cap=-2.0), "cap"), (dict(scale=float("inf")), "scale"), (dict(scale=1e7, cap=1.0), "millionth")):
        with pytest.raises(kb.KimodoError, match=text):
            kb.attention_scored(q, k, v, **bad)
    with pytest.raises(kb.KimodoError, match="strides"):
        kb.attention_scored(q, k[:1].expand(2, -1, -1, -1), v)
    with pytest.raises(kb.KimodoError, match="16-byte aligned"):
        kb.attention_scored(q.flatten()[4:4 + 256].view(1, 1, 4, 64), k[:1], v[:1])
    with pytest.raises(kb.KimodoError, match="head_dim"):
        kb.attention_scored(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous())
