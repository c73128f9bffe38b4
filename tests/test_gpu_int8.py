"""The 8-bit projections (rows in 8-bit integers, RMS norm, product) against their
definitions in 64 bits."""
import pytest
import torch

import transformer_denoiser_b200 as kb
from gpu_fixtures import require_cuda
from operator_refs import BF16_HALF, check_rows, gemm_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _fp32_default():
    """Tensors drawn here are fp32 whatever default another module has set."""
    was = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(was)


def _gen(seed):
    require_cuda()
    return torch.Generator().manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g)


ROWS = [(1, 1), (1, 8), (3, 7), (5, 16), (1, 1024), (151, 1024), (4, 1025), (9, 1032), (2, 4096), (3, 4097), (1, 5000),
        (2, 16384), (2, 16391), (1, 32768), (2, 32767), (1003, 279)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_quantize_int8(rows, cols, dtype):
    g = _gen(rows * 7 + cols)
    x = (_normal(g, rows, cols) * torch.exp(_normal(g, rows, 1) * 3)).to(dtype)
    q, scale = kb.quantize_int8(x.cuda())
    check_rows(q, scale, x.double(), (rows, cols))


def test_quantize_int8_strided_and_misaligned_rows():
    g = _gen(5)
    base = _normal(g, 40, 300).cuda()
    for x in (base[:, 3:260], base[::3, :256], base[1:, :7], base.bfloat16()[:, 1:200], base.flatten()[1:1 + 39 * 300].view(39, 300)):
        q, scale = kb.quantize_int8(x)
        check_rows(q, scale, x.double(), tuple(x.shape))


def test_quantize_int8_rows_of_zeros_nonfinite_and_extreme_values():
    _gen(0)
    x = torch.zeros(9, 64)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = torch.arange(64) * 1e-42          # subnormal: 127 / max overflows
    x[4] = torch.linspace(-1, 1, 64) * 3e38
    x[5] = -2.0
    x[6, 0] = 1e-45
    x[7] = torch.arange(64) * 1e-38
    q, scale = (t.cpu() for t in kb.quantize_int8(x.cuda()))
    assert (q[0] == 0).all() and scale[0] == 0
    for r in (1, 2):
        assert (q[r] == 0).all() and torch.isnan(scale[r])
    keep = [0, 4, 5, 7, 8]
    check_rows(q[keep], scale[keep], x[keep].double(), "extremes")
    u = x[3].double() * 127 / x[3].double().abs().max()
    assert (q[3].double() - u).abs().max() <= 0.5 + 3.1e-5
    assert q[6, 0] == 127 and (q[5] == -127).all()


def _norm_case(rows, cols, dtype, rdtype, seed, scale=1.0):
    g = _gen(seed)
    x = (_normal(g, rows, cols) * scale).to(dtype)
    r = None if rdtype is None else (_normal(g, rows, cols) * scale).to(rdtype)
    gamma = 1 + 0.2 * _normal(g, cols)
    return x, r, gamma


def _check_norm(x, r, gamma, eps, q, s, out, what):
    h = x.float() if r is None else x.float() + r.float()
    if r is not None:
        assert torch.equal(out.cpu(), h.to(r.dtype)), what
    h = h.double()
    t = h * gamma.double() / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    # a thread adds at most 32 squares in order, then 5 + 32 partial sums
    check_rows(q, s, t, what, sum_terms=70)


@pytest.mark.parametrize("rdtype", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (302, 1024), (7, 1023), (3, 8), (2, 1), (5, 2730), (2, 16384), (1, 32767)])
def test_rms_norm_int8(rows, cols, dtype, rdtype):
    x, r, gamma = _norm_case(rows, cols, dtype, rdtype, rows + cols)
    q, s, out = kb.rms_norm_int8(x.cuda(), gamma.cuda(), None if r is None else r.cuda(), 1e-6)
    _check_norm(x, r, gamma, 1e-6, q, s, out, (rows, cols))


def test_rms_norm_int8_residual_in_place():
    x, r, gamma = _norm_case(33, 1024, torch.bfloat16, torch.float32, 3)
    xc, gc = x.cuda(), gamma.cuda()
    want = kb.rms_norm_int8(xc, gc, r.cuda(), 1e-5)
    res = r.cuda()
    got = kb.rms_norm_int8(xc, gc, res, 1e-5, residual_out=res)
    assert got[2] is res
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1e-25, 1e25, 1e37])
def test_rms_norm_int8_extreme_magnitudes(scale):
    """Squares that underflow (eps rules) and squares past the largest float."""
    x, _, gamma = _norm_case(4, 512, torch.float32, None, 11, scale)
    q, s, _ = kb.rms_norm_int8(x.cuda(), gamma.cuda(), None, 1e-6)
    _check_norm(x, None, gamma, 1e-6, q, s, None, scale)


@pytest.mark.parametrize("cols", [512, 333])
@pytest.mark.parametrize("scale,eps", [(1e-25, 0.0), (1e-20, 1e-38), (1e-32, 0.0), (1e-17, 1e-36), (1e-36, 1e-33)])
def test_rms_norm_int8_tiny_rows_without_eps(scale, eps, cols):
    """Squares that underflow and an eps that does not hide it."""
    x, _, gamma = _norm_case(4, cols, torch.float32, None, 13, scale)
    eps = float(torch.tensor(eps))   # the value that the call takes
    q, s, _ = kb.rms_norm_int8(x.cuda(), gamma.cuda(), None, eps)
    _check_norm(x, None, gamma, eps, q, s, None, (scale, eps))


def test_rms_norm_int8_zero_and_nonfinite_rows():
    x, _, gamma = _norm_case(5, 300, torch.float32, None, 12)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 299] = float("-inf")
    for eps in (1e-6, 0.0):
        q, s, _ = (None if t is None else t.cpu() for t in kb.rms_norm_int8(x.cuda(), gamma.cuda(), None, eps))
        assert (q[0] == 0).all() and s[0] == 0
        assert (q[1:3] == 0).all() and torch.isnan(s[1:3]).all()
        _check_norm(x[3:], None, gamma, eps, q[3:], s[3:], None, eps)


def _int8(g, rows, cols, dev="cuda"):
    """Random int8 rows on 16-byte boundaries; what lies past the columns is not zero."""
    ld = (cols + 15) // 16 * 16
    return torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int8).to(dev)[:, :cols]


GEMM = [
    # M, N, K
    (1, 1, 1), (1, 4096, 4096), (1, 129, 31), (2, 64, 128), (5, 1003, 1999), (16, 256, 64), (17, 300, 129), (31, 31, 31),
    (64, 512, 4096), (65, 33, 1000), (100, 274, 1024), (128, 128, 128), (130, 1040, 320), (257, 2048, 1024),
    (362, 2048, 1024), (700, 77, 515), (1283, 1024, 1024), (2049, 511, 257), (4833, 1003, 1999), (300, 1024, 16384),
    (17406, 16, 16), (3, 2049, 127), (9000, 130, 48),
]
EPI = [(kb.EPI_BIAS, False), (kb.EPI_BIAS, True), (kb.EPI_BIAS_GELU, False), (kb.EPI_BIAS_SILU, False),
       (kb.EPI_BIAS_RESID, True)]


def _check_gemm(out, a, sa, w, sw, bias, epi, resid, what):
    ref, err = gemm_ref(a, sa, w, sw, bias, epi, resid)
    tol = err if out.dtype == torch.float32 else err * 1.01 + BF16_HALF * ref.abs()
    bad = (out.double() - ref).abs() > tol + 1e-30
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())


@pytest.mark.parametrize("epi,out_f32", EPI)
@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_int8(M, N, K, epi, out_f32):
    g = _gen(M * 3 + N * 5 + K)
    a, w = _int8(g, M, K), _int8(g, N, K)
    sa = (torch.rand(M, generator=g) + 0.5).cuda() / 64
    sw = (torch.rand(N, generator=g) + 0.5).cuda() / (64 * K ** 0.5)
    bias = _normal(g, N).cuda() if N % 2 else None
    resid = _normal(g, M, N).cuda() if epi == kb.EPI_BIAS_RESID else None
    out = kb.gemm_int8(a, sa, w, sw, bias, epi, out_f32, resid)
    torch.cuda.synchronize()
    _check_gemm(out, a, sa, w, sw, bias, epi, resid, (M, N, K))


@pytest.mark.parametrize("M,N,K", [(1, 40, 131071), (300, 40, 131071)])
def test_gemm_int8_largest_sums(M, N, K):
    """All -128 times all -128 over the largest K: the largest sum that 32 bits hold."""
    _gen(0)
    ld = (K + 15) // 16 * 16
    a = torch.full((M, ld), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, ld), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(max(M, N), device="cuda")
    out = kb.gemm_int8(a, one[:M].clone(), w, one[:N].clone(), None, kb.EPI_BIAS, True)
    assert (out == float(K * 16384)).all()


def test_gemm_int8_writes_only_its_output():
    """Rows and columns around a strided output keep their values; the residual may be the output."""
    g = _gen(9)
    for M, N, K in ((5, 70, 256), (300, 70, 256)):
        a, w = _int8(g, M, K), _int8(g, N, K)
        sa, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda") / 1000
        buf = torch.full((M + 4, N + 9), 7.0, device="cuda")
        view = buf[2:2 + M, 5:5 + N]
        kb.gemm_int8(a, sa, w, sw, None, kb.EPI_BIAS_RESID, True, view, out=view)
        torch.cuda.synchronize()
        _check_gemm(view, a, sa, w, sw, None, kb.EPI_BIAS_RESID, torch.full((M, N), 7.0, device="cuda"), (M, N, K))
        buf[2:2 + M, 5:5 + N] = 7.0
        assert (buf == 7.0).all()


def test_gemm_int8_replayed_and_on_another_stream():
    """A captured call replays on new inputs; a call on a side stream gives the same bits."""
    g = _gen(21)
    M, N, K = 77, 333, 777
    a, w = _int8(g, M, K), _int8(g, N, K)
    sa, sw = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    want = kb.gemm_int8(a, sa, w, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = kb.gemm_int8(a, sa, w, sw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kb.gemm_int8(a, sa, w, sw)
    sa2 = sa * 2
    want2 = kb.gemm_int8(a, sa2, w, sw)
    sa.copy_(sa2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)
    kb.kernel_status()


def test_offsets_past_32_bits():
    """Rows further than 2^31 elements from the first: input rows, product rows, output rows."""
    g = _gen(31)
    ld = (1 << 30) + 16
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(3, ld)[:, 8:1000]
    x.copy_(_normal(g, 3, 992).bfloat16())
    q, scale = kb.quantize_int8(x)
    check_rows(q, scale, x.double(), "far rows")
    M, N, K = 70000, 40, 64
    a, w = _int8(g, M, K), _int8(g, N, K)
    sa, sw = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    out = buf[:M * 40000].view(M, 40000)[:, 39000:39000 + N]
    kb.gemm_int8(a, sa, w, sw, out=out)
    _check_gemm(out[-200:], a[-200:], sa[-200:], w, sw, None, kb.EPI_BIAS, None, "far rows")
    del buf, out, x


def test_rows_wider_than_the_largest_are_refused():
    _gen(0)
    with pytest.raises(kb.KimodoError, match="cols must be"):
        kb.quantize_int8(torch.zeros(1, 32769, device="cuda"))


def test_binding_checks_shapes_types_and_strides():
    g = _gen(1)
    x = _normal(g, 4, 32).cuda()
    with pytest.raises(ValueError, match="bf16 or fp32"):
        kb.quantize_int8(x.half())
    with pytest.raises(ValueError, match="2-D"):
        kb.quantize_int8(x[0])
    with pytest.raises(ValueError, match="unit column stride"):
        kb.quantize_int8(x.t())
    with pytest.raises(ValueError, match="gamma"):
        kb.rms_norm_int8(x, torch.ones(31, device="cuda"))
    with pytest.raises(ValueError, match="residual must have"):
        kb.rms_norm_int8(x, torch.ones(32, device="cuda"), x[:3])
    with pytest.raises(ValueError, match="residual_out needs"):
        kb.rms_norm_int8(x, torch.ones(32, device="cuda"), residual_out=x)
    with pytest.raises(ValueError, match="gamma must be on cuda"):
        kb.rms_norm_int8(x, torch.ones(32))
    a, w = _int8(g, 4, 32), _int8(g, 8, 32)
    s4, s8 = torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        kb.gemm_int8(a[:, :16], s4, w, s8)
    with pytest.raises(ValueError, match="w_scale"):
        kb.gemm_int8(a, s4, w, s4)
    with pytest.raises(ValueError, match="int8"):
        kb.gemm_int8(a.to(torch.uint8), s4, w, s8)
    with pytest.raises(ValueError, match="out must be"):
        kb.gemm_int8(a, s4, w, s8, out=torch.empty(4, 8, device="cuda"))
    with pytest.raises(kb.KimodoError, match="16-byte aligned rows"):
        kb.gemm_int8(torch.zeros(4, 24, dtype=torch.int8, device="cuda"), s4,
                     torch.zeros(8, 24, dtype=torch.int8, device="cuda"), s8)
    with pytest.raises(kb.KimodoError, match="needs resid"):
        kb.gemm_int8(a, s4, w, s8, epilogue=kb.EPI_BIAS_RESID, out_f32=True)


def test_two_threads_on_two_streams():
    """Calls from two host threads at once, each on its own stream, give what one thread gets."""
    import threading
    g = _gen(77)
    a, w = _int8(g, 130, 640), _int8(g, 257, 640)
    sa, sw = torch.rand(130, generator=g).cuda(), torch.rand(257, generator=g).cuda()
    x = _normal(g, 130, 640).cuda()
    want = kb.gemm_int8(a, sa, w, sw)
    wq, ws = kb.quantize_int8(x)
    torch.cuda.synchronize()
    bad = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                out = kb.gemm_int8(a, sa, w, sw)
                q, s = kb.quantize_int8(x)
                st.synchronize()
                if not (torch.equal(out, want) and torch.equal(q, wq) and torch.equal(s, ws)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
