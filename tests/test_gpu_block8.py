"""8-bit matrices and their products against the definitions in 64 bits."""
import pytest
import torch

import exact_tensor_network_gb300 as tn

import block8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()
    tn.tn_block8_check()


def _x(R, C, dtype=torch.bfloat16, seed=0, wide=True):
    g = torch.Generator().manual_seed(seed * 1000 + R * 7 + C)
    x = torch.randn(R, C, generator=g)
    if wide and R and C:
        x *= torch.exp(2 * torch.randn(1, C, generator=g))
        x[torch.rand(R, generator=g) < 0.1] = 0
    return x.to(dtype)


def _same(got, want_codes, want_scales):
    assert torch.equal(got.scales.cpu().double().nan_to_num(-7), want_scales.nan_to_num(-7))
    assert torch.equal(got.codes.cpu().float().double(), want_codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 127), (3, 128), (128, 129), (130, 4), (257, 300), (16, 1030), (1, 4096)])
def test_quantize(R, C, square, dtype):
    x = _x(R, C, dtype)
    rows, cols = tn.quantize8(x.cuda(), square=square, layout="both")
    _same(rows, *ref.quantize(x, square))
    _same(cols, *ref.quantize(x.t(), square))
    for layout, both in (("rows", rows), ("columns", cols)):
        one = tn.quantize8(x.cuda(), square=square, layout=layout)
        assert torch.equal(one.codes.view(torch.uint8), both.codes.view(torch.uint8))
        assert torch.equal(one.scales, both.scales)


LINEAR = [(1, 128, 128), (1, 300, 4096), (2, 1, 1), (16, 129, 257), (17, 1000, 640), (33, 200, 2048), (64, 256, 1024),
          (65, 515, 384), (128, 128, 8192), (129, 257, 130), (300, 700, 1111), (1000, 131, 256), (700, 64, 512),
          (2048, 2500, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("R,N,K", LINEAR)
def test_linear(R, N, K, powers, dtype):
    x, w = _x(R, K, torch.bfloat16, 1), _x(N, K, torch.float32, 2) * K ** -0.5
    q = tn.quantize8(w.cuda(), square=True)
    y = tn.linear8(x.cuda(), tn.Blocks8(q.codes, q.scales, powers), dtype=dtype)
    c, far = ref.product_bound(ref.values(*ref.quantize(x, False)), ref.values(*ref.quantize(w, True)), dtype)
    assert y.shape == (R, N) and y.dtype is dtype
    assert ((y.cpu().double() - c).abs() <= far).all()


@pytest.mark.parametrize("R,N,K", [(1, 128, 64), (5, 130, 256), (128, 256, 384), (300, 515, 260), (1000, 64, 130),
                                   (4096, 640, 512)])
def test_linear_grad(R, N, K):
    x, dy, w = _x(R, K, torch.bfloat16, 3), _x(R, N, torch.bfloat16, 4) * 2.0 ** -8, _x(N, K, torch.float32, 5)
    wt = tn.quantize8(w.cuda(), square=True, layout="columns")
    dx, dw = tn.linear8_grad(x.cuda(), dy.cuda(), wt)
    v = [ref.values(*ref.quantize(m, s)) for m, s in ((dy, False), (w.t(), True), (dy.t(), False), (x.t(), False))]
    for got, (c, far) in ((dx, ref.product_bound(v[0], v[1], torch.bfloat16)),
                          (dw, ref.product_bound(v[2], v[3], torch.float32))):
        assert ((got.cpu().double() - c).abs() <= far).all()


@pytest.mark.parametrize("R,N,K", [(3, 200, 300), (40, 700, 512), (200, 300, 1024), (2000, 1500, 640)])
def test_any_scales(R, N, K):
    """Scales that are no powers of two, of rows and of squares, in either layout."""
    g = torch.Generator().manual_seed(R)
    a, b = tn.quantize8(_x(R, K, seed=6).cuda()), tn.quantize8(_x(N, K, seed=7).cuda(), square=True)
    fa, fb = torch.rand(a.scales.shape, generator=g) + 0.5, torch.rand(b.scales.shape, generator=g) + 0.5
    a = tn.Blocks8(a.codes, (a.scales.cpu() * fa).cuda(), False)
    b = tn.Blocks8(b.codes, (b.scales.cpu() * fb).cuda().t().contiguous().t(), False)
    y = tn.product8(a, b, dtype=torch.float32)
    c, far = ref.product_bound(ref.values(a.codes.cpu().float(), a.scales.cpu()),
                               ref.values(b.codes.cpu().float(), b.scales.cpu()), torch.float32)
    assert ((y.cpu().double() - c).abs() <= far).all()
    # both operands with a scale a row
    z = tn.product8(a, a, dtype=torch.float32)
    v = ref.values(a.codes.cpu().float(), a.scales.cpu())
    c, far = ref.product_bound(v, v, torch.float32)
    assert ((z.cpu().double() - c).abs() <= far).all()
