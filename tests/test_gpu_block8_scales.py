"""Products with scales far from 1 against the definitions in 64 bits; sums that are exact; and what is
reported."""
import threading

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


def _codes(R, K, seed, small):
    """Codes of the smallest numbers, or of all sizes."""
    g = torch.Generator().manual_seed(seed + R)
    if small:
        x = torch.randint(-3, 4, (R, K), generator=g).float() * 2.0 ** -9
    else:
        x = torch.randn(R, K, generator=g) * 60
    codes = torch.zeros(R, -(-K // 16) * 16, dtype=torch.float8_e4m3fn)
    codes[:, :K] = x.to(torch.float8_e4m3fn)
    return codes


SIZES = [(3, 200, 300), (40, 700, 512), (200, 300, 1024), (300, 1000, 384), (2000, 1500, 640)]


@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("ea,eb,small", [(70, 60, True), (-70, -70, False), (-120, 110, False), (110, -120, False),
                                         (120, 4, True), (4, 120, True), (-140, 100, False), (100, -140, False),
                                         (-149, 126, False), (126, -149, False)])
@pytest.mark.parametrize("R,N,K", SIZES)
def test_scales_far_from_one(R, N, K, ea, eb, small, square, powers):
    """Whatever their product is on the way: a value that fp32 holds is that value.  Scales within a factor of 4 of
    2^ea and 2^eb."""
    if powers and min(ea, eb) < -126:
        pytest.skip("no powers of two that a matrix may have")
    g = torch.Generator().manual_seed(R + N)
    m = [tn.Blocks8(None, None)] * 2
    for i, (rows, e, tall) in enumerate(((R, ea, 1), (N, eb, 128 if square else 1))):
        s = torch.randint(-1 if e > -149 else 0, 2, (-(-rows // tall), -(-K // 128)), generator=g)
        s = torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s + e)
        if not powers and e > -120:
            s *= 1 + torch.rand(s.shape, generator=g, dtype=torch.float64) / 2
        m[i] = (_codes(rows, K, 90 + i, small), s.float())
    vals = [ref.values(c[:, :K].float(), s) for c, s in m]
    y = tn.product8(*(tn.Blocks8(c.cuda()[:, :K], s.cuda(), powers) for c, s in m), dtype=torch.float32)
    c, far = ref.product_bound(*vals, torch.float32)
    assert c.abs().max() < 2.0 ** 127 and c.abs().max() > 2.0 ** -126
    assert ((y.cpu().double() - c).abs() <= far).all()


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("R,N,K", SIZES + [(1, 333, 2000), (129, 257, 8192), (500, 500, 8192), (1000, 5003, 1112)])
def test_whole_numbers(R, N, K, powers):
    """Sums of whole numbers below 2^24 are exact, whichever way a product takes: no addend is lost."""
    g = torch.Generator().manual_seed(K)
    a = torch.randint(-8, 9, (R, K), generator=g).float()
    b = torch.randint(-8, 9, (N, K), generator=g).float()
    m = []
    for x in (a, b):
        codes = torch.zeros(x.shape[0], -(-K // 16) * 16, dtype=torch.float8_e4m3fn)
        codes[:, :K] = x.to(torch.float8_e4m3fn)
        m.append(tn.Blocks8(codes.cuda()[:, :K], torch.ones(x.shape[0], -(-K // 128), device="cuda"), powers))
    y = tn.product8(*m, dtype=torch.float32)
    assert torch.equal(y.cpu().double(), a.double() @ b.double().t())


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,N,K", [(1, 130, 4096), (5, 131, 4100), (33, 77, 6000), (100, 333, 5000), (130, 130, 8192),
                                   (257, 1, 8192), (1, 1, 16384), (61, 257, 2048)])
def test_ragged_tiles_of_clusters(R, N, K, dtype, powers):
    """Tiles that a cluster shares and that the output ends in: only some lanes of a warp store at the end.  Whole numbers
    below 2^16, so that a rounding to the output's type is all."""
    g = torch.Generator().manual_seed(K + N)
    a, b = torch.randint(-1, 2, (R, K), generator=g).float(), torch.randint(-1, 2, (N, K), generator=g).float()
    q = [tn.quantize8(x.cuda()) for x in (a, b)]
    q = [tn.Blocks8(x.codes, x.scales, powers) for x in q]
    want = (a.double() @ b.double().t()).float().to(dtype)
    for _ in range(5):
        whole = torch.full((R + 2, N + 5), 3.25, dtype=dtype, device="cuda")
        y = tn.product8(*q, out=whole[1:-1, 2:N + 2])
        assert torch.equal(y.cpu(), want)
        whole[1:-1, 2:N + 2] = 3.25
        assert (whole == 3.25).all()


def test_reports_reach_every_thread():
    """A thread's question takes no report away from another, and is answered once."""
    q = tn.quantize8(_codes(40, 256, 95, False).float().cuda())
    bad = q.scales.clone()
    bad[3, 1] = 1.5
    seen = []

    def ask():
        try:
            tn.tn_block8_check()
            seen.append(tn.TN_OK)
        except tn.TNError as e:
            seen.append(e.status)

    def other(n):
        t = threading.Thread(target=lambda: [ask() for _ in range(n)])
        t.start()
        t.join()

    torch.cuda.synchronize()
    ask()
    assert seen == [tn.TN_OK]
    tn.product8(q._replace(scales=bad), q)
    torch.cuda.synchronize()
    other(2)
    assert seen[1:] == [tn.TN_EDEVICE, tn.TN_OK]
    ask()
    ask()
    assert seen[3:] == [tn.TN_EDEVICE, tn.TN_OK]
