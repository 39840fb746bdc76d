"""The 8-bit matrices as programs use them: what no number is, layouts, memory around the
outputs, empty ones, scales that are not what they are said to be, streams and graphs; and
a head that is served and trained with them and the operators of rows."""
import math

import pytest
import torch

import exact_tensor_network_gb300 as tn

import block8_reference as ref
from outcome_reference import Row
from test_gpu_block8 import _same, _x
from test_gpu_sampling import _compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()
    tn.tn_block8_check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("square", [False, True])
def test_numbers_at_the_ends(square, dtype):
    """Blocks with infinities and NaN, the smallest and the largest numbers, zeros of both signs, and
    a largest entry at and just above 448 times a power of two."""
    f = torch.finfo(dtype)
    x = _x(300, 700, dtype, 8, wide=False)
    x[0, 3], x[1, 200], x[2, 699] = math.nan, math.inf, -math.inf
    x[140, :128] = f.max
    x[140, 5] = -f.max
    x[141, :128] = 0
    x[141, 7] = f.tiny * 2.0 ** -3      # below the normal numbers
    x[142, :128] = -0.0
    for i, v in enumerate((448.0, 448.0 * (1 + 2 * f.eps), 224.0 * (1 - f.eps), 2.0 ** -9 * 448)):
        x[143 + i, :] = x[143 + i, :].clamp(-1, 1) * 2.0 ** -12
        x[143 + i, ::130] = v
    rows, cols = tn.quantize8(x.cuda(), square=square, layout="both")
    _same(rows, *ref.quantize(x, square))
    _same(cols, *ref.quantize(x.t(), square))
    assert rows.scales.cpu()[0, 0].isnan() and (rows.codes.float()[0, :128] == 0).all()


@pytest.mark.parametrize("layout", ["columns", "offset", "steps", "row steps", "one row", "one column"])
@pytest.mark.parametrize("which", ["rows", "columns", "both"])
@pytest.mark.parametrize("square", [False, True])
def test_layouts_of_x(layout, which, square):
    w = _x(400, 530, torch.bfloat16, 9).cuda()
    x = {"columns": w.t().contiguous().t(), "offset": w[3:, 1:], "steps": w[:, ::3], "row steps": w[::2, 2:],
         "one row": w[:1].expand(200, 530), "one column": w[:, 5:6].expand(400, 260)}[layout]
    got = tn.quantize8(x, square=square, layout=which)
    host = x.cpu()
    if which == "columns":
        got = (got,)
    elif which == "rows":
        got = (got,)
    for b, y in zip(got, {"rows": (host,), "columns": (host.t(),), "both": (host, host.t())}[which]):
        _same(b, *ref.quantize(y, square))


@pytest.mark.parametrize("R,C", [(1, 5), (130, 200), (257, 130)])
@pytest.mark.parametrize("square", [False, True])
def test_memory_around_the_codes(R, C, square):
    """Padding, rows before and behind, and what lies between scales are left alone."""
    x = _x(R, C, torch.float32, 10)
    both = []
    for shape in ((R, C), (C, R)):
        tall = -(-shape[0] // 128) if square else shape[0]
        codes = torch.full((shape[0] + 2, -(-shape[1] // 16) * 16 + 32), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.full((tall + 2, 2 * -(-shape[1] // 128) + 1), 7.0, device="cuda")
        both.append((codes, scales, tn.Blocks8(codes.view(torch.float8_e4m3fn)[1:-1, 16:16 + shape[1]],
                                               scales[1:-1, 1::2])))
    out = tn.quantize8(x.cuda(), square=square, layout="both", out=tuple(b[2] for b in both))
    for (codes, scales, b), o, y in zip(both, out, (x, x.t())):
        assert o.codes.data_ptr() == b.codes.data_ptr()
        _same(b, *ref.quantize(y, square))
        keep = torch.ones_like(codes, dtype=torch.bool)
        keep[1:-1, 16:16 + y.shape[1]] = False
        assert (codes[keep] == 0x55).all()
        keep = torch.ones_like(scales, dtype=torch.bool)
        keep[1:-1, 1::2] = False
        assert (scales[keep] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("R,N,K", [(1, 333, 512), (20, 130, 130), (100, 77, 2000), (200, 301, 256), (700, 515, 1000),
                                   (2500, 245, 384)])
def test_memory_around_the_product(R, N, K, powers, dtype):
    """An output of odd stride that starts off 16-byte boundaries, within other memory; scales laid out
    row by row."""
    x, w = _x(R, K, seed=11), _x(N, K, seed=12)
    a, b = tn.quantize8(x.cuda()), tn.quantize8(w.cuda(), square=True)
    a = tn.Blocks8(a.codes, a.scales.contiguous(), powers)
    whole = torch.full((R + 2, N + 6), 3.25, dtype=dtype, device="cuda")
    y = tn.product8(a, b, out=whole[1:-1, 1:N + 1])
    c, far = ref.product_bound(ref.values(*ref.quantize(x, False)), ref.values(*ref.quantize(w, True)), dtype)
    # some of these products lie beyond fp16: 65520 is halfway between the largest number, 65504, and the next step,
    # 65536, so what is as large or larger is rounded to an infinity, and what lies within `far` of it may be either
    over = 65520.0 if dtype is torch.float16 else math.inf
    y64 = y.cpu().double()
    near, inf = (y64 - c).abs() <= far, y64 == c.sign() * math.inf
    assert torch.where(c.abs() - far >= over, inf, near | (inf & (c.abs() + far >= over))).all()
    keep = torch.ones_like(whole, dtype=torch.bool)
    keep[1:-1, 1:N + 1] = False
    assert (whole[keep] == 3.25).all()
    # the same into memory of its own, bit for bit
    assert torch.equal(tn.product8(a, b, dtype=dtype), y)


def test_empty():
    for R, C in ((0, 300), (300, 0), (0, 0)):
        for square in (False, True):
            rows, cols = tn.quantize8(torch.zeros(R, C, device="cuda"), square=square, layout="both")
            assert rows.codes.shape == (R, C) and cols.codes.shape == (C, R)
    for R, N, K in ((0, 5, 128), (5, 0, 128), (3, 200, 0), (300, 700, 0)):
        for powers in (True, False):
            w = tn.quantize8(torch.ones(N, K, device="cuda"), square=True)
            y = tn.linear8(torch.ones(R, K, device="cuda"), tn.Blocks8(w.codes, w.scales, powers))
            assert y.shape == (R, N) and (y == 0).all()
        wt = tn.quantize8(torch.ones(N, K, device="cuda"), square=True, layout="columns")
        dx, dw = tn.linear8_grad(torch.ones(R, K, device="cuda"), torch.ones(R, N, device="cuda"), wt)
        assert dx.shape == (R, K) and dw.shape == (N, K)
        assert (dx == N).all() and (dw == R).all()


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("R,N,K", [(1, 200, 512), (40, 300, 1024), (300, 700, 640)])
def test_what_is_no_number(R, N, K, powers):
    """Rows of x and blocks of w with a NaN make NaN of what is computed from them, and of nothing else."""
    x, w = _x(R, K, seed=13, wide=False), _x(N, K, seed=14, wide=False)
    x[R // 2, K - 1] = math.inf
    w[N - 1, 3] = math.nan
    q = tn.quantize8(w.cuda(), square=True)
    y = tn.linear8(x.cuda(), tn.Blocks8(q.codes, q.scales, powers)).cpu()
    nan = torch.zeros(R, N, dtype=torch.bool)
    nan[R // 2] = True
    nan[:, (N - 1) // 128 * 128:] = True
    assert torch.equal(y.isnan(), nan)


def test_scales_that_are_no_powers():
    """Said to be powers of two: reported, NaN there, right elsewhere; nothing with powers=False."""
    x, w = _x(100, 512, seed=15, wide=False), _x(260, 512, seed=16, wide=False)
    a, b = tn.quantize8(x.cuda()), tn.quantize8(w.cuda(), square=True)
    good = tn.product8(a, b, dtype=torch.float32)
    torch.cuda.synchronize()
    tn.tn_block8_check()
    for bad in (1.5, -1.0, 0.0, 2.0 ** -130, math.inf):
        scales = a.scales.clone()
        scales[7, 2] = bad
        y = tn.product8(tn.Blocks8(a.codes, scales), b, dtype=torch.float32)
        torch.cuda.synchronize()
        with pytest.raises(tn.TNError) as e:
            tn.tn_block8_check()
        assert e.value.status == tn.TN_EDEVICE
        tn.tn_block8_check()
        assert y[7].isnan().all()
        keep = torch.arange(100, device="cuda") != 7
        assert torch.equal(y[keep], good[keep])
    scales = a.scales.clone()
    scales[7, 2] *= 1.5
    y = tn.product8(tn.Blocks8(a.codes, scales, False), b, dtype=torch.float32)
    c, far = ref.product_bound(ref.values(a.codes.cpu().float(), scales.cpu()),
                               ref.values(b.codes.cpu().float(), b.scales.cpu()), torch.float32)
    assert ((y.cpu().double() - c).abs() <= far).all()
    torch.cuda.synchronize()
    tn.tn_block8_check()


def test_far_entries():
    """Matrices of more than 2^31 entries, in and out."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory")
    R, C = 66000, 33000
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    tail = _x(100, C, seed=17)
    x[-100:] = tail.cuda()
    rows, cols = tn.quantize8(x, layout="both")
    codes, scales = ref.quantize(tail, False)
    _same(tn.Blocks8(rows.codes[-100:], rows.scales[-100:]), codes, scales)
    first = R // 128 * 128 - 128        # the last columns' blocks of 128 rows
    codes, scales = ref.quantize(x[first:, -300:].cpu().t(), False)
    _same(tn.Blocks8(cols.codes[-300:, first:], cols.scales[-300:, first // 128:]), codes, scales)
    del x, rows, cols
    a, w = _x(50000, 128, seed=18, wide=False), _x(45000, 128, seed=19, wide=False)
    q = tn.quantize8(w.cuda(), square=True)
    out = tn.linear8(a.cuda(), q)
    c, far = ref.product_bound(ref.values(*ref.quantize(a[-70:], False)), q.values().double().cpu(), torch.bfloat16)
    assert ((out[-70:].cpu().double() - c).abs() <= far).all()


@pytest.mark.parametrize("R,N,K", [(1, 500, 1024), (64, 700, 512), (300, 640, 256)])
def test_streams_and_graphs(R, N, K):
    """Two captures of the calls, replayed in turn with new inputs in the same memory, and a call
    on a stream of its own."""
    x, dy, w = _x(R, K, seed=20).cuda(), _x(R, N, seed=21).cuda(), _x(N, K, seed=22).cuda()
    q, qt = tn.quantize8(w, square=True), tn.quantize8(w, square=True, layout="columns")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    first = tn.linear8(x, q, stream=s)
    graphs, outs = [], []
    with torch.cuda.stream(s):
        tn.linear8_grad(x, dy, qt)
        s.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append((tn.linear8(x, q), *tn.linear8_grad(x, dy, qt)))
            graphs.append(g)
    assert torch.equal(first, tn.linear8(x, q))
    for seed in range(3):
        x.copy_(_x(R, K, seed=30 + seed))
        dy.copy_(_x(R, N, seed=40 + seed))
        for g in graphs + graphs[::-1]:
            g.replay()
        want = (tn.linear8(x, q), *tn.linear8_grad(x, dy, qt))
        for o in outs:
            for got, y in zip(o, want):
                assert torch.equal(got, y)


def test_two_streams_at_once():
    """The calls keep nothing: products on two streams, with no order between them."""
    x = [_x(200, 1024, seed=50 + i).cuda() for i in range(2)]
    w = [tn.quantize8(_x(1000, 1024, seed=60 + i).cuda(), square=True) for i in range(2)]
    want = [tn.linear8(a, b) for a, b in zip(x, w)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(tn.linear8(x[i], w[i]))
    torch.cuda.synchronize()
    for g, y in zip(got, want):
        assert all(torch.equal(a, y) for a in g)


def test_refusals():
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    w = tn.quantize8(torch.zeros(8, 256, device="cuda"), square=True)
    wt = tn.quantize8(torch.zeros(8, 256, device="cuda"), square=True, layout="columns")
    q = tn.quantize8(x)
    bad = [lambda: tn.quantize8(x.double()), lambda: tn.quantize8(x[0]), lambda: tn.quantize8(torch._neg_view(x)),
           lambda: tn.quantize8(x, out=w), lambda: tn.quantize8(x, out=q._replace(powers=False)),
           lambda: tn.quantize8(x, out=q._replace(scales=q.scales.double())),
           lambda: tn.linear8(x[:, :128], w), lambda: tn.linear8(x, w._replace(codes=w.codes.view(torch.uint8))),
           lambda: tn.linear8(x, w._replace(scales=w.scales[:, :1])), lambda: tn.linear8(x, w, dtype=torch.float64),
           lambda: tn.linear8(x, w, out=torch.zeros(4, 9, device="cuda", dtype=torch.bfloat16)),
           lambda: tn.linear8(x, w, out=torch.zeros(8, 4, device="cuda", dtype=torch.bfloat16).t()),
           lambda: tn.linear8(x, w, out=torch.zeros(1, 8, device="cuda", dtype=torch.bfloat16).expand(4, 8)),
           lambda: tn.linear8(x, w._replace(codes=w.codes.cpu())), lambda: tn.linear8_grad(x, x[:, :8], w),
           lambda: tn.linear8_grad(x, x[:3, :8], wt), lambda: tn.product8(q, wt)]
    for call in bad:
        with pytest.raises((ValueError, tn.TNError)):
            call()
    # codes whose rows do not start at 16-byte boundaries
    with pytest.raises(tn.TNError):
        tn.product8(q._replace(codes=torch.zeros(4, 260, device="cuda").to(torch.float8_e4m3fn)[:, 4:]), w)


# ---- together --------------------------------------------------------------------

def test_a_head_is_served():
    """A batch of states through a head in 8 bits, its rows of logits to outcomes: the products against the
    definition, the draws against that of the logits the head made; captured, with new states in a second run."""
    R, K, n = 6, 512, 5000
    w = _x(n, K, torch.float32, 70, wide=False) * 0.1
    q = tn.quantize8(w.cuda(), square=True)
    op = tn.Sampler(n, torch.bfloat16, max_rows=R)
    op.bind_workspace()
    x, u = _x(R, K, seed=71, wide=False).cuda(), torch.rand(R, generator=torch.Generator().manual_seed(3)).cuda()
    kw = dict(temperature=0.8, top_k=50, top_p=0.95)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        op.sample(tn.linear8(x, q), u, **kw)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            logits = tn.linear8(x, q)
            got = op.sample(logits, u, **kw)
    for seed in (71, 72):
        x.copy_(_x(R, K, seed=seed, wide=False))
        g.replay()
        torch.cuda.synchronize()
        c, far = ref.product_bound(ref.values(*ref.quantize(x.cpu(), False)), ref.values(*ref.quantize(w, True)),
                                   torch.bfloat16)
        assert ((logits.cpu().double() - c).abs() <= far).all()
        _compare(got, logits, u, **kw)
    op.check()


def test_a_head_is_trained():
    """The distillation loss of a head's logits and its gradients at states and weights: the loss and its gradient at
    the logits against the 64-bit ones, the two products against the definition, and the whole against
    differences of the loss.

    Differences: the loss of the matrices that the codes stand for is smooth in dx and dW's place, and
    dx, dW are products of quantised dy with exact operands (x and W are such that their codes are exact).  A code is off
    by 2^-4 of the entry, or by half the smallest step, 2^-10 s, where s <= max / 224.  Along a direction that moves the
    logits by dz, the sum of |dy| |dz| 2^-4 and that of 2^-10 / 224 max |dy| |dz| bound what it makes of it; dy and dx
    in bf16 add 2^-8 of the first each.  The differences' own error is of the order (h dz)^2, below 2^-7."""
    R, K, n, k = 8, 256, 640, 16
    g = torch.Generator().manual_seed(80)
    # small whole numbers: exact in e4m3 with whatever power of two
    x = torch.randint(-7, 8, (R, K), generator=g).to(torch.bfloat16)
    w = torch.randint(-7, 8, (n, K), generator=g).float() * 2.0 ** -7
    ids = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(R)])
    teacher = torch.randn(R, k, generator=g)
    each = torch.rand(R, generator=g)
    q, qt = tn.quantize8(w.cuda(), square=True), tn.quantize8(w.cuda(), square=True, layout="columns")
    assert torch.equal(q.values().cpu(), w) and torch.equal(qt.values().cpu(), w.t())
    logits = tn.linear8(x.cuda(), q, dtype=torch.float32)
    z = x.double() @ w.double().t()
    assert torch.equal(logits.cpu().double(), z)        # whole numbers of 2^-7 below 2^24: exact
    op = tn.Outcomes(n, torch.float32, max_rows=R)
    step = op.distill_step(logits, ids.cuda(), teacher.cuda(), each.cuda())
    loss = lambda m: [Row(m[r].numpy().astype("float32"), None, 1.0).distill(ids[r].numpy(), teacher[r].double().numpy())
                      for r in range(R)]
    want = loss(z)
    assert all(abs(a - b) <= 1e-5 * max(1, abs(b)) for a, b in zip(step.loss.tolist(), want))
    dy = step.grad.to(torch.bfloat16)
    dx, dw = tn.linear8_grad(x.cuda(), dy, qt)
    v = [ref.values(*ref.quantize(m, s)) for m, s in ((dy.cpu(), False), (w.t(), True), (dy.cpu().t(), False), (x.t(), False))]
    for got, (c, far) in ((dx, ref.product_bound(v[0], v[1], torch.bfloat16)),
                          (dw, ref.product_bound(v[2], v[3], torch.float32))):
        assert ((got.cpu().double() - c).abs() <= far).all()
    exact = step.grad.double().cpu()
    h = 1e-3
    for over_x in (True, False):
        d = torch.randn((R, K) if over_x else (n, K), generator=g).double()
        dz = d @ w.double().t() if over_x else x.double() @ d.t()
        up, down = loss(z + h * dz), loss(z - h * dz)
        slope = sum(each[r].item() * (up[r] - down[r]) for r in range(R)) / (2 * h)
        got = ((dx if over_x else dw).double().cpu() * d).sum().item()
        size = (exact.abs() * dz.abs()).sum().item()
        far = (2.0 ** -4 + 3 * 2.0 ** -7) * size + 2.0 ** -10 / 224 * exact.abs().max().item() * dz.abs().sum().item()
        assert abs(got - slope) <= far, (over_x, got, slope, far)
