"""The sampler as programs call it: layouts and masks, invalid numbers, rows without a
distribution, many rows, streams and graphs; against the definitions."""
import math

import numpy as np
import pytest
import torch

import exact_tensor_network_gb300 as tn

from test_gpu_sampling import TYPES, _compare, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _u(R, D, seed=0, dtype=torch.float32):
    return torch.rand(R, D, generator=torch.Generator().manual_seed(seed), dtype=dtype)


SIZES = [40, 300, 900, 1500, 3500, 9001, 40003]


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("layout", ["offset", "columns", "steps", "one"])
@pytest.mark.parametrize("filters", [{}, {"top_k": 30, "top_p": 0.9}], ids=str)
def test_layouts_and_masks(type_, n, layout, filters):
    R = 3
    whole = _rows(type_, R, 2 * n + 3, 2).cuda()
    rows = {"offset": whole[:, 1:n + 1], "columns": whole[:, :n].t().contiguous().t(), "steps": whole[:, :2 * n:2],
            "one": whole[:1, :n].expand(R, n)}[layout]
    m = torch.rand(R, 2 * n, generator=torch.Generator().manual_seed(n)).cuda() < 0.6
    mask = {"offset": m[:, 3:n + 3], "columns": m[:, :n].t().contiguous().t(), "steps": m[0, :2 * n:2].to(torch.uint8) * 3,
            "one": m[:, :1]}[layout]
    u = _u(R, 2)
    op = tn.Sampler(n, TYPES[type_], max_rows=R)
    got = op.sample(rows, u.cuda(), mask=mask, **filters)
    op.check()
    _compare(got, rows, u, mask=mask.bool(), **filters)


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("filters", [{}, {"top_p": 0.9}, {"top_k": 7}, {"min_p": 0.01}], ids=str)
def test_rows_without_a_distribution(n, filters):
    """Masked to nothing, only -inf, a NaN or +inf that counts and one that does not, one entry, and a mask
    written as the type's lowest value."""
    x = _rows("bf16", 8, n, 4)
    mask = torch.ones(8, n, dtype=torch.bool)
    mask[0] = False
    x[1] = -math.inf
    x[2, n // 2] = math.nan
    x[3, n - 1] = math.inf
    x[4, 3], mask[4, 3] = math.nan, False
    x[5, :n - 1] = -math.inf
    x[6, ::2] = torch.finfo(torch.bfloat16).min
    x[7, 1:] = torch.finfo(torch.bfloat16).min
    u = _u(8, 1)
    op = tn.Sampler(n, torch.bfloat16, max_rows=8)
    got = op.sample(x.cuda(), u.cuda(), mask=mask.cuda(), **filters)
    op.check()
    _compare(got, x, u, mask=mask, **filters)
    assert got.kept[:4].tolist() == [0] * 4 and got.kept[5].item() == 1


@pytest.mark.parametrize("n", SIZES)
def test_invalid_numbers(n):
    """Reported, and the other rows and draws are right."""
    R = 10
    x = _rows("f32", R, n, 5)
    u = _u(R, 3, dtype=torch.float64)
    t, p, m = torch.ones(R), torch.full((R,), 0.8), torch.zeros(R)
    t[0], t[1], t[2] = -1.0, math.nan, math.inf
    p[3] = math.nan
    m[4], m[5] = 1.5, math.nan
    good = u.clone()
    u[6, 1], u[7, 0], u[8, 2] = 1.0, -1e-300, math.nan
    op = tn.Sampler(n, torch.float32, max_rows=R)
    got = op.sample(x.cuda(), u.cuda(), t.cuda(), None, p.cuda(), m.cuda())
    torch.cuda.synchronize()
    with pytest.raises(tn.TNError) as e:
        op.check()
    assert e.value.status == tn.TN_EDEVICE
    op.check()                          # reported once
    assert (got.ids[:6] == -1).all() and got.logp[:6].isnan().all() and (got.kept[:6] == 0).all()
    for r, d in ((6, 1), (7, 0), (8, 2)):
        assert got.ids[r, d] == -1 and got.logp[r, d].isnan()
        one = op.sample(x[r:r + 1].cuda(), good[r:r + 1].cuda(), None, None, 0.8)
        got.ids[r, d], got.logp[r, d] = one.ids[0, d], one.logp[0, d]
    _compare(tn.Samples(got.ids[6:], got.logp[6:], got.kept[6:]), x[6:], good[6:], top_p=0.8)
    op.check()


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("n", [50, 2000, 30000])
@pytest.mark.parametrize("scale,filters", [(1.0, {"temperature": 1e-30}), (1.0, {"temperature": 1e30, "top_k": 9}),
                                           (2.0, {"temperature": 0.5, "top_p": 0.6}), (0.5, {"min_p": 0.2}),
                                           (2.0 ** -40, {"top_p": 0.3}), (2.0 ** 40, {"top_p": 0.99}),
                                           (1.0, {"temperature": -0.0}), (1.0, {"top_k": 2 ** 40, "top_p": 0.75})], ids=str)
def test_extreme_parameters(type_, n, scale, filters):
    rows, u = _rows(type_, 2, n, 6), _u(2, 2)
    op = tn.Sampler(n, TYPES[type_], max_rows=2, scale=scale)
    got = op.sample(rows.cuda(), u.cuda(), **filters)
    op.check()
    _compare(got, rows, u, scale=scale, **filters)


def _many(got, rows, u, top_k=0, top_p=1.0):
    """All rows at once in 64 bits (sums to 2^-50, so that an outcome is off only where u or top_p
    lies that near to a border)."""
    x = rows.double().cpu().numpy()
    w = np.exp(x - x.max(1, keepdims=True))
    at = np.argsort(-x, axis=1, kind="stable")
    s = np.take_along_axis(w, at, 1)
    if top_k:
        s[:, top_k:] = 0
    c = np.cumsum(s, 1)
    kept = np.minimum((c < np.float64(np.float32(top_p)) * c[:, -1:]).sum(1) + 1, top_k or x.shape[1]) if top_p < 1 \
        else np.full(len(x), min(top_k or x.shape[1], x.shape[1]))
    s[np.arange(x.shape[1])[None] >= kept[:, None]] = 0
    left = np.zeros_like(w)
    np.put_along_axis(left, at, s, 1)
    c = np.cumsum(left, 1)
    ids = np.stack([np.searchsorted(c[r], u[r] * c[r, -1], side="right") for r in range(len(x))])
    assert (got.kept.cpu().numpy() == kept).all() and (got.ids.cpu().numpy() == ids).all()
    logp = np.log(np.take_along_axis(left, ids, 1) / c[:, -1:])
    assert (np.abs(got.logp.cpu().numpy() - logp) <= 2.0 ** -24 * np.abs(logp) + 1e-12).all()


@pytest.mark.parametrize("type_,R,n", [("f32", 20000, 100), ("bf16", 5000, 700), ("f16", 3000, 1200), ("f32", 2500, 2000),
                                       ("bf16", 2501, 2048), ("bf16", 1300, 4095), ("bf16", 700, 6001), ("f16", 400, 9000),
                                       ("f32", 310, 20001)])
@pytest.mark.parametrize("filters", [{}, {"top_k": 40}, {"top_p": 0.85}, {"top_k": 100, "top_p": 0.7}], ids=str)
def test_many_rows(type_, R, n, filters):
    rows, u = _rows(type_, R, n, 7), _u(R, 1, n, torch.float64)
    op = tn.Sampler(n, TYPES[type_], max_rows=R)
    _many(op.sample(rows.cuda(), u.cuda(), **filters), rows, u.numpy(), **filters)


@pytest.mark.parametrize("n", [40, 900, 3500, 40003])
@pytest.mark.parametrize("D", [0, 1, 8, 16, 17, 33, 100])
def test_numbers_of_draws(n, D):
    rows, u = _rows("f32", 2, n, 8), _u(2, D, 1, torch.float64)
    op = tn.Sampler(n, torch.float32, max_rows=2)
    got = op.sample(rows.cuda(), u.cuda(), top_p=0.9)
    assert got.ids.shape == (2, D)
    if D:
        _many(got, rows, u.numpy(), top_p=0.9)
    else:
        assert got.kept.tolist() == op.sample(rows.cuda(), _u(2, 1).cuda(), top_p=0.9).kept.tolist()
    # fewer rows than the handle is for, and none
    one = op.sample(rows[1].cuda(), u[1:].cuda(), top_p=0.9)
    assert torch.equal(one.ids[0], got.ids[1]) and torch.equal(one.logp[0], got.logp[1])
    assert op.sample(rows[:0].cuda(), u[:0].cuda(), top_p=0.9).ids.shape == (0, D)
    op.check()


def test_far_entries():
    """Rows that lie more than 2^31 entries apart, and indices beyond 2^30."""
    n = 1_200_000_000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    rows = torch.zeros(3, n, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor([[0.0, 0.75], [0.25, 0.5], [0.125, 0.99900000041]], dtype=torch.float64, device="cuda")
    op = tn.Sampler(n, torch.bfloat16, max_rows=3)
    got = op.sample(rows, u)
    # all weights equal: u n is a whole number, or lies far from one
    want = torch.floor(u.cpu() * n).long()
    assert torch.equal(got.ids.cpu(), want) and (got.kept == n).all()
    assert (got.logp + math.log(n)).abs().max() <= 2.0 ** -24 * math.log(n) + 1e-12
    at = torch.arange(10, device="cuda") * 119_999_999 + 5
    rows[2, at] = 1.0
    got = op.sample(rows[2], u[2:], top_k=7)
    assert got.kept.item() == 7 and got.ids.tolist() == [[at[int(0.125 * 7)].item(), at[6].item()]]
    op.check()


@pytest.mark.parametrize("n", [64, 2048, 32768])
def test_streams_and_graphs(n):
    """A handle's call captured twice, into graphs that share its workspace and are replayed in turn with
    new numbers in the same memory; and calls on a stream of their own."""
    R = 5
    rows, u = _rows("bf16", R, n, 9).cuda(), _u(R, 2).cuda()
    op = tn.Sampler(n, torch.bfloat16, max_rows=R)
    op.bind_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    first = op.sample(rows, u, top_k=50, top_p=0.9, stream=s)
    outs, graphs = [], []
    with torch.cuda.stream(s):
        outs = [op.sample(rows, u, top_k=50, top_p=0.9), op.sample(rows, u, 0.7)]
        s.synchronize()
        for i, kw in enumerate(({"top_k": 50, "top_p": 0.9}, {"temperature": 0.7})):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                op.sample(rows, u, out=outs[i], **kw)
            graphs.append(g)
    _compare(first, rows, u, top_k=50, top_p=0.9)
    for seed in range(3):
        rows.copy_(_rows("bf16", R, n, 10 + seed))
        u.copy_(_u(R, 2, 20 + seed))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        _compare(outs[0], rows, u, top_k=50, top_p=0.9)
        _compare(outs[1], rows, u, temperature=0.7)
    again = op.sample(rows, u, 0.7)
    assert torch.equal(again.ids, outs[1].ids) and torch.equal(again.logp, outs[1].logp)
    op.check()


def test_refusals():
    x, u = torch.zeros(4, 100, device="cuda"), torch.zeros(4, 2, device="cuda")
    op = tn.Sampler(100, torch.float32, max_rows=4)
    out = op.sample(x, u)
    bad = [dict(rows=x[:, :99]), dict(rows=x.half()), dict(rows=x.cpu()), dict(rows=torch._neg_view(x)), dict(u=u.cpu()),
           dict(u=u.half()), dict(u=u[:3]), dict(u=torch.zeros(4, 4, device="cuda")[:, ::2]), dict(u=u[None]),
           dict(mask=x), dict(mask=torch.ones(4, 100, dtype=torch.bool)), dict(temperature=torch.ones(4)),
           dict(temperature=torch.ones(3, device="cuda")), dict(top_k=torch.ones(4, device="cuda")),
           dict(top_p=torch.ones(8, device="cuda")[::2]), dict(min_p=torch.ones(4, device="cuda").double()),
           dict(out=out._replace(ids=out.ids.int())), dict(out=out._replace(kept=out.kept[:3])),
           dict(out=out._replace(logp=out.logp.t()))]
    for kw in bad:
        with pytest.raises(ValueError):
            op.sample(**{"rows": x, "u": u, **kw})
    with pytest.raises(tn.TNError):
        op.sample(torch.zeros(5, 100, device="cuda"), torch.zeros(5, device="cuda"))       # more rows than it is for
    with pytest.raises(tn.TNError):
        op.sample(torch.zeros(4, 1, device="cuda").expand(4, 100), u)                       # one entry for all columns
    op.check()


@pytest.mark.parametrize("type_,n", [("bf16", 2000003), ("f16", 1 << 21), ("f32", 5000011)])
@pytest.mark.parametrize("filters", [{"top_p": 0.9}, {"top_p": 0.4}, {"top_k": 5000, "top_p": 0.5}, {"top_k": 3000}], ids=str)
def test_very_long_rows(type_, n, filters):
    """16-bit logits of rows this long have thousands of equal entries wherever a filter cuts."""
    rows, u = _rows(type_, 2, n, 12), _u(2, 3, 4, torch.float64)
    op = tn.Sampler(n, TYPES[type_], max_rows=2)
    _many(op.sample(rows.cuda(), u.cuda(), **filters), rows, u.numpy(), **filters)
    op.check()


@pytest.mark.parametrize("n", [9001, 60000, 400001])
@pytest.mark.parametrize("filters", [{"top_p": 0.1}, {"top_p": 0.7}, {"top_p": 0.95}, {"top_k": 7}, {"top_k": 4000},
                                     {"top_k": 5000, "top_p": 0.6}, {"top_k": 8000, "top_p": 0.9}], ids=str)
@pytest.mark.parametrize("draws", [2, 20])
def test_few_different_values(n, filters, draws):
    """Rows of four values, among whose equal entries every filter cuts."""
    g = torch.Generator().manual_seed(n)
    rows = torch.tensor([-1.0, 0.25, 1.5, 3.0])[torch.multinomial(torch.tensor([0.5, 0.3, 0.15, 0.05]), 3 * n, True,
                                                                  generator=g)].view(3, n)
    rows[2, : n // 3] = -math.inf
    u = _u(3, draws, 7, torch.float64)
    for dtype in (torch.float32, torch.bfloat16):
        op = tn.Sampler(n, dtype, max_rows=3)
        got = op.sample(rows.to(dtype).cuda(), u.cuda(), **filters)
        _many(got, rows, u.numpy(), **filters)
        # min_p that cuts above what is equal
        got = op.sample(rows.to(dtype).cuda(), u.cuda(), min_p=0.5, **filters)
        most = (rows == 3.0).sum(1)
        assert (got.kept.cpu() <= most).all() and (got.kept > 0).all()
        for r in range(3):
            assert (rows[r, got.ids[r].cpu()] == 3.0).all()
        op.check()
