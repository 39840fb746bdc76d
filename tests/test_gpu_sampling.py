"""Draws against the definitions with exact sums."""
import itertools
import math

import numpy as np
import pytest
import torch

import exact_tensor_network_gb300 as tn

import sampling_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"c64": torch.complex64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _rows(type_, R, n, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed * 77 + n)
    if type_ == "c64":
        return torch.view_as_complex(torch.randn(R, n, 2, generator=g) * 0.1)
    return (torch.randn(R, n, generator=g) * spread).to(TYPES[type_])


def _numpy(rows):
    return rows.cpu().numpy() if rows.is_complex() else rows.float().cpu().numpy()


def _compare(got, rows, u, scale=1.0, mask=None, **filters):
    x, u = _numpy(rows), u.cpu().numpy()
    if u.ndim == 1:
        u = u[:, None]
    ids, logp, kept = got.ids.cpu().numpy().reshape(u.shape), got.logp.cpu().numpy().reshape(u.shape), got.kept.cpu().numpy()
    if mask is not None:
        mask = mask.expand(x.shape).cpu().numpy()
    for r in range(x.shape[0]):
        own = {k: (v[r].item() if torch.is_tensor(v) else v) for k, v in filters.items()}
        entries = ref.left(x[r], None if mask is None else mask[r], scale, **own)
        assert kept[r] == (0 if isinstance(entries, str) else len(entries)), r
        for d in range(u.shape[1]):
            e, lp = ref.draw(entries, u[r, d])
            assert ids[r, d] == e, (r, d)
            if math.isnan(lp):
                assert math.isnan(logp[r, d])
            elif math.isinf(lp):
                assert logp[r, d] == lp
            else:       # one rounding to fp32 of a number computed in 64 bits
                assert abs(logp[r, d] - lp) <= 2.0 ** -24 * abs(lp) + 1e-12, (r, d)


FILTERS = [{}, {"temperature": 0.7}, {"temperature": 0.0}, {"top_k": 1}, {"top_k": 5}, {"top_k": 50, "temperature": 1.3},
           {"top_p": 0.9}, {"top_p": 0.3, "temperature": 0.5}, {"min_p": 0.1}, {"top_k": 20, "top_p": 0.8},
           {"top_k": 40, "top_p": 0.95, "min_p": 0.05, "temperature": 0.8}, {"top_p": 0.0}, {"min_p": 1.0},
           {"top_k": 10 ** 6, "top_p": 1.0}, {"top_p": 0.999}]


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("n", [1, 2, 7, 64, 100, 1000, 4099])
@pytest.mark.parametrize("filters", FILTERS, ids=str)
def test_sample(type_, n, filters):
    R = 4
    rows = _rows(type_, R, n)
    u = torch.rand(R, 5, generator=torch.Generator().manual_seed(n), dtype=torch.float64)
    u[0, 0] = 0.0
    op = tn.Sampler(n, TYPES[type_], max_rows=R)
    got = op.sample(rows.cuda(), u.cuda(), **filters)
    torch.cuda.synchronize()
    op.check()
    _compare(got, rows, u, **filters)


LONG = [{}, {"temperature": 0.8, "top_k": 40, "top_p": 0.95}, {"top_p": 0.9}, {"top_k": 300}, {"top_p": 0.5, "min_p": 1e-3},
        {"temperature": 0.0}, {"top_k": 6000, "top_p": 0.9}, {"top_k": 5000}, {"top_k": 9000, "top_p": 0.5, "temperature": 0.6},
        {"top_k": 20000, "top_p": 0.997}, {"top_k": 3000, "top_p": 0.1, "min_p": 0.01}]


@pytest.mark.parametrize("filters", LONG, ids=str)
@pytest.mark.parametrize("type_,n", [("bf16", 32768), ("f16", 50001), ("f32", 70003), ("c64", 40000), ("bf16", 300007),
                                     ("f32", 1 << 18), ("c64", 270001)])
def test_long_rows(type_, n, filters):
    R = 3
    rows = _rows(type_, R, n, 1)
    u = torch.rand(R, 2, generator=torch.Generator().manual_seed(n))
    op = tn.Sampler(n, TYPES[type_], max_rows=R)
    got = op.sample(rows.cuda(), u.cuda(), **filters)
    _compare(got, rows, u, **filters)


def test_every_row_its_own():
    R, n = 64, 20011
    rows = _rows("bf16", R, n, 3)
    g = torch.Generator().manual_seed(5)
    t = torch.rand(R, generator=g) + 0.5
    t[::7] = 0.0
    k = torch.randint(-1, 100, (R,), generator=g, dtype=torch.int32)
    p = torch.rand(R, generator=g) * 1.2
    m = torch.rand(R, generator=g) * 0.1 - 0.02
    mask = torch.rand(R, n, generator=g) < 0.5
    mask[11] = False
    rows[:, ::3][~mask[:, ::3]] = float("nan")
    rows[13, 5], mask[13, 5] = float("nan"), True
    u = torch.rand(R, generator=g)
    op = tn.Sampler(n, torch.bfloat16, max_rows=R)
    got = op.sample(rows.cuda(), u.cuda(), t.cuda(), k.cuda(), p.cuda(), m.cuda(), mask=mask.cuda())
    assert got.ids.shape == (R,)
    _compare(got, rows, u, mask=mask, temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("type_", ["f32", "c64"])
@pytest.mark.parametrize("n", [1000, 1 << 15, 1 << 18])
@pytest.mark.parametrize("filters", [{}, {"top_p": 0.5}, {"top_k": 777}, {"top_k": 900, "top_p": 0.25}, {"min_p": 0.5}], ids=str)
def test_equal_entries(type_, n, filters):
    """Uniform states: every cut goes through equal entries, by index, and u on a border belongs to
    the entry behind it."""
    rows = torch.full((2, n), 0.25, dtype=TYPES[type_])
    rows[1, n // 2:] *= 0.5
    u = torch.tensor([[0.0, 0.25, 0.5, 1 - 2.0 ** -24]] * 2)
    op = tn.Sampler(n, TYPES[type_], max_rows=2)
    got = op.sample(rows.cuda(), u.cuda(), **filters)
    _compare(got, rows, u, **filters)


def test_many_draws():
    n, D = 100003, 1000
    rows = _rows("c64", 2, n, 9)
    u = torch.rand(2, D, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    op = tn.Sampler(n, torch.complex64, max_rows=2)
    got = op.sample(rows.cuda(), u.cuda(), top_p=0.7)
    w = _numpy(rows)
    w = (w.real * w.real + w.imag * w.imag).astype(np.float64)
    for r in range(2):
        at = np.argsort(-w[r], kind="stable")
        kept = int(np.searchsorted(np.cumsum(w[r][at]), np.float64(np.float32(0.7)) * w[r].sum())) + 1
        left = np.zeros(n)
        left[at[:kept]] = w[r][at[:kept]]
        c = np.cumsum(left)
        assert got.kept[r].item() == kept
        assert (got.ids[r].cpu().numpy() == np.searchsorted(c, u[r].numpy() * c[-1], side="right")).all()
