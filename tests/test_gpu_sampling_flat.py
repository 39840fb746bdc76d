"""Draws from rows whose weights lie close together: high temperatures, logits of little spread,
amplitudes near the type's smallest numbers; against the definitions."""
import math

import numpy as np
import pytest
import torch

import exact_tensor_network_gb300 as tn

from test_gpu_sampling import TYPES, _compare, _rows
from test_gpu_sampling_use import _many, _u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _holes(type_, n, seed):
    """Rows off 16-byte boundaries, with absent entries of every kind, and their mask."""
    rows = _rows(type_, 3, n + 4, seed).cuda()
    rows[:, 5::7] = 0 if type_ == "c64" else -math.inf
    mask = torch.rand(3, n, generator=torch.Generator().manual_seed(n)).cuda() < 0.6
    return rows[:, 1:n + 1], mask


@pytest.mark.parametrize("n", [50, 300, 2000, 9001, 40003])
@pytest.mark.parametrize("filters", [{"temperature": 300.0, "min_p": 0.05}, {"temperature": 1e30, "min_p": 0.05},
                                     {"temperature": 1e30, "min_p": 0.05, "top_p": 0.9},
                                     {"temperature": 1e30, "min_p": 0.05, "top_k": 5000},
                                     {"temperature": 11.0, "min_p": 1e-30}, {"temperature": 120.0, "min_p": 1e-3},
                                     {"temperature": 300.0, "min_p": 0.05, "top_p": 0.9}], ids=str)
def test_min_p_below_every_amplitude(n, filters):
    """What is absent is not left where min_p cuts below the smallest number."""
    rows, mask = _holes("c64", n, 30)
    u = _u(3, 5, n, torch.float64)
    u[0, 0], u[1, 0] = 0.0, 1 - 2.0 ** -53
    op = tn.Sampler(n, torch.complex64, max_rows=3)
    got = op.sample(rows, u.cuda(), mask=mask, **filters)
    op.check()
    _compare(got, rows, u, mask=mask, **filters)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("n", [50, 2000, 9001, 40003, 300007])
@pytest.mark.parametrize("filters", [{}, {"min_p": 0.05}, {"min_p": 1.0}, {"top_k": 9}, {"top_p": 0.5, "min_p": 1.0},
                                     {"top_k": 5000, "top_p": 0.5}], ids=str)
def test_temperature_that_leaves_no_difference(type_, n, filters):
    """scale / temperature is 0 in fp32: all present entries weigh the same."""
    rows, mask = _holes(type_, n, 31)
    u = _u(3, 5, n, torch.float64)
    op = tn.Sampler(n, TYPES[type_], max_rows=3, scale=2.0 ** -40)
    got = op.sample(rows, u.cuda(), mask=mask, temperature=1e38, **filters)
    op.check()
    _compare(got, rows, u, scale=2.0 ** -40, mask=mask, temperature=1e38, **filters)


@pytest.mark.parametrize("n", [50, 2000, 9001, 40003, 300007])
def test_logits_further_apart_than_numbers_reach(n):
    """A difference beyond fp32 counts as the largest number, which at such a temperature is next to nothing."""
    rows = torch.full((2, n), -3e38)
    rows[:, n // 3] = 3e38
    u = _u(2, 50, n, torch.float64)
    op = tn.Sampler(n, torch.float32, max_rows=2)
    got = op.sample(rows.cuda(), u.cuda(), temperature=3e38)
    beta = float(np.float32(1) / np.float32(3e38))
    w = np.full(n, math.exp(-beta * float(np.finfo(np.float32).max)))
    w[n // 3] = 1.0
    c = np.cumsum(w)
    want = np.searchsorted(c, u.numpy() * c[-1], side="right")
    assert (got.ids.cpu().numpy() == want).all() and (got.kept == n).all()
    logp = np.log(w[want] / c[-1])
    assert (np.abs(got.logp.cpu().numpy() - logp) <= 2.0 ** -24 * np.abs(logp) + 1e-12).all()
    # (they weigh e^-1.134 of the largest; order values would say e^-2)
    assert (op.sample(rows.cuda(), u.cuda(), temperature=3e38, min_p=0.2).kept == n).all()
    assert (op.sample(rows.cuda(), u.cuda(), temperature=3e38, min_p=0.33).kept == 1).all()
    op.check()


@pytest.mark.parametrize("n", [50, 2000, 9001, 40003, 300007])
@pytest.mark.parametrize("largest", [0.0, 1.0])
@pytest.mark.parametrize("filters", [{"temperature": 0.5}, {"temperature": 1.5}, {"temperature": 100.0},
                                     {"temperature": 100.0, "min_p": 0.3}, {"temperature": 1.5, "top_p": 0.8},
                                     {"temperature": 100.0, "top_k": 3000, "top_p": 0.5}], ids=str)
def test_amplitudes_of_subnormal_probability(n, largest, filters):
    """|a|^2 below 2^-126, in all of a row or next to an amplitude of 1 (which at a high temperature is not
    much more)."""
    rows = _rows("c64", 2, n, 32) * 1e-19
    if largest:
        rows[:, n // 2] = largest
    u = _u(2, 5, n, torch.float64)
    op = tn.Sampler(n, torch.complex64, max_rows=2)
    got = op.sample(rows.cuda(), u.cuda(), **filters)
    op.check()
    _compare(got, rows, u, **filters)


@pytest.mark.parametrize("n", [60, 900, 9001, 40003])
@pytest.mark.parametrize("temperature", [1e-2, 1e-5, 1e-6, 2e-7, 1e-7])
def test_amplitudes_next_to_each_other_at_a_low_temperature(n, temperature):
    """Nearly uniform states whose small differences a low temperature makes large: |a|^2 within 8 temperatures of
    the largest, at many sizes of it."""
    R, g = 4000 if n < 1000 else 200, torch.Generator().manual_seed(n)
    size = torch.exp2(torch.linspace(-120, -66, R, dtype=torch.float64))[:, None]
    w = size * (1 - min(8 * temperature, 0.5) * torch.rand(R, n, generator=g, dtype=torch.float64))
    rows = torch.complex(w.sqrt().float(), torch.zeros(R, n))
    u = _u(R, 4, n, torch.float64)
    op = tn.Sampler(n, torch.complex64, max_rows=R)
    got = op.sample(rows.cuda(), u.cuda(), temperature=temperature)
    v = (rows.real * rows.real).double().numpy()
    beta = float(np.float32(1) / np.float32(temperature))
    top = v.max(1, keepdims=True)
    x = beta * np.log1p((v - top) / top)
    c = np.cumsum(np.exp(x), 1)
    ids = np.stack([np.searchsorted(c[r], u[r].numpy() * c[r, -1], side="right") for r in range(R)])
    assert (got.ids.cpu().numpy() == ids).all() and (got.kept == n).all()
    logp = np.take_along_axis(x, ids, 1) - np.log(c[:, -1:])
    # beta times the rounding of a 64-bit logarithm of up to 63, on either side
    far = 2.0 ** -24 * np.abs(logp) + 1e-12 + beta * 64 * 2.0 ** -52
    assert (np.abs(got.logp.cpu().numpy() - logp) <= far).all()
    op.check()


@pytest.mark.parametrize("n", [900, 9001, 40003, 300007])
@pytest.mark.parametrize("each", [1.4e19, 1e-12])
def test_amplitudes_whose_sum_is_beyond_numbers(n, each):
    """Two amplitudes whose |a|^2 add up to more than fp32 holds, and n - 2 others of 2^-30 of that: a draw that aims
    into the middle of one of those finds it.  And the same far below."""
    rows = torch.full((2, n), each * 2.0 ** -15, dtype=torch.complex64)
    rows[:, :2] = each
    v = (rows.real * rows.real).double()
    at = torch.randint(2, n, (2, 40), generator=torch.Generator().manual_seed(n))
    c = v.cumsum(1)
    u = (c.gather(1, at) - 0.5 * v.gather(1, at)) / c[:, -1:]
    got = tn.Sampler(n, torch.complex64, max_rows=2).sample(rows.cuda(), u.cuda())
    assert torch.equal(got.ids.cpu(), at) and (got.kept == n).all()
    assert (got.logp.cpu() - (v.gather(1, at) / c[:, -1:]).log()).abs().max() <= 2.0 ** -24 * 32 + 1e-12


@pytest.mark.parametrize("type_,n", [("f32", 40003), ("bf16", 40003), ("f16", 131072), ("f32", 131072), ("f32", 300007),
                                     ("bf16", 1 << 20)])
@pytest.mark.parametrize("spread", [1e-4, 0.01, 0.1])
@pytest.mark.parametrize("filters", [{"top_p": 0.9}, {"top_k": 1000}, {"top_k": 5000, "top_p": 0.6}], ids=str)
def test_logits_of_little_spread(type_, n, spread, filters):
    """A head at its start: more entries in the bin where a filter cuts than are sorted."""
    rows, u = _rows(type_, 3, n, 33, spread), _u(3, 12, n, torch.float64)
    op = tn.Sampler(n, TYPES[type_], max_rows=3)
    _many(op.sample(rows.cuda(), u.cuda(), **filters), rows, u.numpy(), **filters)
    op.check()
