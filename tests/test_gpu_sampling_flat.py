"""Draws from rows whose weights lie close together: high temperatures, logits of little spread,
amplitudes near the type's smallest numbers; against the definitions."""
import math

import pytest
import torch

import exact_tensor_network_gb300 as tn

from test_gpu_sampling import _compare, _rows
from test_gpu_sampling_use import _u

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
