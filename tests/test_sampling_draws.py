"""The number of draws that a sampler is made for: the most a call may ask of a row."""
import math

import pytest
import torch

import exact_tensor_network_gb300 as tn
from exact_tensor_network_gb300 import build as tnbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    tnbuild.build()


def test_made_with_a_number_of_draws():
    op = tn.Sampler(50, torch.float32, max_rows=3, draws=7, scale=0.5)
    assert (op.cols, op.max_rows, op.draws, op.scale) == (50, 3, 7, 0.5)
    assert tn.Sampler(50).draws is None and tn.Sampler(50, draws=0).draws == 0
    # the workspace is the same whatever the number
    assert op.workspace_bytes == tn.Sampler(50, torch.float32, 3, 0.5).workspace_bytes


@pytest.mark.parametrize("draws", [-1, 1.5, math.nan])
def test_numbers_that_are_refused(draws):
    with pytest.raises(ValueError):
        tn.Sampler(50, torch.float32, draws=draws)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [50, 40003])
def test_calls_are_held_to_it(n):
    rows = torch.randn(2, n, generator=torch.Generator().manual_seed(n)).cuda()
    u = torch.rand(2, 20, generator=torch.Generator().manual_seed(1)).cuda()
    want = tn.Sampler(n, torch.float32, max_rows=2).sample(rows, u, top_p=0.9)
    op = tn.Sampler(n, torch.float32, max_rows=2, draws=20)
    for D in (20, 3, 0):
        got = op.sample(rows, u[:, :D].contiguous(), top_p=0.9)
        assert torch.equal(got.ids, want.ids[:, :D]) and torch.equal(got.logp, want.logp[:, :D])
        assert torch.equal(got.kept, want.kept)
    assert torch.equal(op.sample(rows, u[:, 0].contiguous(), top_p=0.9).ids, want.ids[:, 0])
    with pytest.raises(ValueError):
        op.sample(rows, torch.zeros(2, 21, device="cuda"))
    one = tn.Sampler(n, torch.float32, max_rows=2, draws=1)
    with pytest.raises(ValueError):
        one.sample(rows, u[:, :2].contiguous())
    none = tn.Sampler(n, torch.float32, max_rows=2, draws=0)
    with pytest.raises(ValueError):
        none.sample(rows, u[:, 0].contiguous())
    op.check()
