"""The example that runs contraction, scores and distillation together."""
import os
import sys

import numpy as np
import pytest

import oracle
from outcome_reference import Row
from workloads import greedy_tree, grid_circuit_network

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def test_leaf_gradients_against_differences():
    """The loss's derivative along random directions of every free leaf, from
    the kernels' gradient and from central differences of the loss in 64 bits.

    Bound: amplitudes are good to 1e-5 of their largest, so the loss's
    gradient at them is good to about 1e-5 times their spread (a few hundred
    between the largest and the smallest outcome of the teacher), and 1e-2
    leaves room for cancellation along one direction."""
    import torch
    import distill_circuit as ex
    import exact_tensor_network_gb300 as tn
    net, _ = grid_circuit_network(2, 3, 3, 5, n_open=5)
    rng = np.random.default_rng(0)
    ids = rng.permutation(32)[:6][None, :]
    logits = rng.standard_normal((1, 6)).astype(np.float32)
    student = ex.Student(net, 0)
    op = tn.Outcomes(32, torch.complex64)
    r = op.distill_step(student.forward(), torch.from_numpy(ids).cuda(), torch.from_numpy(logits).cuda(),
                        torch.ones(1, device="cuda"))
    grads = student.backward(r.grad)
    tree = greedy_tree(net, 0)

    def loss(data):
        a = oracle.contract(net.tensors, net.extents, net.open_modes, data, tree)
        return Row(np.asarray(a).reshape(-1), None, 1.0).distill(ids[0], logits[0].astype(np.float64))

    base = [d.astype(np.complex128) for d in net.data]
    assert abs(r.loss.item() - loss(base)) <= 1e-3 * max(1.0, abs(loss(base)))
    h = 1e-5
    for i, g in zip(student.free, grads):
        d = rng.standard_normal(base[i].shape) + 1j * rng.standard_normal(base[i].shape)
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * d, base[i] - h * d
        want = (loss(up) - loss(down)) / (2 * h)
        got = (g.cpu().numpy().astype(np.complex128).conj() * d).sum().real
        size = np.linalg.norm(g.cpu().numpy()) * np.linalg.norm(d)
        assert abs(got - want) <= 1e-2 * max(size, 1e-3), (i, got, want)


def test_shallow_circuit_learns():
    import distill_circuit as ex
    r = ex.run(steps=40, fine=10)
    assert r["losses"][-1] < 0.8 * r["losses"][0]
    assert r["likelihoods"][-1] > r["likelihoods"][0]
    assert 0 < r["heavy_mass"] < 1 and 0 < r["student_mass"] < 1
    assert 0 < r["student_entropy"] < np.log(1024) + 1e-3
