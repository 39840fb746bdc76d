"""A shallow circuit learns the heavy outcomes of a deep one.

    python examples/distill_circuit.py [--steps 80]

1. The deep circuit's network is contracted over ``n_open`` qubits: one row of
   2^n amplitudes.  ``Outcomes.score`` gives its heavy outcomes, their log
   probabilities and the entropy.
2. A shallow circuit with free (not unitary) two-qubit tensors is trained on
   them.  Each step contracts its network to a row of amplitudes,
   ``Outcomes.distill_step`` makes the loss and its gradient at the amplitudes,
   and a contraction for every free tensor carries that back: an amplitude is
   linear in every leaf, so the leaf's gradient is the network without the leaf,
   conjugated and closed with the amplitudes' gradient.
3. The likelihood of outcomes sampled from the deep circuit is raised with a
   small bonus on the entropy (``Outcomes.score``, ``Outcomes.score_grad``).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_tensor_network_gb300 as tn                                   # noqa: E402
from workloads import greedy_tree, grid_circuit_network                   # noqa: E402
from workloads.network import Network                                     # noqa: E402


class Student:
    """A network whose leaves of order 4 can be trained."""

    def __init__(self, net, seed=0):
        self.leaves = [torch.from_numpy(d).cuda().contiguous() for d in net.data]
        self.free = [i for i, t in enumerate(net.tensors) if len(t) == 4]
        self.plan = tn.Plan.from_network(net, greedy_tree(net, seed))
        self.row = torch.empty(self.plan.out_shape, dtype=torch.complex64, device="cuda")
        self.back = {}
        for i in self.free:
            rest = net.tensors[:i] + net.tensors[i + 1:] + [list(net.open_modes)]
            part = Network(rest, net.extents, list(net.tensors[i]))
            self.back[i] = tn.Plan.from_network(part, greedy_tree(part, seed))

    def forward(self):
        """[1, 2^n] amplitudes."""
        self.plan.execute(self.leaves, self.row)
        return self.row.view(1, -1)

    def backward(self, grad):
        """Gradients of the free leaves from that of the amplitudes."""
        conj = [x.conj().resolve_conj() for x in self.leaves]
        out = []
        for i in self.free:
            g = torch.empty_like(self.leaves[i])
            self.back[i].execute(conj[:i] + conj[i + 1:] + [grad.reshape(-1)], g)
            out.append(g)
        return out


def run(rows=3, cols=4, deep=8, shallow=4, n_open=10, heavy=64, steps=80, fine=20, lr=0.05, seed=0,
        report=None):
    """The losses of both phases, and what was found on the way."""
    torch.manual_seed(seed)
    net, _ = grid_circuit_network(rows, cols, deep, seed, n_open=n_open)
    plan = tn.Plan.from_network(net, greedy_tree(net, seed))
    target = torch.empty(plan.out_shape, dtype=torch.complex64, device="cuda")
    plan.execute([torch.from_numpy(d).cuda().contiguous() for d in net.data], target)
    target = target.view(1, -1)

    op = tn.Outcomes(target.shape[1], torch.complex64, top=heavy)
    found = op.score(target)
    ids, logits = found.top_ids, found.top_logp
    mass = logits.exp().sum().item()

    student = Student(grid_circuit_network(rows, cols, shallow, seed + 1, n_open=n_open)[0], seed)
    free = [student.leaves[i] for i in student.free]
    optimiser = torch.optim.Adam(free, lr=lr)
    one = torch.ones(1, device="cuda")

    def update(grads):
        for x, g in zip(free, grads):
            x.grad = g
        optimiser.step()

    losses, likelihoods = [], []
    for i in range(steps):
        r = op.distill_step(student.forward(), ids, logits, one)
        update(student.backward(r.grad))
        losses.append(r.loss)
    learnt = op.score(student.forward(), ids)

    given = torch.multinomial(target.abs().square(), 256, replacement=True)
    g_logp = torch.full((1, 256), -1 / 256, device="cuda")
    g_entropy = torch.full((1,), -0.02, device="cuda")
    for i in range(fine):
        amplitudes = student.forward()
        s = op.score(amplitudes, given)
        grad = op.score_grad(amplitudes, given, s.logz, s.entropy, g_logp, g_entropy)
        update(student.backward(grad))
        likelihoods.append(s.logp.mean())
    last = op.score(student.forward(), given)
    likelihoods.append(last.logp.mean())
    op.check()
    result = {
        "entropy": found.entropy.item(), "heavy_mass": mass,
        "losses": torch.cat(losses).tolist(), "student_mass": learnt.logp.exp().sum().item(),
        "likelihoods": torch.stack(likelihoods).tolist(), "student_entropy": last.entropy.item(),
    }
    if report:
        report(f"deep circuit: entropy {result['entropy']:.4f}, its {heavy} heaviest outcomes hold {mass:.4f}")
        report(f"distance from their distribution: {result['losses'][0]:.4f} -> {result['losses'][-1]:.4f} "
               f"in {steps} steps; the shallow circuit gives them {result['student_mass']:.4f}")
        report(f"log likelihood of 256 samples: {result['likelihoods'][0]:.4f} -> "
               f"{result['likelihoods'][-1]:.4f} in {fine} steps, entropy {result['student_entropy']:.4f}")
    return result


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=80)
    p.add_argument("--fine", type=int, default=20)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args()
    run(steps=a.steps, fine=a.fine, seed=a.seed, report=print)


if __name__ == "__main__":
    main()
