"""The routed readout of examples/: its hand-written backward pass against differences of its forward pass, and the fit."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradient_against_differences():
    """Central differences along random directions of each parameter, with the experts that the routers chose kept (a
    changed choice is a jump of the loss, which no gradient has).  The checkpoints hold a value to 1/127 of the
    largest of its 32 neighbours, so weight gradients of the layers that read them are off by a few parts in a
    thousand of the gradient's size; the others by fp32 rounding of the loss (U 2^-24 of its terms over the step)."""
    import routed_readout as R
    m, x, types, target = R.teacher()
    net = R.Readout(m, x.shape[1], 2)

    chosen = None

    def loss():
        off = net.forward(x, types, chosen) - target
        return off, float((off.double() ** 2).mean())

    off, _ = loss()
    chosen = [kept[2] for kept in net.kept[1:]]
    grads = net.backward(2 * off / len(off))
    assert set(grads) == set(net.p)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    for name, g in grads.items():
        v = torch.sign(torch.randn(g.shape, generator=gen, device="cuda")) * g.abs()     # mostly along the gradient's size
        v = g / g.norm() + 0.3 * v / v.norm()
        kept, h = net.p[name], 2e-3
        net.p[name] = kept + h * v
        _, up = loss()
        net.p[name] = kept - h * v
        _, down = loss()
        net.p[name] = kept
        slope, mine = (up - down) / (2 * h), float((g * v).sum())
        print(f"[readout] {name}: {mine:.6e} differences {slope:.6e}", flush=True)
        assert abs(mine - slope) <= 0.03 * abs(slope) + 1e-4, name


def test_fit_learns():
    import routed_readout as R
    losses = R.fit(steps=120)
    print(f"[readout] {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    assert losses[-1] < 0.25 * losses[0] and all(v == v for v in losses)
    assert R.fit(steps=5) == losses[:5]      # the same bits again
