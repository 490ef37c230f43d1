"""CPU checks of the row operators' boundary and of the plain implementations their GPU tests compare with."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

from tests import rows_util as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "molecular_dynamics_cell_amd", "libmpnn.so")


def test_null_context_is_refused():
    from molecular_dynamics_cell_amd import binding
    if not os.path.exists(LIB):
        from molecular_dynamics_cell_amd import build
        build.build(verbose=False)
    L = binding.lib()
    assert L.mpnn_route_plan(None, 1, 1, 1, None, None, None, None) == -1
    assert L.mpnn_route_scatter(None, 0, 1, 1, 1, None, 1, None, None, 1, None) == -1
    assert L.mpnn_route_combine(None, 0, 1, 1, 1, None, None, None, 1, None, None) == -1
    assert L.mpnn_route_combine_backward(None, 0, 1, 1, 1, None, 1, None, None, None, 1, None, None, None) == -1
    assert L.mpnn_norm_residual(None, None, 1, None, 1, None, 1, None, 1, None, None) == -1
    assert L.mpnn_norm_residual_backward(None, None, 1, *[None] * 3, 1, None, 1, None, 1, *[None] * 8) == -1
    assert L.mpnn_checkpoint_save(None, 0, 1, 1, None, 1, None, None) == -1
    assert L.mpnn_checkpoint_load(None, 0, 1, 1, None, None, None) == -1
    assert L.mpnn_checkpoint_silu(None, 0, 1, 1, None, 1, None, None, None, None, None) == -1
    assert L.mpnn_checkpoint_silu_backward(None, 0, 1, 1, None, 1, None, None, None) == -1
    assert L.mpnn_checkpoint_weight_grad(None, 0, 1, 1, 1, 1, None, None, 1, None, None, None, None) == -1


def test_plain_checkpoint():
    """By hand: 127/64 sits on the largest code, the next value up needs the next step; nothing beyond half a step."""
    x = torch.tensor([[1.984375, -1.0, 0.015625, 0.0078125], [1.9843751, -1.0, 0.015625, 0.046875]])
    codes, scales = R.save(x)
    assert scales.tolist() == [[121], [122]]
    assert codes[0].tolist() == [127, -64, 1, 0] and codes[1].tolist() == [64, -32, 0, 2]   # ties to even
    assert R.load(codes, scales)[0].tolist() == [1.984375, -1.0, 0.015625, 0.0]
    v = torch.randn(50, 70, generator=torch.Generator().manual_seed(1))
    back = R.load(*R.save(v))
    largest = torch.nn.functional.pad(v.double().abs(), (0, 26)).reshape(50, 3, 32).amax(-1).repeat_interleave(32, 1)[:, :70]
    assert ((back - v.double()).abs() <= largest / 127).all()
    assert torch.equal(back.bfloat16().double(), back)


def test_plain_plan():
    e = torch.tensor([[2, 0], [-1, 2], [0, 9]], dtype=torch.int32)
    offsets, source, position = R.plan(e, 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert source.tolist() == [1, 4, 0, 3, 2, 5]
    assert position.tolist() == [[2, 0], [4, 3], [1, 5]]


@pytest.mark.parametrize("layer", [False, True])
def test_plain_norm_gradient(layer):
    """normed_back against differences of normed."""
    g = torch.Generator().manual_seed(2)
    v, d, t = (torch.randn(4, 11, generator=g, dtype=torch.float64) for _ in range(3))
    hat, inv = R.normed(v, layer, 1e-5)
    h = 1e-6
    slope = ((R.normed(v + h * t, layer, 1e-5)[0] - R.normed(v - h * t, layer, 1e-5)[0]) / (2 * h) * d).sum()
    assert abs(float((R.normed_back(d, hat, inv, layer) * t).sum() - slope)) < 1e-7


def test_plain_silu_slope():
    z = torch.linspace(-20, 20, 81, dtype=torch.float64)
    assert torch.allclose(R.silu_slope(z), (R.silu(z + 1e-5) - R.silu(z - 1e-5)) / 2e-5, atol=1e-9)
    assert np.isfinite(R.silu(z).numpy()).all()


class Unlaunched:
    """The methods of a context without a library behind them: what they refuse by themselves."""

    def __new__(cls):
        from molecular_dynamics_cell_amd import rows
        m = rows.RowOperators()
        m.h, m._at, m._stream = None, torch.device("cpu"), None
        return m


def test_tensors_that_require_a_gradient_are_refused():
    """A result without a gradient in place of one that a caller would train through; without gradients nothing is refused."""
    m, x, w = Unlaunched(), torch.zeros(6, 8), torch.ones(8)
    position, offsets = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    weight, rows = torch.zeros(3, 2), torch.zeros(3, 8)
    held = (torch.zeros(6, 8, dtype=torch.int8), torch.zeros(6, 1, dtype=torch.uint8))
    seg = torch.tensor([0, 6], dtype=torch.int32)
    calls = [lambda g: m.route_scatter(g(rows), position, offsets), lambda g: m.route_combine(g(x), position, offsets),
             lambda g: m.route_combine(x, position, offsets, g(weight)),
             lambda g: m.route_combine_backward(g(rows), None, position, offsets),
             lambda g: m.norm_residual(g(x)), lambda g: m.norm_residual(x, g(x)), lambda g: m.norm_residual(x, x, g(x)),
             lambda g: m.norm_residual(x, pre_weight=g(w)), lambda g: m.norm_residual(x, x, scale=g(w)),
             lambda g: m.norm_residual(g(x[:, ::2])),
             lambda g: m.norm_residual_backward(g(x), x, x), lambda g: m.checkpoint_save(g(x)), lambda g: m.checkpoint_silu(g(x)),
             lambda g: m.checkpoint_silu_backward(g(x), held), lambda g: m.checkpoint_weight_grad(g(x), held, seg)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call(lambda t: t.clone().requires_grad_())
        for enabled in (True, False):         # past the refusal: there is no library to reach, which is another error
            with torch.set_grad_enabled(enabled), pytest.raises(Exception) as e:
                call(lambda t: t if enabled else t.clone().requires_grad_())
            assert "requires a gradient" not in str(e.value)


def test_gate_without_columns_is_refused():
    m, x = Unlaunched(), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="gate"):
        m.norm_residual(x, x, x[:, :0])
    with pytest.raises(ValueError, match="gate"):
        m.norm_residual_backward(x, x, x, x, x[:, :0])
