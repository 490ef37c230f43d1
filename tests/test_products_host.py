"""CPU checks of the boundary of the products by expert, 4-bit rows and embedding rows, and of the plain implementations
that their GPU tests compare with."""
import os

import pytest
import torch

from tests import products_util as P
from tests.test_rows_host import LIB, Unlaunched


def test_null_context_is_refused():
    from molecular_dynamics_cell_amd import binding
    if not os.path.exists(LIB):
        from molecular_dynamics_cell_amd import build
        build.build(verbose=False)
    L = binding.lib()
    assert L.mpnn_expert_product(None, 0, 1, 1, 1, 1, None, None, 1, None, 1, None, None, 0, None) == -1
    assert L.mpnn_expert_input_grad(None, 0, 1, 1, 1, 1, None, None, 1, None, None) == -1
    assert L.mpnn_expert_weight_grad(None, 0, 1, 1, 1, 1, None, None, 1, None, 1, None, 1, None, None) == -1
    assert L.mpnn_micro_save(None, 0, 1, 1, None, 1, None, None) == -1
    assert L.mpnn_micro_load(None, 0, 1, 1, None, None, None) == -1
    assert L.mpnn_micro_product(None, 0, 0, 1, 1, 1, 1, None, None, 1, None, None, 1, None, None, None, 0, None) == -1
    assert L.mpnn_embed(None, 0, 1, 1, 1, None, None, 1.0, None) == -1
    assert L.mpnn_embed_plan(None, 1, 1, None, None, None) == -1
    assert L.mpnn_embed_backward(None, 0, 1, 1, 1, None, 1, None, None, 1.0, None) == -1


def test_plain_micro():
    """By hand: ties go to the even code, 7 steps to 6, and 8 steps are the next step's 4."""
    x = torch.tensor([[4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, 7.0], [8.0, 0.5, 1.5, 2.5, 3.5, 5.0, 7.0, 10.0, -0.52, 14.0]])
    codes, scales = P.micro_save(x)
    assert scales.tolist() == [[127], [128]] and codes.shape == (2, 16)
    assert P.micro_load(codes, scales, 10)[0].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5, 6.0]
    assert torch.equal(P.micro_load(codes, scales, 10)[1], 2 * P.micro_load(codes, scales, 10)[0])
    assert int(codes[0, 0]) == 6 and int(codes[0, 4]) == 9 | 7 << 4 and int(codes[0, 5:].sum()) == 0
    v = torch.randn(20, 70, generator=torch.Generator().manual_seed(1))
    v[3, 40], v[4, 2] = float("nan"), float("-inf")
    codes, scales = P.micro_save(v)
    back = P.micro_load(codes, scales, 70)
    assert back[3, 32:64].isnan().all() and back[4, :32].isnan().all() and int(back.isnan().sum()) == 64
    assert torch.equal(torch.nan_to_num(back.bfloat16().double()), torch.nan_to_num(back))
    # the largest of a group has 4 .. 8 steps: within a step of a held value but for those that 6 steps stand for
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :70]
    off = ((back - v.double()).abs() / step)[~back.isnan()]
    assert float(off.max()) <= 2.0


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    x, dy, w, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((9, 5), (9, 4), (3, 4, 5), (3, 4)))
    offsets = torch.tensor([1, 4, 4, 8], dtype=torch.int32)
    v, u, c = (torch.randn(*t.shape, generator=g, dtype=torch.float64) for t in (x, w, b))

    def value(t):
        return float((P.product(x + t * v, w + t * u, offsets, b + t * c, "none", 9)[0] * dy).sum())

    dx, _ = P.input_grad(dy, w, offsets)
    dw, _, db, _, counts = P.weight_grad(dy, x, offsets)
    assert counts == [3, 0, 4] and abs((value(1.0) - value(-1.0)) / 2 - float((dx * v).sum() + (dw * u).sum() + (db * c).sum())) < 1e-12
    index, table = torch.tensor([2, -1, 0, 2, 5], dtype=torch.int32), torch.randn(3, 4, generator=g, dtype=torch.float64)
    d = torch.randn(5, 4, generator=g, dtype=torch.float64)
    got, _, rows = P.embed_grad(index, d, 3, -2.0)
    assert rows.tolist() == [1, 0, 2]
    t = torch.randn(3, 4, generator=g, dtype=torch.float64)
    assert abs(float(((P.embed(index, table + t, -2.0) - P.embed(index, table, -2.0)) * d).sum() - (got * t).sum())) < 1e-12
    offsets, source = P.embed_plan(index, 3)
    assert offsets.tolist() == [0, 1, 1, 3] and source.tolist() == [2, 0, 3, 1, 4]


def calls(m):
    """A call of each method, by the tensor that it is given through g."""
    x, w, b = torch.zeros(6, 8), torch.zeros(2, 5, 8), torch.zeros(2, 5)
    dy, seg = torch.zeros(6, 5), torch.tensor([0, 2, 6], dtype=torch.int32)
    held = (torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 1, dtype=torch.uint8), 8)
    index = torch.zeros(6, dtype=torch.int32)
    return [lambda g: m.expert_product(g(x), w, seg), lambda g: m.expert_product(x, g(w), seg),
            lambda g: m.expert_product(x, w, seg, g(b)), lambda g: m.expert_product_backward(g(dy), x, w, seg),
            lambda g: m.expert_product_backward(dy, g(x), None, seg), lambda g: m.expert_product_backward(dy, None, g(w), seg),
            lambda g: m.micro_save(g(x)), lambda g: m.micro_product(g(x), held, seg), lambda g: m.micro_product(x, held, seg, g(b)),
            lambda g: m.embed(index, g(x)), lambda g: m.embed_backward(g(x), seg, index)]


def test_tensors_that_require_a_gradient_are_refused():
    for call in calls(Unlaunched()):
        with pytest.raises(ValueError, match="requires a gradient"):
            call(lambda t: t.clone().requires_grad_())
        for enabled in (True, False):
            with torch.set_grad_enabled(enabled), pytest.raises(Exception) as e:
                call(lambda t: t if enabled else t.clone().requires_grad_())
            assert "requires a gradient" not in str(e.value)


def test_refused_by_the_binding():
    m = Unlaunched()
    x, w, seg = torch.zeros(6, 8), torch.zeros(2, 5, 8), torch.tensor([0, 2, 6], dtype=torch.int32)
    held = (torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(10, 1, dtype=torch.uint8), 8)
    source = torch.zeros(12, dtype=torch.int32)
    bad = [lambda: m.expert_product(x, w[0], seg), lambda: m.expert_product(x, w[:1], seg), lambda: m.expert_product(x, w.bfloat16(), seg),
           lambda: m.expert_product(x[:, :7], w, seg), lambda: m.expert_product(x, w, seg.long()), lambda: m.expert_product(x, w, seg[:1]),
           lambda: m.expert_product(x, w, seg, torch.zeros(2, 4)), lambda: m.expert_product(x, w, seg, torch.zeros(2, 5).double()),
           lambda: m.expert_product(x, w, seg, act="relu"), lambda: m.expert_product(x.double(), w.double(), seg),
           lambda: m.expert_product(x, w, seg, source=source[:11]), lambda: m.expert_product(x, w, seg, source=source[:0]),
           lambda: m.expert_product(x, w, seg, source=source.reshape(6, 2)), lambda: m.expert_product(x, w, seg, source=source.long()),
           lambda: m.expert_product_backward(x[:, :5], None, None, seg), lambda: m.expert_product_backward(x[:, :5], x[:5], w, seg),
           lambda: m.expert_product_backward(x[:, :4], x, w, seg), lambda: m.expert_product_backward(x[:, :5], x[0], w, seg),
           lambda: m.expert_product_backward(x[:, :5], x, w, seg, source=source),
           lambda: m.micro_save(x[0]), lambda: m.micro_load(held, torch.float16), lambda: m.micro_load((held[0][:, :15], held[1], 8)),
           lambda: m.micro_load((held[0], held[1], 33)), lambda: m.micro_load((held[0], held[1][:9], 8)),
           lambda: m.micro_product(x, (held[0][:9], held[1][:9], 8), seg), lambda: m.micro_product(x[:, :7], held, seg),
           lambda: m.micro_product((held[0], held[1], 9), held, seg), lambda: m.micro_product(x, held, seg, dtype=torch.float64),
           lambda: m.micro_product(x, held, seg, torch.zeros(2, 4)), lambda: m.micro_product(x, held, seg, act="gelu"),
           lambda: m.embed(torch.zeros(3), x), lambda: m.embed(source.reshape(6, 2), x), lambda: m.embed(source, x.double()),
           lambda: m.embed(source, x[0]), lambda: m.embed_plan(source.long(), 3), lambda: m.embed_plan(source.reshape(6, 2), 3),
           lambda: m.embed_backward(x, seg, source), lambda: m.embed_backward(x, seg[:1], source[:6]),
           lambda: m.embed_backward(x[0], seg, source[:6])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
