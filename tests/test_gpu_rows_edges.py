"""Row operators on the GPU where they go wrong most easily, against plain 64-bit implementations."""
import ctypes as C

import pytest
import torch

from molecular_dynamics_cell_amd import binding
from molecular_dynamics_cell_amd import inputs as I
from tests import rows_util as R
from tests.rows_util import U, check, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]
EPS = 1e-5


@pytest.fixture(scope="module")
def m():
    ctx = binding.MPNN(I.make_params(1), DEV)
    yield ctx
    torch.cuda.synchronize()
    ctx.close()


@pytest.fixture(autouse=True)
def say_name(request):
    print(f"[rows] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, size=1.0, at=0.0):
    return (torch.randn(*shape, generator=g) * size + at).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k,width", [(5, 1, 16), (40, 3, 100), (33, 2, 3), (64, 8, 1024)])
@pytest.mark.parametrize("routed", ["more", "most", "fewer", "negative"])
def test_counts_that_are_not_the_rows(m, n, k, width, routed, dtype):
    """Offsets of a longer plan, or of none: a place counts only below the routed pairs and inside the n k rows.  The rows
    are the front of a longer tensor of NaN, so that a place read past them would show."""
    g = rng(n * width)
    pairs = n * k
    behind = torch.full((4 * pairs, width), float("nan"), dtype=dtype, device=DEV)
    rows = behind[:pairs]
    rows.copy_(normal(g, pairs, width, dtype=dtype))
    position = torch.randperm(3 * pairs, generator=g)[:pairs].to(torch.int32).reshape(n, k).to(DEV)   # a part of a longer plan
    position[0, 0] = -1
    last = {"more": 3 * pairs, "most": 2 ** 31 - 1, "fewer": pairs // 2, "negative": -7}[routed]
    offsets = torch.tensor([0, last], dtype=torch.int32, device=DEV)
    live = min(max(last, 0), pairs)
    on = ((position >= 0) & (position < live)).cpu().unsqueeze(-1)
    taken = torch.where(on, f64(rows)[position.cpu().long().clamp(0, pairs - 1)], 0.0)
    weight = normal(g, n, k)
    terms = taken * f64(weight).unsqueeze(-1)
    check("out", m.route_combine(rows, position, offsets, weight), terms.sum(1), (k + 1) * U * terms.abs().sum(1), dtype)
    dout = normal(g, n, width, dtype=dtype)
    _, dweight = m.route_combine_backward(dout, rows, position, offsets, weight)
    products = f64(dout).unsqueeze(1) * taken
    check("dweight", dweight, products.sum(-1), (width + 1) * U * products.abs().sum(-1))
