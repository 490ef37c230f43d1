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


def test_rows_sent_out_by_more_threads_than_a_launch_holds(m):
    """268,500,007 rows of one value to five places: 2^32 threads and more."""
    n, k = 268500007, 5
    x = (torch.arange(n, dtype=torch.int32, device=DEV) % 251).to(torch.bfloat16).unsqueeze(1)
    position = torch.arange(n * k, dtype=torch.int32, device=DEV).reshape(n, k)
    offsets = torch.tensor([0, n * k], dtype=torch.int32, device=DEV)
    rows = m.route_scatter(x, position, offsets)
    assert torch.equal(rows.reshape(n, k), x.expand(n, k))
    del rows
    # the weights' gradient <dout, row> and the rows' own, against the same call on the last rows alone
    dout, weight = x, torch.full((n, k), 0.5, device=DEV)
    rows = x.expand(n, k).reshape(n * k, 1)
    dy, dweight = m.route_combine_backward(dout, rows, position, offsets, weight)
    assert torch.equal(dy.reshape(n, k), (x * 0.5).expand(n, k))
    assert torch.equal(dweight, (x.float() * x.float()).expand(n, k))


def test_rows_added_up_by_more_threads_than_a_launch_holds(m):
    """16,780,000 rows of 1,032 columns, a block each, from three slots; a few rows have places, the others are zeros.  (The
    sorted rows are only those below the routed count, which is all that may be read.)"""
    n, k, width = 16780000, 3, 1032
    g = rng(7)
    rows = normal(g, 16, width, dtype=torch.bfloat16)
    position = torch.full((n, k), -1, dtype=torch.int32, device=DEV)
    some = torch.tensor([0, 1, 8388607, 8388608, 16777206, 16777207, 16777208, 16777209, 16777215, 16777216, n - 1])
    places = torch.randint(0, 16, (len(some), k), generator=g, dtype=torch.int32)
    position[some.to(DEV)] = places.to(DEV)
    offsets = torch.tensor([0, 16], dtype=torch.int32, device=DEV)
    weight = torch.ones(n, k, device=DEV)
    out = torch.full((n, width), float("nan"), dtype=torch.bfloat16, device=DEV)
    L = binding.lib()
    assert L.mpnn_route_combine(m.h, 1, n, k, width, rows.data_ptr(), position.data_ptr(), offsets.data_ptr(), 1,
                                weight.data_ptr(), out.data_ptr()) == 0, L.mpnn_last_error(m.h)
    torch.cuda.synchronize()
    taken = f64(rows)[places.long()]
    check("out", out[some.to(DEV)], taken.sum(1), 4 * U * taken.abs().sum(1), torch.bfloat16)
    out[some.to(DEV)] = 0
    assert int(out.view(torch.int32).count_nonzero()) == 0


class Pieces:
    """Allocator hooks that hand out pieces of one tensor and note what is taken and given back; nothing is used twice."""

    def __init__(self, m, megabytes=256):
        self.base = torch.empty(megabytes << 20, dtype=torch.uint8, device=DEV)
        self.at, self.taken, self.back = 0, [], []

        def alloc(nbytes, user):
            p = self.base.data_ptr() + self.at
            self.at += (int(nbytes) + 255) // 256 * 256
            assert self.at <= self.base.numel()
            self.taken.append(p)
            return p

        self.hooks = (binding._ALLOC_FN(alloc), binding._FREE_FN(lambda p, user: self.back.append(p)))
        assert binding.lib().mpnn_set_allocator(m.h, *self.hooks, None) == 0


def uneven(g, n, E):
    return torch.randint(-1, E, (n, 1), generator=g, dtype=torch.int32).to(DEV)


def test_scratch_of_a_captured_call_stays():
    """A graph keeps its scratch's address: later eager calls, larger ones too, neither give that memory back nor use it."""
    m = binding.MPNN(I.make_params(1), DEV)
    pieces = Pieces(m)
    g = rng(1)
    e, big = uneven(g, 9000, 300), uneven(g, 200000, 1000)
    x, dy = normal(g, 3000, 100), normal(g, 3000, 40)
    held, seg = m.checkpoint_save(x), torch.tensor([0, 3000], dtype=torch.int32, device=DEV)

    def step():
        return [*m.route_plan(e, 300), *m.norm_residual_backward(x, x, x, x)[3:], *m.checkpoint_weight_grad(dy, held, seg)]

    step()
    home, graph = m._stream, torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    try:
        with torch.cuda.graph(graph):
            m.set_stream(torch.cuda.current_stream())
            kept = step()
    finally:
        m.set_stream(home)
    step()
    eager = len(pieces.taken)
    m.route_plan(big, 1000)
    torch.cuda.synchronize()
    assert len(pieces.taken) > eager                     # the larger plan took a larger block,
    recorded = [p for p in pieces.taken if p not in pieces.back]
    assert len(recorded) >= 2                            # beside the graph's, which was not given back
    offsets, source, position = m.route_plan(big, 1000)
    side = torch.cuda.Stream()
    for seed in range(4):
        e.copy_(uneven(rng(seed), 9000, 300))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):                    # replays beside eager calls on the context's stream
            for _ in range(5):
                graph.replay()
        for _ in range(5):
            again = m.route_plan(big, 1000)
        torch.cuda.synchronize()
        assert torch.equal(again[0], offsets) and torch.equal(again[1], source) and torch.equal(again[2], position)
        for a, b in zip([t.clone() for t in kept], step()):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    del graph
    m.close()
    assert sorted(pieces.taken) == sorted(pieces.back)


def test_scratch_of_each_stream():
    """Calls on two streams, neither waiting for the other, do not share scratch; every block goes back in the end."""
    m = binding.MPNN(I.make_params(1), DEV)
    pieces = Pieces(m)
    g = rng(2)
    plans = [uneven(g, 200000 + 5000 * i, 700) for i in range(2)]
    want = [R.plan(e, 700) for e in plans]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):
        for e, s in zip(plans, streams):
            with torch.cuda.stream(s):
                m.set_stream(s)
                got.append(m.route_plan(e, 700))
    assert len(pieces.taken) == 2 and not pieces.back
    torch.cuda.synchronize()
    for i, (offsets, source, position) in enumerate(got):
        for a, b in zip((offsets, source, position), want[i % 2]):
            assert (a.cpu().numpy() == b).all()
    del got
    m.close()
    assert sorted(pieces.taken) == sorted(pieces.back)


def same_kind(got, want):
    """Not-a-numbers and infinities in the same places, of the same sign."""
    got = f64(got)
    assert torch.equal(got.isnan(), want.isnan()), (got.isnan().sum(), want.isnan().sum())
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[got.isinf()] > 0, want[want.isinf()] > 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", [6, 30, 108, 312, 1000, 1400, 5000])
def test_one_infinity_in_a_row(m, width, kind, dtype):
    """An rms row with an infinity is the bias elsewhere (1 over an infinite root is 0), whichever column holds it: rows that
    do not fill their lanes hold some columns twice.  A layer row is NaN throughout."""
    g = rng(width)
    columns = sorted({0, 1, width // 2, *range(max(0, width - 12), width)})
    n = len(columns) + 1                                    # the last row is finite
    at = (torch.arange(n - 1, device=DEV), torch.tensor(columns, device=DEV))
    w = {k: normal(g, width, size=0.3, at=0.0 if "bias" in k else 1.0)
         for k in ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")}
    w64 = {k: f64(v) for k, v in w.items()}
    x, block = normal(g, n, width, dtype=dtype), normal(g, n, width, dtype=dtype)
    size = (width + 64) * U * 16      # of a finite row: sums of `width` terms and the rest of the formula, values of size < 16
    block[at] = float("inf")
    block[0, columns[0]] = float("-inf")
    for gate in (None, normal(g, n, 1, dtype=dtype), normal(g, n, width, dtype=dtype)):
        r, h = m.norm_residual(x, block, gate, **w, kind=kind, eps=EPS)
        r64, h64 = R.residual(f64(x), f64(block), f64(gate), w64, kind == "layer", EPS)
        check("r", r, r64, size, dtype)
        check("h", h, h64, size * 4, dtype)
    x[at] = float("inf")
    _, h = m.norm_residual(x, pre_weight=w["pre_weight"], pre_bias=w["pre_bias"], kind=kind, eps=EPS)
    check("h of x", h, R.normed(f64(x), kind == "layer", EPS)[0] * w64["pre_weight"] + w64["pre_bias"], size, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [6, 30, 108, 312, 1000, 1400, 5000])
def test_one_infinity_in_a_gradient(m, width, dtype):
    """An infinity in dr: where the formula has infinities and where NaN, in any column."""
    g = rng(width)
    columns = sorted({0, width // 2, *range(max(0, width - 9), width)})
    n = len(columns)
    dr, block = normal(g, n, width, dtype=dtype), normal(g, n, width, dtype=dtype)
    block[block == 0] = 1.0
    dr[torch.arange(n, device=DEV), torch.tensor(columns, device=DEV)] = float("inf")
    gate = normal(g, n, 1, dtype=dtype)
    dx, dblock, dgate, *_ = m.norm_residual_backward(dr, None, None, block, gate, kind="rms", eps=EPS)
    hat, inv = R.normed(f64(block), False, EPS)
    sig = torch.sigmoid(f64(gate))
    same_kind(dx, f64(dr))
    same_kind(dblock, R.normed_back(f64(dr) * sig, hat, inv, False))
    same_kind(dgate, (f64(dr) * hat * sig * (1 - sig)).sum(-1, keepdim=True))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", ["row", "element"])
@pytest.mark.parametrize("n,width", [(13, 108), (13, 312), (9, 1024), (7, 1400)])
def test_gate_gradient_far_from_zero(m, n, width, form, dtype):
    """sigma'(g) = sigma(g) sigma(-g) to fp32 accuracy at both signs: |g| 2^-24 from the exponent's argument and a few
    units from the rest, relative to total scale u sigma (1 - sigma) term by term."""
    g = rng(width)
    far = torch.tensor([8.0, 12.0, 15.0, 17.5, 20.0, 30.0, 80.0])
    far = torch.cat([far, -far])
    gate = far[torch.randint(0, len(far), (n, 1 if form == "row" else width), generator=g)].to(dtype).to(DEV)
    dr, dh, r, block = (normal(g, n, width, dtype=dtype) for _ in range(4))
    _, _, dgate, *_ = m.norm_residual_backward(dr, dh, r, block, gate, kind="rms", eps=EPS)
    rhat, rinv = R.normed(f64(r), False, EPS)
    hat, inv = R.normed(f64(block), False, EPS)
    total = f64(dr) + R.normed_back(f64(dh), rhat, rinv, False)
    size = f64(dr).abs() + R.normed_back_size(f64(dh).abs(), rhat, rinv) * (1 + rinv * f64(r).abs().mean(-1, keepdim=True))
    g64 = f64(gate)
    slope = 1 / (1 + torch.exp(-g64)) / (1 + torch.exp(g64))
    us = hat.abs() + inv * f64(block).abs().mean(-1, keepdim=True)
    want, bound = total * hat * slope, (4 * width + 64 + 4 * g64.abs()) * U * size * us * slope
    if form == "row":
        want, bound = want.sum(-1, keepdim=True), bound.sum(-1, keepdim=True)
    check("dgate", dgate, want, bound, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate_kind", ["none", "row", "element"])
@pytest.mark.parametrize("width", [30, 108, 312, 1000, 1400, 2600, 5000, 8192])
def test_in_place_rows_of_several_waves(m, width, gate_kind, dtype):
    """r = x and dx = dr give the bits of separate arrays, also where lanes of another wave hold the same columns."""
    g = rng(width)
    n = 700
    x, block, dr, dh = (normal(g, n, width, dtype=dtype) for _ in range(4))
    gate = {"none": None, "row": normal(g, n, 1, dtype=dtype), "element": normal(g, n, width, dtype=dtype)}[gate_kind]
    p, _ = m._norm(x, width, gate, "layer", EPS, [])
    ptr, wide = None if gate is None else gate.data_ptr(), 0 if gate is None else gate.shape[1]
    r, h = m.norm_residual(x, block, gate, kind="layer", eps=EPS)
    dx, dblock, dgate, *_ = m.norm_residual_backward(dr, dh, r, block, gate, kind="layer", eps=EPS)
    h2, db = torch.empty_like(x), torch.empty_like(x)
    dg = None if gate is None else torch.empty_like(gate)
    L = binding.lib()
    assert L.mpnn_norm_residual(m.h, C.byref(p), n, x.data_ptr(), width, block.data_ptr(), width, ptr, wide, x.data_ptr(),
                                h2.data_ptr()) == 0
    assert L.mpnn_norm_residual_backward(m.h, C.byref(p), n, dr.data_ptr(), dh.data_ptr(), r.data_ptr(), width, block.data_ptr(),
                                         width, ptr, wide, dr.data_ptr(), db.data_ptr(), None if dg is None else dg.data_ptr(),
                                         *[None] * 5) == 0
    torch.cuda.synchronize()
    assert torch.equal(x, r) and torch.equal(h2, h) and torch.equal(dr, dx) and torch.equal(db, dblock)
    assert dg is None or torch.equal(dg, dgate)


def test_torch_allocator_follows_the_stream(monkeypatch):
    """Scratch taken from torch's allocator is memory of the stream that the call runs on, captured calls' included, and all
    of it goes back."""
    g = rng(3)
    e, n, E = uneven(g, 50000, 400), 50000, 400
    want = R.plan(e, E)
    streams, side = [], torch.cuda.Stream()
    real = torch.cuda.caching_allocator_alloc

    def noted(size, device=None, stream=None):
        streams.append(stream.cuda_stream)
        return real(size, device, stream)

    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", noted)
    torch.cuda.synchronize()
    m = binding.MPNN(I.make_params(1), DEV)
    m.use_torch_allocator()
    home = m._stream
    first = m.route_plan(e, E)
    m.set_stream(side)
    with torch.cuda.stream(side):
        second = m.route_plan(e, E)
    torch.cuda.synchronize()
    assert streams == [home.cuda_stream, side.cuda_stream]
    graph = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(graph):
            recording = torch.cuda.current_stream()
            m.set_stream(recording)
            third = m.route_plan(e, E)
    finally:
        m.set_stream(home)
    assert streams[2:] == [recording.cuda_stream]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for got in (first, second, third, m.route_plan(e, E)):
            for a, b in zip(got, want):
                assert (a.cpu().numpy() == b).all()
    assert len(streams) == 3
    del graph, got, third
    m.close()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,pad,shift", [(64, 64, 0), (108, 20, 4), (64, 1, 1), (312, 9, 3), (33, 7, 2), (1024, 1024, 0),
                                             (1400, 3, 1), (5000, 8, 8)])
@pytest.mark.parametrize("kind,gate", [("rms", "element"), ("layer", "row"), ("layer", "none")])
def test_strided_rows_bit_for_bit(m, width, pad, shift, kind, gate, dtype):
    """The layout in memory changes no lane's work and no order of a sum: column blocks give the dense rows' bits."""
    g = rng(width)
    n, k = 50, 2

    def pair(w=width):
        part = normal(g, n, w + pad + shift, dtype=dtype)[:, shift:shift + w]
        return part, part.contiguous()

    (x, xd), (b, bd), (dy, dyd) = pair(), pair(), pair()
    t, td = {"none": (None, None), "row": pair(1), "element": pair()}[gate]
    for p, q in zip(m.norm_residual(x, b, t, kind=kind), m.norm_residual(xd, bd, td, kind=kind)):
        assert torch.equal(p, q)
    for p, q in zip(m.norm_residual_backward(dyd, xd, x, b, t, kind=kind), m.norm_residual_backward(dyd, xd, xd, bd, td, kind=kind)):
        assert (p is None and q is None) or torch.equal(p, q)
    offsets, source, position = m.route_plan(torch.randint(-1, 3, (n, k), generator=g, dtype=torch.int32).to(DEV), 3)
    y = normal(g, n * k, width, dtype=dtype)
    for p, q in zip(m.route_combine_backward(dy, y, position, offsets), m.route_combine_backward(dyd, y, position, offsets)):
        assert torch.equal(p, q)
    held, seg = m.checkpoint_save(x), torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    for p, q in zip(m.checkpoint_weight_grad(dy, held, seg), m.checkpoint_weight_grad(dyd, held, seg)):
        assert torch.equal(p, q)
