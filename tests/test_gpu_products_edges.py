"""Products by expert, 4-bit rows and embedding rows on the GPU where they go wrong most easily, against plain 64-bit
implementations.  The bounds are those of test_gpu_products.py."""
import pytest
import torch

from molecular_dynamics_cell_amd import binding
from molecular_dynamics_cell_amd import inputs as I
from tests import products_util as P
from tests.rows_util import U, check, f64
from tests.test_gpu_products import act_bound, bound, ends, rows

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def m():
    ctx = binding.MPNN(I.make_params(1), DEV)
    yield ctx
    torch.cuda.synchronize()
    ctx.close()


@pytest.fixture(autouse=True)
def say_name(request):
    print(f"[products] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, size=1.0):
    return (torch.randn(*shape, generator=g) * size).to(dtype).to(DEV)


# ---------------------------------------------------------------------------------------------------------------
# products by expert
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n_x", [0, 5])
@pytest.mark.parametrize("dtype", [0, 1])
def test_no_rows_with_a_source(m, dtype, n_x):
    """A batch without rows whose source is an array all the same: gradients of zeros, nothing else written."""
    L = binding.lib()
    offsets, source = (torch.zeros(9, dtype=torch.int32, device=DEV) for _ in range(2))
    x, dw, db, y = (torch.full((600,), 7.0, device=DEV) for _ in range(4))
    o, s, p = offsets.data_ptr(), source.data_ptr(), x.data_ptr()
    assert L.mpnn_expert_weight_grad(m.h, dtype, 0, 16, 8, 2, o, p, 8, p, 16, s, n_x, dw.data_ptr(), db.data_ptr()) == 0
    assert L.mpnn_expert_weight_grad(m.h, dtype, 0, 16, 8, 2, o, None, 8, None, 16, s, n_x, dw[300:].data_ptr(), None) == 0
    assert L.mpnn_expert_product(m.h, dtype, 0, 16, 8, 2, o, p, 16, s, n_x, p, None, 0, y.data_ptr()) == 0
    assert L.mpnn_micro_product(m.h, dtype, 0, 0, 16, 8, 2, o, p, 16, None, s, n_x, p, p, None, 0, y.data_ptr()) == 0
    torch.cuda.synchronize()
    assert (dw[:256] == 0).all() and (dw[256:300] == 7).all() and (dw[300:556] == 0).all() and (dw[556:] == 7).all()
    assert (db[:16] == 0).all() and (db[16:] == 7).all() and (y == 7).all() and (x == 7).all()


def test_as_many_rows_as_there_may_be(m):
    """2^31 - 1 rows of one column, the last rows' places first: small whole numbers, whose sums are exact."""
    n, some = 2 ** 31 - 1, 100000
    whole = torch.full((n + 16, 1), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = whole[:n]
    x.zero_()
    mine, other = (torch.arange(some) % 7 - 2).bfloat16(), (torch.arange(some) % 5 - 1).bfloat16()
    x[-some:] = mine.to(DEV).unsqueeze(1)
    dy = torch.zeros(n, 1, dtype=torch.bfloat16, device=DEV)
    dy[:some] = other.to(DEV).unsqueeze(1)
    source = torch.arange(n, dtype=torch.int32, device=DEV)
    source.neg_().add_(n - 1)
    offsets = torch.tensor([0, 1000, n], dtype=torch.int32, device=DEV)
    w = torch.tensor([3.0, -2.0], dtype=torch.bfloat16, device=DEV).reshape(2, 1, 1)
    _, dw, db = m.expert_product_backward(dy, x, None, offsets, source=source)
    pairs = mine.flip(0).double() * other.double()
    assert f64(dw).reshape(-1).tolist() == [float(pairs[:1000].sum()), float(pairs[1000:].sum())]
    assert f64(db).reshape(-1).tolist() == [float(other[:1000].double().sum()), float(other[1000:].double().sum())]
    factor = torch.where(torch.arange(some) < 1000, 3.0, -2.0).double()
    y = m.expert_product(x, w, offsets, source=source)
    assert torch.equal(f64(y[:some])[:, 0], factor * mine.flip(0).double()) and float(y[-1000:].float().abs().max()) == 0
    del y
    y = m.expert_product(x, w, offsets)
    assert torch.equal(f64(y[-some:])[:, 0], -2.0 * mine.double()) and float(y[:1000].float().abs().max()) == 0
    del y
    dx = m.expert_product_backward(x, None, w, offsets)[0]
    assert torch.equal(f64(dx[-some:])[:, 0], -2.0 * mine.double())


TOP = torch.finfo(torch.float32).max
# straight from memory, tiles, and wide tiles where the type has them
SIZES = [(24, 100, 60), (3000, 33, 600), (7000, 128, 256), (5000, 264, 392)]


def agrees(name, got, want, b, dtype):
    """Within the bound, and infinite exactly where a 64-bit result does not fit the type, with its sign."""
    want = torch.where(want.abs() > torch.finfo(dtype).max, torch.sign(want) * float("inf"), want)
    assert torch.equal(f64(got).isinf(), want.isinf()), name
    check(name, got, want, torch.where(want.isinf(), 0.0, b), dtype)


def large(g, *shape, at, dtype):
    """Positive values between `at` and twice it, whose roundings to fewer bits are off either way."""
    return ((1 + torch.rand(*shape, generator=g)) * at).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [1e25, 2.0 ** 66])
@pytest.mark.parametrize("n,width,out", SIZES)
def test_products_that_overflow(m, n, width, out, at, dtype):
    """Finite values whose product does not fit: an infinity with the product's sign, not a NaN; their neighbours stay."""
    g, c, o = rng(n + out), width - 1, out // 3
    x, w, dy = rows(g, n, width, dtype), normal(g, 2, out, width, dtype=dtype), rows(g, n, out, dtype)
    offsets, few = ends([n // 2, n - n // 2]), slice(0, n, 3)
    x[few, c], dy[few, o] = large(g, len(x[few]), at=at, dtype=dtype), large(g, len(x[few]), at=at, dtype=dtype)
    w[:, :out // 2, c] = large(g, 2, out // 2, at=at, dtype=dtype)
    for act in ("none", "silu"):
        bias = None if act == "none" else normal(g, 2, out)
        want, size = P.product(x, w, offsets, bias, act, n)
        agrees("y", m.expert_product(x, w, offsets, bias, act=act), want, act_bound(bound(width, size, dtype, dtype), want, act), dtype)
    w[:, :out // 4, c] *= -1
    want, size = P.product(x, w, offsets, None, "none", n)
    agrees("y of either sign", m.expert_product(x, w, offsets), want, bound(width, size, dtype, dtype), dtype)
    dx, dw, db = m.expert_product_backward(dy, x, w, offsets)
    want, size = P.input_grad(dy, w, offsets)
    agrees("dx", dx, want, bound(out, size, dtype, dtype), dtype)
    want, size, db64, dbs, count = P.weight_grad(dy, x, offsets)
    agrees("dweight", dw, want, bound(max(count), size, dtype, dtype), torch.float32)
    check("dbias", db, db64, (max(count) + 2) * U * dbs)


@pytest.mark.parametrize("n,width,out", SIZES)
def test_products_just_below_the_largest(m, n, width, out):
    """Two values whose first terms' product is 2^128, but not their own."""
    g, c, o, r = rng(n + out), width // 2, out - 1, n // 3
    x, w, dy = rows(g, n, width), normal(g, 2, out, width), rows(g, n, out)
    near = (2 - 2.0 ** -12) * 2.0 ** 63
    x[r, c], w[:, o, c], dy[r, o] = near, near, near
    offsets, b = ends([n // 2, n - n // 2]), normal(g, 2, out)
    f32 = torch.float32
    for act in ("none", "silu"):
        want, size = P.product(x, w, offsets, b, act, n)
        assert 0.999 * TOP < want[r, o] < TOP
        agrees("y", m.expert_product(x, w, offsets, b, act=act), want, act_bound(bound(width, size, f32, f32), want, act), f32)
    dx, dw, _ = m.expert_product_backward(dy, x, w, offsets)
    want, size = P.input_grad(dy, w, offsets)
    agrees("dx", dx, want, bound(out, size, f32, f32), f32)
    want, size, _, _, count = P.weight_grad(dy, x, offsets)
    agrees("dweight", dw, want, bound(max(count), size, f32, f32), f32)


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "micro"])
@pytest.mark.parametrize("rows_at,weights_at", [(1e25, 1e25), (1e10, 2.0 ** 110), (2.0 ** 110, 1e10)])
@pytest.mark.parametrize("n,width,out", SIZES)
def test_products_by_held_weights_that_overflow(m, n, width, out, rows_at, weights_at, kind):
    g, c = rng(n + out), width - 1
    dtype = torch.float32 if kind == "float32" else torch.bfloat16
    x, w = rows(g, n, width, dtype), normal(g, 2 * out, width)
    x[::3, c], w[:out // 2, c] = large(g, len(x[::3]), at=rows_at, dtype=dtype), -large(g, out // 2, at=weights_at, dtype=torch.float32)
    held, offsets = m.micro_save(w), ends([n // 2, n - n // 2])
    taken = m.micro_save(x) if kind == "micro" else x
    x64 = P.micro_load(taken.codes, taken.scales, width) if kind == "micro" else f64(x)
    want, size = P.product(x64, P.micro_load(held.codes, held.scales, width).reshape(2, out, width), offsets, None, "none", n)
    for t in TYPES:
        agrees("y", m.micro_product(taken, held, offsets, dtype=t), want, bound(width, size, dtype, torch.bfloat16), t)


def same_places(name, got, want, b, dtype=torch.float32):
    """Not-a-numbers and infinities where 64 bits have them, the others within the bound."""
    got64, fine = f64(got), want.isfinite()
    assert torch.equal(got64.isnan(), want.isnan()) and torch.equal(got64[want.isinf()], want[want.isinf()]), name
    check(name, torch.where(fine, got64, 0.0), torch.where(fine, want, 0.0), torch.where(fine, b, 0.0), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("by_source", [False, True])
@pytest.mark.parametrize("n,width,out", SIZES + [(2000, 264, 136), (2200, 136, 800)])
def test_values_that_are_not_finite_in_tiles(m, n, width, out, by_source, dtype):
    """Infinities and NaN in an expert's first and last rows, in last columns and weights: where the formula has them (0 times an
    infinity is not a number), in their rows, columns and experts alone."""
    g, inf, nan = rng(n + width), float("inf"), float("nan")
    x, w, dy = rows(g, n, width, dtype), normal(g, 3, out, width, dtype=dtype), rows(g, n, out, dtype)
    cut = [2, 2 + n // 3, 2 + n // 3, n - 5]
    offsets = torch.tensor(cut, dtype=torch.int32, device=DEV)
    x[:2], x[-5:], dy[:2], dy[-5:] = nan, inf, inf, nan              # rows of no expert
    source = torch.randperm(n, generator=g).to(torch.int32).to(DEV) if by_source else torch.arange(n, dtype=torch.int32, device=DEV)
    xs = x.clone()                                                   # sorted
    xs[cut[0], width - 1], xs[cut[1] - 1, 0], xs[cut[3] - 1, width // 2] = inf, nan, -inf
    xs[cut[2] + 1, 3] = 0.0
    w[0, out - 1, 1], w[2, 4, width - 1], w[2, 5, 3] = -inf, nan, inf
    w[1] = nan                                                       # of the expert without rows
    dy[cut[0], 7], dy[cut[1] - 1, out - 1], dy[cut[3] - 1, 0] = inf, -inf, nan
    x[source.long()] = xs
    given = {"source": source} if by_source else {}
    x64, w64, dy64 = f64(xs), f64(w), f64(dy)
    y64, dx64, b64 = torch.zeros(n, out, dtype=torch.float64), torch.zeros(n, width, dtype=torch.float64), [torch.zeros(n, v, dtype=torch.float64) for v in (out, width)]
    dw64, db64, dws, dbs = [], [], [], []
    for e, r in P.segments(offsets, n):
        y64[r], b64[0][r] = x64[r] @ w64[e].T, x64[r].abs() @ w64[e].abs().T
        dx64[r], b64[1][r] = dy64[r] @ w64[e], dy64[r].abs() @ w64[e].abs()
        dw64.append(dy64[r].T @ x64[r]), dws.append(dy64[r].abs().T @ x64[r].abs())
        db64.append(dy64[r].sum(0)), dbs.append(dy64[r].abs().sum(0))
    same_places("y", m.expert_product(x, w, offsets, **given), y64, bound(width, b64[0], dtype, dtype), dtype)
    dx, dw, db = m.expert_product_backward(dy, x, w, offsets, **given)
    same_places("dx", dx, dx64, bound(out, b64[1], dtype, dtype), dtype)
    same_places("dweight", dw, torch.stack(dw64), bound(n, torch.stack(dws), dtype, dtype))
    same_places("dbias", db, torch.stack(db64), (n + 2) * U * torch.stack(dbs))


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("n,width,out", SIZES)
def test_values_that_round_to_an_infinity(m, n, width, out, act):
    """fp32 values above bf16's largest, in sums that fit: their results, with bias and activation, and both gradients."""
    g, f32, huge = rng(3 * n + out), torch.float32, 3.395e38
    x, w, dy = rows(g, n, width), (torch.rand(2, out, width, generator=g) * 1.8 - 0.9).to(DEV), rows(g, n, out)
    offsets, bias = ends([n // 2, n - n // 2]), normal(g, 2, out)
    for r, q in ((1, 3), (n - 1, n - 4)):
        x[r, width - 1], dy[q, out // 2] = huge, -huge
        dy[r], x[q] = (torch.rand(out, generator=g) * 1.8 - 0.9).to(DEV), (torch.rand(width, generator=g) * 1.8 - 0.9).to(DEV)
    want, size = P.product(x, w, offsets, bias, act, n)
    assert int((want.abs() > 1e37).sum()) > out // 4
    agrees("y", m.expert_product(x, w, offsets, bias, act=act), want, act_bound(bound(width, size, f32, f32), want, act), f32)
    held = m.micro_save(w.reshape(-1, width))
    w64 = P.micro_load(held.codes, held.scales, width).reshape(w.shape)
    want, size = P.product(x, w64, offsets, bias, act, n)
    b = act_bound(bound(width, size, f32, torch.bfloat16), want, act)
    for t in TYPES:
        agrees("y by held weights", m.micro_product(x, held, offsets, bias, act=act, dtype=t), want, b, t)
    dx, dw, _ = m.expert_product_backward(dy, x, w, offsets)
    want, size = P.input_grad(dy, w, offsets)
    assert int((want.abs() > 1e37).sum()) > width // 4
    agrees("dx", dx, want, bound(out, size, f32, f32), f32)
    want, size, _, _, count = P.weight_grad(dy, x, offsets)
    assert int((want.abs() > 1e37).sum()) > (width + out) // 4
    agrees("dweight", dw, want, bound(max(count), size, f32, f32), f32)


# ---------------------------------------------------------------------------------------------------------------
# embedding rows
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 5, 40, 136])
@pytest.mark.parametrize("ends", [[10, 500, 1000], [30, 31, 31, 900], [64, 1000], [200, 1000], [63, 129, 700], [65, 130, 140], [700, 1000], [960, 1000],
                                  [999, 1000], [1000, 1000], [300, 600, 2000], [-5, -3, 70, 800], [64, 128, 193, 193, 1000]])
def test_embed_gradient_of_entries_from_later_places_on(m, ends, width, dtype):
    """Rows before the first entry's are no entry's, wherever it starts in a window of 64 places; what earlier calls left in the
    scratch reaches nothing."""
    g, n = rng(width + ends[0]), 1000
    source = torch.randperm(n, generator=g).to(torch.int32).to(DEV)
    dout = normal(g, n, width, dtype=dtype)
    whole = torch.tensor([0, n // 3, n], dtype=torch.int32, device=DEV)
    m.embed_backward(torch.full_like(dout, float("nan")), whole, source)
    cut = [min(max(v, 0), n) for v in ends]
    kept = dout.clone()
    dout[source[:cut[0]].long()], dout[source[cut[-1]:].long()] = float("nan"), float("nan")
    got = m.embed_backward(dout, torch.tensor(ends, dtype=torch.int32, device=DEV), source, -0.5)
    d = f64(kept)[source.cpu().long()]
    want, size = (torch.stack([v[a:b].sum(0) for a, b in zip(cut, cut[1:])]) * s for v, s in ((d, -0.5), (d.abs(), 0.5)))
    check("dtable", got, want, (n + 2) * U * size)


@pytest.mark.parametrize("dtype", TYPES)
def test_embed_gradient_of_a_shard(m, dtype):
    """A slice of the plan's offsets gives those entries' gradients, the same bits."""
    g, n, entries = rng(4), 30000, 40
    index = (torch.rand(n, generator=g) ** 3 * (entries + 2) - 1).floor().to(torch.int32).to(DEV)
    offsets, source = m.embed_plan(index, entries)
    dout = normal(g, n, 72, dtype=dtype)
    whole = m.embed_backward(dout, offsets, source, 1.5)
    for a, b in ((0, 1), (1, 2), (1, 40), (2, 9), (7, 40), (39, 40)):
        m.embed_backward(torch.full_like(dout, float("nan")), offsets, source)
        assert torch.equal(m.embed_backward(dout, offsets[a:b + 1], source, 1.5), whole[a:b]), (a, b)


def test_embed_of_as_many_rows_as_there_may_be(m):
    """2^31 - 1 rows: places next to the end of 32 bits, sums of small whole numbers (exact)."""
    n, tail = 2 ** 31 - 1, 200000
    index = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    last = torch.zeros(tail, dtype=torch.int32)
    last[-60:-1], last[-1] = 1, 2
    index[-tail:] = last.to(DEV)
    table = torch.tensor([[2.0], [3.0], [5.0]], dtype=torch.bfloat16, device=DEV)
    out = m.embed(index, table)
    assert torch.equal(out[-tail:].cpu(), table.cpu()[last.long()]) and float(out[:1000].abs().max()) == 0
    # the plan puts the rows of no entry last; offsets of the same rows in their own order put the entries last
    offsets, source = m.embed_plan(index, 3)
    assert offsets.tolist() == [0, tail - 60, tail - 1, tail]
    assert torch.equal(source[:tail], torch.arange(n - tail, n, dtype=torch.int32, device=DEV)) and int(source[-1]) == n - tail - 1
    out.zero_()
    values = (torch.arange(tail) % 7 - 2).to(torch.bfloat16)
    out[-tail:] = values.to(DEV).unsqueeze(1)
    want = torch.stack([v.double().sum() for v in (values[:-60], values[-60:-1], values[-1:])])
    assert torch.equal(f64(m.embed_backward(out, offsets, source))[:, 0], want)
    torch.arange(n, out=source)
    late = torch.tensor([n - tail, n - 60, n - 1, n], dtype=torch.int32, device=DEV)
    assert torch.equal(f64(m.embed_backward(out, late, source))[:, 0], want)
