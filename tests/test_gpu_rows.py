"""Row operators (rows by expert, norms around a gated residual block, 8-bit checkpoints, their weight gradient)
against plain 64-bit implementations, on the GPU.

Bounds: fp32 arithmetic adds at most U = 2^-24 of the magnitudes involved per operation.  A sum of m terms taken
lane by lane and then over lanes differs from the exact one by at most m U times the sum of magnitudes; each result
is rounded once more to its type."""
import numpy as np
import pytest
import torch

from molecular_dynamics_cell_amd import binding
from molecular_dynamics_cell_amd import inputs as I
from tests import rows_util as R
from tests.rows_util import U, check, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]
WIDTHS = [1, 3, 6, 30, 64, 108, 127, 312, 1000, 1024, 2048, 4096, 4100, 8192]


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


# ---------------------------------------------------------------------------------------------------------------
# rows by expert
# ---------------------------------------------------------------------------------------------------------------
def experts(g, n, k, E, how):
    e = torch.randint(0, E, (n, k), generator=g, dtype=torch.int32)
    if how == "dropped":
        e[torch.rand(n, k, generator=g) < 0.3] = -1
        e[torch.rand(n, k, generator=g) < 0.05] = E
        e[::5] = -7                                   # rows without any expert
    elif how == "none":
        e[:] = -1
    elif how == "one":
        e[:] = E - 1
    return e.to(DEV)


@pytest.mark.parametrize("n,k,E,how", [(0, 1, 3, "all"), (1, 1, 1, "all"), (1, 8, 64, "dropped"), (63, 1, 2, "all"), (65, 3, 7, "dropped"),
                                       (108, 2, 4, "all"), (4096, 1, 5, "dropped"), (4097, 1, 5, "one"), (1365, 3, 1024, "all"),
                                       (5000, 7, 33, "dropped"), (30011, 2, 300, "dropped"), (20000, 8, 1, "none"), (131072, 4, 64, "all"),
                                       (2000003, 1, 6, "dropped"), (300007, 8, 1024, "dropped")])
def test_plan(m, n, k, E, how):
    e = experts(rng(n + E), n, k, E, how)
    offsets, source, position = R.plan(e, E)
    got = m.route_plan(e, E)
    for a, b in zip(got, (offsets, source, position)):
        assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k,E,width,how", [(1, 1, 1, 1, "all"), (1, 8, 64, 4096, "dropped"), (108, 2, 4, 64, "dropped"),
                                             (257, 3, 5, 30, "dropped"), (130, 2, 5, 108, "all"), (77, 1, 5, 312, "dropped"),
                                             (33, 4, 9, 1000, "dropped"), (19, 6, 9, 1027, "all"), (5, 64, 70, 127, "dropped"),
                                             (9, 2, 3, 8193, "dropped"), (40, 2, 3, 3, "none"), (1025, 1, 2, 6, "one"), (3, 2, 2, 20000, "dropped")])
def test_there_and_back(m, n, k, E, width, how, dtype):
    g = rng(n * width + k)
    e = experts(g, n, k, E, how)
    x, weight = normal(g, n, width, dtype=dtype), normal(g, n, k)
    dout = normal(g, n, width, dtype=dtype)
    offsets, source, position = m.route_plan(e, E)
    used, pairs = int(offsets[-1]), n * k
    live = (position < used).cpu().unsqueeze(-1)
    rows = m.route_scatter(x, position, offsets)
    want = f64(x)[source.cpu().long() // k]
    want[used:] = 0
    assert torch.equal(f64(rows), want)
    # the experts' rows: what stands at dropped places and in dropped weights must not reach any sum
    y = normal(g, pairs, width, dtype=dtype)
    y[used:] = float("nan")
    weight[~live.squeeze(-1).to(DEV)] = float("inf")
    w64 = torch.where(live, f64(weight).unsqueeze(-1), 0.0)
    taken = torch.where(live, f64(y)[position.cpu().long()], 0.0)
    out = m.route_combine(y, position, offsets, weight)
    check("out", out, (taken * w64).sum(1), (k + 1) * U * (taken * w64).abs().sum(1), dtype)
    plain = m.route_combine(y, position, offsets)
    check("unweighted", plain, taken.sum(1), k * U * taken.abs().sum(1), dtype)
    assert torch.equal(plain[~live.any(1).squeeze(-1).to(DEV)].cpu(), torch.zeros(int((~live.any(1)).sum()), width, dtype=dtype))
    # gradient
    dy, dweight = m.route_combine_backward(dout, y, position, offsets, weight)
    want = torch.zeros(pairs, width, dtype=torch.float64)
    want[position.cpu().long().reshape(-1)] = (f64(dout).unsqueeze(1) * w64).reshape(pairs, width)
    check("dsorted", dy, want, U * want.abs(), dtype)
    terms = f64(dout).unsqueeze(1) * taken
    check("dweight", dweight, terms.sum(-1), (width + 1) * U * terms.abs().sum(-1))
    only, none = m.route_combine_backward(dout, None, position, offsets)
    want[position.cpu().long().reshape(-1)] = (f64(dout).unsqueeze(1) * live).reshape(pairs, width)
    assert none is None and torch.equal(f64(only), want)
    # differences: <dout, combine(y + t v, weight + t s)> is linear in each of y and weight
    v, s = torch.randn(pairs, width, generator=g, dtype=torch.float64), torch.randn(n, k, generator=g, dtype=torch.float64)
    s = s * live.squeeze(-1)

    def value(t):
        moved = torch.where(live, (torch.nan_to_num(f64(y)) + t * v)[position.cpu().long()], 0.0)
        return float((f64(dout).unsqueeze(1) * moved * (w64 + t * s.unsqueeze(-1))).sum())

    slope = (value(1.0) - value(-1.0)) / 2      # exact for a quadratic
    mine = float((f64(dy)[:used] * v[:used]).sum() + (f64(dweight) * s).sum())
    size = float((f64(dy)[:used] * v[:used]).abs().sum() + (terms.abs().sum(-1) * s.abs()).sum())
    assert abs(mine - slope) <= (2 * R.HALF[dtype] + (width + 1) * U) * size + 1e-12


def test_places_out_of_range_are_ignored(m):
    x = torch.ones(4, 16, device=DEV)
    position = torch.tensor([[0], [-5], [2], [1 << 30]], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    out = m.route_combine(x, position, offsets)
    assert torch.equal(out.cpu(), torch.tensor([1.0, 0.0, 1.0, 0.0]).unsqueeze(1).expand(4, 16))
    rows = m.route_scatter(x, position, offsets)
    dy, dw = m.route_combine_backward(x, x, position, offsets)
    assert torch.equal(rows[[0, 2]].cpu(), x[:2].cpu()) and torch.equal(dy[[0, 2]].cpu(), x[:2].cpu())
    assert dw.flatten().tolist() == [16.0, 0.0, 16.0, 0.0]


# ---------------------------------------------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------------------------------------------
VECTORS = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")
PLAIN = {"post_weight": 1.0, "post_bias": 0.0, "scale": 1.0, "pre_weight": 1.0, "pre_bias": 0.0}
EPS = 1e-5


def norm_inputs(g, n, width, dtype, gate, vectors):
    x, block = normal(g, n, width, dtype=dtype, size=2.0), normal(g, n, width, dtype=dtype, size=3.0, at=0.5)
    gate = {"none": None, "row": normal(g, n, 1, dtype=dtype), "element": normal(g, n, width, dtype=dtype, size=2.0)}[gate]
    w = {name: normal(g, width, size=0.3, at=0.0 if "bias" in name else 1.0) for name in VECTORS} if vectors else {}
    w64 = {name: f64(w[name]) if vectors else PLAIN[name] for name in VECTORS}
    return x, block, gate, w, w64


def hat_error(v, hat, inv, width):
    """Error of a normed value: mean and mean square are sums of `width` terms, then a handful of operations."""
    return (width + 16) * U * (inv * v.abs().mean(-1, keepdim=True) + inv * v.abs() + hat.abs())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,gate,vectors", [("rms", "element", True), ("layer", "row", True), ("layer", "none", False)])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("n", [1, 37])
def test_norm_residual(m, n, width, kind, gate, vectors, dtype):
    g = rng(n + width)
    x, block, gate, w, w64 = norm_inputs(g, n, width, dtype, gate, vectors)
    block[n // 2] = 0                              # a row of zeros: N is 0, or the bias
    layer = kind == "layer"
    r, h = m.norm_residual(x, block, gate, **w, kind=kind, eps=EPS)
    r64, h64 = R.residual(f64(x), f64(block), f64(gate), w64, layer, EPS)
    hat, inv = R.normed(f64(block), layer, EPS)
    sig = 1.0 if gate is None else torch.sigmoid(f64(gate))
    added = torch.as_tensor(w64["scale"]).abs() * sig
    pw, pb = (torch.as_tensor(w64[k], dtype=torch.float64).abs() for k in ("post_weight", "post_bias"))
    er = added * (hat_error(f64(block), hat, inv, width) * pw + 16 * U * (hat.abs() * pw + pb)) + 2 * U * (f64(x).abs() + r64.abs())
    check("r", r, r64, er, dtype)
    rhat, rinv = R.normed(r64, layer, EPS)
    eh = hat_error(r64, rhat, rinv, width) + rinv * (er + er.mean(-1, keepdim=True)) + rhat.abs() * rinv * er.mean(-1, keepdim=True) * 4
    qw = torch.as_tensor(w64["pre_weight"], dtype=torch.float64).abs()
    check("h", h, h64, eh * qw + 4 * U * (h64.abs() + torch.as_tensor(w64["pre_bias"]).abs()), dtype)
    # a norm alone; the sum alone
    same, alone = m.norm_residual(x, pre_weight=w.get("pre_weight"), pre_bias=w.get("pre_bias"), kind=kind, eps=EPS)
    xhat, xinv = R.normed(f64(x), layer, EPS)
    want = xhat * w64["pre_weight"] + w64["pre_bias"]
    check("h of x", alone, want, hat_error(f64(x), xhat, xinv, width) * qw + 4 * U * want.abs(), dtype)
    assert torch.equal(same, x)
    only, none = m.norm_residual(x, block, gate, **w, kind=kind, eps=EPS, want_h=False)
    assert none is None
    check("r alone", only, r64, er, dtype)


def norm_gradient(x64, dr, dh, r, block, gate, w, layer):
    """Gradients and, for each, the sum of magnitudes behind it (both 64 bits)."""
    rhat, rinv = R.normed(r, layer, EPS)
    total, size = torch.zeros_like(r), torch.zeros_like(r)
    if dr is not None:
        total, size = total + dr, size + dr.abs()
    if dh is not None:
        total = total + R.normed_back(dh * w["pre_weight"], rhat, rinv, layer)
        size = size + R.normed_back_size((dh * w["pre_weight"]).abs(), rhat, rinv) * (1 + rinv * r.abs().mean(-1, keepdim=True))
    hat, inv = R.normed(block, layer, EPS)
    sig = torch.ones(1, dtype=torch.float64) if gate is None else torch.sigmoid(gate)
    u = hat * w["post_weight"] + w["post_bias"]
    us = hat.abs() * torch.as_tensor(w["post_weight"]).abs() + torch.as_tensor(w["post_bias"]).abs() + inv * block.abs().mean(-1, keepdim=True)
    s = torch.as_tensor(w["scale"], dtype=torch.float64)
    pw = torch.as_tensor(w["post_weight"], dtype=torch.float64)
    du, dus = total * s * sig, size * s.abs() * sig
    out = {"dx": (total, size),
           "dblock": (R.normed_back(du * pw, hat, inv, layer),
                      R.normed_back_size(dus * pw.abs(), hat, inv) * (1 + inv * block.abs().mean(-1, keepdim=True)))}
    if gate is not None:
        d, ds = total * s * u * sig * (1 - sig), size * s.abs() * us * sig
        out["dgate"] = (d.sum(-1, keepdim=True), ds.sum(-1, keepdim=True)) if gate.shape[1] == 1 and r.shape[1] > 1 else (d, ds)
    hs = hat.abs() + inv * block.abs().mean(-1, keepdim=True)
    out["dpost_weight"] = ((du * hat).sum(0), (dus * hs).sum(0))
    out["dpost_bias"] = (du.sum(0), dus.sum(0))
    out["dscale"] = ((total * sig * u).sum(0), (size * sig * us).sum(0))
    if dh is not None:
        out["dpre_weight"] = ((dh * rhat).sum(0), (dh.abs() * (rhat.abs() + rinv * r.abs().mean(-1, keepdim=True))).sum(0))
        out["dpre_bias"] = (dh.sum(0), dh.abs().sum(0))
    return out


NAMES = ("dx", "dblock", "dgate", "dpost_weight", "dpost_bias", "dscale", "dpre_weight", "dpre_bias")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,gate,vectors,given", [("rms", "element", True, "both"), ("layer", "row", True, "both"),
                                                     ("layer", "none", False, "dh"), ("rms", "element", True, "dr")])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("n", [1, 67])
def test_norm_residual_backward(m, n, width, kind, gate, vectors, given, dtype):
    g = rng(n + width)
    r, block, gate, w, w64 = norm_inputs(g, n, width, dtype, gate, vectors)
    layer = kind == "layer"
    dr = normal(g, n, width, dtype=dtype) if given != "dh" else None
    dh = normal(g, n, width, dtype=dtype) if given != "dr" else None
    got = dict(zip(NAMES, m.norm_residual_backward(dr, dh, r, block, gate, **w, kind=kind, eps=EPS)))
    want = norm_gradient(None, f64(dr), f64(dh), f64(r), f64(block), f64(gate), w64, layer)
    for name in NAMES:
        if name not in want:
            assert got[name] is None
            continue
        value, size = want[name]
        rowwise = name in ("dx", "dblock", "dgate")
        terms = 4 * width + 64 + (0 if rowwise else n)
        check(name, got[name], value, terms * U * size, dtype if rowwise else torch.float32)
    # a norm alone
    if dh is not None:
        dx, a, b, c, d, e, dpw, dpb = m.norm_residual_backward(dr, dh, r, pre_weight=w.get("pre_weight"), kind=kind, eps=EPS)
        assert (a, b, c, d, e) == (None,) * 5
        check("dx alone", dx, want["dx"][0], (4 * width + 64) * U * want["dx"][1], dtype)
        for name, v in (("dpre_weight", dpw), ("dpre_bias", dpb)):
            check(name, v, want[name][0], (4 * width + 64 + n) * U * want[name][1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,width", [(3, 1400), (5, 2600), (2, 6144), (1300, 1400), (700, 5000), (600, 8192), (9000, 96)])
def test_norms_of_wide_and_many_rows(m, n, width, dtype):
    """Rows of every number of waves, and more rows than groups run at once."""
    test_norm_residual(m, n, width, "layer", "element", True, dtype)
    test_norm_residual_backward(m, n, width, "rms", "element", True, "both", dtype)
    test_norm_residual_backward(m, n, width, "layer", "row", True, "both", dtype)


@pytest.mark.parametrize("kind,gate", [("rms", "element"), ("layer", "row"), ("layer", "none")])
def test_norm_gradient_against_differences(m, kind, gate):
    """Central differences of the 64-bit forward pass along random directions, for each input in turn."""
    n, width, layer = 9, 108, kind == "layer"
    g = rng(5)
    x, block, gate, w, w64 = norm_inputs(g, n, width, torch.float32, gate, True)
    at = {"x": f64(x), "block": f64(block), **w64}
    if gate is not None:
        at["gate"] = f64(gate)

    def forward(v):
        return R.residual(v["x"], v["block"], v.get("gate"), {k: v[k] for k in VECTORS}, layer, EPS)

    dr, dh = normal(g, n, width), normal(g, n, width)
    r = forward(at)[0].float().to(DEV)
    got = dict(zip(NAMES, m.norm_residual_backward(dr, dh, r, block, gate, **w, kind=kind, eps=EPS)))
    for name in at:
        v = torch.randn(at[name].shape, generator=g, dtype=torch.float64)

        def value(t):
            a, b = forward({**at, name: at[name] + t * v})
            return float((a * f64(dr)).sum() + (b * f64(dh)).sum())

        h = 1e-4      # error of the difference: h^2 of third derivatives, and 1e-16 / h of the values
        slope = (value(h) - value(-h)) / (2 * h)
        mine = float((f64(got["d" + name]) * v).sum())
        size = float((f64(got["d" + name]) * v).abs().sum())
        assert abs(mine - slope) <= 2e-6 * size + 1e-9, (name, mine, slope, size)


def test_norm_rows_that_are_not_finite_stay_apart(m):
    g = rng(3)
    x, block, gate, w, _ = norm_inputs(g, 40, 312, torch.float32, "element", True)
    clean = m.norm_residual(x, block, gate, **w, eps=EPS)
    block[7, 5], block[9, 0], x[11, 311] = float("nan"), float("inf"), float("nan")
    gate[13], gate[14] = float("inf"), float("-inf")
    r, h = m.norm_residual(x, block, gate, **w, eps=EPS)
    for row, out in ((7, r), (9, r), (7, h), (9, h), (11, h)):
        assert out[row].isnan().any()
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[[7, 9, 11, 13, 14]] = False
    assert torch.equal(r[keep], clean[0][keep]) and torch.equal(h[keep], clean[1][keep])
    assert torch.equal(r[14], x[14]) and r[13].isfinite().all() and h[13:15].isfinite().all()
    dx, dblock, dgate, *_ = m.norm_residual_backward(x, x, x, block, gate, **w, eps=EPS)
    assert (dgate[13:15] == 0).all() and (dblock[14] == 0).all() and dx[keep].isfinite().all() and dblock[keep].isfinite().all()


# ---------------------------------------------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,width", [(1, 1), (1, 4096), (3, 31), (5, 32), (7, 33), (108, 64), (65, 108), (33, 312), (17, 127), (9, 1000),
                                     (4, 8192), (2, 20001), (3000, 6)])
def test_checkpoint(m, n, width, dtype):
    g = rng(n * width)
    x = normal(g, n, width, dtype=dtype) * torch.exp(3 * normal(g, n, 1)).to(dtype)
    codes, scales = R.save(x)
    held = m.checkpoint_save(x)
    assert np.array_equal(held.codes.cpu().numpy(), codes) and np.array_equal(held.scales.cpu().numpy(), scales)
    back = R.load(codes, scales)
    for t in TYPES:
        assert torch.equal(f64(m.checkpoint_load(held, t)), back)
    groups = torch.nn.functional.pad(f64(x).abs(), (0, -width % 32)).reshape(n, -1, 32).amax(-1)
    assert ((back - f64(x)).abs() <= groups.repeat_interleave(32, 1)[:, :width] / 127).all()
    # with silu, and its gradient
    dy = normal(g, n, width, dtype=dtype)
    y, z_held, y_held = m.checkpoint_silu(x, save_output=True)
    y2, z2, none = m.checkpoint_silu(x)
    assert none is None and torch.equal(y, y2)
    for a in (z_held, z2):
        assert np.array_equal(a.codes.cpu().numpy(), codes) and np.array_equal(a.scales.cpu().numpy(), scales)
    y64 = R.silu(f64(x))
    # exp(-z) is off by U |z| for its argument's rounding and a few U of its own
    ey = (f64(x).abs() + 8) * U * y64.abs() + 2.0 ** -121   # exp(88.8) is infinite: y is 0 there, not 2.6e-37
    check("y", y, y64, ey, dtype)
    yback = R.load(y_held.codes.cpu(), y_held.scales.cpu())
    step = torch.from_numpy(np.exp2(y_held.scales.cpu().numpy().astype(np.float64) - 127)).repeat_interleave(32, 1)[:, :width]
    assert ((yback - y64).abs() <= step / 2 + ey + 2.0 ** -100).all()
    largest = torch.nn.functional.pad(y64.abs(), (0, -width % 32)).reshape(n, -1, 32).amax(-1).repeat_interleave(32, 1)[:, :width]
    assert (step <= largest / 63.4 + 2.0 ** -100).all()
    dz = m.checkpoint_silu_backward(dy, held)
    slope = R.silu_slope(back)
    sig = torch.sigmoid(back)
    size = f64(dy).abs() * sig * (1 + back.abs() * (1 - sig))
    check("dz", dz, f64(dy) * slope, (back.abs() + 12) * U * size + 2.0 ** -118, dtype)
    h = 1e-5      # the difference is off by h^2 of third derivatives and 2^-52 |z| / h
    check("differences", dz, f64(dy) * (R.silu(back + h) - R.silu(back - h)) / (2 * h),
          (1e-9 + 1e-10 * back.abs()) * f64(dy).abs() + (back.abs() + 12) * U * size + 2.0 ** -118, dtype)


def test_checkpoint_extremes(m):
    top = float(np.finfo(np.float32).max)
    rows = torch.zeros(14, 64)
    for i, v in enumerate([0.0, 1e-45, 1e-38, 2.0 ** -101, 2.0 ** -100, 2.0 ** -95, 1.984375, 1.9843751, 127.0, 2.0 ** 126, top]):
        rows[i, :32] = v * torch.linspace(-1, 1, 32)
        rows[i, 31] = v
    rows[11, 3], rows[12, 40], rows[13, 0] = float("nan"), float("inf"), float("-inf")
    rows[11, 32:], rows[12, :32] = 1.0, -2.0
    x = rows.to(DEV)
    codes, scales = R.save(x)
    held = m.checkpoint_save(x)
    assert np.array_equal(held.codes.cpu().numpy(), codes) and np.array_equal(held.scales.cpu().numpy(), scales)
    back = f64(m.checkpoint_load(held))
    assert back[:11].isfinite().all()
    assert back[11, :32].isnan().all() and (back[11, 32:] == 1).all() and back[12, 32:].isnan().all() and (back[12, :32] == -2).all()
    assert back[13, :32].isnan().all() and (back[13, 32:] == 0).all()
    y, z_held, y_held = m.checkpoint_silu(x, save_output=True)
    assert np.array_equal(z_held.scales.cpu().numpy(), scales) and y[:11].isfinite().all()
    dz = m.checkpoint_silu_backward(torch.ones_like(x), held)
    assert dz[:11].isfinite().all() and dz[11, :32].isnan().all() and (dz[11, 32:] - 0.9276705).abs().max() < 1e-5


WEIGHT_GRADS = [(0, 8, 8, [0, 0]), (1, 1, 1, [1]), (5, 3, 30, [2, 0, 3]), (64, 64, 64, [64]), (108, 64, 108, [50, 58]), (300, 33, 65, [300]),
                (1000, 128, 312, [1, 0, 599, 400]), (777, 17, 127, [100, 0, 0, 677]), (5000, 130, 40, [4999, 1]), (640, 256, 96, [640]),
                (2050, 1, 1000, [2050]), (2050, 1000, 3, [1025, 1025]), (900, 260, 520, [30] * 30), (40000, 64, 108, [30000, 10000])]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,out,width,counts", WEIGHT_GRADS)
def test_weight_grad(m, n, out, width, counts, dtype):
    g = rng(n + out + width)
    dy = normal(g, n, out, dtype=dtype)
    x = normal(g, n, width) * torch.exp(normal(g, n, 1))
    held = m.checkpoint_save(x)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    dweight, dbias = m.checkpoint_weight_grad(dy, held, offsets)
    x64, dy64 = R.load(held.codes.cpu(), held.scales.cpu()), f64(dy)
    at = 0
    for e, c in enumerate(counts):
        a, b = dy64[at:at + c], x64[at:at + c]
        at += c
        check("dweight", dweight[e], a.T @ b, (c + 8) * U * (a.abs().T @ b.abs()))
        check("dbias", dbias[e], a.sum(0), (c + 8) * U * a.abs().sum(0))
    again = m.checkpoint_weight_grad(dy, held, offsets)
    assert torch.equal(again[0], dweight) and torch.equal(again[1], dbias)


@pytest.mark.parametrize("n,out,width,experts_", [(600, 1030, 1030, 7), (1100, 1024, 1024, 8), (500, 130, 1000, 64), (400, 40, 200, 66),
                                                  (300, 300, 140, 1)])
def test_weight_grad_experts_of_unlike_length(m, n, out, width, experts_):
    """One piece an expert: the order in which experts start changes no result, empty ones and equal lengths included."""
    g = rng(n + experts_)
    share = torch.rand(experts_, generator=g, dtype=torch.float64).pow(3)
    share[experts_ // 2] = 0.0 if experts_ > 1 else 1.0
    ends = torch.round(torch.cumsum(share, 0) / share.sum() * n).long()
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), ends]).to(DEV, torch.int32)
    dy, held = normal(g, n, out, dtype=torch.bfloat16), m.checkpoint_save(normal(g, n, width))
    dweight, dbias = m.checkpoint_weight_grad(dy, held, offsets)
    x64, dy64 = R.load(held.codes.cpu(), held.scales.cpu()), f64(dy)
    for e in range(experts_):
        a, b = dy64[offsets[e]:offsets[e + 1]], x64[offsets[e]:offsets[e + 1]]
        check("dweight", dweight[e], a.T @ b, (len(a) + 8) * U * (a.abs().T @ b.abs()))
        check("dbias", dbias[e], a.sum(0), (len(a) + 8) * U * a.abs().sum(0))


def test_weight_grad_special_values(m):
    """A held NaN reaches its column only, a row outside every segment nothing; differences of a loss."""
    g = rng(9)
    n, out, width = 200, 24, 70
    dy, x = normal(g, n, out), normal(g, n, width)
    x[150, 40] = float("nan")                          # its group of columns 32 .. 63 reads back as NaN
    x[5, 3], dy[195] = float("nan"), float("inf")      # rows of no expert
    held = m.checkpoint_save(x)
    offsets = torch.tensor([10, 100, 190], dtype=torch.int32, device=DEV)
    dweight, dbias = m.checkpoint_weight_grad(dy, held, offsets)
    bad = dweight.isnan().cpu()
    assert bad[1, :, 32:64].all() and int(bad.sum()) == out * 32 and dbias.isfinite().all()
    x64, dy64 = R.load(held.codes.cpu(), held.scales.cpu()), f64(dy)
    # L(W) = sum of dy . (x W^T) over expert 0 is linear in W: a difference along V is exact
    V = torch.randn(out, width, generator=g, dtype=torch.float64)
    slope = float((dy64[10:100] * (x64[10:100] @ V.T)).sum())
    size = float((dy64[10:100].abs() * (x64[10:100].abs() @ V.abs().T)).sum())
    assert abs(float((f64(dweight[0]) * V).sum()) - slope) <= 98 * U * size
    check("dbias", dbias[0], dy64[10:100].sum(0), 98 * U * dy64[10:100].abs().sum(0))


# ---------------------------------------------------------------------------------------------------------------
# layouts, streams, graphs, long arrays
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,pad,shift", [(64, 64, 0), (108, 20, 4), (64, 1, 1), (312, 9, 3), (33, 7, 2), (1024, 1024, 0)])
def test_strided_rows(m, width, pad, shift, dtype):
    """Column blocks of a wider tensor, aligned or not, give the dense rows' results bit for bit."""
    g = rng(width)
    n, k = 50, 2
    e = experts(g, n, k, 3, "dropped")
    offsets, source, position = m.route_plan(e, 3)

    def pair():
        wide = normal(g, n, width + pad + shift, dtype=dtype)
        part = wide[:, shift:shift + width]
        return part, part.contiguous()

    (x, xd), (b, bd), (t, td), (dy, dyd) = pair(), pair(), pair(), pair()
    y = normal(g, n * k, width, dtype=dtype)
    assert torch.equal(m.route_scatter(x, position, offsets), m.route_scatter(xd, position, offsets))
    a, b2 = m.route_combine_backward(dy, y, position, offsets), m.route_combine_backward(dyd, y, position, offsets)
    assert torch.equal(a[0], b2[0])
    check("dweight", a[1], f64(b2[1]), 1e-4 * width ** 0.5)
    tol = dict(rtol=1e-2 if dtype == torch.bfloat16 else 1e-5, atol=1e-2 if dtype == torch.bfloat16 else 1e-5)
    for p, q in zip(m.norm_residual(x, b, t, kind="layer"), m.norm_residual(xd, bd, td, kind="layer")):
        assert torch.allclose(p.float(), q.float(), **tol)
    for p, q in zip(m.norm_residual_backward(dyd, xd, x, b, t), m.norm_residual_backward(dyd, xd, xd, bd, td)):
        assert torch.allclose(p.float(), q.float(), rtol=tol["rtol"], atol=10 * tol["atol"])
    for p, q in zip(m.checkpoint_save(x), m.checkpoint_save(xd)):
        assert torch.equal(p, q)
    held = m.checkpoint_save(x)
    for p, q in zip(m.checkpoint_silu(x)[1], held):
        assert torch.equal(p, q)
    assert torch.equal(m.checkpoint_silu_backward(dy, held), m.checkpoint_silu_backward(dyd, held))
    seg = torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    for p, q in zip(m.checkpoint_weight_grad(dy, held, seg), m.checkpoint_weight_grad(dyd, held, seg)):
        assert torch.allclose(p, q, rtol=1e-4, atol=1e-4)


def test_in_place(m):
    g = rng(2)
    x, block, gate, w, _ = norm_inputs(g, 100, 108, torch.float32, "element", True)
    p, kept = m._norm(x, 108, gate, "rms", EPS, [(k, w[k]) for k in VECTORS])
    r, h = m.norm_residual(x, block, gate, **w, eps=EPS)
    dr, dh = normal(g, 100, 108), normal(g, 100, 108)
    got = m.norm_residual_backward(dr, dh, r, block, gate, **w, eps=EPS)
    L, h2, db, dg = binding.lib(), torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    import ctypes as C
    inplace = x.clone()
    assert L.mpnn_norm_residual(m.h, C.byref(p), 100, inplace.data_ptr(), 108, block.data_ptr(), 108, gate.data_ptr(), 108,
                                inplace.data_ptr(), h2.data_ptr()) == 0
    assert L.mpnn_norm_residual_backward(m.h, C.byref(p), 100, dr.data_ptr(), dh.data_ptr(), r.data_ptr(), 108, block.data_ptr(), 108,
                                         gate.data_ptr(), 108, dr.data_ptr(), db.data_ptr(), dg.data_ptr(), None, None, None, None, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(inplace, r) and torch.equal(h2, h)
    assert torch.equal(dr, got[0]) and torch.equal(db, got[1]) and torch.equal(dg, got[2])


def test_other_stream(m):
    """Tensors made on a side stream behind a long-running producer, used there right after."""
    g = rng(4)
    n, width = 4000, 312
    x, e = normal(g, n, width), experts(g, n, 2, 5, "dropped")
    offsets, source, position = m.route_plan(e, 5)
    want = m.route_combine(m.route_scatter(x * 3, position, offsets), position, offsets)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big = torch.randn(4096, 4096, device=DEV)
            for _ in range(20):
                big = big @ big * 1e-2
            y = x * 3
            got = m.route_combine(m.route_scatter(y, position, offsets), position, offsets)
            del y
            out = got + 0
        side.synchronize()
        assert torch.equal(out, want)


def test_graph_replays(m):
    """Every call captured once and replayed with new inputs between eager work."""
    g = rng(6)
    n, k, E, width = 9000, 2, 6, 108
    e = experts(g, n, k, E, "dropped")
    x, block, gate, w, _ = norm_inputs(g, n, width, torch.float32, "element", True)
    weight, dy = normal(g, n, k), normal(g, n * k, 64)

    def step():
        offsets, source, position = m.route_plan(e, E)
        rows = m.route_scatter(x, position, offsets)
        y, zh, yh = m.checkpoint_silu(rows, save_output=True)
        out = m.route_combine(y, position, offsets, weight)
        r, h = m.norm_residual(x, out, gate, **w)
        back = m.norm_residual_backward(h, r, r, out, gate, **w)
        dsorted, dweight = m.route_combine_backward(back[1], y, position, offsets, weight)
        dz = m.checkpoint_silu_backward(dsorted, zh)
        return [offsets, source, position, out, r, h, *back, dweight, dz, *m.checkpoint_weight_grad(dy, yh, offsets)]

    step()
    home = m._stream
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    try:
        with torch.cuda.graph(graph):
            m.set_stream(torch.cuda.current_stream())
            kept = step()
    finally:
        m.set_stream(home)
    for seed in range(4):
        g2 = rng(100 + seed)
        e.copy_(experts(g2, n, k, E, "dropped"))
        x.copy_(normal(g2, n, width))
        weight.copy_(normal(g2, n, k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        for a, b in zip(got, step()):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())


def test_long_arrays(m):
    """More than 2^32 bytes and 2^31 values: the last rows are right."""
    n, width = 270011, 8192
    x = torch.empty(n, width, dtype=torch.bfloat16, device=DEV)
    x.copy_((torch.arange(n, device=DEV) % 251).unsqueeze(1) + (torch.arange(width, device=DEV) % 3).unsqueeze(0))
    e = torch.ones(n, 1, dtype=torch.int32, device=DEV)
    e[-1] = 0
    offsets, source, position = m.route_plan(e, 2)
    rows = m.route_scatter(x, position, offsets)
    assert torch.equal(rows[0], x[-1]) and torch.equal(rows[1:][-5:], x[-6:-1]) and torch.equal(rows[-1], x[-2])
    out = m.route_combine(rows, position, offsets)
    assert torch.equal(out[-100:], x[-100:]) and torch.equal(out[:5], x[:5])
    del rows, out
    tail = x[-64:].contiguous()
    held, some = m.checkpoint_save(x), m.checkpoint_save(tail)
    assert torch.equal(held.codes[-64:], some.codes) and torch.equal(held.scales[-64:], some.scales)
    r, h = m.norm_residual(x, x)
    r2, h2 = m.norm_residual(tail, tail)
    close = dict(rtol=2.0 ** -7, atol=1e-3)     # an ulp of bf16, should a launch of another size sum in another order
    assert torch.allclose(r[-64:], r2, **close) and torch.allclose(h[-64:], h2, **close)
    del r, h
    got, want = m.norm_residual_backward(x, x, x, x), m.norm_residual_backward(tail, tail, tail, tail)
    assert torch.allclose(got[0][-64:], want[0], **close) and torch.allclose(got[1][-64:], want[1], **close)
    del got
    dy = x[:, :16]
    dw, db = m.checkpoint_weight_grad(dy, held, torch.tensor([n - 64, n], dtype=torch.int32, device=DEV))
    dw2, db2 = m.checkpoint_weight_grad(tail[:, :16], some, torch.tensor([0, 64], dtype=torch.int32, device=DEV))
    assert torch.allclose(dw, dw2, rtol=256 * U) and torch.equal(db, db2)


# ---------------------------------------------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------------------------------------------
def refused(code, call, *args, **kw):
    with pytest.raises(binding.MPNNError) as e:
        call(*args, **kw)
    assert e.value.code == code and str(e.value)


def test_refusals(m):
    x = torch.zeros(4, 16, device=DEV)
    e = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    offsets, source, position = m.route_plan(e, 3)
    refused(-1, m.route_plan, e, 0)
    refused(-1, m.route_plan, e, 1025)
    refused(-1, m.route_plan, torch.zeros(1, 65, dtype=torch.int32, device=DEV), 4)
    refused(-1, m.norm_residual, x, eps=0.0)
    refused(-1, m.norm_residual, x, eps=float("nan"))
    refused(-1, m.norm_residual, x, eps=1e-60)
    refused(-1, m.norm_residual, x, gate=x)
    refused(-1, m.norm_residual, x, x, x[:, :3])
    refused(-1, m.norm_residual, torch.zeros(2, 8193, device=DEV))
    bad = [lambda: m.route_plan(e.long(), 3), lambda: m.route_plan(e[0], 3), lambda: m.route_scatter(x.double(), position, offsets),
           lambda: m.route_scatter(x[:3], position, offsets), lambda: m.route_combine(x, position, offsets),
           lambda: m.route_combine(torch.zeros(8, 16, device=DEV), position, offsets, torch.zeros(4, 3, device=DEV)),
           lambda: m.route_combine(torch.zeros(8, 16), position, offsets),
           lambda: m.norm_residual(x, x.bfloat16()), lambda: m.norm_residual(x, x[:, :8]), lambda: m.norm_residual(x, want_h=False),
           lambda: m.norm_residual(x, kind="batch"), lambda: m.norm_residual(x, pre_weight=torch.ones(16, device=DEV).double()),
           lambda: m.norm_residual_backward(None, None, x), lambda: m.norm_residual_backward(x, x, None),
           lambda: m.checkpoint_save(x[0]), lambda: m.checkpoint_load(m.checkpoint_save(x), torch.float64),
           lambda: m.checkpoint_silu_backward(x[:, :8], m.checkpoint_save(x)),
           lambda: m.checkpoint_weight_grad(x[:2], m.checkpoint_save(x), offsets)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    # through the C ABI, where the binding cannot make the mistake
    L, p = binding.lib(), x.data_ptr()
    assert L.mpnn_route_scatter(m.h, 0, 4, 2, 16, p, 15, position.data_ptr(), offsets.data_ptr(), 3, p) == -1
    assert L.mpnn_route_scatter(m.h, 2, 4, 2, 16, p, 16, position.data_ptr(), offsets.data_ptr(), 3, p) == -1
    assert L.mpnn_route_scatter(m.h, 0, 4, 2, 16, None, 16, position.data_ptr(), offsets.data_ptr(), 3, p) == -1
    assert b"null" in L.mpnn_last_error(m.h)
    assert L.mpnn_route_plan(m.h, 1 << 31, 1, 3, p, p, p, p) == -4
    assert L.mpnn_route_combine(m.h, 0, -1, 2, 16, p, p, p, 3, None, p) == -1
    assert L.mpnn_checkpoint_silu(m.h, 0, 4, 16, p, 16, p, p, p, p, None) == -1
    assert L.mpnn_checkpoint_weight_grad(m.h, 0, 4, 16, 16, 0, p, p, 16, p, p, p, None) == -1
    assert L.mpnn_route_combine_backward(m.h, 0, 4, 2, 16, p, 16, None, position.data_ptr(), offsets.data_ptr(), 3, None, p, p) == -1
    # the context is usable afterwards
    assert m.route_scatter(x, position, offsets).shape == (8, 16)
    assert m.checkpoint_save(torch.zeros(0, 40, device=DEV)).scales.shape == (0, 2)
    assert m.norm_residual(torch.zeros(0, 40, device=DEV))[1].shape == (0, 40)
    got = m.norm_residual_backward(torch.zeros(0, 40, device=DEV), torch.zeros(0, 40, device=DEV), torch.zeros(0, 40, device=DEV),
                                   torch.zeros(0, 40, device=DEV))
    assert all((v == 0).all() for v in got[3:])
