"""Plain 64-bit implementations of the row operators and the error bounds of the tests, on the CPU."""
import numpy as np
import torch

U = 2.0 ** -24          # half an ulp of fp32, relative
UB = 2.0 ** -8           # of bf16: its 8 significant bits put values of [1, 2) 2^-7 apart
HALF = {torch.float32: U, torch.bfloat16: UB}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(name, got, want, bound, dtype=torch.float32):
    """|got - want| <= bound, plus the rounding of the result to its type; not-a-numbers in the same places."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(want) + HALF[dtype] * want.abs() * (1 + 1e-6)
    bad = ~((got - want).abs() <= bound) & ~(got.isnan() & want.isnan()) & ~(got == want)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


def plan(expert, n_experts):
    flat = expert.cpu().numpy().reshape(-1)
    key = np.where((flat >= 0) & (flat < n_experts), flat, n_experts)
    source = np.argsort(key, kind="stable")
    position = np.empty_like(source)
    position[source] = np.arange(len(source))
    offsets = np.searchsorted(key[source], np.arange(n_experts + 1))
    return offsets, source, position.reshape(tuple(expert.shape))


def normed(v, layer, eps):
    v = v - v.mean(-1, keepdim=True) if layer else v
    inv = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * inv, inv


def residual(x, block, gate, w, layer, eps):
    """(r, h) in 64 bits; w: dict of the five vectors."""
    r = x
    if block is not None:
        g = 1.0 if gate is None else 1 / (1 + torch.exp(-gate))
        r = x + w["scale"] * g * (normed(block, layer, eps)[0] * w["post_weight"] + w["post_bias"])
    return r, normed(r, layer, eps)[0] * w["pre_weight"] + w["pre_bias"]


def normed_back(d, hat, inv, layer):
    m = d.mean(-1, keepdim=True) if layer else 0.0
    return inv * (d - m - hat * (d * hat).mean(-1, keepdim=True))


def normed_back_size(d, hat, inv):
    """Sum of the magnitudes that normed_back adds up, for magnitudes d."""
    return inv * (d + d.mean(-1, keepdim=True) + hat.abs() * (d * hat.abs()).mean(-1, keepdim=True))


def save(x):
    """(codes, bytes) of rows in 8 bits, by exact arithmetic in 64 bits."""
    x = f64(x).numpy()
    n, w = x.shape
    groups = -(-w // 32)
    v = np.zeros((n, groups * 32))
    v[:, :w] = x
    v = v.reshape(n, groups, 32)
    largest = np.abs(v).max(-1)
    fine = np.isfinite(largest)
    m, e = np.frexp(np.where(fine, largest, 0.0))           # largest = m 2^e, 1/2 <= m < 1
    e = np.where(largest == 0, -100, np.clip(e - 1 - 6 + (2 * m > 127 / 64), -100, 121))
    with np.errstate(invalid="ignore"):
        codes = np.clip(np.rint(v / np.exp2(e)[..., None]), -127, 127)
    codes = np.where(fine[..., None], codes, 0)
    return codes.reshape(n, -1)[:, :w].astype(np.int8), np.where(fine, e + 127, 255).astype(np.uint8)


def load(codes, scales):
    codes, scales = np.asarray(codes), np.asarray(scales)
    step = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return torch.from_numpy(codes.astype(np.float64) * np.repeat(step, 32, 1)[:, :codes.shape[1]])


def silu(z):
    return z / (1 + torch.exp(-z))


def silu_slope(z):
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))
