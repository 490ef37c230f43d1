"""Plain 64-bit implementations of the products by expert, 4-bit rows and embedding rows, on the CPU."""
import torch

from tests.rows_util import f64, silu

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
MIDDLES = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
GROUP = 32


def taken(x, source, n):
    """The rows of x at the n sorted places."""
    x = f64(x)
    return x if source is None else x[source.cpu().long() // (n // len(x))]


def segments(offsets, n):
    """(expert, rows) of every expert's rows, offsets clamped to 0 .. n."""
    ends = offsets.cpu().long().clamp(0, n).tolist()
    return [(e, slice(ends[e], max(ends[e], ends[e + 1]))) for e in range(len(ends) - 1)]


def product(x, weight, offsets, bias, act, n, source=None):
    """(y, the sums of the magnitudes that a row's sums have): zeros in rows of no expert."""
    x, w = taken(x, source, n), f64(weight)
    y, size = torch.zeros(n, w.shape[1], dtype=torch.float64), torch.zeros(n, w.shape[1], dtype=torch.float64)
    for e, rows in segments(offsets, n):
        y[rows], size[rows] = x[rows] @ w[e].T, x[rows].abs() @ w[e].abs().T
        if bias is not None:
            y[rows] += f64(bias)[e]
            size[rows] += f64(bias)[e].abs()
        if act == "silu":
            y[rows] = silu(y[rows])
    return y, size


def input_grad(dy, weight, offsets):
    dy, w = f64(dy), f64(weight)
    dx, size = (torch.zeros(len(dy), w.shape[2], dtype=torch.float64) for _ in range(2))
    for e, rows in segments(offsets, len(dy)):
        dx[rows], size[rows] = dy[rows] @ w[e], dy[rows].abs() @ w[e].abs()
    return dx, size


def weight_grad(dy, x, offsets, source=None):
    """(dweight, its magnitudes, dbias, its magnitudes, rows of each expert)."""
    dy = f64(dy)
    x = taken(x, source, len(dy))
    got = [(dy[r].T @ x[r], dy[r].abs().T @ x[r].abs(), dy[r].sum(0), dy[r].abs().sum(0), r.stop - r.start)
           for _, r in segments(offsets, len(dy))]
    return [torch.stack([g[i] for g in got]) for i in range(4)] + [[g[4] for g in got]]


def micro_save(x):
    """(codes, scales) by exact arithmetic in 64 bits."""
    x = f64(x)
    n, w = x.shape
    groups = -(-w // GROUP)
    v = torch.nn.functional.pad(x, (0, groups * GROUP - w)).reshape(n, groups, GROUP)
    largest = v.abs().amax(-1)
    fine = torch.isfinite(largest)
    exponent = torch.where(fine & (largest > 0), torch.frexp(torch.where(fine, largest, 1.0))[1] - 3, -100).clamp(min=-100)
    steps = torch.where(fine.unsqueeze(-1), v, 0.0) * torch.exp2(-exponent.double()).unsqueeze(-1)
    a = steps.abs().unsqueeze(-1)
    tie_up = torch.tensor([False, True, False, True, False, True, False])        # to the even code
    code = ((a > MIDDLES) | ((a == MIDDLES) & tie_up)).sum(-1) + 8 * (steps < 0)
    code = code.reshape(n, groups * GROUP)
    return (code[:, ::2] | code[:, 1::2] << 4).to(torch.uint8), torch.where(fine, exponent + 127, 255).to(torch.uint8)


def micro_load(codes, scales, width):
    codes, scales = codes.cpu().long(), scales.cpu().long()
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    value = LEVELS[code & 7] * torch.where(code > 7, -1.0, 1.0)
    step = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return (value * step.repeat_interleave(GROUP, 1))[:, :width]


def embed(index, table, scale):
    index, table = index.cpu().long(), f64(table)
    there = (index >= 0) & (index < len(table))
    return torch.where(there.unsqueeze(1), table[index.clamp(0, len(table) - 1)] * scale, 0.0)


def embed_plan(index, entries):
    index = index.cpu().long()
    key = torch.where((index >= 0) & (index < entries), index, entries)
    key, source = torch.sort(key, stable=True)
    return torch.searchsorted(key, torch.arange(entries + 1)), source


def embed_grad(index, dout, entries, scale):
    """(dtable, the sums of the magnitudes, rows of each entry)."""
    index, dout = index.cpu().long(), f64(dout)
    at = torch.where((index >= 0) & (index < entries), index, entries)
    sums = [torch.zeros(entries + 1, dout.shape[1], dtype=torch.float64).index_add_(0, at, v)[:entries] * abs(scale) for v in (dout, dout.abs())]
    return sums[0] * (1 if scale >= 0 else -1), sums[1], torch.bincount(at, minlength=entries + 1)[:entries]
