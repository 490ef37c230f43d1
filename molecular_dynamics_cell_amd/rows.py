"""The row operators of include/mpnn.h as methods of binding.MPNN: argument checks, output tensors
and the calls.  Rows are 2-D tensors [n, width] of float32 or bfloat16 on the context's device; a
row tensor may have any row stride (a column block of a wider tensor), other layouts are copied.

Work runs on the context's stream.  When torch's current stream is another one, the call waits for
it, and it waits for the call, so tensors may be made and used there.  The methods are no autograd
functions (each gradient is a method of its own): with gradients enabled a tensor that requires one is
refused, rather than its gradient dropped; call them under torch.no_grad().

Calls may be captured into a graph (with the captured stream as the context's: set_stream), which may
be replayed as long as the context lives; replay the graphs captured from one context one after another
(they share its scratch for captured calls)."""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

GROUP = 32      # columns that share one scale of a checkpoint
_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
_KIND = {"rms": 0, "layer": 1}
_CALLS = {}     # the library's functions by name, once they have been used

# the handle of torch's current stream on a device (a stream object for each call costs 2 us)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class Norm(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("width", C.c_int32), ("kind", C.c_int32), ("gate_width", C.c_int32),
                ("eps", C.c_double), ("post_weight", C.c_void_p), ("post_bias", C.c_void_p),
                ("scale", C.c_void_p), ("pre_weight", C.c_void_p), ("pre_bias", C.c_void_p)]


class Checkpoint(NamedTuple):
    """Rows held in 8 bits: codes int8 [n, width], scales uint8 [n, ceil(width / 32)]."""
    codes: torch.Tensor
    scales: torch.Tensor


def _ptr(t):
    return None if t is None else t.data_ptr()


class RowOperators:
    # A small call is bound by what happens here, so checks are few comparisons and a dense tensor is taken as it is.
    def _rows(self, name, t, n=None, width=None, dtype=None):
        """The tensor as rows with a row stride: (tensor, stride)."""
        shape = t.shape
        if len(shape) != 2 or t.dtype not in _DTYPE or (dtype is not None and t.dtype != dtype) or \
                (n is not None and shape[0] != n) or (width is not None and shape[1] != width):
            raise ValueError(f"{name}: expected rows [{'n' if n is None else n}, {'width' if width is None else width}] "
                             f"of {dtype or 'float32 or bfloat16'}, got {tuple(shape)} of {t.dtype}")
        if t.device != self._at:
            raise ValueError(f"{name}: on {t.device}, the context is on {self._at}")
        rows, columns = shape
        if t.is_contiguous():
            return t, columns
        down, across = t.stride()
        if (across != 1 and columns > 1) or (down < columns and rows > 1):
            return t.contiguous(), columns
        return t, max(down, columns)

    def _dense(self, name, t, shape, dtype):
        if t.dtype is dtype and t.shape == shape and t.device == self._at:
            return t if t.is_contiguous() else t.contiguous()
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
        raise ValueError(f"{name}: on {t.device}, the context is on {self._at}")

    @staticmethod
    def _new(like, *shape, dtype=None):
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)

    def _call(self, name, tensors, *args):
        """One library call on the context's stream, ordered with torch's current stream."""
        if torch.is_grad_enabled():
            for t in tensors:
                if t is not None and t.requires_grad:
                    raise ValueError(f"{name[5:]}: a tensor requires a gradient, which the result would not carry; call it "
                                     "under torch.no_grad() and take gradients from the methods for them")
        call = _CALLS.get(name)
        if call is None:
            from . import binding
            call = _CALLS[name] = getattr(binding.lib(), name)
        own = self._stream
        apart = _current_stream(self._at.index) != own.cuda_stream
        if apart:
            current = torch.cuda.current_stream(self._at)
            own.wait_stream(current)
        code = call(self.h, *args)
        if apart:
            current.wait_stream(own)
            for t in tensors:
                if t is not None:
                    t.record_stream(own)
        if code:
            self._check(code)

    # ---- rows by expert ----
    def route_plan(self, expert: torch.Tensor, n_experts: int):
        """Stable order by expert of the pairs (row, slot) of expert int32 [n, k] (values outside
        0 .. n_experts - 1: dropped): offsets [n_experts + 1], source [n k], position [n, k], int32."""
        if expert.dim() != 2:
            raise ValueError(f"expert: expected [n, k], got {tuple(expert.shape)}")
        n, k = expert.shape
        expert = self._dense("expert", expert, (n, k), torch.int32)
        offsets = self._new(expert, max(int(n_experts), 0) + 1)
        source, position = self._new(expert, n * k), self._new(expert, n, k)
        self._call("mpnn_route_plan", (expert, offsets, source, position), n, k, int(n_experts), _ptr(expert),
                   _ptr(offsets), _ptr(source), _ptr(position))
        return offsets, source, position

    def _places(self, position, offsets, n=None):
        if position.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2 or (n is not None and position.shape[0] != n):
            raise ValueError(f"position [n, k] and offsets [n_experts + 1]: got {tuple(position.shape)}, {tuple(offsets.shape)}")
        return (self._dense("position", position, position.shape, torch.int32),
                self._dense("offsets", offsets, offsets.shape, torch.int32))

    def route_scatter(self, x: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor):
        """x [n, width] to its places: sorted [n k, width], zeros where a pair was dropped."""
        x, ld = self._rows("x", x)
        n, width = x.shape
        position, offsets = self._places(position, offsets, n)
        k = position.shape[1]
        out = self._new(x, n * k, width)
        self._call("mpnn_route_scatter", (x, position, offsets, out), _DTYPE[x.dtype], n, k, width, _ptr(x), ld,
                   _ptr(position), _ptr(offsets), offsets.shape[0] - 1, _ptr(out))
        return out

    def route_combine(self, rows: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor,
                      weight: torch.Tensor = None):
        """Sorted rows [n k, width] back to their rows, weighted by weight float32 [n, k]: [n, width]."""
        position, offsets = self._places(position, offsets)
        n, k = position.shape
        if rows.dim() != 2 or rows.dtype not in _DTYPE:
            raise ValueError(f"rows: expected [n k, width] of float32 or bfloat16, got {tuple(rows.shape)} of {rows.dtype}")
        width = rows.shape[1]
        rows = self._dense("rows", rows, (n * k, width), rows.dtype)
        weight = None if weight is None else self._dense("weight", weight, (n, k), torch.float32)
        out = self._new(rows, n, width)
        self._call("mpnn_route_combine", (rows, position, offsets, weight, out), _DTYPE[rows.dtype], n, k, width,
                   _ptr(rows), _ptr(position), _ptr(offsets), offsets.shape[0] - 1, _ptr(weight), _ptr(out))
        return out

    def route_combine_backward(self, dout: torch.Tensor, rows: torch.Tensor, position: torch.Tensor,
                               offsets: torch.Tensor, weight: torch.Tensor = None):
        """Gradient of route_combine: (dsorted [n k, width], dweight float32 [n, k]); rows None: no dweight."""
        dout, ld = self._rows("dout", dout)
        n, width = dout.shape
        position, offsets = self._places(position, offsets, n)
        k = position.shape[1]
        rows = None if rows is None else self._dense("rows", rows, (n * k, width), dout.dtype)
        weight = None if weight is None else self._dense("weight", weight, (n, k), torch.float32)
        dsorted = self._new(dout, n * k, width)
        dweight = None if rows is None else self._new(dout, n, k, dtype=torch.float32)
        self._call("mpnn_route_combine_backward", (dout, rows, position, offsets, weight, dsorted, dweight),
                   _DTYPE[dout.dtype], n, k, width, _ptr(dout), ld, _ptr(rows), _ptr(position), _ptr(offsets),
                   offsets.shape[0] - 1, _ptr(weight), _ptr(dsorted), _ptr(dweight))
        return dsorted, dweight

    # ---- norms around a block ----
    def _norm(self, x, width, gate, kind, eps, vectors):
        if kind not in _KIND:
            raise ValueError(f"kind: expected 'rms' or 'layer', got {kind!r}")
        kept = [None if v is None else self._dense(name, v, (width,), torch.float32) for name, v in vectors]
        gate_width = 0 if gate is None else gate.shape[1] if gate.dim() == 2 else -1
        return Norm(_DTYPE[x.dtype], width, _KIND[kind], gate_width, float(eps), *[_ptr(v) for v in kept]), kept

    def _block_and_gate(self, like, block, gate):
        n, width = like.shape
        block, ldb = (None, 0) if block is None else self._rows("block", block, n, width, like.dtype)
        gate, ldg = (None, 0) if gate is None else self._rows("gate", gate, n, None, like.dtype)
        if gate is not None and gate.shape[1] == 0:     # its null pointer would stand for no gate
            raise ValueError(f"gate: expected [{n}, {width}] or [{n}, 1], got {tuple(gate.shape)}")
        return block, ldb, gate, ldg

    def norm_residual(self, x: torch.Tensor, block: torch.Tensor = None, gate: torch.Tensor = None, *,
                      post_weight=None, post_bias=None, scale=None, pre_weight=None, pre_bias=None, kind="rms",
                      eps=1e-5, want_h=True):
        """r = x + scale * sigma(gate) * N_post(block) and h = N_pre(r), gate [n, width] or [n, 1]:
        (r, h).  Without a block r is x itself; h is None unless wanted."""
        x, ldx = self._rows("x", x)
        n, width = x.shape
        block, ldb, gate, ldg = self._block_and_gate(x, block, gate)
        p, kept = self._norm(x, width, gate, kind, eps,
                             (("post_weight", post_weight), ("post_bias", post_bias), ("scale", scale),
                              ("pre_weight", pre_weight), ("pre_bias", pre_bias)))
        if block is None and not want_h:
            raise ValueError("neither a block to add nor h wanted")
        r = None if block is None else self._new(x, n, width)
        h = self._new(x, n, width) if want_h else None
        self._call("mpnn_norm_residual", (x, block, gate, r, h, *kept), C.byref(p), n, _ptr(x), ldx, _ptr(block), ldb,
                   _ptr(gate), ldg, _ptr(r), _ptr(h))
        return (x if r is None else r), h

    def norm_residual_backward(self, dr: torch.Tensor, dh: torch.Tensor, r: torch.Tensor, block: torch.Tensor = None,
                               gate: torch.Tensor = None, *, post_weight=None, post_bias=None, scale=None,
                               pre_weight=None, pre_bias=None, kind="rms", eps=1e-5):
        """Gradient of norm_residual at r (dr or dh may be None): (dx, dblock, dgate, dpost_weight,
        dpost_bias, dscale, dpre_weight, dpre_bias), the last five float32 [width]; None where there is
        no block, gate or dh."""
        like = dr if dr is not None else dh
        if like is None:
            raise ValueError("dr and dh are both None")
        if like.dim() != 2 or like.dtype not in _DTYPE:
            raise ValueError(f"dr, dh: expected [n, width] of float32 or bfloat16, got {tuple(like.shape)} of {like.dtype}")
        n, width = like.shape
        dr = None if dr is None else self._dense("dr", dr, (n, width), like.dtype)
        dh = None if dh is None else self._dense("dh", dh, (n, width), like.dtype)
        if dh is not None and r is None:
            raise ValueError("dh needs r")
        r, ldr = (None, 0) if dh is None else self._rows("r", r, n, width, like.dtype)
        block, ldb, gate, ldg = self._block_and_gate(like, block, gate)
        p, kept = self._norm(like, width, gate, kind, eps,
                             (("post_weight", post_weight), ("post_bias", post_bias), ("scale", scale),
                              ("pre_weight", pre_weight), ("pre_bias", pre_bias)))
        dx = self._new(like, n, width)
        dblock = None if block is None else self._new(like, n, width)
        dgate = None if gate is None else self._new(like, n, gate.shape[1])
        post = self._new(like, 3, width, dtype=torch.float32) if block is not None else (None,) * 3
        pre = self._new(like, 2, width, dtype=torch.float32) if dh is not None else (None,) * 2
        sums = [*post, *pre]
        self._call("mpnn_norm_residual_backward", (dr, dh, r, block, gate, dx, dblock, dgate, *sums, *kept), C.byref(p), n,
                   _ptr(dr), _ptr(dh), _ptr(r), ldr, _ptr(block), ldb, _ptr(gate), ldg, _ptr(dx), _ptr(dblock),
                   _ptr(dgate), *[_ptr(v) for v in sums])
        return (dx, dblock, dgate, *sums)

    # ---- activation checkpoints ----
    def _new_checkpoint(self, x):
        n, width = x.shape
        return Checkpoint(self._new(x, n, width, dtype=torch.int8),
                          self._new(x, n, -(-width // GROUP), dtype=torch.uint8))

    def _held(self, saved, n=None, width=None):
        codes, scales = saved
        if codes.dim() != 2 or (n is not None and codes.shape[0] != n) or (width is not None and codes.shape[1] != width):
            raise ValueError(f"codes: expected [{n}, {width}], got {tuple(codes.shape)}")
        n, width = codes.shape
        return (self._dense("codes", codes, (n, width), torch.int8),
                self._dense("scales", scales, (n, -(-width // GROUP)), torch.uint8))

    def checkpoint_save(self, x: torch.Tensor) -> Checkpoint:
        """x [n, width] in 8 bits, one power-of-two step per 32 columns of a row."""
        x, ld = self._rows("x", x)
        n, width = x.shape
        held = self._new_checkpoint(x)
        self._call("mpnn_checkpoint_save", (x, *held), _DTYPE[x.dtype], n, width, _ptr(x), ld, _ptr(held.codes),
                   _ptr(held.scales))
        return held

    def checkpoint_load(self, saved, dtype=torch.float32) -> torch.Tensor:
        """The values that a checkpoint holds (exact in either type)."""
        if dtype not in _DTYPE:
            raise ValueError(f"dtype: expected float32 or bfloat16, got {dtype}")
        codes, scales = self._held(saved)
        n, width = codes.shape
        out = self._new(codes, n, width, dtype=dtype)
        self._call("mpnn_checkpoint_load", (codes, scales, out), _DTYPE[dtype], n, width, _ptr(codes), _ptr(scales),
                   _ptr(out))
        return out

    def checkpoint_silu(self, z: torch.Tensor, save_output=False):
        """y = silu(z) with the checkpoint of z and, if asked for, of y: (y, z held, y held or None)."""
        z, ld = self._rows("z", z)
        n, width = z.shape
        y, held = self._new(z, n, width), self._new_checkpoint(z)
        also = self._new_checkpoint(z) if save_output else None
        codes, scales = (None, None) if also is None else also
        self._call("mpnn_checkpoint_silu", (z, y, *held, codes, scales), _DTYPE[z.dtype], n, width, _ptr(z), ld, _ptr(y),
                   _ptr(held.codes), _ptr(held.scales), _ptr(codes), _ptr(scales))
        return y, held, also

    def checkpoint_silu_backward(self, dy: torch.Tensor, saved) -> torch.Tensor:
        """dz = dy silu'(z) for the z that the checkpoint holds."""
        dy, ld = self._rows("dy", dy)
        n, width = dy.shape
        codes, scales = self._held(saved, n, width)
        dz = self._new(dy, n, width)
        self._call("mpnn_checkpoint_silu_backward", (dy, codes, scales, dz), _DTYPE[dy.dtype], n, width, _ptr(dy), ld,
                   _ptr(codes), _ptr(scales), _ptr(dz))
        return dz

    def checkpoint_weight_grad(self, dy: torch.Tensor, saved, offsets: torch.Tensor):
        """Weight and bias gradients of y = x W_e^T + b_e per expert, x held by the checkpoint, rows
        offsets[e] .. offsets[e + 1] - 1 of expert e: (dweight [E, n_out, width], dbias [E, n_out]), float32."""
        dy, ld = self._rows("dy", dy)
        n, n_out = dy.shape
        codes, scales = self._held(saved, n)
        width = codes.shape[1]
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError(f"offsets: expected [n_experts + 1], got {tuple(offsets.shape)}")
        offsets = self._dense("offsets", offsets, offsets.shape, torch.int32)
        experts = offsets.shape[0] - 1
        dweight = self._new(dy, experts, n_out, width, dtype=torch.float32)
        dbias = self._new(dy, experts, n_out, dtype=torch.float32)
        self._call("mpnn_checkpoint_weight_grad", (dy, codes, scales, offsets, dweight, dbias), _DTYPE[dy.dtype], n, n_out,
                   width, experts, _ptr(offsets), _ptr(dy), ld, _ptr(codes), _ptr(scales), _ptr(dweight), _ptr(dbias))
        return dweight, dbias
