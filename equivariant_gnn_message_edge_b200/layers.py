"""Node-level operators around the convolution, for a training step of a stack
of layers (contracts in include/eqconv.h):

    emb = Embedding(n_types, C)                     # first features from node types
    norm = BlockNorm("0e+1o+2e", C, gate="sigmoid") # norms, gate and residual around a layer
    x0 = emb(types, table)                          # differentiable in table
    x, h = norm(x, b, gate, w_post, w_pre, scale)   # differentiable in x, b, gate, w_post, w_pre
    total = clip_gradients([p.grad for p in params], max_norm=10.0)

Tensors are fp32, bf16 or fp16 and live on the operator's device (the current
one when it was made); every step runs in libeqconv's kernels on the current
stream, or on ``stream``, and nothing waits for the GPU.  The autograd forms
are once differentiable: a second derivative raises.  To capture a backward
pass into a CUDA graph, release eager autograd graphs of the same leaves first
and take the gradients with torch.autograd.grad.
"""
from __future__ import annotations

import array
import contextlib
import functools
import itertools

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

_TYPES = {torch.float32: B.EQCONV_F32, torch.bfloat16: B.EQCONV_BF16, torch.float16: B.EQCONV_F16}
_GATES = {"none": B.EQCONV_GATE_NONE, "sigmoid": B.EQCONV_GATE_SIGMOID, "silu": B.EQCONV_GATE_SILU,
          "tanh": B.EQCONV_GATE_TANH}
_NOTHING = contextlib.nullcontext()
_KINDS = {torch.Tensor, torch.nn.Parameter}


@functools.lru_cache(None)
def _device(index: int):
    return torch.device("cuda", index)


def _type_code(dtype) -> int:
    if dtype not in _TYPES:
        raise ValueError(f"expected torch.float32, bfloat16 or float16, got {dtype}")
    return _TYPES[dtype]


def _on(device: int, stream):
    """The context in which outputs and workspaces are made and kernels are
    launched: the operator's device, and the given stream, so that memory made
    there is not handed to another stream while it is in use."""
    if stream is None:
        return _NOTHING if torch.cuda.current_device() == device else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _check(name, t, shape, dtype, device: int):
    """The tensor's address, if it is what the operator takes."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device and t.shape == shape and \
            t.is_contiguous():
        return t.data_ptr()
    _refuse(name, t, shape, dtype, device)
    raise ValueError(f"{name} must be contiguous")


def _refuse(name, t, shape, dtype, device: int):
    """Raises what is wrong with a tensor's kind, place, type or shape, if anything is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a CUDA tensor, got {type(t)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must live on cuda:{device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


class Embedding:
    """Rows of a table of types, y[i] = scale * table[ids[i]], and the table's
    gradient.  table [n_types][C] of ``dtype``; y of ``out_dtype`` (the same,
    or 16 bits from an fp32 table).  ``padding``: the type whose row gets no
    gradient.  ids: int32 or int64, any shape; ids out of range give zero rows
    and set the plan's status (binding.eqconv_get_device_error)."""

    def __init__(self, n_types: int, C: int, dtype=torch.float32, out_dtype=None, padding: int | None = None):
        out_dtype = dtype if out_dtype is None else out_dtype
        self.n_types, self.C, self.dtype, self.out_dtype, self.padding = int(n_types), int(C), dtype, out_dtype, padding
        if padding is not None and not 0 <= padding < n_types:
            raise ValueError(f"padding must be a type in 0..{n_types - 1}, got {padding}")
        self.plan = B.eqconv_embedding_plan_create(n_types, C, _type_code(dtype), _type_code(out_dtype),
                                                   -1 if padding is None else padding)
        self.device = torch.cuda.current_device()

    def __reduce__(self):       # a copy has a plan of its own, on the device that is current where it is made
        return type(self), (self.n_types, self.C, self.dtype, self.out_dtype, self.padding)

    def __del__(self):
        try:
            B.eqconv_plan_destroy(self.plan)
        except Exception:
            pass

    def _ids(self, ids):
        """(ids, contiguous; their bits)"""
        if not isinstance(ids, torch.Tensor):
            raise TypeError(f"ids: expected a CUDA tensor, got {type(ids)}")
        if ids.get_device() != self.device:
            raise ValueError(f"ids must live on cuda:{self.device}, got {ids.device}")
        if ids.dtype is torch.int64:
            return ids if ids.is_contiguous() else ids.contiguous(), 64
        if ids.dtype is torch.int32:
            return ids if ids.is_contiguous() else ids.contiguous(), 32
        raise ValueError(f"ids: expected int32 or int64, got {ids.dtype}")

    def _rows(self, name, t, shape, dtype):
        """(address, row stride) of a tensor of rows [C]; the row stride is
        None when the rows are not evenly spaced runs of C elements."""
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == self.device and
                t.shape == shape):
            _refuse(name, t, shape, dtype, self.device)
        if t.is_contiguous():
            return t.data_ptr(), self.C
        if t.dim() == 2 and (t.stride(1) == 1 or self.C == 1):
            return t.data_ptr(), t.stride(0) if shape[0] > 1 else self.C
        return t.data_ptr(), None

    def forward_raw(self, ids, table, scale: float = 1.0, out=None, stream=None):
        """out: rows may be spaced, as x[:, 0, :] of node features [N][D][C]."""
        tp, ts = self._rows("table", table, (self.n_types, self.C), self.dtype)
        if ts is None or ts < self.C:
            raise ValueError("table must have contiguous rows that do not overlap")
        with _on(self.device, stream):
            ids, bits = self._ids(ids)
            shape = ids.shape + (self.C,)
            if out is None:
                out = table.new_empty(shape, dtype=self.out_dtype)
                op, os = out.data_ptr(), self.C
            else:
                op, os = self._rows("out", out, shape, self.out_dtype)
                if os is None or os < self.C:
                    raise ValueError("out must have contiguous, evenly spaced rows that do not overlap")
            B.eqconv_embedding(self.plan, ids.numel(), ids.data_ptr(), bits, tp, ts, scale, op, os)
        return out

    def backward_raw(self, ids, gy, scale: float = 1.0, out=None, workspace=None, stream=None):
        """dtable [n_types][C] from gy (the shape of y)."""
        with _on(self.device, stream):
            ids, bits = self._ids(ids)
            gp, gs = self._rows("gy", gy, ids.shape + (self.C,), self.out_dtype)
            if gs is None or gs < 0:
                gy = gy.contiguous()
                gp, gs = gy.data_ptr(), self.C
            N = ids.numel()
            if out is None:
                out = gy.new_empty((self.n_types, self.C), dtype=self.dtype)
                dp = out.data_ptr()
            else:
                dp = _check("out", out, (self.n_types, self.C), self.dtype, self.device)
            nbytes = B.eqconv_embedding_workspace_bytes(self.plan, N)
            if workspace is None and nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=ids.device)
            if workspace is not None:
                nbytes = workspace.numel() * workspace.element_size()
            B.eqconv_embedding_backward(self.plan, N, ids.data_ptr(), bits, gp, gs, scale, dp, workspace, nbytes)
        return out

    def __call__(self, ids, table, scale: float = 1.0):
        return _EmbeddingFn.apply(self, ids, table, scale)


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, op: Embedding, ids, table, scale):
        ctx.op, ctx.scale = op, scale
        ctx.save_for_backward(ids)
        if table.dim() == 2 and (table.stride(1) != 1 or table.stride(0) < table.shape[1]):
            table = table.contiguous()          # columns apart, or rows that repeat or overlap
        return op.forward_raw(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        (ids,) = ctx.saved_tensors
        return None, None, ctx.op.backward_raw(ids, gy, ctx.scale), None


class BlockNorm:
    """The norms before and after a layer with its gate and residual:

        u = b / rms(b) * w_post,  x_out = x + scale * a(gate) * u,  h = x_out / rms(x_out) * w_pre

    rms over a node's rows of one degree.  x, b [N][D][C] of ``dtype`` with
    D = (L+1)^2 rows ("0e": D = 1, the plain row norm), gate [N][L+1][C] of
    ``dtype`` (None with gate="none"), w_post, w_pre [L+1][C] fp32.  Without b
    (and gate, w_post) it is the norm before a first layer; without w_pre the
    end of a last one."""

    def __init__(self, irreps: str, C: int, gate: str = "sigmoid", eps: float = 1e-6, dtype=torch.float32):
        if gate not in _GATES:
            raise ValueError(f"gate must be one of {sorted(_GATES)}, got {gate!r}")
        self.irreps, self.C, self.gate, self.eps, self.dtype = irreps, int(C), gate, float(eps), dtype
        self.plan = B.eqconv_block_norm_plan_create(irreps, C, _type_code(dtype), _GATES[gate], eps)
        self.device = torch.cuda.current_device()
        self.D = B.eqconv_plan_info(self.plan)["D_in"]
        self.L = int(round(self.D ** 0.5)) - 1

    def __reduce__(self):       # as the embedding's
        return type(self), (self.irreps, self.C, self.gate, self.eps, self.dtype)

    def __del__(self):
        try:
            B.eqconv_plan_destroy(self.plan)
        except Exception:
            pass

    def _inputs(self, x, b, gate, w_post, w_pre):
        dev, T = self.device, self.dtype
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            raise ValueError("x must be a tensor [N][D][C]")
        N = x.shape[0]
        rows, flat, w = (N, self.D, self.C), (N, self.L + 1, self.C), (self.L + 1, self.C)
        if (b is None) != (w_post is None):
            raise ValueError("b and w_post come together")
        if b is None and gate is not None:
            raise ValueError("a gate needs b")
        if b is not None and (gate is None) != (self.gate == "none"):
            raise ValueError(f"gate={self.gate!r} was chosen: a gate tensor is " +
                             ("not taken" if self.gate == "none" else "needed"))
        if w_post is None and w_pre is None:
            raise ValueError("nothing to compute: w_post and w_pre are both None")
        f32 = torch.float32
        return N, (_check("x", x, rows, T, dev), None if b is None else _check("b", b, rows, T, dev),
                   None if gate is None else _check("gate", gate, flat, T, dev),
                   None if w_post is None else _check("w_post", w_post, w, f32, dev),
                   None if w_pre is None else _check("w_pre", w_pre, w, f32, dev))

    def forward_raw(self, x, b, gate, w_post, w_pre, scale: float = 1.0, save: bool = False, out=None, stream=None):
        """(x_out, h, stats); x_out is None without b, h without w_pre, stats
        without ``save`` (they are what backward_raw needs).  out: (x_out, h)."""
        N, ptrs = self._inputs(x, b, gate, w_post, w_pre)
        with _on(self.device, stream):
            if out is not None:
                x_out, h = out
                if (x_out is None) != (b is None) or (h is None) != (w_pre is None):
                    raise ValueError("out: (x_out, h), each given where it is computed")
                for name, t in (("x_out", x_out), ("h", h)):
                    if t is not None:
                        _check(name, t, x.shape, self.dtype, self.device)
            else:
                x_out = None if b is None else torch.empty_like(x)
                h = None if w_pre is None else torch.empty_like(x)
            stats = torch.empty((2, N, self.L + 1), dtype=torch.float32, device=x.device) if save else None
            B.eqconv_block_norm(self.plan, N, *ptrs, scale, None if x_out is None else x_out.data_ptr(),
                                None if h is None else h.data_ptr(), None if stats is None else stats.data_ptr())
        return x_out, h, stats

    def backward_raw(self, x, b, gate, w_post, w_pre, stats, g_x, g_h, scale: float = 1.0, need_dw: bool = True,
                     workspace=None, stream=None):
        """(dx, db, dgate, dw_post, dw_pre) from the gradients of x_out and h
        (None: zero); None in the places of inputs that are None, and for the
        weights without ``need_dw``.  The others are always computed."""
        N, ptrs = self._inputs(x, b, gate, w_post, w_pre)
        dev = self.device
        if (g_x is not None and b is None) or (g_h is not None and w_pre is None):
            raise ValueError("a gradient of an output that was not computed")
        sp = _check("stats", stats, (2, N, self.L + 1), torch.float32, dev)
        gxp = None if g_x is None else _check("g_x", g_x, x.shape, self.dtype, dev)
        ghp = None if g_h is None else _check("g_h", g_h, x.shape, self.dtype, dev)
        with _on(dev, stream):
            dx = torch.empty_like(x)
            db = None if b is None else torch.empty_like(b)
            dgate = None if gate is None else torch.empty_like(gate)
            dw_post = torch.empty_like(w_post) if need_dw and w_post is not None else None
            dw_pre = torch.empty_like(w_pre) if need_dw and w_pre is not None else None
            nbytes = B.eqconv_block_norm_workspace_bytes(self.plan, N)
            if workspace is None:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
            p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
            B.eqconv_block_norm_backward(self.plan, N, *ptrs, scale, sp, gxp, ghp, dx.data_ptr(), p(db), p(dgate),
                                         p(dw_post), p(dw_pre), workspace,
                                         workspace.numel() * workspace.element_size())
        return dx, db, dgate, dw_post, dw_pre

    def __call__(self, x, b=None, gate=None, w_post=None, w_pre=None, scale: float = 1.0):
        """(x_out, h); x_out is x itself without b, h is None without w_pre."""
        x_out, h = _BlockNormFn.apply(self, scale, x, b, gate, w_post, w_pre)
        return (x if b is None else x_out), h


class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, op: BlockNorm, scale, *args):
        args = [None if t is None else t.contiguous() for t in args]
        x_out, h, stats = op.forward_raw(*args, scale=scale, save=True)
        ctx.op, ctx.scale = op, scale
        ctx.save_for_backward(*args, stats)
        ctx.set_materialize_grads(False)
        return x_out, h

    @staticmethod
    @once_differentiable
    def backward(ctx, g_x, g_h):
        *args, stats = ctx.saved_tensors
        if g_x is None and g_h is None:
            return (None,) * 7
        g = [None if t is None else t.contiguous() for t in (g_x, g_h)]
        need = ctx.needs_input_grad[5] or ctx.needs_input_grad[6]
        return (None, None) + ctx.op.backward_raw(*args, stats, *g, scale=ctx.scale, need_dw=need)


def _tensor_list(grads, out):
    """(packed array of eqconv_tensor_t, its length, the device's index, the tensors written)"""
    if isinstance(grads, torch.Tensor):
        raise TypeError("expected a list of tensors")
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"out: expected {len(grads)} tensors, got {len(outs)}")
    every = grads if out is None else grads + outs
    if not set(map(type, every)) <= _KINDS:
        for i, t in enumerate(every):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"tensor {i % len(grads)}: expected a CUDA tensor, got {type(t)}")
    places = set(map(torch.Tensor.get_device, every))
    dev = places.pop() if places else torch.cuda.current_device()
    if places or dev < 0:
        raise ValueError("expected CUDA tensors of one device, got " + ", ".join(sorted({str(t.device) for t in every})))
    kinds, sizes = [g.dtype for g in grads], list(map(torch.Tensor.numel, grads))
    types = list(map(_TYPES.get, kinds))
    if None in types:
        raise ValueError(f"tensor {types.index(None)}: expected torch.float32, bfloat16 or float16, got "
                         f"{kinds[types.index(None)]}")
    if out is not None and (kinds != [o.dtype for o in outs] or sizes != list(map(torch.Tensor.numel, outs))):
        raise ValueError("out: expected the types and sizes of the inputs")
    if not all(map(torch.Tensor.is_contiguous, every)):
        for i, (g, o) in enumerate(zip(grads, outs)):
            if not torch.ops.aten.is_non_overlapping_and_dense(g):
                raise ValueError(f"tensor {i}: its elements must fill its memory without gaps or repeats")
            if g.shape != o.shape or g.stride() != o.stride():
                raise ValueError(f"out {i}: expected the shape and strides of its input")
    at = list(map(torch.Tensor.data_ptr, grads))
    to = at if out is None else list(map(torch.Tensor.data_ptr, outs))
    # four 64-bit words are one eqconv_tensor_t
    return array.array("q", itertools.chain.from_iterable(zip(at, to, sizes, types))), len(grads), dev, outs


def gradient_norm(grads, stream=None):
    """sqrt of the sum of all elements' squares, over a list of tensors: a
    0-dimensional fp32 tensor on their device."""
    arr, n, dev, _ = _tensor_list(grads, None)
    with _on(dev, stream):
        rows = arr.buffer_info()[0]
        nbytes = B.eqconv_clip_workspace_bytes(n, rows)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=_device(dev))
        norm = ws.new_empty((), dtype=torch.float32)
        B.eqconv_gradient_norm(n, rows, norm, ws, nbytes)
    return norm


def clip_gradients(grads, max_norm: float, out=None, eps: float = 1e-6, stream=None):
    """Scales a list of tensors by k = min(1, max_norm / (norm + eps)) with
    norm their norm together, in place or into ``out`` (a list of tensors like
    them), and returns norm (a 0-dimensional fp32 tensor).  A tensor may not
    be in the list twice, nor share memory with another."""
    arr, n, dev, outs = _tensor_list(grads, out)
    with _on(dev, stream):
        rows = arr.buffer_info()[0]
        nbytes = B.eqconv_clip_workspace_bytes(n, rows)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=_device(dev))
        norm = ws.new_empty((), dtype=torch.float32)
        B.eqconv_clip_gradients(n, rows, max_norm, eps, norm, ws, nbytes)
    torch.autograd.graph.increment_version(outs)      # as any in-place operation does
    return norm
