"""The layers whose weight gradients the framework reduces: an embedding's lookup
with its gradient by sorted tokens, and experts' matrix products over ragged runs
of rows.  They read a step's BF16 copies and write gradients where the step reads
them: ``DeviceState.grad_view`` is a tensor's place in a bucket buffer, and a
``TensorGroup`` takes any of these gradients as it is.

    by_row = RowOrder(tokens, 16384, 1024)                  # once
    table = st.flat_view(st.p_bf16, i).view(16384, 1024)
    x = lookup(table, ids, scale)
    ...
    by_row.sort(ids)
    by_row.lookup_grad(dx, scale, out=st.grad_view(bufs, i, slot, (16384, 1024)))

A call runs on ``stream``, by default the current one; ordering it after the work
that made its inputs is the caller's, as with any operation on another stream.
Memory is not: what a call uses on a stream other than the current one is kept until
that stream is done with it.  Nothing here takes part in autograd: forward and
gradient are calls of their own.  Tensors whose gradient autograd would lose that
way are refused while it records (those that require one, and those with a
forward-mode tangent): call under ``torch.no_grad()`` or with detached tensors, or
from a ``torch.autograd.Function``.
"""
from __future__ import annotations

import types

import torch
from torch.autograd import forward_ad

from . import binding as B

_TYPES = {torch.bfloat16: B.GRO_BF16, torch.float32: B.GRO_FP32}
_IDS = {torch.int32: B.GRO_INT32, torch.int64: B.GRO_INT64}


# No tensor has a tangent while no level is entered (-1); a torch that does not say is asked of every tensor.
_levels = forward_ad if hasattr(forward_ad, "_current_level") else types.SimpleNamespace(_current_level=0)


def _not_recorded(what: str, t) -> None:
    """Nothing that autograd follows would be lost in a call that it does not see."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and the layers take no part in autograd: call under torch.no_grad() "
                         f"or with detached tensors")
    if forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{what} has a forward-mode tangent, which the layers' results would not have")


def _matrix(what: str, t, device, dtypes=_TYPES) -> B.gro_matrix:
    """A matrix of one of these types on this GPU (its index) whose rows' elements lie side by side."""
    if t.requires_grad or _levels._current_level >= 0:
        _not_recorded(what, t)
    kind = dtypes.get(t.dtype)
    shape, step = t.shape, t.stride()
    if len(shape) != 2 or kind is None or t.get_device() != device or (shape[1] > 1 and step[1] != 1):
        raise ValueError(f"{what}: a matrix of {' or '.join(map(str, dtypes))} on cuda:{device}, rows' elements side by "
                         f"side, is needed, got {t.dtype} {tuple(shape)}, strides {step}, on {t.device}")
    rows, cols = shape
    return B.gro_matrix(t.data_ptr(), rows, cols, step[0] if rows > 1 else cols, kind, 0)


def _experts(what: str, t, device, dtypes=_TYPES) -> B.gro_experts:
    if t.requires_grad or _levels._current_level >= 0:
        _not_recorded(what, t)
    kind = dtypes.get(t.dtype)
    if t.dim() != 3 or kind is None or t.get_device() != device or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{what}: [experts, outer, inner] of {' or '.join(map(str, dtypes))} on cuda:{device}, rows' "
                         f"elements side by side, is needed, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on "
                         f"{t.device}")
    n, outer, inner = t.shape
    row = t.stride(1) if outer > 1 else inner
    return B.gro_experts(t.data_ptr(), outer, inner, row, t.stride(0) if n > 1 else outer * row, n, kind, 0)


def _index(what: str, t, device, dtypes, n=None) -> int:
    """The kind of a contiguous list of whole numbers on this GPU."""
    kind = dtypes.get(t.dtype)
    if kind is None or t.dim() != 1 or t.get_device() != device or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what}: {'' if n is None else f'{n} '}contiguous {' or '.join(map(str, dtypes))} on "
                         f"cuda:{device} are needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return kind


def _flat(ids):
    return ids if ids.dim() == 1 and ids.is_contiguous() else ids.contiguous().view(-1)


def _gpu(t) -> int:
    device = t.get_device()
    if device < 0:
        raise ValueError(f"the layers' tensors are on a GPU, got {t.device}")
    return device


def _call(device, stream, tensors, made, fn, *args) -> None:
    """fn(..., stream handle) with the tensors' GPU current.  A stream that is not the current one waits for tensors
    that this call has ``made`` on the current one, and the tensors it uses are recorded with the allocator."""
    s = torch.cuda.current_stream(device)
    if stream is not None and stream != s:
        if made:
            stream.wait_stream(s)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        s = stream
    if torch.cuda.current_device() == device:
        fn(*args, s.cuda_stream)
    else:
        with torch.cuda.device(device):
            fn(*args, s.cuda_stream)


_count = torch.autograd.graph.increment_version


def _wrote(out) -> None:
    """An operation in place on the caller's tensor, as autograd counts them."""
    _count(out)


def _aligned(room) -> int:
    return (room.data_ptr() + 255) // 256 * 256


def _room(nbytes: int, device):
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=torch.device("cuda", device)) if nbytes else None


def lookup(table, ids, scale: float = 1.0, first_row: int = 0, out=None, dtype=None, stream=None):
    """``scale * table[ids - first_row]`` (gro_lookup), zeros for ids of another shard of the table; ids of any
    shape, the result has it with the table's width behind.  ``out``: a matrix of a row for each id, or one is
    allocated in ``dtype``, by default the table's."""
    device = _gpu(table)
    flat = _flat(ids)
    kind = _index("ids", flat, device, _IDS)
    n = flat.numel()
    rows = torch.empty((n, table.shape[-1]), dtype=dtype or table.dtype, device=table.device) if out is None else out
    m, o = _matrix("table", table, device), _matrix("out", rows, device)
    if o.rows != n:
        raise ValueError(f"out: {n} rows are needed, got {o.rows}")
    _call(device, stream, (table, flat, rows), out is None or flat is not ids, B.gro_lookup, m, first_row,
          flat.data_ptr(), kind, scale, o)
    if out is None:
        return rows.view(*ids.shape, o.cols)
    _wrote(out)
    return out


class RowOrder:
    """Positions sorted by the row of a table that they name, for up to ``n`` ids and a table (or a shard of one) of
    ``n_rows``, with what ``sort`` and ``lookup_grad`` (of up to ``width`` columns) need allocated once.  ``order``
    and ``starts`` are those of the last ``sort``: also an expert's runs of rows, for the products below, from a
    router's choices with ``n_rows`` experts.  One sort or gradient at a time: on another stream than the last
    call's, order it after that one."""

    def __init__(self, n: int, n_rows: int, width: int = 0, device="cuda"):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"the layers' tensors are on a GPU, got {device}")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self._gpu = self.device.index
        self.n, self.n_rows, self.width, self.used = int(n), int(n_rows), int(width), 0
        self._sort_bytes = B.gro_row_sort_workspace(self.n, self.n_rows)
        self._bytes = max(self._sort_bytes, B.gro_lookup_grad_workspace(self.n, self.width))
        self.workspace = torch.empty(self._bytes + 256, dtype=torch.uint8, device=self.device)
        self._ws = _aligned(self.workspace)
        self._order = torch.zeros(self.n, dtype=torch.int32, device=self.device)
        self.starts = torch.zeros(self.n_rows + 1, dtype=torch.int32, device=self.device)
        born = torch.cuda.current_stream(self.device)
        born.synchronize()                  # so that any stream may be the first to use them
        self._seen = {born.cuda_stream}     # streams that need no (further) recording of the object's own memory

    @property
    def order(self):
        """A position for each id of the last sort; those behind ``starts[-1]`` say nothing."""
        return self._order[:self.used]

    def _run(self, stream, tensors, made, fn, *args) -> None:
        s = torch.cuda.current_stream(self._gpu) if stream is None else stream
        if s.cuda_stream not in self._seen:
            for t in (self._order, self.starts, self.workspace):
                t.record_stream(s)
            self._seen.add(s.cuda_stream)
        _call(self._gpu, stream, tensors, made, fn, *args)

    def sort(self, ids, first_row: int = 0, stream=None):
        """gro_row_sort: (order, starts) of these ids, read in order of their elements."""
        flat = _flat(ids)
        kind = _index("ids", flat, self._gpu, _IDS)
        n = flat.numel()
        if n > self.n:
            raise ValueError(f"{n} ids, {self.n} at most")
        self._run(stream, (flat,), flat is not ids, B.gro_row_sort, flat.data_ptr(), kind, n, first_row, self.n_rows,
                  self._order.data_ptr(), self.starts.data_ptr(), self._ws, self._bytes)
        self.used = n
        return self.order, self.starts

    def lookup_grad(self, dy, scale: float = 1.0, out=None, accumulate: bool = False, dtype=None, stream=None):
        """gro_lookup_grad of the last sorted ids: ``out[r] = scale * sum of dy[i]`` over row r's positions, written
        or (``accumulate``) added.  ``dy``: a row for each id.  ``out``: [n_rows, width], or one is allocated in
        ``dtype``, by default dy's."""
        if dy.dim() < 2:
            raise ValueError(f"dy: a row for each id is needed, got {tuple(dy.shape)}")
        flat = dy if dy.dim() == 2 else dy.flatten(0, -2)
        d = _matrix("dy", flat, self._gpu)
        if accumulate and out is None:
            raise ValueError("accumulate adds to an array that is given")
        given = out is not None
        if not given:
            out = torch.empty((self.n_rows, flat.shape[1]), dtype=dtype or flat.dtype, device=self.device)
        o = _matrix("out", out, self._gpu)
        if d.rows != self.used or o.rows != self.n_rows or d.cols > self.width:
            raise ValueError(f"{self.used} ids were sorted for {self.n_rows} rows of up to {self.width} elements, got "
                             f"dy {tuple(dy.shape)} and out {tuple(out.shape)}")
        self._run(stream, (flat, out), not given or flat is not dy, B.gro_lookup_grad, d,
                  self._order.data_ptr(), self.starts.data_ptr(), scale, bool(accumulate), o, self._ws, self._bytes)
        if given:
            _wrote(out)
        return out


_BF16 = {torch.bfloat16: B.GRO_BF16}
_I32 = {torch.int32: B.GRO_INT32}


def _product(fn, in_name, rows, weight, starts, out, out_name, cols, dtype, stream):
    device = _gpu(rows)
    w = _experts("weight", weight, device, _BF16)
    _index("starts", starts, device, _I32, w.n_experts + 1)
    given = out is not None
    if not given:  # rows that no expert has are not written by the product
        out = torch.zeros((rows.shape[0], getattr(w, cols)), dtype=dtype or rows.dtype, device=rows.device)
    x, y = _matrix(in_name, rows, device, _BF16), _matrix(out_name, out, device)
    nbytes = B.gro_experts_workspace(w.n_experts, x.rows, w.inner, w.outer)
    room = _room(nbytes, device)
    _call(device, stream, (rows, weight, starts, out, room), not given or room is not None, fn, x, w, starts.data_ptr(), y,
          _aligned(room) if nbytes else 0, nbytes)
    if given:
        _wrote(out)
    return out


def experts_forward(x, weight, starts, out=None, dtype=None, stream=None):
    """y = x W_e^T for the rows ``starts[e]:starts[e + 1]`` of each expert (gro_experts_forward).  ``x`` [rows, inner] and
    ``weight`` [experts, outer, inner] BF16, ``starts`` int32 on the GPU, ``out`` [rows, outer] BF16 or FP32; one of
    zeros is allocated in ``dtype``, by default BF16, when it is not given.  Rows of no expert stay as they were."""
    return _product(B.gro_experts_forward, "x", x, weight, starts, out, "y", "outer", dtype, stream)


def experts_input_grad(dy, weight, starts, out=None, dtype=None, stream=None):
    """dx = dy W_e (gro_experts_input_grad); ``dy`` [rows, outer], ``out`` [rows, inner], else as experts_forward."""
    return _product(B.gro_experts_input_grad, "dy", dy, weight, starts, out, "dx", "inner", dtype, stream)


def experts_weight_grad(dy, x, starts, out=None, accumulate: bool = False, dtype=None, stream=None):
    """dW_e = dy^T x over each expert's rows (gro_experts_weight_grad), written or (``accumulate``) added; zeros, or
    what was there, for an expert without rows.  ``out`` [experts, outer, inner] BF16 or FP32, or one is allocated in
    ``dtype``, by default BF16."""
    device = _gpu(dy)
    d, r = _matrix("dy", dy, device, _BF16), _matrix("x", x, device, _BF16)
    _index("starts", starts, device, _I32)
    if accumulate and out is None:
        raise ValueError("accumulate adds to an array that is given")
    given = out is not None
    if not given:
        out = torch.empty((max(starts.numel() - 1, 0), d.cols, r.cols), dtype=dtype or dy.dtype, device=dy.device)
    w = _experts("out", out, device)
    _index("starts", starts, device, _I32, w.n_experts + 1)
    nbytes = B.gro_experts_workspace(w.n_experts, d.rows, w.inner, w.outer)
    room = _room(nbytes, device)
    _call(device, stream, (dy, x, starts, out, room), not given or room is not None, B.gro_experts_weight_grad, d, r,
          starts.data_ptr(), bool(accumulate), w, _aligned(room) if nbytes else 0, nbytes)
    if given:
        _wrote(out)
    return out
