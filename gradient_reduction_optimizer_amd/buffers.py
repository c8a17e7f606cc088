"""Device-memory plumbing around a plan: PyTorch allocates the buffers the
C ABI asks for, and copies per-tensor gradients into the bucket buffers.

Nothing here computes any part of the path; it only allocates and moves
bytes (the kernels in libgro.so do the work).
"""
from __future__ import annotations

from itertools import compress
from operator import attrgetter, eq
from typing import List, Optional, Sequence, Tuple

from . import binding as B


class Plan:
    """Owns a plan handle and caches its info, tensor rows and buckets."""

    def __init__(self, tensors: Sequence, R: int, bucket_elems: int):
        self.handle = B.gro_plan_create(tensors, R, bucket_elems)
        self.R = int(R)
        # this rank's shard index per tensor, as registered (-1 unless Shard)
        self.shard_index = [int(B._attr(t, "shard_index", -1)) for t in tensors]
        self.info = B.gro_plan_get_info(self.handle)
        self.tensors = [B.gro_plan_tensor(self.handle, i) for i in range(self.info["n_tensors"])]
        self.buckets = [B.gro_plan_bucket(self.handle, b) for b in range(self.info["n_buckets"])]

    def close(self) -> None:
        if self.handle:
            B.gro_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def segments(self, i: int) -> List[Tuple[int, int, int, int]]:
        """Where tensor i's elements sit in the bucket buffers:
        [(bucket, offset in bucket, offset in tensor, count)]."""
        t = self.tensors[i]
        out = []
        if t["n_buckets"] <= 0:
            return out
        start, end = t["flat_offset"], t["flat_offset"] + t["numel"]
        for b in range(t["first_bucket"], t["first_bucket"] + t["n_buckets"]):
            bk = self.buckets[b]
            lo, hi = max(start, bk["flat_base"]), min(end, bk["flat_base"] + bk["len"])
            if hi > lo:
                out.append((b, lo - bk["flat_base"], lo - start, hi - lo))
        return out


class DeviceState:
    """FP32 accumulator / master / m / v, the BF16 parameter copy and the
    workspace for one plan, allocated with torch on ``device`` and bound.
    With ``static_workspace`` no workspace is allocated: the plan is bound
    to the library's own per-GPU workspace (gro_plan_bind_static).  With
    ``coded_moments`` the moments are held in 8 bits: ``m_code`` and
    ``v_code`` are code bytes, ``m_scale`` and ``v_scale`` the blocks' scales,
    ``coded`` their four pointers, for gro_clip_adamw_coded, and there are
    no ``m`` and ``v``."""

    def __init__(self, plan: Plan, device="cuda", with_bf16: bool = True, stream=None,
                 static_workspace: bool = False, coded_moments: bool = False):
        import torch
        self.plan = plan
        self.device = torch.device(device)
        n = max(int(plan.info["n_flat"]), 1)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.acc = torch.zeros(n, **f32)
        self.master = torch.zeros(n, **f32)
        self.coded = None
        if coded_moments:
            self.m = self.v = None
            self.m_code = torch.zeros(n, dtype=torch.uint8, device=self.device)
            self.v_code = torch.zeros(n, dtype=torch.uint8, device=self.device)
            self.m_scale = torch.zeros(-(-n // B.GRO_CODED_BLOCK), **f32)
            self.v_scale = torch.zeros(-(-n // B.GRO_CODED_BLOCK), **f32)
            self.coded = tuple(t.data_ptr() for t in (self.m_code, self.v_code, self.m_scale, self.v_scale))
        else:
            self.m = torch.zeros(n, **f32)
            self.v = torch.zeros(n, **f32)
        self.p_bf16 = torch.zeros(n, dtype=torch.bfloat16, device=self.device) if with_bf16 else None
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        if not static_workspace:
            nbytes = int(plan.info["workspace_bytes"])
            self.workspace = torch.zeros(nbytes + 256, dtype=torch.uint8, device=self.device)
        # the arrays' memory and zeros are the current stream's
        self._keep(x for x in vars(self).values() if isinstance(x, torch.Tensor))
        self.stream.wait_stream(torch.cuda.current_stream(self.device))
        if static_workspace:
            self.workspace, self.ws_ptr, self.ws_bytes = None, None, 0
            B.gro_plan_bind_static(plan.handle, self.stream.cuda_stream)
            return
        base = self.workspace.data_ptr()
        self.ws_ptr = (base + 255) // 256 * 256
        self.ws_bytes = nbytes
        B.gro_plan_bind(plan.handle, self.ws_ptr, nbytes, self.stream.cuda_stream)

    def _keep(self, tensors) -> None:
        """Tensors of the current stream that the state's stream uses: their
        memory is not handed out again before that stream is done with it."""
        import torch
        if self.stream != torch.cuda.current_stream(self.device):
            for t in tensors:
                t.record_stream(self.stream)

    def moments(self):
        """The moments as flat FP32 arrays (m, v): the state's own, or, held in
        8 bits, decoded ones (zeros between buckets), on the current stream
        after the work that the state's stream has been given.  The state's
        stream waits for the decoding, whose codes its next step writes."""
        import torch
        here = torch.cuda.current_stream(self.device)
        here.wait_stream(self.stream)
        if self.coded is None:
            return self.m, self.v
        m, v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        B.gro_moments_decode(self.plan.handle, self.coded, m.data_ptr(), v.data_ptr(), here.cuda_stream)
        self.stream.wait_stream(here)
        return m, v

    def set_moments(self, m, v) -> None:
        """Take flat FP32 moments over, encoded if the state holds 8 bits, on
        the current stream, which the state's stream then waits for."""
        import torch
        for name, t in (("m", m), ("v", v)):
            if t.dtype != torch.float32 or t.shape != self.master.shape:
                raise ValueError(f"{name}: flat FP32 moments have shape {tuple(self.master.shape)}, "
                                 f"got {t.dtype} {tuple(t.shape)}")
        here = torch.cuda.current_stream(self.device)
        here.wait_stream(self.stream)
        if self.coded is None:
            self.m.copy_(m)
            self.v.copy_(v)
        else:
            m, v = m.to(self.device).contiguous(), v.to(self.device).contiguous()
            B.gro_moments_encode(self.plan.handle, m.data_ptr(), v.data_ptr(), self.coded, here.cuda_stream)
        self.stream.wait_stream(here)

    def grad_buffers(self) -> List:
        """One [slots, slot_stride] buffer per bucket (zeros, written on the
        current stream), BF16 or FP32 as the bucket's gradient type says."""
        import torch
        bufs = [torch.zeros((bk["slots"], bk["slot_stride"]),
                            dtype=torch.float32 if bk["grad_dtype"] == B.GRO_GRAD_FP32 else torch.bfloat16,
                            device=self.device)
                for bk in self.plan.buckets]
        self._keep(bufs)
        return bufs

    def pack(self, bufs: List, i: int, slot_grads: Sequence) -> None:
        """Copy tensor i's per-slot gradients (1-D, length numel, the
        bucket's type) into the bucket buffers."""
        for b, dst, src, cnt in self.plan.segments(i):
            for r, g in enumerate(slot_grads):
                bufs[b][r, dst:dst + cnt].copy_(g[src:src + cnt], non_blocking=True)

    def flat_view(self, arr, i: int):
        """Tensor i's slice of a flat array (acc, master, m, v, p_bf16)."""
        t = self.plan.tensors[i]
        off = t["flat_offset"]
        return arr[off:off + t["numel"]] if off >= 0 else arr[:0]


def _check_array(what: str, t, dtype, shape, device) -> None:
    """A contiguous tensor of this type and shape on this GPU.  A flat one of as
    many elements has them in the same order, and so does any for a flat shape."""
    if (t.dtype != dtype or t.numel() != shape.numel() or t.get_device() != device.index or not t.is_contiguous()
            or (t.shape != shape and t.dim() != 1 and len(shape) != 1)):
        raise ValueError(f"{what}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


class TensorGroup:
    """Many FP32 master tensors stepped at once where they lie, bound to a
    workspace of its own: gro_group_norm and gro_group_clip_adamw.

    ``masters``: contiguous FP32 tensors of one GPU.  A tensor's copy, moments
    and gradients have its shape, or they or it are flat.  Per tensor, as one value
    for all or a list: ``state_bits`` (32 or 8: how the moments are held),
    ``no_decay``, ``grad_dtype`` (torch.bfloat16 or torch.float32).
    ``params_bf16``: BF16 copies to update along, None for a tensor without.
    ``states``: per tensor (m, v) or, in 8 bits, (m, v, m_scale, v_scale);
    zeros are allocated when it is not given.  The tensors stay the caller's;
    the group keeps references to them.

    A call runs on ``stream``, by default the current one; ordering it after
    the work that made its inputs is the caller's, as with any operation on
    another stream.  Memory is not: whatever the group or the caller lets go of
    stays as it is until the enqueued work is done with it.  A captured graph
    holds pointers only: group and gradients are kept as long as it is replayed."""

    def __init__(self, masters: Sequence, state_bits=32, no_decay=False, grad_dtype=None,
                 params_bf16: Optional[Sequence] = None, states: Optional[Sequence] = None):
        import torch
        self.handle = 0
        n = len(masters)
        per_tensor = lambda x: list(x) if isinstance(x, (list, tuple)) else [x] * n  # noqa: E731
        bits = per_tensor(state_bits)
        no_decay = per_tensor(no_decay)
        grad_dtype = per_tensor(torch.bfloat16 if grad_dtype is None else grad_dtype)
        copies = [None] * n if params_bf16 is None else list(params_bf16)
        for what, x in (("state_bits", bits), ("no_decay", no_decay), ("grad_dtype", grad_dtype),
                        ("params_bf16", copies), ("states", bits if states is None else states)):
            if len(x) != n:
                raise ValueError(f"{what}: {len(x)} entries for {n} tensors")
        if any(b not in (8, 32) for b in bits):
            raise ValueError("state_bits is 8 or 32")
        if any(d not in (torch.bfloat16, torch.float32) for d in grad_dtype):
            raise ValueError("grad_dtype is torch.bfloat16 or torch.float32")
        self.device = masters[0].device if n else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError(f"a group's tensors are on a GPU, got {self.device}")
        self.masters, self.copies, self.bits, self.grad_dtype = list(masters), copies, bits, grad_dtype
        self.states = []
        rows = []
        kinds = {32: (torch.float32,) * 2, 8: (torch.uint8,) * 2 + (torch.float32,) * 2}
        for i, p in enumerate(masters):
            k = p.numel()
            _check_array(f"master {i}", p, torch.float32, p.shape, self.device)
            if copies[i] is not None:
                _check_array(f"params_bf16 {i}", copies[i], torch.bfloat16, p.shape, self.device)
            dtypes = kinds[bits[i]]
            blocks = torch.Size([-(-k // B.GRO_CODED_BLOCK)])
            shapes = (p.shape, p.shape, blocks, blocks)[:len(dtypes)]
            if states is None:
                st = tuple(torch.zeros(s.numel(), dtype=d, device=self.device) for s, d in zip(shapes, dtypes))
            else:
                st = tuple(states[i])
                if len(st) != len(dtypes):
                    raise ValueError(f"states {i}: {len(dtypes)} tensors are needed, got {len(st)}")
                for t, s, d in zip(st, shapes, dtypes):
                    _check_array(f"states {i}", t, d, s, self.device)
            self.states.append(st)
            rows.append([p.data_ptr(), *[t.data_ptr() for t in st], *[0] * (4 - len(st)),
                         0 if copies[i] is None else copies[i].data_ptr()])
        self.handle = B.gro_group_create([dict(numel=p.numel(), no_decay=bool(nd), coded_moments=b == 8,
                                               fp32_grad=gd == torch.float32)
                                          for p, nd, b, gd in zip(masters, no_decay, bits, grad_dtype)])
        self.info = B.gro_group_get_info(self.handle)
        nbytes = int(self.info["workspace_bytes"])
        self.workspace = torch.zeros(nbytes + 256, dtype=torch.uint8, device=self.device)
        self._shapes = [p.shape for p in masters]
        self._shaped = [p.dim() != 1 for p in masters]
        self._flat = [not x for x in self._shaped]
        self._fit = (list(compress(self._shapes, self._shaped)),
                     [p.numel() for p in compress(masters, self._flat)])
        self._on = [self.device.index] * n
        born = torch.cuda.current_stream(self.device.index).cuda_stream
        # waits for the current stream, and so for the zeros above too
        self._call(B.gro_group_bind, rows, (self.workspace.data_ptr() + 255) // 256 * 256, nbytes, born)
        self._seen = {born}       # streams that need no (further) recording of the group's own memory
        self._grads, self._grads_on = None, None
        # views of one allocation share their version counter
        roots = {id(r): r for t in (*self.masters, *copies) if t is not None for r in (t if t._base is None else t._base,)}
        self._written = self._all = list(roots.values())
        self._count = torch.autograd.graph.increment_version

    def close(self) -> None:
        if self.handle:
            B.gro_group_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def norm(self, grads: Sequence, window_size: int = 1, stream=None) -> None:
        """gro_group_norm of ``grads`` (one per tensor, None for a tensor left
        out of this step) on ``stream``, by default the current one."""
        ptrs = self._pointers(grads)
        s = self._use(stream, grads)
        self._call(B.gro_group_norm, ptrs, window_size, s)
        self._grads, self._grads_on = list(grads), s  # in place until clip_adamw has been enqueued
        self._written = self._all if 0 not in ptrs else [t for q, (p, c) in zip(ptrs, zip(self.masters, self.copies))
                                                         if q for t in (p, c) if t is not None]

    def _pointers(self, grads: Sequence) -> List[int]:
        """The gradients' pointers, 0 for None, after checking each: property
        by property over the whole list, which for 4000 tensors took 0.6 to 0.7 ms of
        the host's time against 1.5 ms tensor by tensor.  Shapes are dropped
        one by one: a list of 4000 made Python's garbage collector run five
        times a call, 1.2 ms."""
        import torch
        if len(grads) != len(self.masters):
            raise ValueError(f"{len(grads)} gradients for {len(self.masters)} tensors")
        T = torch.Tensor
        try:
            shapes, counts = self._fit
            if (all(map(eq, map(T.size, compress(grads, self._shaped)), shapes))
                    and list(map(T.numel, compress(grads, self._flat))) == counts
                    and list(map(T.get_device, grads)) == self._on
                    and list(map(attrgetter("dtype"), grads)) == self.grad_dtype and all(map(T.is_contiguous, grads))):
                return list(map(T.data_ptr, grads))
        except TypeError:  # None among them
            pass
        ptrs = []
        for i, g in enumerate(grads):
            if g is not None:
                _check_array(f"gradient {i}", g, self.grad_dtype[i], self._shapes[i], self.device)
            ptrs.append(0 if g is None else g.data_ptr())
        return ptrs

    def _call(self, fn, *args):
        """fn(handle, ...) with the group's device current."""
        import torch
        if torch.cuda.current_device() == self.device.index:
            return fn(self.handle, *args)
        with torch.cuda.device(self.device):
            return fn(self.handle, *args)

    def _use(self, stream, grads, recorded=None) -> int:
        """The handle of the stream that a call runs on.  Memory that the call
        uses there is recorded with the allocator, so that it is not handed
        out again before that stream is done with it: the group's own once per
        stream, gradients in every call, unless they are ``recorded`` on that
        stream already or both it and the current one are the default stream
        (0), where gradients usually come from and recording 4000 of them would
        take longer than the checks."""
        import torch
        here = torch.cuda.current_stream
        s = here(self.device.index) if stream is None else stream
        handle = s.cuda_stream
        if handle not in self._seen:
            for t in (self.workspace, *self.masters, *self.copies, *(x for st in self.states for x in st)):
                if t is not None:
                    t.record_stream(s)
            self._seen.add(handle)
        if grads is not None and handle != recorded and (
                handle or (stream is not None and here(self.device.index).cuda_stream)):
            for g in grads:
                if g is not None:
                    g.record_stream(s)
        return handle

    def clip_adamw(self, max_norm: float, hp: dict, step: int, stream=None) -> None:
        """gro_group_clip_adamw of the gradients given to ``norm``, on
        ``stream``, by default the current one.  Counts as an operation in
        place on the masters and copies it writes, so that autograd refuses a
        backward pass through a graph that saved them from before (a replay of
        a captured step does not: nothing tells autograd of it)."""
        s = self._use(stream, self._grads, self._grads_on)
        try:
            self._call(B.gro_group_clip_adamw, max_norm, hp, step, s)
        except B.GroError as e:
            if e.code == B.GRO_E_HIP:   # some kinds of tensors may have been updated
                self._count(self._written)
            raise
        self._count(self._written)
        self._grads, self._grads_on, self._written = None, None, self._all

    def get_norm(self):
        """(norm, norm_sq, finite) of the last ``norm``; waits for its stream."""
        return self._call(B.gro_group_get_norm)
