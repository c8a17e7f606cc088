"""CPU: what the layers' entry points refuse -- every refusal comes before any
device work, so the pointers are made up -- what they say of workspaces, and what the
Python calls check of tensors, on host tensors that say they are on GPU 0."""
import pytest
import torch

from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd import layers as L
from gradient_reduction_optimizer_amd.buffers import DeviceState, Plan

A, BB, C, D, WS = 1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32     # made-up arrays far apart
BF16, FP32 = B.GRO_BF16, B.GRO_FP32


def M(at, rows, cols, stride=None, type=BF16, reserved=0):
    return B.gro_matrix(at, rows, cols, cols if stride is None else stride, type, reserved)


def W(at, n, outer, inner, stride=None, expert=None, type=BF16, reserved=0):
    stride = inner if stride is None else stride
    return B.gro_experts(at, outer, inner, stride, outer * stride if expert is None else expert, n, type, reserved)


def refused(fn, *args, kind="invalid"):
    with pytest.raises(B.GroError) as e:
        fn(*args)
    assert e.value.kind == kind and str(e.value)


def test_row_sort_refuses():
    ok = dict(ids=A, type=B.GRO_INT64, n=100, first=0, rows=10, order=BB, starts=C, ws=WS, bytes=1 << 30)

    def sort(**k):
        a = {**ok, **k}
        B.gro_row_sort(a["ids"], a["type"], a["n"], a["first"], a["rows"], a["order"], a["starts"], a["ws"], a["bytes"], 0)

    for bad in (dict(type=2), dict(type=-1), dict(n=-1), dict(n=2 ** 31), dict(rows=-1), dict(rows=B.GRO_MAX_TABLE_ROWS + 1),
                dict(first=-1), dict(first=2 ** 63 - 5), dict(ids=0), dict(ids=A + 4), dict(type=B.GRO_INT32, ids=A + 2),
                dict(order=0), dict(order=BB + 2), dict(starts=0), dict(starts=C + 1), dict(order=A), dict(order=A + 796),
                dict(starts=A - 40), dict(starts=BB + 396), dict(starts=BB - 40), dict(n=9000, ws=0),
                dict(n=9000, ws=WS + 128), dict(n=9000, bytes=B.gro_row_sort_workspace(9000, 10) - 1), dict(n=9000, ws=A),
                dict(n=9000, ws=BB), dict(n=9000, ws=C), dict(n=9000, ws=BB - 256)):
        refused(lambda bad=bad: sort(**bad))


def test_lookup_refuses():
    ok = dict(table=M(A, 50, 8), first=0, ids=BB, type=B.GRO_INT64, out=M(C, 20, 8))

    def lookup(**k):
        a = {**ok, **k}
        B.gro_lookup(a["table"], a["first"], a["ids"], a["type"], 1.0, a["out"], 0)

    for bad in (dict(table=M(A, 50, 9)), dict(table=M(A + 1, 50, 8)), dict(table=M(A + 2, 50, 8, type=FP32)),
                dict(table=M(0, 50, 8)), dict(table=M(A, 50, 8, 7)), dict(table=M(A, 50, 8, -8)), dict(table=M(A, 50, 8, type=2)),
                dict(table=M(A, 50, 8, reserved=1)), dict(table=M(A, -1, 8)), dict(table=M(A, 50, 8, 2 ** 41)),
                dict(table=M(A, B.GRO_MAX_TABLE_ROWS + 1, 8)), dict(out=M(0, 20, 8)), dict(out=M(C, 20, 8, 4)),
                dict(out=M(C, 2 ** 31, 8)), dict(out=M(A, 20, 8)), dict(out=M(A + 798, 20, 8)), dict(out=M(BB, 20, 8)),
                dict(out=M(BB - 318, 20, 8)), dict(ids=0), dict(ids=BB + 4), dict(type=7), dict(first=-1),
                # rows that begin within the table's, though both lie 32 elements apart
                dict(table=M(A, 50, 8, 32), out=M(A + 14, 20, 8, 32)), dict(table=M(A + 14, 50, 8, 32), out=M(A, 20, 8, 32)),
                # and 50 elements around the end of its row
                dict(table=M(A, 50, 8, 32), out=M(A + 2 * 26, 20, 8, 32))):
        refused(lambda bad=bad: lookup(**bad))


def test_lookup_grad_refuses():
    need = B.gro_lookup_grad_workspace(1000, 8)
    ok = dict(dy=M(A, 1000, 8), order=BB, starts=C, accumulate=0, out=M(D, 30, 8), ws=WS, bytes=need)

    def grad(**k):
        a = {**ok, **k}
        B.gro_lookup_grad(a["dy"], a["order"], a["starts"], 1.0, a["accumulate"], a["out"], a["ws"], a["bytes"], 0)

    assert need > 0
    for bad in (dict(dy=M(A, 1000, 9)), dict(dy=M(0, 1000, 8)), dict(dy=M(A, 1000, 8, type=3)), dict(order=0), dict(order=BB + 1),
                dict(starts=0), dict(starts=C + 2), dict(accumulate=2), dict(out=M(D, 30, 8, 7)), dict(out=M(A, 30, 8)),
                dict(out=M(BB, 30, 8)), dict(out=M(C, 30, 8)), dict(out=M(D, B.GRO_MAX_TABLE_ROWS + 1, 8)),
                dict(dy=M(A, 1, (1 << 24) + 1), out=M(D, 1, (1 << 24) + 1), bytes=1 << 40), dict(ws=0), dict(ws=WS + 64), dict(bytes=need - 1), dict(ws=A), dict(ws=BB), dict(ws=C), dict(ws=D)):
        refused(lambda bad=bad: grad(**bad))


def test_products_refuse():
    ok = dict(rows=M(A, 100, 8), w=W(BB, 4, 16, 8), starts=C, out=M(D, 100, 16))
    back = dict(rows=M(A, 100, 16), w=W(BB, 4, 16, 8), starts=C, out=M(D, 100, 8))

    def call(fn, base, **k):
        a = {**base, **k}
        fn(a["rows"], a["w"], a["starts"], a["out"], a.get("ws", 0), a.get("bytes", 0), 0)

    shared = (dict(w=W(0, 4, 16, 8)), dict(w=W(BB + 1, 4, 16, 8)), dict(w=W(BB, 4, 16, 8, 7)), dict(w=W(BB, 4, 16, 8, expert=127)),
              dict(w=W(BB, -1, 16, 8)), dict(w=W(BB, B.GRO_MAX_EXPERTS + 1, 16, 8)), dict(w=W(BB, 4, 16, 8, type=FP32)),
              dict(w=W(BB, 4, 16, 8, reserved=1)), dict(w=W(BB, 4, 16, 8, expert=2 ** 40)), dict(starts=0), dict(starts=C + 2),
              dict(w=W(BB, 4, 17, 9)))
    for bad in (*shared, dict(rows=M(A, 100, 8, type=FP32)), dict(rows=M(A, 99, 8)), dict(rows=M(A, 100, 16)),
                dict(out=M(D, 100, 8)), dict(out=M(A, 100, 16)), dict(out=M(BB, 100, 16)), dict(out=M(BB + 1022, 100, 16)),
                dict(out=M(C, 100, 16)), dict(out=M(D, 100, 16, 8)), dict(out=M(D, 100, 16, type=5))):
        refused(lambda bad=bad: call(B.gro_experts_forward, ok, **bad))
    for bad in (*shared, dict(rows=M(A, 100, 16, type=FP32)), dict(rows=M(A, 100, 8)), dict(out=M(D, 100, 16))):
        refused(lambda bad=bad: call(B.gro_experts_input_grad, back, **bad))
    # few tiles and a long sum, which is taken in parts
    need = B.gro_experts_workspace(1, 20, 8192, 64)
    long = dict(rows=M(A, 20, 8192), w=W(BB, 1, 64, 8192), out=M(D, 20, 64), ws=WS, bytes=need)
    assert need >= 2 * 20 * 64 * 4
    for bad in (dict(ws=0), dict(ws=WS + 8), dict(bytes=need - 1 if need == 32 * 20 * 64 * 4 else 0), dict(ws=A), dict(ws=BB),
                dict(ws=C - 256), dict(ws=D)):
        refused(lambda bad=bad: call(B.gro_experts_forward, ok, **{**long, **bad}))
    huge = dict(rows=M(A, 2 ** 31 - 2 ** 17, 64), w=W(BB, 1, 2 ** 24, 64), out=M(1 << 50, 2 ** 31 - 2 ** 17, 2 ** 24))
    refused(lambda: call(B.gro_experts_forward, ok, **huge))


def test_weight_gradient_refuses():
    ok = dict(dy=M(A, 100, 16), x=M(BB, 100, 8), starts=C, accumulate=0, dw=W(D, 4, 16, 8, type=FP32), ws=WS, bytes=1 << 30)

    def grad(**k):
        a = {**ok, **k}
        B.gro_experts_weight_grad(a["dy"], a["x"], a["starts"], a["accumulate"], a["dw"], a["ws"], a["bytes"], 0)

    for bad in (dict(dy=M(A, 99, 16)), dict(dy=M(A, 100, 8)), dict(x=M(BB, 100, 16)), dict(dy=M(A, 100, 16, type=FP32)),
                dict(x=M(BB, 100, 8, type=FP32)), dict(starts=0), dict(accumulate=-1), dict(dw=W(D, 4, 16, 8, type=4)),
                dict(dw=W(A, 4, 16, 8)), dict(dw=W(BB, 4, 16, 8)), dict(dw=W(C, 4, 16, 8)), dict(dw=W(D, 4, 16, 8, expert=100)),
                dict(dw=W(D, 4, 16, 8, 4)), dict(dw=W(D, 4, 15, 8))):
        refused(lambda bad=bad: grad(**bad))
    # long runs and few tiles are summed in parts
    need = B.gro_experts_workspace(1, 1 << 20, 64, 64)
    assert need > 0
    if need:
        long = dict(dy=M(A, 1 << 20, 64), x=M(BB, 1 << 20, 64), dw=W(D, 1, 64, 64), bytes=need)
        for bad in (dict(ws=0), dict(ws=WS + 8), dict(bytes=need - 1), dict(ws=A), dict(ws=BB), dict(ws=C - 256), dict(ws=D)):
            refused(lambda bad=bad: grad(**{**long, **bad}))


def test_workspaces():
    for fn, bad in ((B.gro_row_sort_workspace, ((-1, 5), (5, -1), (2 ** 31, 5), (5, B.GRO_MAX_TABLE_ROWS + 1))),
                    (B.gro_lookup_grad_workspace, ((-1, 5), (5, -1), (2 ** 31, 5))),
                    (B.gro_experts_workspace, ((-1, 5, 5, 5), (5000, 5, 5, 5), (5, -1, 5, 5), (5, 5, -1, 5),
                                                           (5, 5, 5, -1), (4096, 5, 2 ** 20, 2 ** 20)))):
        for args in bad:
            refused(fn, *args)
    assert B.gro_row_sort_workspace(0, 0) == 0 and B.gro_row_sort_workspace(8192, 1000) == 0
    sizes = [B.gro_row_sort_workspace(n, r) for n, r in ((8193, 0), (8193, 1000), (8193, 2000), (1 << 20, 2000), (2 ** 31 - 2 ** 16, 2000))]
    assert sizes == sorted(sizes) and all(s >= 8 * 8193 for s in sizes[2:]) and sizes[-1] >= 8 * (2 ** 31 - 2 ** 16)


def test_a_workspace_serves_shorter_lists():
    lengths = sorted(m + d for m in (511, 4096, 8192, 65_536, 131_072, 1 << 20, 1 << 21) for d in (-1, 0, 1, 4096))
    for rows in (0, 3, 1000, 1024, 1025, 30_000, 1 << 20):
        sizes = [B.gro_row_sort_workspace(n, rows) for n in lengths]
        assert sizes == sorted(sizes)
    for cols in (0, 1, 2048):
        sizes = [B.gro_lookup_grad_workspace(n, cols) for n in lengths]
        assert sizes == sorted(sizes)


@pytest.fixture
def on_gpu(monkeypatch):
    """Host tensors that say they are on GPU 0, and the library's calls as a list."""
    calls = []

    class Stream:
        cuda_stream = 7

        def synchronize(self):
            pass

    class Device:
        def __init__(self, *a):
            pass

        __enter__ = __exit__ = lambda *a: None

    current = Stream()
    for name in ("zeros", "empty"):
        fn = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, device=None, fn=fn, **k: fn(*a, **k))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", 0)))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    for name in ("gro_lookup", "gro_row_sort", "gro_lookup_grad", "gro_experts_forward", "gro_experts_input_grad",
                 "gro_experts_weight_grad"):
        monkeypatch.setattr(B, name, lambda *a, name=name: calls.append((name, a)))
    return calls


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_python_calls_check_their_tensors(on_gpu):
    ids, table = torch.zeros(6, dtype=torch.int64), bf(10, 8)
    for bad in (lambda: L.lookup(table.half(), ids), lambda: L.lookup(table.t(), ids), lambda: L.lookup(table[0], ids),
                lambda: L.lookup(table, ids.float()), lambda: L.lookup(table, ids, out=bf(5, 8)),
                lambda: L.lookup(table, ids, out=bf(6, 8).double())):
        with pytest.raises(ValueError):
            bad()
    by = L.RowOrder(6, 10, 8)
    for bad in (lambda: by.sort(torch.zeros(7, dtype=torch.int64)), lambda: by.sort(ids.short()),
                lambda: by.lookup_grad(bf(6, 8))):           # nothing sorted yet
        with pytest.raises(ValueError):
            bad()
    by.sort(ids)
    for bad in (lambda: by.lookup_grad(bf(5, 8)), lambda: by.lookup_grad(bf(6, 9)), lambda: by.lookup_grad(bf(8)),
                lambda: by.lookup_grad(bf(6, 8), out=bf(9, 8)), lambda: by.lookup_grad(bf(6, 8), accumulate=True),
                lambda: by.lookup_grad(bf(8, 6).t())):
        with pytest.raises(ValueError):
            bad()
    starts, w = torch.zeros(4, dtype=torch.int32), bf(3, 16, 8)
    for bad in (lambda: L.experts_forward(bf(5, 8).float(), w, starts), lambda: L.experts_forward(bf(5, 8), w.float(), starts),
                lambda: L.experts_forward(bf(5, 8), w, starts[:3]), lambda: L.experts_forward(bf(5, 8), w, starts.long()),
                lambda: L.experts_forward(bf(5, 8), w.transpose(1, 2), starts), lambda: L.experts_forward(bf(5, 8), w[0], starts),
                lambda: L.experts_forward(bf(5, 8), w, starts, out=bf(16, 5).t()),
                lambda: L.experts_weight_grad(bf(5, 16), bf(5, 8), starts, accumulate=True),
                lambda: L.experts_weight_grad(bf(5, 16), bf(5, 8), starts, out=bf(2, 16, 8)),
                lambda: L.experts_weight_grad(bf(5, 16).float(), bf(5, 8), starts)):
        with pytest.raises(ValueError):
            bad()
    assert [c[0] for c in on_gpu] == ["gro_row_sort"]


def test_python_calls_hand_over_what_the_tensors_are(on_gpu):
    big = bf(3, 40, 32)
    w = big[:, 4:20, 8:16]
    x, y = bf(5, 24)[:, 8:16], bf(5, 20)[:, :16]
    starts = torch.zeros(4, dtype=torch.int32)
    assert L.experts_forward(x, w, starts, out=y) is y
    name, (mx, mw, s, my, ws, nbytes, stream) = on_gpu.pop()
    assert name == "gro_experts_forward" and s == starts.data_ptr() and stream == 7
    assert (mx.data, mx.rows, mx.cols, mx.stride, mx.type) == (x.data_ptr(), 5, 8, 24, BF16)
    assert (mw.data, mw.outer, mw.inner, mw.stride, mw.expert_stride, mw.n_experts) == (w.data_ptr(), 16, 8, 32, 1280, 3)
    assert (my.data, my.rows, my.cols, my.stride) == (y.data_ptr(), 5, 16, 20)
    version = y._version
    L.experts_forward(x, w, starts, out=y)
    assert y._version == version + 1, "an operation in place, as autograd counts them"
    # a single row or matrix may have any stride
    L.experts_forward(bf(1, 8).as_strided((1, 8), (3, 1)), bf(1, 16, 8).as_strided((1, 16, 8), (5, 8, 1)), starts[:2])
    _, (mx, mw, *_) = on_gpu.pop()
    assert mx.stride == 8 and mw.expert_stride == 128
    # ids of any shape, also not contiguous
    ids = torch.arange(12).view(3, 4).t()
    assert L.lookup(bf(20, 8), ids).shape == (4, 3, 8)


def every_call(t, rows=lambda: bf(5, 8), back=lambda: bf(5, 16), matrices=lambda: bf(3, 16, 8)):
    """Each call with one of its tensors made by ``t``, and which: inputs and results."""
    ids, starts = torch.zeros(5, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)
    by = L.RowOrder(5, 10, 8)
    by.sort(ids)
    return {"table": lambda: L.lookup(t(bf(10, 8)), ids), "rows": lambda: L.lookup(bf(10, 8), ids, out=t(rows())),
            "dy": lambda: by.lookup_grad(t(rows())), "dy of the ids' shape": lambda: by.lookup_grad(t(bf(1, 5, 8))),
            "row gradient": lambda: by.lookup_grad(rows(), out=t(bf(10, 8))),
            "x": lambda: L.experts_forward(t(rows()), matrices(), starts), "w": lambda: L.experts_forward(rows(), t(matrices()), starts),
            "y": lambda: L.experts_forward(rows(), matrices(), starts, out=t(back())),
            "dy of rows": lambda: L.experts_input_grad(t(back()), matrices(), starts),
            "dx": lambda: L.experts_input_grad(back(), matrices(), starts, out=t(rows())),
            "dy of weights": lambda: L.experts_weight_grad(t(back()), rows(), starts),
            "x of weights": lambda: L.experts_weight_grad(back(), t(rows()), starts),
            "dw": lambda: L.experts_weight_grad(back(), rows(), starts, out=t(matrices()))}


def test_a_gradient_that_autograd_would_lose_is_refused(on_gpu):
    """The results take no part in autograd's graph: what would have to is refused, as torch refuses it for out=, and
    taken where nothing is recorded."""
    by = every_call(lambda t: t.requires_grad_())
    del on_gpu[:]
    for name, call in by.items():
        with pytest.raises(ValueError, match="autograd"):
            call()
        assert not on_gpu, name
        with torch.no_grad():
            call()
        with torch.inference_mode():
            call()
        assert len(on_gpu) == 2, name
        del on_gpu[:]
    for call in every_call(lambda t: t.requires_grad_().detach()).values():
        call()
    # so are they in an operation of the caller's own, whose forward and backward are recorded as one
    ids = torch.zeros(5, dtype=torch.int64)

    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table):
            return L.lookup(table, ids)

        @staticmethod
        def backward(ctx, dy):
            order = L.RowOrder(5, 10, 8)
            order.sort(ids)
            return order.lookup_grad(dy)

    table = bf(10, 8).requires_grad_()
    Lookup.apply(table).float().square().sum().backward()
    assert table.grad.shape == (10, 8)


@pytest.fixture
def forward_mode():
    """torch compiles its own formulas for it at the first level, which it cannot once functions are replaced."""
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        forward_ad.make_dual(torch.zeros(1), torch.ones(1))
    return forward_ad


def test_a_tangent_is_refused(forward_mode, on_gpu):
    forward_ad = forward_mode
    with forward_ad.dual_level():
        for name, call in every_call(lambda t: forward_ad.make_dual(t, torch.ones_like(t))).items():
            del on_gpu[:]
            with pytest.raises(ValueError, match="tangent"):
                call()
            assert not on_gpu, name
        for call in every_call(lambda t: t).values():
            call()


def test_rows_without_elements(on_gpu):
    """A gradient of width 0 in the ids' shape has a row for each id all the same."""
    by = L.RowOrder(6, 10, 0)
    by.sort(torch.zeros(2, 3, dtype=torch.int64))
    assert L.lookup(bf(10, 0), torch.zeros(2, 3, dtype=torch.int64)).shape == (2, 3, 0)
    for dy in (bf(2, 3, 0), bf(6, 0), bf(1, 2, 3, 0)):
        assert by.lookup_grad(dy).shape == (10, 0)
        _, (d, *_) = on_gpu.pop()
        assert (d.rows, d.cols) == (6, 0)
    by.sort(torch.zeros(0, 3, dtype=torch.int64))
    assert by.lookup_grad(bf(0, 3, 0)).shape == (10, 0)
    with pytest.raises(ValueError):
        by.lookup_grad(bf(2, 3, 0))
    # and several rows of a width, contiguous and not
    by = L.RowOrder(6, 10, 8)
    by.sort(torch.zeros(2, 3, dtype=torch.int64))
    base = bf(2, 6, 8)
    for dy, stride in ((base[:, ::2], 16), (base[:, :3], 8), (bf(2, 3, 8), 8), (bf(3, 2, 8).transpose(0, 1), 8)):
        by.lookup_grad(dy)
        _, (d, *_) = on_gpu.pop()
        assert (d.rows, d.cols, d.stride) == (6, 8, stride)


def test_a_view_of_a_gradient_slot():
    plan = Plan([dict(param_id=0, shape=(30, 4), placement="replicate"), dict(param_id=1, shape=(100, 8), placement="shard",
                                                                              shard_index=0),
                 dict(param_id=2, shape=(5,), placement="replicate", frozen=True)], 2, 500)
    st = object.__new__(DeviceState)
    st.plan = plan
    bufs = [torch.zeros(b["slots"], b["slot_stride"]) for b in plan.buckets]
    view = DeviceState.grad_view(st, bufs, 0, 1, (30, 4))
    view.fill_(3.0)
    other = [torch.zeros_like(b) for b in bufs]
    DeviceState.pack(st, other, 0, [torch.zeros(120), torch.full((120,), 3.0)])
    assert view.shape == (30, 4) and all(torch.equal(a, b) for a, b in zip(bufs, other))
    assert DeviceState.grad_view(st, bufs, 0, 0).shape == (120,)
    for i, slot in ((1, 0), (2, 0), (0, 2), (0, -1)):       # two buckets, no bucket, no such slot
        with pytest.raises(ValueError):
            DeviceState.grad_view(st, bufs, i, slot)
