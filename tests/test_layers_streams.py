"""CPU: the order and the memory of the layers' calls on streams of their own, on
stand-ins for streams that note what is asked of them, with host tensors that say
they are on GPU 0.  No kernel runs."""
import pytest
import torch

from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd import layers as L

BF16, I32 = torch.bfloat16, torch.int32


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waited, self.kept, self.calls = handle, [], [], []

    def wait_stream(self, other):
        # before the call, or it orders nothing
        self.waited.append((other, len(self.calls)))

    def synchronize(self):
        pass


class Streams:
    def __init__(self):
        self.default, self.side, self.third = Stream(0), Stream(7), Stream(9)
        self.now, self.entered, self.device = self.default, [], 0

    def clear(self):
        for s in (self.default, self.side, self.third):
            for notes in (s.waited, s.kept, s.calls):
                notes.clear()


@pytest.fixture
def gpu0(monkeypatch):
    st = Streams()

    class Device:
        def __init__(self, device):
            st.entered.append(device)

        __enter__ = __exit__ = lambda *a: None

    for name in ("zeros", "empty"):
        fn = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, device=None, fn=fn, **k: fn(*a, **k))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", 0)))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: s.kept.append(t.untyped_storage().data_ptr()))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: st.device)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: st.now)
    by_handle = {s.cuda_stream: s for s in (st.default, st.side, st.third)}
    for name in ("gro_lookup", "gro_row_sort", "gro_lookup_grad", "gro_experts_forward", "gro_experts_input_grad",
                 "gro_experts_weight_grad"):
        monkeypatch.setattr(B, name, lambda *a, name=name: by_handle[a[-1]].calls.append((name, a)))
    return st


def bf(*shape):
    return torch.zeros(shape, dtype=BF16)


def memory(*tensors):
    return {t.untyped_storage().data_ptr() for t in tensors}


def room_of(call):
    """Where a product's call has its workspace: the address, 256-byte aligned, within the allocation."""
    return call[1][-3], call[1][-2]


def products(given, few):
    """(call of a stream, operands, result) of the three products; few rows and long sums have a workspace."""
    rows, inner, outer = (20, 8192, 64) if few else (20, 8, 16)
    starts, w = torch.tensor([0, rows], dtype=I32), bf(1, outer, inner)
    x, dy = bf(rows, inner), bf(rows, outer)
    if few:
        long, wide = torch.tensor([0, 1 << 16], dtype=I32), bf(1 << 16, 64)
        back = (bf(20, 8192), bf(1, 8192, 64))
    else:
        long, wide, back = starts, x, (dy, w)
    y, dx, dw = (torch.zeros(s, dtype=BF16) if given else None for s in
                 ((rows, outer), (back[0].shape[0], back[1].shape[2]), (1, wide.shape[1], wide.shape[1])))
    return ((lambda s: L.experts_forward(x, w, starts, out=y, stream=s), (x, w, starts)),
            (lambda s: L.experts_input_grad(back[0], back[1], starts, out=dx, stream=s), (*back, starts)),
            (lambda s: L.experts_weight_grad(wide, wide, long, out=dw, stream=s), (wide, long)))


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("few", [True, False])
def test_products_on_another_stream(gpu0, given, few):
    """Operands, result and workspace are kept for the stream, which waits exactly where the call has allocated
    (the allocator may have handed out memory of the current stream's past work, and results start as zeros)."""
    for k, (call, operands) in enumerate(products(given, few)):
        gpu0.clear()
        out = call(gpu0.side)
        name, args = gpu0.side.calls[0]
        at, nbytes = room_of((name, args))
        assert (nbytes > 0) == few, "the sizes of a case with a workspace"
        assert len(gpu0.side.calls) == 1 and not gpu0.default.calls
        assert gpu0.side.waited == ([] if given and not few else [(gpu0.default, 0)])
        kept = set(gpu0.side.kept)
        assert memory(*operands, out) <= kept
        rooms = kept - memory(*operands, out)
        assert len(rooms) == (1 if few else 0)
        if few:
            assert at % 256 == 0 and 0 <= at - rooms.pop() < 256
        assert not gpu0.default.kept and not gpu0.default.waited


def test_lookups_on_another_stream(gpu0):
    table, ids, out = bf(10, 8), torch.zeros(6, dtype=torch.int64), bf(6, 8)
    L.lookup(table, ids, out=out, stream=gpu0.side)
    assert memory(table, ids, out) == set(gpu0.side.kept) and not gpu0.side.waited
    gpu0.clear()
    got = L.lookup(table, ids, stream=gpu0.side)
    assert memory(table, ids, got) == set(gpu0.side.kept) and gpu0.side.waited == [(gpu0.default, 0)]
    gpu0.clear()                    # ids that are put in order first, on the current stream
    L.lookup(table, torch.zeros(6, 2, dtype=I32)[:, 0], out=out, stream=gpu0.side)
    assert len(set(gpu0.side.kept)) == 3 and gpu0.side.waited == [(gpu0.default, 0)]
    (name, args), = gpu0.side.calls
    assert args[2] in gpu0.side.kept, "the copy is kept, not the list it was made from"


@pytest.mark.parametrize("how", ["none given", "the current one given", "current"])
def test_the_current_stream_needs_neither(gpu0, how):
    if how == "current":
        gpu0.now = gpu0.side
    stream = gpu0.now if how == "the current one given" else None
    for call, _ in products(False, True):
        call(stream)
    L.lookup(bf(10, 8), torch.zeros(6, dtype=torch.int64), stream=stream)
    by = L.RowOrder(6, 10, 8)
    by.sort(torch.zeros(6, 1, dtype=torch.int64), stream=stream)
    by.lookup_grad(bf(6, 8), stream=stream)
    assert len(gpu0.now.calls) == 6
    for s in (gpu0.default, gpu0.side, gpu0.third):
        assert not s.kept and not s.waited


def test_a_row_orders_own_memory(gpu0):
    """Workspace, order and starts are kept for each stream that uses them, given or current, once."""
    by = L.RowOrder(600, 10, 8)
    own = memory(by.workspace, by._order, by.starts)
    ids, dy, out = torch.zeros(600, dtype=torch.int64), bf(600, 8), bf(10, 8)
    by.sort(ids)
    by.lookup_grad(dy, out=out)
    assert not gpu0.default.kept, "where it was allocated"
    by.sort(ids, stream=gpu0.side)
    assert own | memory(ids) == set(gpu0.side.kept) and not gpu0.side.waited
    gpu0.clear()
    by.lookup_grad(dy, out=out, stream=gpu0.side)
    assert memory(dy, out) == set(gpu0.side.kept) and not gpu0.side.waited
    gpu0.clear()
    given = by.lookup_grad(dy, stream=gpu0.side)
    assert memory(dy, given) == set(gpu0.side.kept) and gpu0.side.waited == [(gpu0.default, 0)]
    gpu0.clear()
    gpu0.now = gpu0.third
    by.lookup_grad(dy, out=out)
    assert own == set(gpu0.third.kept)
    gpu0.clear()
    by.sort(ids)
    assert not gpu0.third.kept and [c[0] for c in gpu0.third.calls] == ["gro_row_sort"]


def test_the_tensors_gpu_is_current_in_the_call(gpu0):
    by = L.RowOrder(6, 10, 8, device="cuda:0")
    gpu0.device = 1
    L.lookup(bf(10, 8), torch.zeros(6, dtype=torch.int64))
    by.sort(torch.zeros(6, dtype=torch.int64))
    assert gpu0.entered == [0, 0]
