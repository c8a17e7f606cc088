"""GPU: lookups, positions by row and the lookup's gradient against plain 64-bit
statements: sizes around tiles, buckets and runs, both id and element types,
strides, alignments, shards of a table, common and absent rows, infinities, empty
lists, captured graphs, other streams."""
import numpy as np
import pytest
import torch

import layers_reference as R
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.layers import RowOrder, lookup

pytestmark = pytest.mark.gpu
BF16, F32, F64 = R.BF16, R.F32, R.F64


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def draw_ids(n, rows, seed, kind="mixed", first=0, dtype=torch.int64):
    """mixed: half of them of a few common rows, others anywhere, some of no row."""
    r = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full(n, first + rows - 1)
    elif kind == "few":
        ids = first + r.integers(0, max(1, min(rows, 7)), size=n) * max(1, rows // 7)
    else:
        ids = first + r.integers(-max(1, rows // 8), rows + max(1, rows // 8), size=n)
        common = r.random(n) < 0.5
        ids[common] = first + (r.random(int(common.sum())) ** 8 * rows).astype(np.int64)
    return torch.from_numpy(ids.astype(np.int64)).to(dtype)


SORTS = [(0, 5), (0, 0), (1, 0), (1, 1), (2, 1), (63, 64), (64, 64), (65, 256), (1000, 257), (1024, 255), (4095, 64),
         (4096, 1000), (8191, 513), (8192, 16_384), (8193, 16_384), (8193, 0), (8200, 1), (12_288, 33), (20_001, 32_000),
         (70_000, 262_144), (70_000, 262_145), (5_000, 1_048_576), (100_003, 1_048_576), (8193, 64), (20_000, 1024),
         (20_000, 1025), (300_000, 16), (1_100_000, 1000), (1_100_000, 40_000)]


@pytest.mark.parametrize("n,rows", SORTS)
def test_positions_by_row(n, rows):
    for kind in ("mixed", "one", "few"):
        for dtype, first in ((torch.int32, 0), (torch.int64, rows)):
            if rows == 0 and kind != "mixed":
                continue
            ids = draw_ids(n, rows, n + rows, kind, first, dtype)
            want, starts = R.row_order(ids, first, rows)
            by = RowOrder(n, rows)
            by._order.fill_(-7)
            by.workspace.fill_(0xA5)
            order, got = by.sort(ids.cuda(), first_row=first)
            m = len(want)
            assert np.array_equal(got.cpu().numpy(), starts), (kind, dtype, "starts")
            assert np.array_equal(order.cpu().numpy()[:m], want), (kind, dtype, "order")
            assert bool((order[m:] == -7).all()), (kind, dtype, "positions behind the last")


def test_many_chunks_of_more_than_a_tile():
    """So many ids that a chunk is several tiles."""
    n, rows = 256 * 4096 * 2 + 5, 3000
    ids = torch.randint(-3, rows + 3, (n,), generator=gen(1))
    key = torch.where((ids >= 0) & (ids < rows), ids, rows)
    want = torch.sort(key, stable=True)[1]
    starts = torch.searchsorted(torch.sort(key)[0], torch.arange(rows + 1))
    order, got = RowOrder(n, rows).sort(ids.cuda())
    assert torch.equal(got.cpu().long(), starts)
    assert torch.equal(order.cpu().long()[:starts[-1]], want[:starts[-1]])


def test_ids_at_the_ends_of_their_types():
    for dtype in (torch.int32, torch.int64):
        lim = torch.iinfo(dtype)
        for n in (9, 9000):
            ids = torch.full((n,), lim.max, dtype=dtype)
            ids[0], ids[3], ids[4], ids[5] = lim.min, 7, -1, 0
            order, starts = RowOrder(n, 8).sort(ids.cuda())
            assert starts.tolist() == [0, 1, 1, 1, 1, 1, 1, 1, 2] and order[:2].tolist() == [5, 3]
    ids = torch.tensor([lim.max, lim.max - 1, lim.max - 2, lim.min, 0])
    order, starts = RowOrder(5, 2).sort(ids.cuda(), first_row=lim.max - 2)
    assert starts.tolist() == [0, 1, 2] and order[:2].tolist() == [2, 1]


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1), (64, 4)])
@pytest.mark.parametrize("table_type,out_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_lookup(table_type, out_type, pad, shift):
    for n, rows, width in ((1, 1, 1), (3, 5, 7), (8, 300, 8), (33, 100, 9), (64, 1000, 64), (5, 17, 333), (130, 64, 512),
                           (7, 9, 1024), (9, 40, 2056), (0, 5, 8), (4, 0, 8), (4, 4, 0)):
        table = torch.randn(rows, width, generator=gen(width)).to(table_type)
        if rows and width:
            table[0, 0], table[-1, -1] = float("inf"), float("nan")
        for dtype, first in ((torch.int32, 0), (torch.int64, 10 ** 10)):
            ids = draw_ids(n, rows, n + width, "mixed", first, dtype)
            t = R.Matrix(table, pad, shift)
            out = R.Matrix(torch.full((n, width), 3.0, dtype=out_type), pad, shift)
            got = lookup(t.view, ids.cuda(), 5.7, first_row=first, out=out.view)
            assert got is out.view
            want = R.lookup(table, ids, 5.7, first)
            # the scale's rounding and the product's in FP32
            R.check_close(got, want, want.abs().nan_to_num(0, 0, 0) * 2.0 ** -23, (n, rows, width, dtype))
            assert out.rest_untouched() and t.rest_untouched()


def test_lookup_allocates_and_keeps_the_ids_shape():
    table = torch.randn(50, 24, generator=gen(2)).to(BF16).cuda()
    ids = torch.randint(0, 50, (3, 4, 5), generator=gen(3)).cuda()
    for i in (ids, ids.transpose(0, 2)):
        got = lookup(table, i)
        assert got.shape == (*i.shape, 24) and got.dtype == BF16 and torch.equal(got, table[i])
        assert torch.equal(lookup(table, i, 2.0, dtype=F32), table[i].float() * 2)


GRADS = [(0, 5, 8), (1, 1, 1), (5, 3, 7), (37, 1001, 333), (64, 2, 64), (300, 40, 24), (1000, 7, 520), (4096, 3, 8),
         (5000, 300, 72), (8193, 2000, 40), (3, 0, 16), (9, 4, 0), (200, 9, 1100)]


@pytest.mark.parametrize("n,rows,width", GRADS)
@pytest.mark.parametrize("kind", ["mixed", "one", "few"])
def test_lookup_grad(n, rows, width, kind):
    if rows == 0 and kind != "mixed":
        return
    ids = draw_ids(n, rows, n, kind)
    order, starts = R.row_order(ids, 0, rows)
    by = RowOrder(n, rows, width)
    by.sort(ids.cuda())
    for k, (dy_type, out_type) in enumerate(((BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16))):
        pad, shift = ((0, 0), (3, 1), (64, 0), (0, 3))[k]
        dy = torch.randn(n, width, generator=gen(n + k)).to(dy_type)
        was = torch.randn(rows, width, generator=gen(k)).to(out_type)
        d = R.Matrix(dy, pad, shift)
        want, slack = R.lookup_grad(dy, order, starts, 0.37)
        first = None
        for accumulate in (False, True, False):
            out = R.Matrix(was, pad, shift)
            by.workspace.fill_(0xFF)        # NaN in every partial sum that is not written
            by.lookup_grad(d.view, 0.37, out=out.view, accumulate=accumulate)
            if accumulate:
                # one more FP32 addition
                R.check_close(out.view, want + was.to(F64), slack + (want.abs() + was.to(F64).abs()) * 2.0 ** -23,
                              (dy_type, out_type, "added"))
                absent = torch.from_numpy(np.diff(starts) == 0)
                assert torch.equal(R.bits(out.view.cpu()[absent]), R.bits(was[absent]))
            else:
                R.check_close(out.view, want, slack, (dy_type, out_type))
                assert first is None or torch.equal(first, R.bits(out.view)), "another sum on the same inputs"
                first = R.bits(out.view)
            assert out.rest_untouched() and d.rest_untouched()


@pytest.mark.parametrize("n,rows,width,kind", [(5, 3, 33, "mixed"), (700, 40, 333, "mixed"), (5_000, 9, 64, "one"), (9_000, 3_000, 72, "few")])
def test_gradient_equals_differences(n, rows, width, kind):
    """d sum(out * r) along a direction, by the lookup at two points.  All values are whole and the scale is 4, so a
    row's sum is at most 9,000 * 2 * 4, below 2^24: every FP32 sum is exact in any order, as are the 64-bit ones."""
    g = gen(n)
    whole = lambda most, *shape: torch.randint(-most, most + 1, shape, generator=g).to(BF16).cuda()  # noqa: E731
    ids = draw_ids(n, rows, n, kind).cuda()
    table, r = whole(2, rows, width), whole(2, n, width)
    by_row = RowOrder(n, rows, width)
    by_row.sort(ids)
    dw = by_row.lookup_grad(r, 4.0, dtype=F32).double()
    f = lambda t: (lookup(t, ids, 4.0, dtype=F32).double() * r.double()).sum()  # noqa: E731
    for _ in range(3):
        e = whole(1, rows, width)
        change = (dw * e.double()).sum()
        got = (f(table + e) - f(table - e)) / 2
        assert float(change) != 0 and float(got) == float(change)


def test_infinities_and_nan_stay_in_their_rows():
    n, rows, width = 600, 5, 40
    ids = torch.arange(n) % 4
    dy = torch.randn(n, width, generator=gen(4)).to(BF16)
    dy[0, 3], dy[1, 4], dy[5, 4] = float("nan"), float("inf"), float("-inf")
    by = RowOrder(n, rows, width)
    by.sort(ids.cuda())
    out = by.lookup_grad(dy.cuda()).float().cpu()
    assert torch.nonzero(out.isnan()).tolist() == [[0, 3], [1, 4]] and bool((out[4] == 0).all())


def test_order_and_starts_out_of_range_are_not_followed():
    """What a caller may hand over by mistake: every access stays inside the arrays."""
    n, rows, width = 100, 6, 16
    dy, out = torch.ones(n, width, dtype=BF16).cuda(), torch.zeros(rows, width).cuda()
    m = lambda t: B.gro_matrix(t.data_ptr(), t.shape[0], width, width, int(t.dtype == F32), 0)  # noqa: E731
    room = torch.zeros(B.gro_lookup_grad_workspace(n, width) + 256, dtype=torch.uint8, device="cuda")
    ws = (room.data_ptr() + 255) // 256 * 256
    s = torch.cuda.current_stream().cuda_stream
    order = torch.arange(n, dtype=torch.int32)
    order[10], order[11], order[12] = -1, n, 2 ** 31 - 1
    starts = torch.tensor([-50, 10, 13, 13, 90, 2 ** 31 - 1, -3], dtype=torch.int32)
    order, starts = order.cuda(), starts.cuda()
    B.gro_lookup_grad(m(dy), order.data_ptr(), starts.data_ptr(), 1.0, False, m(out), ws, room.numel() - 256, s)
    # rows 0..5: [0, 10), [10, 13) none of which is a position, none, [13, 90), [90, 100), [100, 100)
    assert out[:, 0].tolist() == [10, 0, 0, 77, 10, 0]


def test_a_captured_sort_and_gradient_replayed(gpu):
    n, rows, width = 9000, 700, 72
    by, ids = RowOrder(n, rows, width), torch.zeros(n, dtype=torch.int64, device="cuda")
    dy = torch.zeros(n, width, dtype=BF16, device="cuda")
    table = torch.randn(rows, width, generator=gen(6)).to(BF16).cuda()
    out, x = torch.zeros(rows, width, device="cuda"), torch.zeros(n, width, dtype=BF16, device="cuda")

    def step():
        by.sort(ids)
        by.lookup_grad(dy, 0.5, out=out)
        lookup(table, ids, 0.5, out=x)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        ids.copy_(draw_ids(n, rows, k, ("mixed", "few", "one", "mixed")[k]))
        dy.copy_(torch.randn(n, width, generator=gen(k)))
        graph.replay()
        torch.cuda.synchronize()
        got, starts, y = out.clone(), by.starts.clone(), x.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(starts, by.starts) and torch.equal(R.bits(got), R.bits(out)) and torch.equal(R.bits(y), R.bits(x))


def test_another_stream_than_the_current_one():
    n, rows, width = 20_000, 500, 64
    ids, dy = draw_ids(n, rows, 8).cuda(), torch.randn(n, width, generator=gen(8)).to(BF16).cuda()
    by = RowOrder(n, rows, width)
    by.sort(ids)
    want = by.lookup_grad(dy, 2.0, dtype=F32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    by.sort(ids.view(-1, 2), stream=side)
    got = by.lookup_grad(dy.view(-1, 2, width), 2.0, dtype=F32, stream=side)
    looked = lookup(want, ids[::2], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    mine = (ids[::2] >= 0) & (ids[::2] < rows)
    assert torch.equal(looked, torch.where(mine[:, None], want[ids[::2].clamp(0, rows - 1)], 0))


@pytest.mark.parametrize("most,rows,lengths", [(70_000, 300, (65_536, 511, 8192, 70_000)),
                                               (1_048_600, 1000, (1_048_576, 12_288, 3)),
                                               (1_048_600, 1025, (1_048_576, 8193))])
def test_one_row_order_for_shorter_lists(most, rows, lengths):
    by = RowOrder(most, rows, 4)
    dy = torch.randint(-3, 4, (most, 4), generator=gen(most)).to(BF16)
    for n in lengths:
        ids = draw_ids(n, rows, n, "mixed")
        want, starts = R.row_order(ids, 0, rows)
        order, got = by.sort(ids.cuda())
        assert np.array_equal(order[:len(want)].cpu().numpy(), want) and np.array_equal(got.cpu().numpy(), starts)
        inside = (ids >= 0) & (ids < rows)
        sums = torch.zeros(rows, 4, dtype=F64).index_add_(0, ids[inside].long(), dy[:n][inside].to(F64))
        out = by.lookup_grad(dy[:n].cuda(), dtype=F32)
        assert torch.equal(out.to(F64).cpu(), sums)         # whole numbers below 2^24: exact in FP32


def test_places_past_32_bits():
    """Results of more than 2^31 elements, 4.5 GB, and rows of a table that lie as far apart."""
    n, rows, width = 1_100_000, 5, 2048
    big = torch.empty(rows, 600_000_000, dtype=BF16, device="cuda")
    table = big[:, -width:]
    table.copy_(torch.randint(-2, 3, (rows, width), generator=gen(3)).to(BF16))
    ids = torch.randint(0, rows, (n,), generator=gen(4)).cuda()
    out = lookup(table, ids)
    del big
    for lo in range(0, n, 100_000):
        assert torch.equal(out[lo:lo + 100_000], table[ids[lo:lo + 100_000]])
    by = RowOrder(n, rows, width)
    by.sort(ids)
    got = by.lookup_grad(out, dtype=F32)
    count = torch.bincount(ids, minlength=rows)
    assert torch.equal(got, table.float() * count[:, None])   # whole numbers below 2^24: exact in FP32
