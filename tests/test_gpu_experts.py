"""GPU: experts' products over ragged runs of rows against plain 64-bit ones:
each direction and result type, runs of no, one and many rows, sizes around tiles,
strides, alignments, rows of no expert, infinities and NaN of other rows, one expert,
many experts, captured graphs, and the layers together with a plan's step."""
import numpy as np
import pytest
import torch

import layers_reference as R
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd import layers as L

pytestmark = pytest.mark.gpu
BF16, F32, F64 = R.BF16, R.F32, R.F64


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def normal(seed, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).to(BF16)


# rows of each expert, rows in front of the first and behind the last, inner, outer
CASES = {
    "one row": ([1], 0, 0, 64, 64),
    "nothing": ([0, 0], 0, 3, 64, 64),
    "no experts": ([], 0, 4, 32, 32),
    "single tokens": ([1, 0, 2, 0, 0, 1, 3], 0, 0, 256, 512),
    "token of a wide expert": ([0, 1, 0, 1], 0, 0, 1024, 1024),
    "small odd": ([3, 0, 17, 5], 2, 6, 33, 31),
    "eights": ([5, 64, 0, 129, 9], 0, 8, 72, 200),
    "around tiles": ([63, 64, 65, 1, 0, 127, 128, 129], 1, 1, 128, 192),
    "large tiles": ([255, 256, 257, 0, 513], 0, 0, 320, 512),
    "wide": ([700, 20], 0, 5, 1032, 776),
    "one long": ([3000], 7, 0, 192, 264),
    "odd and long": ([1500, 0, 1000], 0, 0, 131, 257),
    "no inner": ([4, 2], 0, 1, 0, 24),
    "no outer": ([4, 2], 0, 1, 24, 0),
    "thin": ([100, 30], 0, 0, 1, 1),
    "many experts": ([(7 * i) % 5 for i in range(200)], 3, 3, 64, 40),
    "few rows, long sums": ([3, 0, 17], 1, 1, 2056, 1320),
    "few odd rows, long sums": ([5, 2], 0, 3, 1031, 519),
    "one wide row": ([1], 0, 0, 4101, 24),
    "long and thin": ([2500, 0, 9], 0, 0, 45, 72),
    "long and narrow": ([0, 3333], 2, 0, 5, 6),
    "a round and a few tiles": ([3000, 0, 257, 5100], 3, 0, 264, 2100),
    "two rounds and a few tiles": ([9000, 255, 256], 0, 9, 72, 3600),
    "batch": ([300, 500, 0, 800, 250], 0, 50, 512, 1024),
}
LAYOUTS = [(0, 0), (8, 0), (64, 8), (3, 1), (0, 5)]


class Case:
    def __init__(self, name, seed=0):
        sizes, self.front, self.behind, self.inner, self.outer = CASES[name]
        self.n = len(sizes)
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + self.front
        self.rows = int(self.starts[-1]) + self.behind
        self.x, self.dy = normal(seed + 1, self.rows, self.inner), normal(seed + 2, self.rows, self.outer)
        self.w = normal(seed + 3, self.n, self.outer, self.inner)
        # what lies outside every expert must not matter
        for t in (self.x, self.dy):
            t[:self.front], t[self.rows - self.behind:] = float("nan"), float("inf")
        self.dstarts = torch.from_numpy(self.starts).cuda()

    def runs(self):
        return [(e, slice(int(self.starts[e]), int(self.starts[e + 1]))) for e in range(self.n)]


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("direction", ["forward", "input"])
def test_products_of_rows(name, direction):
    c = Case(name)
    src, width = (c.x, c.outer) if direction == "forward" else (c.dy, c.inner)
    want, slack = torch.zeros(c.rows, width, dtype=F64), torch.zeros(c.rows, width, dtype=F64)
    for e, at in c.runs():
        want[at], slack[at] = R.product(src[at], c.w[e].t() if direction == "forward" else c.w[e])
    call = L.experts_forward if direction == "forward" else L.experts_input_grad
    inside = torch.zeros(c.rows, dtype=torch.bool)
    inside[c.front:c.rows - c.behind] = True
    for k, (pad, shift) in enumerate(LAYOUTS):
        dtype = (BF16, F32)[k % 2]
        s, w = R.Matrix(src, pad, shift), R.Matrix(c.w, pad, shift)
        was = torch.full((c.rows, width), 7.0, dtype=dtype)
        out = R.Matrix(was, pad, shift)
        assert call(s.view, w.view, c.dstarts, out=out.view) is out.view
        R.check_close(out.view.cpu()[inside], want[inside], slack[inside], (name, pad, shift, dtype))
        assert bool((out.view.cpu()[~inside] == 7).all()), "rows of no expert"
        assert out.rest_untouched()
    got = call(src.cuda(), c.w.cuda(), c.dstarts, dtype=F32)
    R.check_close(got.cpu()[inside], want[inside], slack[inside], (name, "allocated"))
    assert bool((got.cpu()[~inside] == 0).all())


@pytest.mark.parametrize("name", CASES)
def test_weight_gradients(name):
    c = Case(name, 10)
    want, slack = (torch.zeros(c.n, c.outer, c.inner, dtype=F64) for _ in "ws")
    for e, at in c.runs():
        want[e], slack[e] = R.product(c.dy[at].t(), c.x[at])
    empty = torch.from_numpy(np.diff(c.starts) == 0)
    for k, (pad, shift) in enumerate(LAYOUTS):
        d, x = R.Matrix(c.dy, pad, shift), R.Matrix(c.x, (pad + 8) % 72, shift)
        for dtype in (BF16, F32):
            was = normal(k, c.n, c.outer, c.inner).to(dtype)
            out = R.Matrix(was, pad, shift)
            L.experts_weight_grad(d.view, x.view, c.dstarts, out=out.view)
            R.check_close(out.view, want, slack, (name, pad, shift, dtype))
            first = R.bits(out.view)
            assert out.rest_untouched()
            out = R.Matrix(was, pad, shift)
            L.experts_weight_grad(d.view, x.view, c.dstarts, out=out.view, accumulate=True)
            R.check_close(out.view, want + was.to(F64), slack + (want.abs() + was.to(F64).abs()) * 2.0 ** -23, (name, "added"))
            assert torch.equal(R.bits(out.view.cpu()[empty]), R.bits(was[empty])) and out.rest_untouched()
            again = L.experts_weight_grad(d.view, x.view, c.dstarts, dtype=dtype)
            assert torch.equal(R.bits(again), first), "another sum on the same inputs"


def test_infinities_and_nan_of_other_rows_do_not_arrive():
    """Rows of an expert's neighbours share tiles with its own."""
    c = Case("around tiles", 20)
    for bad in range(c.n):
        at = slice(int(c.starts[bad]), int(c.starts[bad + 1]))
        x, dy = c.x.clone(), c.dy.clone()
        x[at], dy[at] = float("nan"), float("inf")
        w = c.w.clone()
        w[bad] = float("nan")
        y = L.experts_forward(x.cuda(), w.cuda(), c.dstarts)
        dx = L.experts_input_grad(dy.cuda(), w.cuda(), c.dstarts)
        dw = L.experts_weight_grad(dy.cuda(), x.cuda(), c.dstarts)
        keep = torch.ones(c.rows, dtype=torch.bool)
        keep[at] = False
        keep[:c.front], keep[c.rows - c.behind:] = False, False
        assert bool(y.cpu()[keep].isfinite().all()) and bool(dx.cpu()[keep].isfinite().all())
        others = [e for e in range(c.n) if e != bad]
        assert bool(dw.cpu()[others].isfinite().all())


def test_starts_out_of_range_are_cut():
    """Runs that leave the rows or go backwards are cut to what exists."""
    x, w = normal(1, 100, 64).cuda(), normal(2, 4, 64, 64).cuda()
    starts = torch.tensor([-5, 40, 30, 2 ** 31 - 1, -7], dtype=torch.int32).cuda()
    y = L.experts_forward(x, w, starts, dtype=F32)
    runs = [(0, 0, 40), (2, 30, 100)]       # expert 1 goes backwards, 3 begins at the end
    for e, lo, hi in runs[1:]:
        want, slack = R.product(x[lo:hi], w[e].t())
        R.check_close(y[40:], want[10:], slack[10:], e)
    dw = L.experts_weight_grad(x, x, starts, dtype=F32)
    for e, lo, hi in runs:
        want, slack = R.product(x[lo:hi].t(), x[lo:hi])
        R.check_close(dw[e], want, slack, ("dw", e))
    assert bool((dw[1] == 0).all()) and bool((dw[3] == 0).all())


def test_runs_over_each_other_end_and_stay_inside():
    """Starts that go up and down give runs over each other, more tiles than rows could have: whatever the rows
    hold then, the calls end and write nothing outside."""
    n, rows = 130, 300
    starts = torch.tensor([0, rows] * (n // 2) + [0], dtype=torch.int32).cuda()
    for inner, outer in ((64, 72), (512, 40)):
        x, w = normal(1, rows, inner).cuda(), normal(2, n, outer, inner).cuda()
        out = R.Matrix(torch.zeros(rows, outer, dtype=F32), 4)
        L.experts_forward(x, w, starts, out=out.view)
        back = R.Matrix(torch.zeros(rows, inner, dtype=F32), 4)
        L.experts_input_grad(normal(3, rows, outer).cuda(), w, starts, out=back.view)
        assert out.rest_untouched() and back.rest_untouched()


def test_columns_side_by_side_in_one_matrix():
    """Input and result as two halves of one matrix's columns, weights as the halves of each expert's rows."""
    c = Case("eights")
    both = torch.zeros(c.rows, c.inner + c.outer, dtype=BF16).cuda()
    both[:, :c.inner] = c.x.cuda()
    pair = torch.zeros(c.n, 2 * c.outer, c.inner, dtype=BF16).cuda()
    pair[:, c.outer:] = c.w.cuda()
    L.experts_forward(both[:, :c.inner], pair[:, c.outer:], c.dstarts, out=both[:, c.inner:])
    want = L.experts_forward(c.x.cuda(), c.w.cuda(), c.dstarts)
    keep = slice(c.front, c.rows - c.behind)
    assert torch.equal(R.bits(both[keep, c.inner:]), R.bits(want[keep]))
    dw = torch.zeros(c.n, 2 * c.outer, c.inner).cuda()
    L.experts_weight_grad(c.dy.cuda(), c.x.cuda(), c.dstarts, out=dw[:, c.outer:])
    assert bool((dw[:, :c.outer] == 0).all())
    assert torch.equal(dw[:, c.outer:], L.experts_weight_grad(c.dy.cuda(), c.x.cuda(), c.dstarts, dtype=F32))


def test_gradients_against_differences():
    """d sum(y * r) along a direction, by the forward product at two points: y is linear in x and in W, so the
    difference over any distance is the gradient's product with the direction."""
    c = Case("eights", 30)
    keep = slice(c.front, c.rows - c.behind)
    x, w, r = c.x.clone(), c.w.clone(), c.dy.clone()
    for t in (x, r):
        t[c.rows - c.behind:] = 0
    x, w, r = x.cuda(), w.cuda(), r.cuda()
    dx = L.experts_input_grad(r, w, c.dstarts, dtype=F32).double()
    dw = L.experts_weight_grad(r, x, c.dstarts, dtype=F32).double()
    f = lambda x, w: (L.experts_forward(x, w, c.dstarts, dtype=F32).double()[keep] * r.double()[keep]).sum()  # noqa: E731
    # steps of whole powers of two on values of few bits stay exact in BF16
    ex, ew = torch.randint(-1, 2, x.shape).to(BF16).cuda(), torch.randint(-1, 2, w.shape).to(BF16).cuda()
    x0, w0 = (t.float().mul(4).round().div(4).to(BF16) for t in (x, w))
    dx0 = L.experts_input_grad(r, w0, c.dstarts, dtype=F32).double()
    dw0 = L.experts_weight_grad(r, x0, c.dstarts, dtype=F32).double()
    scale = float((x0.double().abs().max() + 1) * (w0.double().abs().max() + 1) * r.double().abs().sum() * c.inner)
    for got, change in (((f(x0 + ex, w0) - f(x0 - ex, w0)) / 2, (dx0 * ex.double())[keep].sum()),
                        ((f(x0, w0 + ew) - f(x0, w0 - ew)) / 2, (dw0 * ew.double()).sum())):
        assert abs(float(got - change)) <= scale * (c.inner + c.outer) * 2.0 ** -23
    assert dx.shape == x.shape and dw.shape == w.shape


def whole(seed, most, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(BF16)


@pytest.mark.parametrize("name", ["small odd", "eights", "around tiles", "many experts", "few rows, long sums", "a round and a few tiles"])
def test_gradients_equal_differences(name):
    """d sum(y * r) along a direction, by the forward product at two points.  All values are whole: |y| is at most
    2 * 3 * 2,056, |dx| 4 * 2,100 and |dw| 4 * 8,357, below 2^24, so every FP32 sum is exact in any order, and so are
    the 64-bit ones of at most 2^25 terms below 2^16; nothing is left for a tolerance."""
    c = Case(name)
    x, w, r = whole(31, 2, c.rows, c.inner).cuda(), whole(32, 2, c.n, c.outer, c.inner).cuda(), whole(33, 2, c.rows, c.outer).cuda()
    dx = L.experts_input_grad(r, w, c.dstarts, dtype=F32).double()
    dw = L.experts_weight_grad(r, x, c.dstarts, dtype=F32).double()
    f = lambda x, w: (L.experts_forward(x, w, c.dstarts, dtype=F32).double() * r.double()).sum()  # noqa: E731
    for seed in (34, 36, 38):
        ex, ew = whole(seed, 1, *x.shape).cuda(), whole(seed + 1, 1, *w.shape).cuda()
        for got, change in (((f(x + ex, w) - f(x - ex, w)) / 2, (dx * ex.double()).sum()),
                            ((f(x, w + ew) - f(x, w - ew)) / 2, (dw * ew.double()).sum())):
            assert float(change) != 0 and float(got) == float(change), (name, seed)


def test_captured_and_replayed():
    """Runs' lengths are read on the device: a replay follows the starts of its time."""
    c = Case("batch", 40)
    x, dy, w = c.x.cuda().nan_to_num(0, 0, 0), c.dy.cuda().nan_to_num(0, 0, 0), c.w.cuda()
    starts = c.dstarts.clone()
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros(w.shape, device="cuda")

    def step():
        L.experts_forward(x, w, starts, out=y)
        L.experts_input_grad(dy, w, starts, out=dx)
        L.experts_weight_grad(dy, x, starts, out=dw, accumulate=True)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k, sizes in enumerate(([300, 500, 0, 800, 250], [0, 0, 0, 0, 1900], [1, 2, 3, 4, 5], [380] * 5)):
        starts.copy_(torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32))
        x.copy_(normal(50 + k, *x.shape))
        got = []
        for run in (graph.replay, step):
            for t in (y, dx, dw):
                t.fill_(0.5)
            run()
            torch.cuda.synchronize()
            got.append([t.clone() for t in (y, dx, dw)])
        assert all(torch.equal(R.bits(a), R.bits(b)) for a, b in zip(*got)), sizes


def test_two_streams_at_once():
    """Calls that overlap, each with results and workspace of its own."""
    c = Case("batch", 60)
    x, dy, w = c.x.cuda().nan_to_num(0, 0, 0), c.dy.cuda().nan_to_num(0, 0, 0), c.w.cuda()
    want = [L.experts_forward(x, w, c.dstarts), L.experts_weight_grad(dy, x, c.dstarts, dtype=F32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in "ab"]
    got = [[L.experts_forward(x, w, c.dstarts, stream=s), L.experts_weight_grad(dy, x, c.dstarts, dtype=F32, stream=s)]
           for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(R.bits(a), R.bits(b)) for a, b in zip(pair, want))


def test_an_embedding_and_experts_through_a_step():
    """One microbatch of a small model through the layers into a plan's buckets and its step, as a user runs it:
    the gradients arrive where gro_accumulate reads them, and the BF16 copies that the step leaves are read next."""
    from gradient_reduction_optimizer_amd.buffers import DeviceState, Plan
    V, H, F, E, T, K = 300, 64, 128, 6, 500, 2
    plan = Plan([dict(param_id=0, shape=(V, H), placement="shard", shard_index=0),
                 dict(param_id=1, shape=(E, F, H), placement="shard", shard_index=0),
                 dict(param_id=2, shape=(E, H, F), placement="shard", shard_index=0, fp32_grad=True)], 2, 1 << 20)
    st = DeviceState(plan, "cuda")
    shapes = [(V, H), (E, F, H), (E, H, F)]
    for i, s in enumerate(shapes):
        st.flat_view(st.master, i).copy_(normal(i, *s).float().reshape(-1).cuda() * 0.1)
    st.p_bf16.copy_(st.master)
    bufs = st.grad_buffers()
    by_token, by_expert = L.RowOrder(T, V, H), L.RowOrder(T * K, E)
    by_source = L.RowOrder(T * K, T, H)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    s = torch.cuda.current_stream().cuda_stream
    for step in (1, 2):
        r = np.random.default_rng(step)
        tokens = torch.from_numpy(r.integers(0, V, T)).cuda()
        choice = torch.from_numpy(np.stack([r.permutation(E)[:K] for _ in range(T)])).to(torch.int32).cuda()
        emb, up, down = (st.flat_view(st.p_bf16, i).view(*q) for i, q in enumerate(shapes))
        h = L.lookup(emb, tokens, 8.0)
        order, starts = by_expert.sort(choice)
        source = (order // K).to(torch.int32)               # the token of each row of the experts
        x = L.lookup(h, source)
        a = L.experts_forward(x, up, starts)
        y = L.experts_forward(a, down, starts)
        dy = (y.float() * 1e-2).to(BF16)                    # of the loss 0.005 * sum(y^2)
        da = L.experts_input_grad(dy, down, starts)
        dx = L.experts_input_grad(da, up, starts)
        L.experts_weight_grad(dy, a, starts, out=st.grad_view(bufs, 2, 0, shapes[2]))
        L.experts_weight_grad(da, x, starts, out=st.grad_view(bufs, 1, 0, shapes[1]))
        by_source.sort(source)
        dh = by_source.lookup_grad(dx)
        by_token.sort(tokens)
        by_token.lookup_grad(dh, 8.0, out=st.grad_view(bufs, 0, 0, (V, H)))

        # the same in 64 bits from the same copies
        p = [t.detach().double().cpu().requires_grad_() for t in (emb, up, down)]
        hh = p[0][tokens.cpu()] * 8.0
        loss = 0
        for t in range(K):
            e = choice[:, t].cpu().long()
            v = torch.bmm(p[2][e], torch.bmm(p[1][e], hh[:, :, None]))
            loss = loss + 0.005 * v.square().sum()
        loss.backward()
        for i, q in enumerate(p):
            got = st.grad_view(bufs, i, 0, shapes[i]).double().cpu()
            # five BF16 roundings in a row at most (h, a, y, dy, da, dx, dh: seven), each 2^-8 of its value, and
            # sums of them: in norm no more than their sum
            off = float((got - q.grad).norm() / q.grad.norm())
            assert off <= 8 * 2.0 ** -8, (step, i, off)
        B.gro_accumulate(plan.handle, 0, plan.info["n_buckets"], [b.data_ptr() for b in bufs], st.acc.data_ptr(), 0, 1, s)
        B.gro_reduce_norm(plan.handle, st.acc.data_ptr(), 1, s)
        norm, _, finite = B.gro_plan_get_norm(plan.handle)
        want = float(sum(q.grad.square().sum() for q in p)) ** 0.5
        assert finite and abs(norm - want) <= 8 * 2.0 ** -8 * want
        before = st.p_bf16.clone()
        B.gro_clip_adamw(plan.handle, st.acc.data_ptr(), 1, 1.0, hp, step, st.master.data_ptr(), st.m.data_ptr(),
                         st.v.data_ptr(), st.p_bf16.data_ptr(), s)
        assert not torch.equal(before, st.p_bf16)


def test_places_past_32_bits():
    """Operands and results whose rows or experts lie more than 2^32 bytes apart; whole numbers, exact in FP32."""
    r = torch.Generator().manual_seed(77)
    few = lambda *shape: torch.randint(-2, 3, shape, generator=r).to(BF16)  # noqa: E731
    n, inner, outer = 1_100_000, 8, 2048
    starts = torch.tensor([0, 3, 700_001, n], dtype=torch.int32).cuda()
    room = torch.zeros(3, 1_300_000_000, dtype=BF16, device="cuda")
    w = room[:, -outer * inner:].view(3, outer, inner)
    w.copy_(few(3, outer, inner))
    x = few(n, inner).cuda()
    y = L.experts_forward(x, w, starts)
    at = [0, 3, 700_001, n]
    for e in range(3):
        for lo in range(at[e], at[e + 1], 100_000):
            hi = min(lo + 100_000, at[e + 1])
            assert torch.equal(y[lo:hi].float(), x[lo:hi].float() @ w[e].float().t())    # at most 32: exact in BF16
    # rows of 4.5 GB as dy: sums over 2048 products up to 64, below 2^24
    dx = L.experts_input_grad(y, w, starts, dtype=F32)
    for lo, hi, e in ((0, 3, 0), (600_000, 700_001, 1), (n - 100_000, n, 2)):
        assert torch.equal(dx[lo:hi].double(), y[lo:hi].double() @ w[e].double())
    # rows 120,000 elements apart as x and their gradients' experts as far as the weights'; the last expert's 20 rows
    m = 20_000
    far = torch.zeros(m, 120_000, dtype=BF16, device="cuda")[:, :64]
    far.copy_(few(m, 64))
    dy = few(m, 128).cuda()
    s2 = torch.tensor([0, 10_000, m - 20, m], dtype=torch.int32).cuda()
    dw = room[:, :128 * 64].view(3, 128, 64)
    L.experts_weight_grad(dy, far, s2, out=dw)
    for e, (lo, hi) in enumerate(((0, 10_000), (10_000, m - 20), (m - 20, m))):
        want = dy[lo:hi].double().t() @ far[lo:hi].double()
        assert torch.equal(dw[e], want.to(BF16))               # FP32 sums below 2^24 are exact, rounded once


def test_more_tiles_than_a_launch_has_lanes_for():
    """2^23 and more tiles of 128 rows, which the workgroups take one after the other: rows of one element, whose
    products by a power of two are exact."""
    cut, n = (1 << 30) - 77, (1 << 30) + 300
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randint(-3, 4, (n, 1), generator=g, dtype=torch.int8, device="cuda").to(BF16)
    w = torch.tensor([2.0, -0.5], device="cuda").to(BF16).view(2, 1, 1)
    starts = torch.tensor([0, cut, n], dtype=torch.int32).cuda()
    y = L.experts_forward(x, w, starts)
    assert torch.equal(y[:cut], x[:cut] * 2) and torch.equal(y[cut:], x[cut:] * -0.5)
    dx = L.experts_input_grad(x, w, starts, out=y.fill_(9))
    assert torch.equal(dx[:cut], x[:cut] * 2) and torch.equal(dx[cut:], x[cut:] * -0.5)


def test_experts_held_apart():
    """Experts that are parameters of their own: a call for each, with its two entries of the starts."""
    c = Case("eights", 80)
    x, dy = c.x.cuda(), c.dy.cuda()
    y, dx = torch.zeros(c.rows, c.outer).cuda(), torch.zeros(c.rows, c.inner).cuda()
    for e, at in c.runs():
        w, dw, two = c.w[e:e + 1].cuda(), torch.full((1, c.outer, c.inner), 3.0).cuda(), c.dstarts[e:e + 2]
        L.experts_forward(x, w, two, out=y)
        L.experts_input_grad(dy, w, two, out=dx)
        L.experts_weight_grad(dy, x, two, out=dw)
        R.check_close(dw[0], *R.product(c.dy[at].t(), c.x[at]), e)
    for e, at in c.runs():
        R.check_close(y[at], *R.product(c.x[at], c.w[e].t()), e)
        R.check_close(dx[at], *R.product(c.dy[at], c.w[e]), e)
    assert bool((y[c.rows - c.behind:] == 0).all()) and bool((dx[c.rows - c.behind:] == 0).all())
