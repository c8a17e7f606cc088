"""GPU: groups of tensors that stay where they lie -- gro_group_norm and
gro_group_clip_adamw, moments in 32 and 8 bits -- against the oracle bit for
bit and against 64-bit arithmetic: sizes around blocks, vectors and chunks,
views at odd offsets, mixed kinds, tensors without a gradient, thousands of
tensors, skipped steps, other streams, captured graphs, refusals."""
import math
import threading

import numpy as np
import pytest
import torch

import oracle.method as M
from coded_reference import F32, HP, check_codes64, check_step64, host, same_bits, step64
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import TensorGroup

pytestmark = pytest.mark.gpu
SIZES = [1, 2, 3, 4, 5, 63, 64, 65, 66, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 8192, 12_289]
BF16, FP32 = torch.bfloat16, torch.float32
GUARD = 8          # poisoned elements around every array


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


class Arena:
    """Arrays cut out of poisoned allocations: each `shift` elements past a
    16-byte boundary and with guard elements on both sides."""

    def __init__(self, shift):
        self.shift, self.all = shift, []

    def cut(self, values):
        n = values.numel()
        back = torch.empty(n + 2 * GUARD + self.shift + 16, dtype=values.dtype, device="cuda")
        back.view(torch.uint8).fill_(0xA5)
        lo = 16 + self.shift
        back[lo:lo + n] = values
        self.all.append((back, lo, n))
        return back[lo:lo + n]

    def guards_untouched(self):
        return all(bool((back[:lo].view(torch.uint8) == 0xA5).all() and (back[lo + n:].view(torch.uint8) == 0xA5).all())
                   for back, lo, n in self.all)


class Case:
    """A group of the given sizes, its state before a step on the host, and
    what the oracle makes of it."""

    def __init__(self, sizes, bits, dtypes, shift=0, seed=0, copies=True, shift_of=None):
        """shift: of every array, or per kind of array from shift_of (p, copy,
        state, grad), which is 0 for those it does not name."""
        self.sizes, self.bits, self.dtypes = sizes, bits, dtypes
        self.rng = np.random.default_rng(seed)
        self.arena = Arena(shift)
        self.shift_of = shift_of
        cut = lambda a, kind="state": self.cut(torch.from_numpy(a).cuda(), kind)  # noqa: E731
        self.p = [cut((self.rng.normal(size=n) * 0.02).astype(F32), "p") for n in sizes]
        self.copy = [cut(np.zeros(n, np.int16), "copy").view(BF16) if copies and i % 4 != 3 else None
                     for i, n in enumerate(sizes)]
        self.states = []
        for n, b in zip(sizes, bits):
            m = (self.rng.normal(size=n) * np.exp(self.rng.normal(size=n)) * 1e-3).astype(F32)
            v = (m.astype(np.float64) ** 2 * np.exp(self.rng.normal(size=n))).astype(F32)
            if b == 8:
                (mc, ms), (vc, vs) = M.encode_m(m), M.encode_v(v)
                self.states.append(tuple(cut(x) for x in (mc, vc, ms, vs)))
            else:
                self.states.append((cut(m), cut(v)))
        self.no_decay = [i % 3 == 0 for i in range(len(sizes))]
        self.group = TensorGroup(self.p, state_bits=bits, no_decay=self.no_decay, grad_dtype=dtypes,
                                 params_bf16=self.copy, states=self.states)

    def cut(self, values, kind):
        if self.shift_of is not None:
            self.arena.shift = self.shift_of.get(kind, 0)
        return self.arena.cut(values)

    def gradients(self, sigma=1e-2, without=()):
        out = []
        for i, (n, d) in enumerate(zip(self.sizes, self.dtypes)):
            g = (self.rng.normal(size=n) * sigma * np.exp(self.rng.normal(size=n))).astype(F32)
            out.append(None if i in without else self.cut(torch.from_numpy(g).cuda().to(d), "grad"))
        return out

    def state(self):
        return [[host(self.p[i]), None if self.copy[i] is None else host(self.copy[i]),
                 *[host(x) for x in self.states[i]]] for i in range(len(self.sizes))]


def oracle_norm(grads, n):
    return math.sqrt(math.fsum(float(x) ** 2 for g in grads if g is not None
                               for x in M.window_gradient(M.as_f32(host(g)), n)))


def check_step(case, before, grads, n, max_norm, step, norm, exact=True, hp=HP):
    coef, taken = M.clip_coefficient(norm, max_norm)
    assert taken
    sc = M.adamw_scalars(*[hp[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")], step)
    after = case.state()
    for i, (got, was, g) in enumerate(zip(after, before, grads)):
        if g is None:
            for x, y in zip(got, was):
                if x is not None:
                    same_bits(x, y, (i, "left out"))
            continue
        g = M.as_f32(host(g))
        dec = not case.no_decay[i]
        if case.bits[i] == 8:
            start = (was[0], M.decode_m(was[2], was[4]), M.decode_v(was[3], was[5]))
            p, coded, bits = M.adamw_update_coded(M.window_gradient(g, n), coef, was[0], tuple(was[2:]), sc, dec)
            for k, name in enumerate(("m", "v", "m_scale", "v_scale")):
                same_bits(got[2 + k], coded[k], (i, case.sizes[i], name))
        else:
            start = (was[0], was[2], was[3])
            p, m, v, bits = M.adamw_update(M.window_gradient(g, n), coef, *start, sc, dec)
            same_bits(got[2], m, (i, case.sizes[i], "m"))
            same_bits(got[3], v, (i, case.sizes[i], "v"))
        same_bits(got[0], p, (i, case.sizes[i], "p"))
        if got[1] is not None:
            same_bits(got[1], bits, (i, case.sizes[i], "copy"))
        if not exact:
            continue
        if case.bits[i] == 32:
            check_step64((got[0], got[2], got[3]), start, g, n, norm, max_norm, HP, step, dec, (i, case.sizes[i]))
        else:
            want, bound = step64(g, n, norm, max_norm, *start, HP, step, dec)
            assert np.all(np.abs(got[0].astype(np.float64) - want[0]) <= bound[0]), i
            check_codes64(got[2], got[4], want[1], bound[1], True, i)
            check_codes64(got[3], got[5], want[2], bound[2], False, i)


def run(case, grads, n, max_norm, step):
    before = case.state()
    case.group.norm(grads, n)
    norm, sq, finite = case.group.get_norm()
    want = oracle_norm(grads, n)
    # squares are exact in FP64; on a value's way to the total lie at most 64 additions in its lane, 6 in the wave, 8 in
    # a lane of the second stage and 6 + 3 twice behind it: under 100 roundings of 2^-53, half as much on the root
    assert finite and abs(norm - want) <= 64 * 2.0 ** -53 * want, (norm, want)
    assert sq == pytest.approx(norm * norm, rel=1e-14)
    case.group.clip_adamw(max_norm, HP, step)
    torch.cuda.synchronize()
    check_step(case, before, grads, n, max_norm, step, norm)


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_match_the_oracle_and_64_bits(bits, dtype, shift):
    case = Case(SIZES, [bits] * len(SIZES), [dtype] * len(SIZES), shift, seed=bits + shift)
    for step, (n, max_norm) in enumerate(((1, 1.0), (3, 0.02), (4, 0.0)), 1):
        run(case, case.gradients(), n, max_norm, step)
    assert case.arena.guards_untouched()


@pytest.mark.parametrize("kind", ["p", "copy", "state", "grad"])
def test_one_misaligned_array(kind):
    """Only one of a tensor's arrays off its vector alignment."""
    sizes = [4096, 4097, 70, 9000]
    for bits, dtype in ((8, BF16), (32, FP32)):
        case = Case(sizes, [bits] * 4, [dtype] * 4, seed=3, shift_of={kind: 1})
        run(case, case.gradients(), 1, 1.0, 1)
        assert case.arena.guards_untouched()


def test_mixed_kinds_and_tensors_without_a_gradient():
    sizes = SIZES + [0, 300, 0, 7]
    bits = [8 if i % 2 else 32 for i in range(len(sizes))]
    dtypes = [FP32 if i % 3 == 0 else BF16 for i in range(len(sizes))]
    case = Case(sizes, bits, dtypes, seed=9)
    run(case, case.gradients(), 2, 1.0, 1)
    run(case, case.gradients(without=(0, 5, 18, 20)), 1, 0.05, 2)
    run(case, case.gradients(), 1, 1.0, 3)                    # back again
    run(case, [None] * len(sizes), 1, 1.0, 4)                 # a norm of 0, nothing changes
    assert case.arena.guards_untouched()


EXTREMES = [dict(beta1=0.0, beta2=0.0), dict(beta2=0.0, eps=0.0), dict(beta1=0.999999, beta2=1 - 2.0 ** -40),
            dict(lr=0.0), dict(lr=100.0, weight_decay=10.0), dict(eps=1e30), dict(weight_decay=0.0, eps=1e-30)]


@pytest.mark.parametrize("extreme", EXTREMES, ids=[",".join(e) for e in EXTREMES])
def test_extreme_hyper_parameters(extreme):
    hp = dict(HP, **extreme)
    case = Case([4096, 5000, 63], [32, 8, 8], [BF16, BF16, FP32], seed=6)
    for step, max_norm, n, sigma in ((1, float("inf"), 7, 1.0), (10 ** 9, -1.0, 1, 1e-18), (2, 1e-30, 2, 1e15)):
        before = case.state()
        grads = case.gradients(sigma=sigma)
        case.group.norm(grads, n)
        norm = case.group.get_norm()[0]
        case.group.clip_adamw(max_norm, hp, step)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            check_step(case, before, grads, n, max_norm, step, norm, exact=False, hp=hp)


def test_one_gradient_for_two_tensors():
    case = Case([500, 500, 77], [32, 8, 8], [BF16] * 3)
    g = case.gradients()
    g[1] = g[0]
    run(case, g, 1, 1.0, 1)


@pytest.mark.parametrize("count", [448, 449, 1000, 2700])
def test_many_tensors(count):
    """More tensors than one launch carries pointers for, most of them small."""
    rng = np.random.default_rng(count)
    sizes = [int(x) for x in np.exp(rng.normal(4.0, 1.5, count)).clip(0, 9000)]
    case = Case(sizes, [8 if rng.random() < 0.5 else 32 for _ in sizes],
                [FP32 if rng.random() < 0.2 else BF16 for _ in sizes], seed=count)
    grads = case.gradients(without=range(3, count, 50))
    before = case.state()
    case.group.norm(grads, 2)
    norm, _, finite = case.group.get_norm()
    want = oracle_norm(grads, 2)
    assert finite and abs(norm - want) <= 64 * 2.0 ** -53 * want
    case.group.clip_adamw(0.5, HP, 3)
    torch.cuda.synchronize()
    check_step(case, before, grads, 2, 0.5, 3, norm, exact=False)
    assert case.arena.guards_untouched()


@pytest.mark.parametrize("chunks", [127, 128, 129, 512, 2048, 2049])
def test_sizes_around_the_launch_rules(chunks):
    """Numbers of chunks where the launches change (a step split four ways, the
    norm's second stage left to the step), of one kind and of two."""
    layouts = [[chunks * 4096 - 5], [(chunks - 1) * 4096, 1], [4096] * 3 + [(chunks - 4) * 4096 - 9, 70]]
    for parts in layouts[:3 if chunks < 600 else 2]:
        case = Case(parts, [8 if i % 2 == 0 else 32 for i in range(len(parts))], [BF16] * len(parts), seed=chunks)
        assert case.group.info["n_chunks"] == chunks
        before = case.state()
        grads = case.gradients()
        case.group.norm(grads, 1)
        norm = case.group.get_norm()[0]
        want = math.sqrt(sum(float(np.sum(M.as_f32(host(g)).astype(np.float64) ** 2)) for g in grads))
        assert abs(norm - want) <= 128 * 2.0 ** -53 * want     # the order of numpy's sum is another one
        case.group.clip_adamw(0.5, HP, 2)
        torch.cuda.synchronize()
        check_step(case, before, grads, 1, 0.5, 2, norm, exact=False)
        assert case.group.get_norm()[0] == norm    # still there after the step


def test_a_captured_norm_with_an_eager_step():
    """The step takes the norm of the gradients that lay there last, whether
    the norm ran eagerly or was replayed, and get_norm reads the same one."""
    case = Case([5000, 300], [8, 32], [BF16, BF16])
    grads = case.gradients()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        case.group.norm(grads, 1)
    for k in range(3):
        for x, y in zip(grads, case.gradients(sigma=10.0 ** -k)):
            x.copy_(y)
        if k == 1:
            case.group.norm(case.gradients(), 1)   # another one in between
            case.group.get_norm()
            torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        before = case.state()
        norm = case.group.get_norm()[0]
        assert abs(norm - oracle_norm(grads, 1)) <= 64 * 2.0 ** -53 * norm
        case.group.clip_adamw(0.5, HP, 2)
        torch.cuda.synchronize()
        check_step(case, before, grads, 1, 0.5, 2, norm)
        case.group.norm(grads, 1)                  # the host's state for the next step


@pytest.mark.parametrize("count", [64, 65])
def test_tensors_around_the_short_argument_list(count):
    case = Case([50 + i for i in range(count)], [8] * count, [BF16] * count, seed=count)
    run(case, case.gradients(without=(count - 1,)), 1, 1.0, 1)
    run(case, case.gradients(), 1, 1.0, 2)


def test_the_norm_does_not_depend_on_alignment_and_repeats():
    """The same values at every element offset: the same bits, each time."""
    rng = np.random.default_rng(1)
    vals = [(rng.normal(size=n)).astype(F32) for n in (100_003, 4096, 17)]
    seen = set()
    for shift in (0, 1, 2, 3):
        case = Case([v.size for v in vals], [32] * 3, [FP32] * 3, shift)
        grads = [case.arena.cut(torch.from_numpy(v).cuda()) for v in vals]
        for _ in range(3):
            case.group.norm(grads, 3)
            seen.add(case.group.get_norm()[0])
    assert len(seen) == 1


def test_a_non_finite_gradient_leaves_everything_as_it_was():
    case = Case([5000, 70, 300], [32, 8, 8], [BF16, BF16, FP32])
    for bad in (float("nan"), float("inf")):
        before = case.state()
        grads = case.gradients()
        grads[2][17] = bad
        case.group.norm(grads, 1)
        assert not case.group.get_norm()[2]
        case.group.clip_adamw(1.0, HP, 1)
        torch.cuda.synchronize()
        for got, was in zip(case.state(), before):
            for x, y in zip(got, was):
                if x is not None:
                    same_bits(x, y, bad)
    grads = case.gradients()
    grads[2] = None
    run(case, grads, 1, 1.0, 1)


def test_an_empty_group_and_empty_tensors():
    for sizes in ([], [0], [0, 0]):
        g = TensorGroup([torch.zeros(n, device="cuda") for n in sizes])
        g.norm([torch.zeros(n, dtype=BF16, device="cuda") for n in sizes])
        assert g.get_norm() == (0.0, 0.0, True)
        g.clip_adamw(1.0, HP, 1)
    torch.cuda.synchronize()


def test_order_of_calls_and_refusals():
    case = Case([300, 70], [8, 32], [BF16, FP32])
    g = case.group
    before = case.state()

    def kind(fn):
        with pytest.raises(B.GroError) as e:
            fn()
        return e.value.kind

    assert kind(lambda: g.clip_adamw(1.0, HP, 1)) == "state"            # no norm yet
    assert kind(g.get_norm) == "state"
    grads = case.gradients()
    assert kind(lambda: g.norm(grads, 0)) == "invalid"
    s = torch.cuda.current_stream().cuda_stream
    ptrs = [x.data_ptr() for x in grads]
    assert kind(lambda: B.gro_group_norm(g.handle, [ptrs[0] + 1, ptrs[1]], 1, s)) == "invalid"
    assert kind(lambda: B.gro_group_norm(g.handle, [ptrs[0], ptrs[1] + 2], 1, s)) == "invalid"
    assert kind(lambda: g.clip_adamw(1.0, HP, 1)) == "state"
    for bad in (grads[:1], [grads[0], grads[0]], [grads[0].float(), grads[1]], [grads[0].cpu(), grads[1]],
                [torch.zeros(600, dtype=BF16, device="cuda")[::2], grads[1]]):
        with pytest.raises(ValueError):
            g.norm(bad, 1)
    g.norm(grads, 1)
    assert kind(lambda: g.clip_adamw(float("nan"), HP, 1)) == "invalid"
    assert kind(lambda: g.clip_adamw(1.0, HP, 0)) == "invalid"
    assert kind(lambda: g.clip_adamw(1.0, dict(HP, lr=-1.0), 1)) == "invalid"
    torch.cuda.synchronize()
    for got, was in zip(case.state(), before):
        for x, y in zip(got, was):
            if x is not None:
                same_bits(x, y, "refused")
    g.clip_adamw(1.0, HP, 1)
    assert kind(lambda: g.clip_adamw(1.0, HP, 2)) == "state"            # one update for one norm
    p = torch.zeros(64, device="cuda")
    for bad in (dict(masters=[p.cpu()]), dict(masters=[p.half()]), dict(masters=[p[::2]]),
                dict(masters=[p], state_bits=16), dict(masters=[p], state_bits=[8, 8]),
                dict(masters=[p], grad_dtype=torch.float16), dict(masters=[p], params_bf16=[p]),
                dict(masters=[p], states=[(p,)]), dict(masters=[p], state_bits=8, states=[(p, p)]),
                dict(masters=[p], states=[(p.double(), p)])):
        with pytest.raises(ValueError):
            TensorGroup(**bad)
    with pytest.raises(B.GroError) as e:
        TensorGroup([p, p])
    assert e.value.kind == "duplicate"
    with pytest.raises(B.GroError) as e:
        TensorGroup([p[:40], p[32:]])
    assert e.value.kind == "duplicate"
    TensorGroup([p[:32], p[32:]])


def test_captured_steps_replay_as_the_eager_ones():
    """Two graphs of one group, captured on gradients of their own, replayed in
    turn with new values, eager steps of the same group between them."""
    sizes = [70_001, 4096, 300, 65]
    bits, dtypes = [8, 32, 8, 32], [BF16, FP32, BF16, BF16]
    eager, graph = (Case(sizes, bits, dtypes, seed=4) for _ in range(2))
    sets = [graph.gradients() for _ in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for grads in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            graph.group.norm(grads, 2)
            graph.group.clip_adamw(1.0, HP, 5)
        graphs.append(g)
    torch.cuda.synchronize()
    for k in range(6):
        for x, y in zip(sets[k % 2], graph.gradients()):
            x.copy_(y)
        graphs[k % 2].replay()
        eager.group.norm(sets[k % 2], 2)
        eager.group.clip_adamw(1.0, HP, 5)
        torch.cuda.synchronize()
        assert graph.group.get_norm() == eager.group.get_norm()
        extra = graph.gradients()
        for c in (eager, graph):
            c.group.norm(extra, 1)
            c.group.clip_adamw(1.0, HP, 5)
        torch.cuda.synchronize()
        for got, want in zip(graph.state(), eager.state()):
            for x, y in zip(got, want):
                if x is not None:
                    same_bits(x, y, k)


def test_groups_on_streams_and_threads_of_their_own():
    sizes = [200_000, 4097, 300]
    cases = [Case(sizes, [8, 32, 8], [BF16] * 3, seed=k) for k in range(4)]
    alone = [Case(sizes, [8, 32, 8], [BF16] * 3, seed=k) for k in range(4)]
    work = [[c.gradients() for _ in range(3)] for c in cases]
    torch.cuda.synchronize()
    errors = []

    def go(case, grads):
        try:
            stream = torch.cuda.Stream()
            for t in range(3):
                case.group.norm(grads[t], 1, stream)
                case.group.clip_adamw(1.0, HP, t + 1, stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=a) for a in zip(cases, work)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for case, other, grads in zip(cases, alone, work):
        for t in range(3):
            other.group.norm(grads[t], 1)
            other.group.clip_adamw(1.0, HP, t + 1)
        torch.cuda.synchronize()
        for got, want in zip(case.state(), other.state()):
            for x, y in zip(got, want):
                if x is not None:
                    same_bits(x, y, "streams")


@pytest.mark.parametrize("given", [True, False], ids=["stream given", "stream current"])
def test_a_group_dropped_with_steps_still_on_another_stream(given):
    """The workspace, the states that the group allocated and the gradients of
    a dropped group stay as they are until its steps are done, whatever is
    allocated and written on the default stream meanwhile."""
    sizes, bits = [3_000_000, 4097, 300], [8, 32, 8]
    stream = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    found = []
    for s in (stream, torch.cuda.current_stream()):
        gen = torch.Generator(device="cuda").manual_seed(8)
        masters = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
        group = TensorGroup(masters, state_bits=bits)
        used = [group.workspace.numel(), *(x.numel() * x.element_size() for st in group.states for x in st)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):                 # some milliseconds in front of the steps
                busy @ busy
        for step in (1, 2, 3):
            grads = [torch.randn(n, generator=gen, device="cuda").to(BF16) for n in sizes]
            ready = torch.cuda.Event()
            ready.record()
            s.wait_event(ready)
            if given:
                group.norm(grads, 1, s)
                group.clip_adamw(1.0, HP, step, s)
            else:
                with torch.cuda.stream(s):
                    group.norm(grads)
                    group.clip_adamw(1.0, HP, step)
        del group, grads
        junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in used + [2 * n for n in sizes]]
        torch.cuda.synchronize()
        found.append([host(p) for p in masters])
        del junk
    for got, want in zip(*found):
        same_bits(got, want, "master")


def test_bound_again_to_moved_states():
    case = Case([500, 90], [8, 32], [BF16, BF16])
    run(case, case.gradients(), 1, 1.0, 1)
    moved = [tuple(x.clone() for x in st) for st in case.states]
    rows = [[p.data_ptr(), *[x.data_ptr() for x in st], *[0] * (4 - len(st)), c.data_ptr()]
            for p, st, c in zip(case.p, moved, case.copy)]
    ws = case.group.workspace
    B.gro_group_bind(case.group.handle, rows, (ws.data_ptr() + 255) // 256 * 256, case.group.info["workspace_bytes"],
                     torch.cuda.current_stream().cuda_stream)
    with pytest.raises(B.GroError):
        case.group.get_norm()
    old = [[host(x) for x in st] for st in case.states]
    kept, case.states = case.states, moved
    run(case, case.gradients(), 1, 1.0, 2)
    for st, was in zip(kept, old):
        for x, y in zip(st, was):
            same_bits(host(x), y, "the old place")


@pytest.mark.parametrize("step,beta2", [(1, 0.5), (9, 0.5), (3, 0.999), (1, 0.9999999)])
def test_every_root_of_two_binades(step, beta2):
    """Root, division by sqrt(bc2) and division of the moments for every FP32
    mantissa at an even and an odd exponent, and at values outside the range
    that the short form takes (zeros, subnormals, up to infinity): the same
    bits as one IEEE operation after the other.  No gradient, no decay, eps 0,
    p = 0, so that p is -step_size * (m / (sqrt(v) / sqrt(bc2)))."""
    bits = np.arange(1 << 24, dtype=np.uint32)
    v = np.concatenate([(bits + np.uint32(0x3f000000)), (bits + np.uint32(0x0f000000)),
                        np.uint32(0x0f800000) - bits[:5000], bits[:5000], np.uint32(0x7f800000) - bits[:5000],
                        np.linspace(0, 0x7f800000, 2_000_003).astype(np.uint32)]).view(F32)
    rng = np.random.default_rng(step)
    m = rng.uniform(-2, 2, v.size).astype(F32)
    hp = dict(HP, beta1=0.5, beta2=beta2, eps=0.0, weight_decay=0.0)
    sc = M.adamw_scalars(*[hp[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")], step)
    with np.errstate(all="ignore"):
        p, mw, vw, _ = M.adamw_update(np.zeros_like(m), F32(1), np.zeros_like(m), m, v, sc, True)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    pd, state = torch.zeros(v.size, device="cuda"), (dev(m), dev(v))
    group = TensorGroup([pd], grad_dtype=FP32, states=[state])
    group.norm([torch.zeros(v.size, device="cuda")])
    group.clip_adamw(1.0, hp, step)
    torch.cuda.synchronize()
    same_bits(host(state[1]), vw, "v")
    same_bits(host(state[0]), mw, "m")
    same_bits(host(pd), p, "p")


@pytest.mark.parametrize("bits,dtype", [(8, BF16), (32, FP32)])
def test_offsets_past_32_bits(bits, dtype):
    """A tensor of more than 2^31 elements: both ends against the oracle."""
    n = 2 ** 31 + 4096 + 77
    ends = [slice(0, 8192), slice(n - 4096 - 77, n)]
    rng = np.random.default_rng(0)
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    copy = torch.zeros(n, dtype=BF16, device="cuda")
    vals = []
    for e in ends:
        size = e.stop - e.start
        vals.append(((rng.normal(size=size) * 0.02).astype(F32), torch.from_numpy((rng.normal(size=size) * 1e-2).astype(F32)).to(dtype)))
        p[e] = torch.from_numpy(vals[-1][0]).cuda()
        g[e] = vals[-1][1].cuda()
    group = TensorGroup([p], state_bits=bits, grad_dtype=dtype, params_bf16=[copy])
    group.norm([g])
    norm = group.get_norm()[0]
    want = oracle_norm([v[1] for v in vals], 1)
    assert abs(norm - want) <= 64 * 2.0 ** -53 * want
    group.clip_adamw(1.0, HP, 1)
    torch.cuda.synchronize()
    coef, _ = M.clip_coefficient(norm, 1.0)
    sc = M.adamw_scalars(*[HP[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")], 1)
    for e, (p0, g0) in zip(ends, vals):
        size = e.stop - e.start
        zero = np.zeros(size, F32)
        pw, mw, vw, bw = M.adamw_update(M.as_f32(host(g0)), coef, p0, zero, zero, sc, True)
        same_bits(host(p[e]), pw, "p")
        same_bits(host(copy[e]), bw, "copy")
        if bits == 32:
            same_bits(host(group.states[0][0][e]), mw, "m")
            same_bits(host(group.states[0][1][e]), vw, "v")
        else:
            blocks = slice(e.start // 64, -(-e.stop // 64))
            for k, want in enumerate((*M.encode_m(mw), *M.encode_v(vw))):
                got = group.states[0][(0, 2, 1, 3)[k]][e if k % 2 == 0 else blocks]
                same_bits(host(got), want, k)
