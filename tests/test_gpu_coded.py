"""GPU: a plan's Adam moments in 8 bits -- gro_moments_encode,
gro_moments_decode, gro_clip_adamw_coded -- against the oracle bit for bit and
against 64-bit arithmetic, over ragged buckets, block tails, special values,
skipped steps, refusals, other streams, captured graphs and checkpoints."""
import numpy as np
import pytest
import torch

import oracle.method as M
from coded_reference import F32, HP, check_codes64, host, same_bits, step64
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd import checkpoint as C
from gradient_reduction_optimizer_amd import synth
from gradient_reduction_optimizer_amd.buffers import DeviceState, Plan

pytestmark = pytest.mark.gpu
POISON = 0xA5


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def specs(sizes, **kw):
    places = ("shard", "replicate", "partial", "reduced")
    return [dict(param_id=i, shape=(n,), placement=places[i % 4], shard_index=0 if i % 4 == 0 else -1,
                 no_decay=i % 3 == 1, **kw) for i, n in enumerate(sizes)]


def plans():
    """(name, tensors, R, bucket capacity): whole chunks, ragged ones, buckets
    of every length around a block and a vector, empty and frozen tensors."""
    yield "ones", specs([1, 1, 1, 1]), 2, 1 << 20
    yield "tails", specs([2, 3, 4, 5, 63, 64, 65, 127, 129, 255, 257]), 2, 64
    yield "chunk", specs([4096]), 1, 1 << 20
    yield "chunks", specs([4095, 4097, 8192, 12289]), 2, 1 << 20
    yield "split", specs([30_001, 7, 0, 10_000]), 3, 4160
    yield "fp32", specs([5000, 4096, 100], fp32_grad=True), 2, 1 << 20
    yield "frozen", specs([100, 200]) + [dict(param_id=9, shape=(50,), placement="replicate", frozen=True)], 2, 1 << 20
    yield "tiny", synth.tiny().tensors, 2, 25_000_000


PLANS = list(plans())
IDS = [p[0] for p in PLANS]


class Side:
    """A plan with poisoned gaps and 8-bit moments, and every bucket's arrays."""

    def __init__(self, tensors, R, cap, seed=0, static=False):
        self.plan = Plan(tensors, R, cap)
        self.st = DeviceState(self.plan, "cuda", static_workspace=static, coded_moments=True)
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.nb = self.plan.info["n_buckets"]
        st = self.st
        self.arrays = [st.acc, st.master, st.p_bf16, st.m_code, st.v_code, st.m_scale, st.v_scale]
        for a in self.arrays:
            a.view(torch.uint8).fill_(POISON)
        for b in range(self.nb):
            for a, scale in ((st.master, False), (st.m_code, False), (st.v_code, False), (st.m_scale, True), (st.v_scale, True)):
                a[self.span(b, scale)] = 0
            s = self.span(b)
            st.master[s] = 0.02 * torch.randn(s.stop - s.start, generator=self.gen, device="cuda")

    def span(self, b, scale=False):
        bk = self.plan.buckets[b]
        lo, hi = bk["flat_base"], bk["flat_base"] + bk["len"]
        return slice(lo // 64, -(-hi // 64)) if scale else slice(lo, hi)

    def gaps_untouched(self):
        for a, scale in zip(self.arrays, (False,) * 5 + (True,) * 2):
            free = torch.ones(a.numel(), dtype=torch.bool, device="cuda")
            for b in range(self.nb):
                free[self.span(b, scale)] = False
            if not bool((a.view(torch.uint8).view(a.numel(), -1)[free] == POISON).all()):
                return False
        return True

    def coded(self, b):
        s, k = self.span(b), self.span(b, True)
        return host(self.st.m_code[s]), host(self.st.v_code[s]), host(self.st.m_scale[k]), host(self.st.v_scale[k])

    def state(self):
        return [host(x) for x in (self.st.master, self.st.p_bf16, self.st.m_code, self.st.v_code, self.st.m_scale, self.st.v_scale)]

    def gradients(self, n, sigma=1e-2):
        """n microbatches of bucket buffers; NaN behind each bucket's end."""
        out = []
        for _ in range(n):
            bufs = self.st.grad_buffers()
            for buf, bk in zip(bufs, self.plan.buckets):
                g = torch.randn(buf.shape, generator=self.gen, device="cuda")
                wide = torch.randn((buf.shape[1] + 255) // 256, generator=self.gen, device="cuda").exp()
                buf.copy_(sigma * g * wide.repeat_interleave(256)[:buf.shape[1]])
                buf[:, bk["len"]:] = float("nan")
            out.append(bufs)
        return out

    def window(self, grads, stream=None):
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
        n, acc, h = len(grads), self.st.acc.data_ptr(), self.plan.handle
        B.gro_accumulate_window(h, 0, self.nb, [b.data_ptr() for bufs in grads for b in bufs], n, acc, s)
        B.gro_reduce_norm(h, acc, n, s)

    def update(self, n, max_norm, step, stream=None, copy=True, hp=HP):
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
        B.gro_clip_adamw_coded(self.plan.handle, self.st.acc.data_ptr(), n, max_norm, hp, step,
                               self.st.master.data_ptr(), self.st.coded, self.st.p_bf16.data_ptr() if copy else 0, s)


@pytest.mark.parametrize("tensors,R,cap", [p[1:] for p in PLANS], ids=IDS)
def test_steps_match_the_oracle_and_64_bits(tensors, R, cap):
    side = Side(tensors, R, cap)
    for step, (n, max_norm) in enumerate(((1, 1.0), (3, 0.05), (2, 0.0)), 1):
        p0 = [host(side.st.master[side.span(b)]) for b in range(side.nb)]
        c0 = [side.coded(b) for b in range(side.nb)]
        side.window(side.gradients(n))
        norm, _, finite = B.gro_plan_get_norm(side.plan.handle)
        assert finite
        side.update(n, max_norm, step)
        torch.cuda.synchronize()
        coef, _ = M.clip_coefficient(norm, max_norm)
        sc = M.adamw_scalars(*[HP[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")], step)
        for b in range(side.nb):
            what = (step, b)
            acc = host(side.st.acc[side.span(b)])
            dec = bool(side.plan.buckets[b]["decayed"])
            p, coded, bits = M.adamw_update_coded(M.window_gradient(acc, n), coef, p0[b], c0[b], sc, dec)
            got = side.coded(b)
            same_bits(host(side.st.master[side.span(b)]), p, (what, "p"))
            same_bits(host(side.st.p_bf16[side.span(b)]), bits, (what, "copy"))
            for k, name in enumerate(("m", "v", "m_scale", "v_scale")):
                same_bits(got[k], coded[k], (what, name))
            start = (p0[b], M.decode_m(c0[b][0], c0[b][2]), M.decode_v(c0[b][1], c0[b][3]))
            exact, bound = step64(acc, n, norm, max_norm, *start, HP, step, dec)
            assert np.all(np.abs(p.astype(np.float64) - exact[0]) <= bound[0]), what
            check_codes64(got[0], got[2], exact[1], bound[1], True, what)
            check_codes64(got[1], got[3], exact[2], bound[2], False, what)
    assert side.gaps_untouched()


def special(n, seed):
    """Moments with zeros, tiny and huge blocks, -0, and in some blocks infinities and NaN."""
    rng = np.random.default_rng(seed)
    m = (rng.normal(size=n) * np.exp(rng.normal(size=n) * 3)).astype(F32)
    v = (rng.normal(size=n) ** 2 * np.exp(rng.normal(size=n) * 6)).astype(F32)
    nb = -(-n // 64)
    kind = np.repeat(rng.integers(0, 10, nb), 64)[:n]
    m[kind == 0] = 0
    v[kind == 0] = 0
    m[kind == 1] *= F32(2.0 ** -104)
    v[kind == 1] *= F32(2.0 ** -130)
    m[kind == 2] *= F32(2.0 ** 100)
    v[kind == 2] *= F32(2.0 ** 90)
    m[kind == 3], v[kind == 3] = -0.0, -0.0
    with_ = lambda k, x, y: (m.__setitem__(np.flatnonzero(kind == k)[::7], x),  # noqa: E731
                             v.__setitem__(np.flatnonzero(kind == k)[::7], y))
    with_(4, np.nan, np.nan)
    with_(5, np.inf, np.inf)
    with_(6, -np.inf, -1.0)
    return m, v


@pytest.mark.parametrize("tensors,R,cap", [p[1:] for p in PLANS], ids=IDS)
def test_encode_and_decode_match_the_oracle(tensors, R, cap):
    side = Side(tensors, R, cap)
    n = side.plan.info["n_flat"]
    m, v = special(n, 3)
    dm, dv = torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda()
    s = torch.cuda.current_stream().cuda_stream
    B.gro_moments_encode(side.plan.handle, dm.data_ptr(), dv.data_ptr(), side.st.coded, s)
    om, ov = torch.full_like(dm, 7.0), torch.full_like(dv, 7.0)
    B.gro_moments_decode(side.plan.handle, side.st.coded, om.data_ptr(), ov.data_ptr(), s)
    torch.cuda.synchronize()
    assert np.array_equal(host(dm).view(np.uint32), m.view(np.uint32))  # inputs are only read
    free = np.ones(n, bool)
    for b in range(side.nb):
        sp = side.span(b)
        free[sp] = False
        mc, vc, ms, vs = side.coded(b)
        want_m, want_v = M.encode_m(m[sp]), M.encode_v(v[sp])
        same_bits(ms, want_m[1], (b, "m_scale"))
        same_bits(vs, want_v[1], (b, "v_scale"))
        # in a block whose scale is NaN every code stands for NaN
        fine_m = ~np.isnan(np.repeat(ms, 64)[:mc.size]) & ~np.isinf(np.repeat(ms, 64)[:mc.size])
        fine_v = ~np.isnan(np.repeat(vs, 64)[:vc.size])
        same_bits(mc[fine_m], want_m[0][fine_m], (b, "m"))
        same_bits(vc[fine_v], want_v[0][fine_v], (b, "v"))
        with np.errstate(invalid="ignore"):
            same_bits(host(om[sp]), M.decode_m(*want_m), (b, "decoded m"))
            same_bits(host(ov[sp]), M.decode_v(*want_v), (b, "decoded v"))
    assert (host(om)[free] == 7.0).all() and (host(ov)[free] == 7.0).all()
    assert side.gaps_untouched()


def test_encoding_what_was_decoded_changes_nothing():
    side = Side(specs([100_003, 4096, 65]), 2, 1 << 20)
    for step in (1, 2):
        side.window(side.gradients(1))
        side.update(1, 1.0, step)
    before = side.state()
    side.st.set_moments(*side.st.moments())
    for got, want in zip(side.state(), before):
        same_bits(got, want, "state")


def test_a_non_finite_norm_leaves_everything_as_it_was():
    for bad in (float("nan"), float("inf")):
        side = Side(specs([5000, 130]), 2, 1 << 20)
        side.window(side.gradients(1))
        side.update(1, 1.0, 1)
        before = side.state()
        grads = side.gradients(1)
        grads[0][1][0, 3] = bad
        side.window(grads)
        assert not B.gro_plan_get_norm(side.plan.handle)[2]
        side.update(1, 1.0, 2)
        for got, want in zip(side.state(), before):
            same_bits(got, want, bad)
        side.window(side.gradients(1))   # the window is over; the next one works
        side.update(1, 1.0, 2)


def test_large_gradients_overflow_v_to_the_largest_finite_one():
    """g^2 beyond FP32 while the FP64 norm is finite: v saturates, clipping off."""
    side = Side(specs([200]), 1, 1 << 20)
    grads = side.gradients(1)
    grads[0][0][0, 5] = 1e25
    side.window(grads)
    side.update(1, 0.0, 1)
    torch.cuda.synchronize()
    mc, vc, ms, vs = side.coded(0)
    assert vs[0] == M.ROOT_MAX and vc[5] == 240 and np.isfinite(M.decode_v(vc, vs)).all()
    assert np.isfinite(host(side.st.master[side.span(0)])).all()
    assert (vc[:64] >= 1).all()


def test_without_a_copy_and_without_eps():
    side = Side(specs([4096 + 70]), 1, 1 << 20)
    hp = dict(HP, eps=0.0)
    side.window(side.gradients(1))
    acc, p0 = host(side.st.acc[side.span(0)]), host(side.st.master[side.span(0)])
    norm = B.gro_plan_get_norm(side.plan.handle)[0]
    before = host(side.st.p_bf16)
    side.update(1, 1.0, 1, copy=False, hp=hp)
    torch.cuda.synchronize()
    assert np.array_equal(host(side.st.p_bf16), before)
    zero = np.zeros(p0.size, F32)
    exact, bound = step64(acc, 1, norm, 1.0, p0, zero, zero, hp, 1, True)
    assert np.all(np.abs(host(side.st.master[side.span(0)]) - exact[0]) <= bound[0])


def test_refusals_change_nothing():
    side = Side(specs([5000, 130]), 2, 1 << 20)
    st, h, s = side.st, side.plan.handle, torch.cuda.current_stream().cuda_stream
    acc, ok = st.acc.data_ptr(), st.coded
    n = side.plan.info["n_flat"]
    m = torch.zeros(n, device="cuda")
    v = torch.zeros(n, device="cuda")
    side.window(side.gradients(1))
    before = side.state()

    def kind(fn):
        with pytest.raises(B.GroError) as e:
            fn()
        return e.value.kind

    def step(coded=ok, acc=acc, master=st.master.data_ptr(), copy=st.p_bf16.data_ptr(), n=1, max_norm=1.0, t=1, hp=HP):
        B.gro_clip_adamw_coded(h, acc, n, max_norm, hp, t, master, coded, copy, s)

    def put(i, x):
        return tuple(x if k == i else p for k, p in enumerate(ok))

    for i in range(4):
        assert kind(lambda: step(coded=put(i, 0))) == "invalid"
        assert kind(lambda: step(coded=put(i, ok[i] + 4))) == "invalid"
        assert kind(lambda: B.gro_moments_encode(h, m.data_ptr(), v.data_ptr(), put(i, 0), s)) == "invalid"
        assert kind(lambda: B.gro_moments_decode(h, put(i, ok[i] + 8), m.data_ptr(), v.data_ptr(), s)) == "invalid"
    assert kind(lambda: step(coded=put(1, ok[0]))) == "invalid"                     # m and v in one array
    assert kind(lambda: step(coded=put(2, ok[3] + 16))) == "invalid"                # scales that overlap
    assert kind(lambda: step(coded=put(0, st.master.data_ptr() + 64))) == "invalid"
    assert kind(lambda: step(coded=put(3, acc))) == "invalid"
    assert kind(lambda: B.gro_moments_decode(h, ok, m.data_ptr(), m.data_ptr(), s)) == "invalid"
    assert kind(lambda: B.gro_moments_encode(h, m.data_ptr(), ok[1], ok, s)) == "invalid"
    assert kind(lambda: B.gro_moments_encode(h, 0, v.data_ptr(), ok, s)) == "invalid"
    assert kind(lambda: B.gro_moments_decode(h, ok, m.data_ptr() + 4, v.data_ptr(), s)) == "invalid"
    assert kind(lambda: step(master=0)) == "invalid" and kind(lambda: step(acc=0)) == "invalid"
    assert kind(lambda: step(copy=st.p_bf16.data_ptr() + 2)) == "invalid"
    assert kind(lambda: step(n=0)) == "invalid" and kind(lambda: step(t=0)) == "invalid"
    assert kind(lambda: step(max_norm=float("nan"))) == "invalid"
    assert kind(lambda: step(hp=dict(HP, beta2=1.0))) == "invalid"
    assert kind(lambda: step(n=2)) == "state"                                       # another window
    assert kind(lambda: step(acc=m.data_ptr())) == "state"                          # not this window's accumulator
    for got, want in zip(side.state(), before):
        same_bits(got, want, "state")
    step()                                                                          # and the right call works
    assert kind(step) == "state"                                                    # the window is over
    lib = B.load()
    assert lib.gro_moments_encode(h, m.data_ptr(), v.data_ptr(), None, s) == B.GRO_E_INVALID
    with pytest.raises(ValueError):
        st.set_moments(m.double(), v)
    with pytest.raises(ValueError):
        st.set_moments(m[:-1], v)


def test_codes_inside_the_workspace_are_refused():
    """They would overwrite the chunk table; nothing is launched."""
    side = Side(specs([100_000]), 1, 1 << 20)
    st, h, s = side.st, side.plan.handle, torch.cuda.current_stream().cuda_stream
    m, v = torch.zeros_like(st.master), torch.zeros_like(st.master)
    side.window(side.gradients(1))
    before = side.state()
    for i in range(4):
        for at in (st.ws_ptr, st.ws_ptr + st.ws_bytes - 256):
            coded = tuple(at if k == i else p for k, p in enumerate(st.coded))
            for call in (lambda: B.gro_moments_encode(h, m.data_ptr(), v.data_ptr(), coded, s),
                         lambda: B.gro_moments_decode(h, coded, m.data_ptr(), v.data_ptr(), s),
                         lambda: B.gro_clip_adamw_coded(h, st.acc.data_ptr(), 1, 1.0, HP, 1, st.master.data_ptr(), coded,
                                                        st.p_bf16.data_ptr(), s)):
                with pytest.raises(B.GroError) as e:
                    call()
                assert e.value.kind == "invalid"
    for flat in (m, v):
        with pytest.raises(B.GroError):
            B.gro_moments_decode(h, st.coded, *[st.ws_ptr if x is flat else x.data_ptr() for x in (m, v)], s)
    torch.cuda.synchronize()
    for got, want in zip(side.state(), before):
        same_bits(got, want, "state")
    side.update(1, 1.0, 1)


def test_an_empty_plan_does_nothing():
    plan = Plan([dict(param_id=1, shape=(0,), placement="replicate")], 2, 1 << 20)
    st = DeviceState(plan, "cuda", coded_moments=True)
    s = torch.cuda.current_stream().cuda_stream
    B.gro_reduce_norm(plan.handle, 0, 1, s)
    B.gro_clip_adamw_coded(plan.handle, 0, 1, 1.0, HP, 1, 0, (0, 0, 0, 0), 0, s)
    B.gro_moments_encode(plan.handle, 0, 0, (0, 0, 0, 0), s)
    B.gro_moments_decode(plan.handle, st.coded, 0, 0, s)


@pytest.mark.parametrize("static", [False, True])
def test_a_captured_step_replays_as_the_eager_one(static):
    """Encode, a step and decode captured together and replayed with new
    gradients, eager work and synchronizations between the replays."""
    tensors = specs([70_001, 4096, 300])
    eager, graph = Side(tensors, 2, 1 << 20, seed=1), Side(tensors, 2, 1 << 20, seed=1, static=static)
    grads = eager.gradients(2)
    out = [[torch.zeros_like(x.st.master) for _ in "mv"] for x in (eager, graph)]

    def run(side, o, s):
        side.window(grads, s)
        side.update(2, 1.0, 5, s)
        B.gro_moments_decode(side.plan.handle, side.st.coded, o[0].data_ptr(), o[1].data_ptr(), s.cuda_stream)
        B.gro_moments_encode(side.plan.handle, o[0].data_ptr(), o[1].data_ptr(), side.st.coded, s.cuda_stream)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        run(graph, out[1], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for k in range(4):
        fresh = eager.gradients(2)
        for a, b in zip(grads, fresh):
            for x, y in zip(a, b):
                x.copy_(y)
        torch.cuda.synchronize()
        run(eager, out[0], torch.cuda.current_stream())
        g.replay()
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(graph.state() + [host(x) for x in out[1]],
                                            eager.state() + [host(x) for x in out[0]])):
            same_bits(got, want, (k, i))
        assert torch.randn(1000, device="cuda").sum().isfinite()


def test_two_plans_on_two_streams():
    sides = [Side(specs([200_000, 4096 + k]), 2, 1 << 20, seed=k) for k in range(2)]
    alone = [Side(specs([200_000, 4096 + k]), 2, 1 << 20, seed=k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in sides]
    work = [[s.gradients(2) for _ in range(3)] for s in sides]
    torch.cuda.synchronize()
    for t in range(3):
        for side, stream, grads in zip(sides, streams, work):
            side.window(grads[t], stream)
            side.update(2, 1.0, t + 1, stream)
    torch.cuda.synchronize()
    for side, other, grads in zip(sides, alone, work):
        for t in range(3):
            other.window(grads[t])
            other.update(2, 1.0, t + 1)
        for got, want in zip(side.state(), other.state()):
            same_bits(got, want, "state")


def test_a_state_on_a_stream_of_its_own():
    """Steps on the state's stream, moments read and set from the current one,
    with nothing of the caller's between them."""
    tensors = specs([3_000_000, 4096])
    stream = torch.cuda.Stream()
    plan = Plan(tensors, 2, 1 << 22)
    st = DeviceState(plan, "cuda", stream=stream, coded_moments=True)
    ref = DeviceState(Plan(tensors, 2, 1 << 22), "cuda", coded_moments=True)
    grads = [torch.randn(b.shape, device="cuda").to(b.dtype) for b in st.grad_buffers()]
    ones = torch.ones_like(st.master)
    torch.cuda.synchronize()
    found = []
    for state, s in ((st, stream), (ref, torch.cuda.current_stream())):
        h, nb, acc = state.plan.handle, plan.info["n_buckets"], state.acc.data_ptr()
        for step in range(1, 6):
            B.gro_accumulate_window(h, 0, nb, [g.data_ptr() for g in grads], 1, acc, s.cuda_stream)
            B.gro_reduce_norm(h, acc, 1, s.cuda_stream)
            B.gro_clip_adamw_coded(h, acc, 1, 1.0, HP, step, state.master.data_ptr(), state.coded,
                                   state.p_bf16.data_ptr(), s.cuda_stream)
            if step == 2:
                state.set_moments(ones * 1e-3, ones * 1e-6)
        found.append([host(x) for x in (*state.moments(), state.master)])
    for got, want in zip(*found):
        same_bits(got, want, "stream")


def test_moments_between_steps_on_a_stream_of_its_own():
    """Moments read from the current stream after every step, the next step
    given to the state's stream at once: each reading is of one step."""
    tensors = specs([3_000_000, 4096])
    stream = torch.cuda.Stream()
    plan = Plan(tensors, 2, 1 << 22)
    st = DeviceState(plan, "cuda", stream=stream, coded_moments=True)
    ref = DeviceState(Plan(tensors, 2, 1 << 22), "cuda", coded_moments=True)
    grads = [torch.randn(b.shape, device="cuda").to(b.dtype) for b in st.grad_buffers()]
    torch.cuda.synchronize()
    found = []
    for state, s in ((st, stream), (ref, torch.cuda.current_stream())):
        h, nb, acc = state.plan.handle, plan.info["n_buckets"], state.acc.data_ptr()
        read = []
        for step in range(1, 6):
            B.gro_accumulate_window(h, 0, nb, [g.data_ptr() for g in grads], 1, acc, s.cuda_stream)
            B.gro_reduce_norm(h, acc, 1, s.cuda_stream)
            B.gro_clip_adamw_coded(h, acc, 1, 1.0, HP, step, state.master.data_ptr(), state.coded,
                                   state.p_bf16.data_ptr(), s.cuda_stream)
            read += state.moments()
        found.append([host(x) for x in read])
    for got, want in zip(*found):
        same_bits(got, want, "moments")


def test_a_state_dropped_with_steps_still_on_its_stream():
    """Codes, scales, accumulator, workspace and gradient buffers of a dropped
    state stay as they are until the steps on its stream are done, whatever is
    allocated and written on the current stream meanwhile."""
    tensors = specs([3_000_000, 4096])
    stream = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    found = []
    for s in (stream, torch.cuda.current_stream()):
        plan = Plan(tensors, 2, 1 << 22)
        st = DeviceState(plan, "cuda", stream=s, coded_moments=True)
        gen = torch.Generator(device="cuda").manual_seed(5)
        grads = st.grad_buffers()
        for g in grads:
            g.copy_(torch.randn(g.shape, generator=gen, device="cuda"))
        master, sizes = st.master, [x.numel() for x in (st.acc, st.m_code, st.m_scale, st.workspace, *grads)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):                 # some milliseconds in front of the steps
                busy @ busy
        h, nb, acc = plan.handle, plan.info["n_buckets"], st.acc.data_ptr()
        for step in (1, 2, 3):
            B.gro_accumulate_window(h, 0, nb, [g.data_ptr() for g in grads], 1, acc, s.cuda_stream)
            B.gro_reduce_norm(h, acc, 1, s.cuda_stream)
            B.gro_clip_adamw_coded(h, acc, 1, 1.0, HP, step, master.data_ptr(), st.coded, st.p_bf16.data_ptr(),
                                   s.cuda_stream)
        del st, grads, g
        junk = [torch.full((n * size,), POISON, dtype=torch.uint8, device="cuda") for n in sizes for size in (1, 2, 4)]
        torch.cuda.synchronize()
        found.append(host(master))
        del junk
    same_bits(found[0], found[1], "master")
    assert found[0].any()


def test_checkpoints_carry_8_bit_moments(tmp_path):
    """Saved after two steps and restored into a fresh state of the same
    layout, the third step is the uninterrupted run's bit for bit; restored
    into FP32 moments, it has exactly the decoded ones; and FP32 moments
    restored into an 8-bit state are the encoded ones, in another layout too."""
    tensors = specs([30_001, 7, 4096, 10_000])
    a = Side(tensors, 2, 1 << 20, seed=2)
    for t in (1, 2):
        a.window(a.gradients(1))
        a.update(1, 1.0, t)
    C.save_device_state(a.st, 2, str(tmp_path / "ck"))
    assert a.st.m is None and a.st.v is None
    with pytest.raises(C.CheckpointError):
        C.save_state(a.plan, a.st.master, a.st.m_code, a.st.v_code, 2, str(tmp_path / "codes"))
    with pytest.raises(C.CheckpointError):
        C.save_state(a.plan, a.st.master, a.st.m, a.st.v, 2, str(tmp_path / "codes"))
    b = Side(tensors, 2, 1 << 20, seed=3)
    assert C.load_device_state(b.st, str(tmp_path / "ck")) == 2
    grads = a.gradients(1)
    for side in (a, b):
        side.window(grads)
        side.update(1, 1.0, 3)
    for k in range(a.nb):
        for got, want in zip(b.coded(k), a.coded(k)):
            same_bits(got, want, k)
        same_bits(host(b.st.master[b.span(k)]), host(a.st.master[a.span(k)]), k)
    plain = DeviceState(Plan(tensors, 2, 4160), "cuda")
    assert C.load_device_state(plain, str(tmp_path / "ck")) == 2
    C.save_device_state(plain, 2, str(tmp_path / "ck32"))
    c = Side(tensors, 2, 1 << 20, seed=4)
    C.load_device_state(c.st, str(tmp_path / "ck"))
    m, v = c.st.moments()
    for i in range(len(tensors)):
        same_bits(host(plain.flat_view(plain.m, i)), host(c.st.flat_view(m, i)), i)
        same_bits(host(plain.flat_view(plain.v, i)), host(c.st.flat_view(v, i)), i)
    d = Side(tensors, 2, 1 << 20, seed=5)
    C.load_device_state(d.st, str(tmp_path / "ck32"))
    for k in range(c.nb):
        for got, want in zip(d.coded(k), c.coded(k)):
            same_bits(got, want, k)


@pytest.mark.parametrize("coded", [True, False])
def test_a_restored_state_has_its_bf16_copy(tmp_path, coded):
    """Loaded into a fresh state: the copy is the saved run's bit for bit at
    once, before any step, and the gaps between the buckets stay."""
    tensors = specs([30_001, 7, 4096, 10_000])
    a = Side(tensors, 2, 1 << 20, seed=2)
    a.window(a.gradients(1))
    a.update(1, 1.0, 1)
    C.save_device_state(a.st, 1, str(tmp_path))
    if coded:
        b = Side(tensors, 2, 1 << 20, seed=3)
        st = b.st
    else:
        b, st = None, DeviceState(Plan(tensors, 2, 1 << 20), "cuda")
    assert C.load_device_state(st, str(tmp_path)) == 1
    torch.cuda.synchronize()
    for k in range(a.nb):
        same_bits(host(st.p_bf16[a.span(k)]), host(a.st.p_bf16[a.span(k)]), k)
    assert b is None or b.gaps_untouched()


def test_offsets_past_32_bits():
    """One bucket of more than 2^31 elements: both ends against the oracle."""
    n = 2 ** 31 + 4096 + 77
    plan = Plan([dict(param_id=0, shape=(n,), placement="reduced", fp32_grad=True)], 1, 1 << 40)
    st = DeviceState(plan, "cuda", with_bf16=True, coded_moments=True)
    g = st.grad_buffers()[0]
    rng = np.random.default_rng(0)
    ends = [slice(0, 8192), slice(n - 4096 - 77, n)]
    vals = {}
    for k, e in enumerate(ends):
        size = e.stop - e.start
        vals[k] = ((rng.normal(size=size) * 1e-2).astype(F32), (rng.normal(size=size) * 0.02).astype(F32))
        g[0, e] = torch.from_numpy(vals[k][0]).cuda()
        st.master[e] = torch.from_numpy(vals[k][1]).cuda()
    s = torch.cuda.current_stream().cuda_stream
    B.gro_accumulate_window(plan.handle, 0, 1, [g.data_ptr()], 1, st.acc.data_ptr(), s)
    B.gro_reduce_norm(plan.handle, st.acc.data_ptr(), 1, s)
    B.gro_clip_adamw_coded(plan.handle, st.acc.data_ptr(), 1, 0.0, HP, 1, st.master.data_ptr(), st.coded,
                           st.p_bf16.data_ptr(), s)
    m, v = st.moments()
    torch.cuda.synchronize()
    sc = M.adamw_scalars(*[HP[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")], 1)
    for k, e in enumerate(ends):
        size = e.stop - e.start
        nb = -(-size // 64)
        zero = (np.zeros(size, np.uint8),) * 2 + (np.zeros(nb, F32),) * 2
        p, coded, bits = M.adamw_update_coded(vals[k][0], F32(1), vals[k][1], zero, sc, True)
        same_bits(host(st.master[e]), p, (k, "p"))
        same_bits(host(st.p_bf16[e]), bits, (k, "copy"))
        same_bits(host(st.m_code[e]), coded[0], (k, "m"))
        same_bits(host(st.v_code[e]), coded[1], (k, "v"))
        same_bits(host(m[e]), M.decode_m(coded[0], coded[2]), (k, "decoded m"))
        same_bits(host(v[e]), M.decode_v(coded[1], coded[3]), (k, "decoded v"))
    assert not bool(st.m_code[10_000:20_000].any())


def test_conversions_of_more_chunks_than_one_launch_takes():
    """Past 2^21 chunks a conversion is several launches: codes on both sides
    of the seam, decoded and encoded again."""
    n = (1 << 33) + 4096 * 3 + 5
    need = n * 10 + n // 8 + (1 << 30)
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip("needs 102 GB of free device memory")
    plan = Plan([dict(param_id=0, shape=(n,), placement="reduced")], 1, 1 << 40)
    assert plan.info["n_chunks"] > 1 << 21
    ws = torch.empty(plan.info["workspace_bytes"] + 256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    B.gro_plan_bind(plan.handle, (ws.data_ptr() + 255) // 256 * 256, plan.info["workspace_bytes"], s)
    flat = plan.info["n_flat"]
    codes = [torch.zeros(flat, dtype=torch.uint8, device="cuda") for _ in "mv"]
    scales = [torch.zeros(flat // 64, device="cuda") for _ in "mv"]
    state = tuple(t.data_ptr() for t in codes + scales)
    rng = np.random.default_rng(0)
    spots = [slice(0, 4096), slice((1 << 33) - 4096, (1 << 33) + 8192), slice(n - 4096 - 5, n)]
    want = []
    for sp in spots:
        x = (rng.normal(size=sp.stop - sp.start) * np.exp(rng.normal(size=sp.stop - sp.start))).astype(F32)
        want.append((M.encode_m(x), M.encode_v(x * x)))
    m, v = (torch.zeros(flat, device="cuda") for _ in "mv")
    try:
        for sp, ((mc, ms), (vc, vs)) in zip(spots, want):
            m[sp] = torch.from_numpy(M.decode_m(mc, ms)).cuda()
            v[sp] = torch.from_numpy(M.decode_v(vc, vs)).cuda()
        B.gro_moments_encode(plan.handle, m.data_ptr(), v.data_ptr(), state, s)
        m.fill_(7.0)
        v.fill_(7.0)
        B.gro_moments_decode(plan.handle, state, m.data_ptr(), v.data_ptr(), s)
        torch.cuda.synchronize()
        for sp, ((mc, ms), (vc, vs)) in zip(spots, want):
            blocks = slice(sp.start // 64, -(-sp.stop // 64))
            same_bits(host(codes[0][sp]), mc, "m")
            same_bits(host(codes[1][sp]), vc, "v")
            same_bits(host(scales[0][blocks]), ms, "m_scale")
            same_bits(host(scales[1][blocks]), vs, "v_scale")
            same_bits(host(m[sp]), M.decode_m(mc, ms), "decoded m")
            same_bits(host(v[sp]), M.decode_v(vc, vs), "decoded v")
        assert not bool(m[(1 << 33) + 8192:n - 4096 - 5].any()) and not bool(codes[1][4096:1 << 20].any())
    finally:
        del m, v, codes, scales
        torch.cuda.empty_cache()
