"""CPU: the order that DeviceState and TensorGroup give to work on streams of
their own, and the memory they keep for it, on stand-ins for streams that note
what is asked of them.  No kernel runs."""
import pytest
import torch

from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import DeviceState, Plan, TensorGroup


class Stream:
    """Work in the order it is enqueued; a wait takes over what the other
    stream has been given so far."""

    def __init__(self, handle):
        self.cuda_stream, self.done, self.kept = handle, [], []

    def wait_stream(self, other):
        self.done += [x for x in other.done if x not in self.done]


@pytest.fixture
def streams(monkeypatch):
    """(current stream, another one); the library's calls are noted on the
    stream whose handle they are given."""
    here, side = Stream(1), Stream(2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here)

    def note(name):
        def call(*args):
            {1: here, 2: side}[args[-1]].done.append(name)
        return call

    for name in ("gro_plan_bind", "gro_moments_decode", "gro_moments_encode"):
        monkeypatch.setattr(B, name, note(name))
    # what the allocator is told of a tensor used on a stream other than the one it was allocated on
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: s.kept.append(t.data_ptr()))
    return here, side


def plan():
    return Plan([dict(param_id=0, shape=(300,), placement="replicate"),
                 dict(param_id=1, shape=(70,), placement="partial")], 2, 1 << 20)


def test_a_step_after_moments_waits_for_the_decoding(streams):
    """The decode runs on the current stream and reads the codes; what the
    state's stream is given next writes them."""
    here, side = streams
    st = DeviceState(plan(), "cpu", stream=side, coded_moments=True)
    side.done.append("step")
    st.moments()
    assert here.done.index("step") < here.done.index("gro_moments_decode")
    assert "gro_moments_decode" in side.done


def test_a_step_after_set_moments_waits_for_the_encoding(streams):
    here, side = streams
    st = DeviceState(plan(), "cpu", stream=side, coded_moments=True)
    side.done.append("step")
    zeros = torch.zeros_like(st.master)
    st.set_moments(zeros, zeros)
    assert here.done.index("step") < here.done.index("gro_moments_encode")
    assert "gro_moments_encode" in side.done


@pytest.mark.parametrize("coded", [False, True])
def test_a_states_memory_outlives_the_work_on_its_stream(streams, coded):
    """Arrays, workspace and gradient buffers are allocated on the current
    stream: dropped with steps still running on the state's stream, they must
    not be handed out again before those are done."""
    here, side = streams
    st = DeviceState(plan(), "cpu", stream=side, coded_moments=coded)
    arrays = [x for x in vars(st).values() if isinstance(x, torch.Tensor)]
    assert len(arrays) == (8 if coded else 6)
    bufs = st.grad_buffers()
    assert {x.data_ptr() for x in arrays + bufs} <= set(side.kept)
    assert not here.kept
    own = DeviceState(plan(), "cpu", coded_moments=coded)      # on the current stream: nothing to record
    own.grad_buffers()
    assert not here.kept


HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture
def host_groups(streams, monkeypatch):
    """Lets TensorGroup run on host tensors that say they are on GPU 0;
    returns (default stream, two others, a function that sets the current one)."""
    default, side, third = Stream(0), streams[1], Stream(3)
    zeros = torch.zeros
    now = [default]
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", 0)))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    for name in ("gro_group_bind", "gro_group_norm", "gro_group_clip_adamw"):
        monkeypatch.setattr(B, name, lambda *a: None)
    return default, side, third, lambda s: now.__setitem__(0, s)


def group_and_gradients():
    masters = [torch.ones(300), torch.ones(70)]
    copies = [torch.ones(300).bfloat16(), None]
    group = TensorGroup(masters, state_bits=[8, 32], params_bf16=copies)
    own = masters + copies[:1] + [t for st in group.states for t in st] + [group.workspace]
    return group, {t.data_ptr() for t in own}, [torch.ones(300).bfloat16(), torch.ones(70).bfloat16()]


def test_a_groups_memory_outlives_the_work_on_another_stream(host_groups):
    """Workspace (the table of the arrays' pointers), states, masters and
    copies on a stream given to the call or current in it: recorded once."""
    default, side, third, enter = host_groups
    group, own, grads = group_and_gradients()
    group.norm(grads)
    group.clip_adamw(1.0, HP, 1)
    assert not default.kept                     # where everything was allocated: nothing to record
    group.norm(grads, 1, side)
    assert own <= set(side.kept)
    enter(third)
    group.clip_adamw(1.0, HP, 2)
    assert own <= set(third.kept)
    del side.kept[:], third.kept[:]
    group.norm(grads, 1, side)
    group.clip_adamw(1.0, HP, 3)
    assert not own & set(side.kept) and not own & set(third.kept)


@pytest.mark.parametrize("how", ["given", "current", "born there", "default given"])
def test_gradients_outlive_the_step_that_reads_them(host_groups, how):
    """clip_adamw lets go of the gradients once it is enqueued, so whichever
    stream it runs on has to be recorded with them."""
    default, side, third, enter = host_groups
    if how == "born there":
        enter(side)
    group, _, grads = group_and_gradients()
    enter(side if how != "given" else default)
    given = {"given": side, "default given": default}.get(how)
    used = default if how == "default given" else side
    ptrs = {g.data_ptr() for g in grads}
    group.norm(grads, 1, given)
    assert ptrs <= set(used.kept)
    group.clip_adamw(1.0, HP, 1, given)
    assert group._grads is None
    del used.kept[:]
    group.norm(grads, 1, given)
    assert ptrs <= set(used.kept)
    del used.kept[:]
    group.clip_adamw(1.0, HP, 2, given)
    assert not used.kept                        # the norm has recorded them on this stream
    group.norm([grads[0], None], 1, given)
    enter(third)                                # a step on a stream that the norm did not run on
    del third.kept[:]
    group.clip_adamw(1.0, HP, 3)
    assert grads[0].data_ptr() in third.kept
