"""CPU: the order that DeviceState and TensorGroup give to work on streams of
their own, and the memory they keep for it, on stand-ins for streams that note
what is asked of them.  No kernel runs."""
import pytest
import torch

from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import DeviceState, Plan


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
