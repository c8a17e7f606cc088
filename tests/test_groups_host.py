"""CPU: what TensorGroup checks of the tensors it is given, and what autograd
learns of the ones it writes, on host tensors that say they are on GPU 0 and
with the library's calls taken out.  No kernel runs."""
import pytest
import torch

from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import TensorGroup

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


class Stream:
    cuda_stream = 0


@pytest.fixture(autouse=True)
def host_groups(monkeypatch):
    """Returns the list of the pointers given to each norm."""
    zeros, given = torch.zeros, []
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", 0)))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(B, "gro_group_bind", lambda *a: None)
    monkeypatch.setattr(B, "gro_group_norm", lambda handle, ptrs, *a: given.append(ptrs))
    monkeypatch.setattr(B, "gro_group_clip_adamw", lambda *a: None)
    return given


def ones(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype)


BF16 = torch.bfloat16


def test_gradients_of_another_shape_are_refused(host_groups):
    """Same elements, another order: the gradient of a transpose."""
    group = TensorGroup([ones(4, 8), ones(32)])
    right = [ones(4, 8, dtype=BF16), ones(32, dtype=BF16)]
    for wrong in ((8, 4), (2, 16), (4, 8, 1), (1, 4, 8), (4, 2, 4)):
        for other in (right[1], None):          # with and without a tensor left out
            with pytest.raises(ValueError, match=r"gradient 0.*\(4, 8\)"):
                group.norm([ones(*wrong, dtype=BF16), other])
    assert not host_groups
    group.norm(right)
    group.norm([right[0], None])
    assert host_groups == [[g.data_ptr() for g in right], [right[0].data_ptr(), 0]]


def test_flat_arrays_are_taken_for_any_shape(host_groups):
    """A flat array of a tensor's elements in order, as a flat gradient buffer
    gives, and a flat master with shaped gradients."""
    group = TensorGroup([ones(4, 8), ones(32), ones()], grad_dtype=BF16,
                        params_bf16=[ones(32, dtype=BF16), ones(4, 8, dtype=BF16), None],
                        states=[(ones(32), ones(4, 8)), (ones(32), ones(32)), (ones(), ones(1))])
    for shapes in (((32,), (4, 8), (1,)), ((4, 8), (32,), ()), ((32,), (2, 16), ())):
        grads = [ones(*s, dtype=BF16) for s in shapes]
        group.norm(grads)
        assert host_groups.pop() == [g.data_ptr() for g in grads]
        group.norm([None, *grads[1:]])
        assert host_groups.pop() == [0] + [g.data_ptr() for g in grads[1:]]


def test_states_and_copies_of_another_shape_are_refused():
    p = ones(4, 8)
    codes = [torch.ones(4, 8, dtype=torch.uint8) for _ in "mv"]
    scales = [ones(1), ones(1)]
    TensorGroup([p], params_bf16=[ones(4, 8, dtype=BF16)], states=[(ones(4, 8), ones(32))])
    TensorGroup([p], state_bits=8, states=[(*codes, *scales)])
    for bad in (dict(params_bf16=[ones(8, 4, dtype=BF16)]), dict(states=[(ones(8, 4), ones(4, 8))]),
                dict(states=[(ones(4, 8), ones(2, 16))]), dict(state_bits=8, states=[(codes[0], codes[1].view(8, 4), *scales)])):
        with pytest.raises(ValueError, match=r"\(4, 8\)"):
            TensorGroup([p], **bad)


def test_a_step_behind_a_saved_tensors_back_is_seen():
    """A backward pass through a graph that saved a master or a copy from
    before the step would use its new values: autograd raises, as it does for
    torch's own operations in place."""
    p, w = ones(4, 8).requires_grad_(), ones(4, 8, dtype=BF16).requires_grad_()
    group = TensorGroup([p, ones(32)], params_bf16=[w, None])
    for saved in (p, w):
        loss = (saved * saved).sum()
        group.norm([ones(4, 8, dtype=BF16), ones(32, dtype=BF16)])
        group.clip_adamw(1.0, HP, 1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        (saved * saved).sum().backward()        # a new graph is as good as ever


def test_only_what_a_step_writes_counts_as_modified():
    """Left out, refused and failing calls leave versions alone; tensors made
    in inference mode have none and are stepped all the same."""
    p, q = ones(4, 8).requires_grad_(), ones(32).requires_grad_()
    with torch.inference_mode():
        r = ones(5)
    group = TensorGroup([p, q, r])
    grads = [ones(4, 8, dtype=BF16), None, ones(5, dtype=BF16)]
    versions = [x._version for x in (p, q)]
    loss = (q * q).sum()
    group.norm(grads)
    assert [x._version for x in (p, q)] == versions          # a norm writes none of them
    group.clip_adamw(1.0, HP, 1)
    assert p._version > versions[0] and q._version == versions[1]
    loss.backward()
    with pytest.MonkeyPatch.context() as m:
        def fails(*a):
            raise B.GroError(B.GRO_E_STATE, "refused")
        m.setattr(B, "gro_group_clip_adamw", fails)
        version = p._version
        with pytest.raises(B.GroError):
            group.clip_adamw(1.0, HP, 2)
        assert p._version == version


def test_views_of_one_allocation_are_seen_too():
    """They share one version counter, which a step raises whichever of them it
    writes; a detached alias shares it as well."""
    flat = ones(64)
    group = TensorGroup([flat[:32], flat[32:], ones(4, 8).detach()])
    alias = group.masters[2].detach()
    before = flat._version, alias._version
    grads = [ones(32, dtype=BF16), ones(32, dtype=BF16), ones(4, 8, dtype=BF16)]
    group.norm(grads)
    group.clip_adamw(1.0, HP, 1)
    assert flat._version > before[0] and alias._version > before[1]
    before = flat._version, alias._version
    group.norm([None, grads[1], None])
    group.clip_adamw(1.0, HP, 2)
    assert flat._version > before[0] and alias._version == before[1]


@pytest.mark.parametrize("code,counts", [(B.GRO_E_HIP, True), (B.GRO_E_STATE, False), (B.GRO_E_INVALID, False)])
def test_a_step_that_failed_on_the_way_counts(monkeypatch, code, counts):
    """A refused call has written nothing; a launch that failed may have left
    other kinds of tensors updated."""
    p = ones(4, 8)
    group = TensorGroup([p])
    group.norm([ones(4, 8, dtype=BF16)])

    def fails(*a):
        raise B.GroError(code, "no")

    monkeypatch.setattr(B, "gro_group_clip_adamw", fails)
    version = p._version
    with pytest.raises(B.GroError):
        group.clip_adamw(1.0, HP, 1)
    assert (p._version > version) == counts
