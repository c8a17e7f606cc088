"""GPU: the short instruction sequences of the 8-bit and group kernels round as
the IEEE operations they stand for: the root of every FP32 value that takes the
short form, and the block reciprocals for every mantissa of a scale.  The
references are computed in 64 bits and rounded once more, which is the same as
rounding once: for a root, a quotient or a reciprocal of 24-bit numbers 50 bits
in between are enough (Figueroa, 1995), FP64 has 53."""
import numpy as np
import pytest
import torch

import oracle.method as M
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import Plan, TensorGroup

pytestmark = pytest.mark.gpu
MANTISSAS = 1 << 23


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def test_the_root_of_every_value_of_the_short_form():
    """All 224 binades from 2^-96 to the largest finite value.  beta2 rounds to
    1 in FP32 and its correction to 1, so v stays as it is, and sqrt(v) / 1
    divides m, which the step halves to the IEEE root: p = -1/2 exactly.  A root
    one step off gives another quotient than 1, for every mantissa."""
    p, m, v = (torch.zeros(MANTISSAS, device="cuda") for _ in "pmv")
    group = TensorGroup([p], no_decay=True, grad_dtype=torch.float32, states=[(m, v)])
    hp = dict(lr=0.5, beta1=0.5, beta2=1 - 2.0 ** -40, eps=0.0, weight_decay=0.0)
    grads = [torch.zeros(MANTISSAS, device="cuda")]
    mantissa = torch.arange(MANTISSAS, dtype=torch.int32, device="cuda")
    for binade in range(127 - 96, 255):
        want = (mantissa + (binade << 23)).view(torch.float32)
        v.copy_(want)
        root = want.double().sqrt().float()
        m.copy_(2 * root)
        p.zero_()
        group.norm(grads)
        group.clip_adamw(0.0, hp, 10 ** 15)
        assert torch.equal(v, want) and torch.equal(m, root), binade
        assert bool((p == -0.5).all()), (binade, int((p != -0.5).sum()))


def near(borders, scale):
    """Blocks whose largest element is `scale` and whose others are at most one
    step from border * scale, where one step of the reciprocal decides: 21 of
    the borders in each block, others in the next."""
    lanes = torch.arange(63, device="cuda")
    which = (lanes // 3 * (len(borders) // 21))[None, :] + \
        (torch.arange(scale.numel(), device="cuda") % (len(borders) // 21))[:, None]
    x = borders[which] * scale[:, None]
    x = (x.view(torch.int32) + (lanes % 3 - 1).to(torch.int32)[None, :]).view(torch.float32)
    return torch.cat([scale[:, None], x], 1)


@pytest.mark.parametrize("exponents", [(0, 0), (-99, -50), (127, 63)], ids=["middle", "low", "high"])
def test_the_reciprocal_of_every_mantissa_of_a_scale(exponents):
    """Codes of moments next to the borders between two codes, for scales of
    every mantissa: those of the IEEE reciprocal.  (With a reciprocal one step
    off, codes differ in 99.6 % of the blocks or more.)"""
    nb = 1 << 19
    plan = Plan([dict(param_id=0, shape=(nb * 64,), placement="reduced")], 1, 1 << 40)
    ws = torch.empty(plan.info["workspace_bytes"] + 256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    B.gro_plan_bind(plan.handle, (ws.data_ptr() + 255) // 256 * 256, plan.info["workspace_bytes"], s)
    codes = [torch.zeros(nb * 64, dtype=torch.uint8, device="cuda") for _ in "mv"]
    scales = [torch.zeros(nb, device="cuda") for _ in "mv"]
    middle = lambda x: torch.from_numpy(((x[1:] + x[:-1]) / 2).astype(np.float32)).cuda()  # noqa: E731
    m_borders = middle(M.e4m3_values()[:127]) / 256
    m_borders = m_borders[m_borders < 1][-105:]             # up to the border below 1, from the normal codes on
    v_borders = middle(M.root_values()[16:241])[-210:]
    for first in range(0, MANTISSAS, nb):
        mantissa = torch.arange(first, first + nb, dtype=torch.int32, device="cuda")
        sm, sv = ((mantissa + ((127 + e) << 23)).view(torch.float32) for e in exponents)
        m, r = near(m_borders, sm), near(v_borders, sv)
        v = r * r
        B.gro_moments_encode(plan.handle, m.data_ptr(), v.data_ptr(),
                             tuple(t.data_ptr() for t in codes + scales), s)
        torch.cuda.synchronize()
        assert torch.equal(scales[0], sm)
        inverse = (256 / sm.double()).float()
        want = (m * inverse[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(codes[0].view(nb, 64), want), (first, "m")
        r = v.double().sqrt().float()
        top = r.amax(1)
        assert torch.equal(scales[1], top) and torch.equal(top, sv)
        inverse = (1 / top.double()).float()
        bits = ((r * inverse[:, None]) * 2.0 ** -112).view(torch.int32)
        want = ((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19).clamp(1, 240).to(torch.uint8)
        assert torch.equal(codes[1].view(nb, 64), want), (first, "v")
