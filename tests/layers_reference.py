"""Plain 64-bit statements of the layers on the host, and matrices cut out of
poisoned memory for the GPU tests of them."""
import numpy as np
import torch

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}      # a rounding is off by at most this, relative to the value
TINY = 2.0 ** -126                                  # below it a type's steps no longer shrink with the value


class Matrix:
    """`values` on the GPU in rows `pad` elements further apart than they are
    long, `shift` elements past a 16-byte boundary, poison everywhere else."""

    def __init__(self, values, pad=0, shift=0):
        *lead, cols = values.shape
        rows = int(np.prod(lead, dtype=np.int64))
        self.row, self.cols, self.rows, self.lo = cols + pad, cols, rows, 64 + shift
        self.back = torch.empty(self.lo + rows * self.row + 64, dtype=values.dtype, device="cuda")
        self.back.view(torch.uint8).fill_(0xA5)
        self.inside = torch.zeros(self.back.numel(), dtype=torch.bool, device="cuda")
        flat = self.back[self.lo:self.lo + rows * self.row].view(rows, self.row)[:, :cols]
        self.inside[self.lo:self.lo + rows * self.row].view(rows, self.row)[:, :cols] = True
        flat.copy_(values.reshape(rows, cols))
        step = [1]
        for n in reversed([*lead[1:], self.row]):
            step.append(step[-1] * n)
        self.view = self.back.as_strided(tuple(values.shape), tuple(reversed(step[:len(values.shape)])), self.lo)
        assert torch.equal(self.view.reshape(-1), values.to("cuda").reshape(-1)) or values.isnan().any()

    def rest_untouched(self):
        size = self.back.element_size()
        return bool((self.back.view(torch.uint8).view(-1, size)[~self.inside] == 0xA5).all())


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def check_close(got, want, slack, what):
    """|got - want| <= half a step of the result's type + slack, element by element; equal where want is infinite,
    NaN where it is NaN."""
    want, slack = want.cpu(), slack.cpu() if isinstance(slack, torch.Tensor) else slack
    x = got.detach().cpu().to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(x), torch.isnan(want)), (what, "NaN")
    infinite = torch.isinf(want)
    assert torch.equal(x[infinite], want[infinite]), (what, "infinite")
    allowed = (want.abs() * HALF_STEP[got.dtype] * (1 + 2.0 ** -10) + slack + TINY * HALF_STEP[got.dtype] * 4)
    bad = fine & ~((x - want).abs() <= allowed)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(), x[bad][:3].tolist(), want[bad][:3].tolist())


def row_order(ids, first, n_rows):
    """(order, starts) by a plain stable sort on the host."""
    local = ids.cpu().numpy().reshape(-1).astype(object) - first
    mine = [i for i, r in enumerate(local) if 0 <= r < n_rows]
    mine.sort(key=lambda i: local[i])               # Python's sort is stable
    count = np.bincount([int(local[i]) for i in mine], minlength=n_rows) if mine else np.zeros(n_rows, np.int64)
    return np.array(mine, np.int32), np.concatenate([[0], np.cumsum(count)]).astype(np.int32)


def lookup(table, ids, scale, first):
    local = ids.cpu().reshape(-1).to(torch.int64) - first
    mine = (local >= 0) & (local < table.shape[0])
    out = torch.zeros(local.numel(), table.shape[1], dtype=F64)
    out[mine] = table.cpu().to(F64)[local[mine]] * scale
    return out


def lookup_grad(dy, order, starts, scale):
    """(sums, what FP32 additions in any order may be off by: n - 1 of them for n summands, and the product's
    and the scale's roundings)."""
    dy = dy.cpu().to(F64)
    out = torch.zeros(len(starts) - 1, dy.shape[1], dtype=F64)
    slack = torch.zeros_like(out)
    for r in range(len(starts) - 1):
        part = dy[torch.from_numpy(order[starts[r]:starts[r + 1]].astype(np.int64))]
        if part.shape[0]:
            out[r] = part.sum(0) * scale
            slack[r] = part.abs().sum(0) * abs(scale) * (part.shape[0] + 2) * 2.0 ** -24
    return out, slack


def product(a, b):
    """(a b, what FP32 sums of k exact products may be off by: every addition at most a whole step)."""
    a, b = a.to("cuda", F64), b.to("cuda", F64)
    return (a @ b).cpu(), (a.abs() @ b.abs()).cpu() * (a.shape[1] + 1) * 2.0 ** -23
