"""Shared by the GPU tests of 8-bit moments and of tensor groups: one step in
64 bits with the error that FP32 arithmetic may add to it, and bit comparisons."""
import numpy as np

import oracle.method as M

F32, F64 = np.float32, np.float64
U = 2.0 ** -24          # half a step of FP32, relative
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def host(t):
    """A device tensor's values on the host, BF16 as its bits."""
    import torch
    t = t.detach().cpu()
    return (t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()).copy()


def same_bits(got, want, what):
    """Equal bit for bit; NaNs may differ in sign and payload."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape and got.dtype == want.dtype, (what, got.shape, want.shape, got.dtype, want.dtype)
    if got.dtype == np.float32:
        bad = (got.view(np.uint32) != want.view(np.uint32)) & ~(np.isnan(got) & np.isnan(want))
    else:
        bad = got != want
    assert not bad.any(), (what, int(bad.sum()), np.flatnonzero(bad)[:5], got[bad][:5], want[bad][:5])


def step64(g, n, norm, max_norm, p, m, v, hp, step, decayed):
    """(p, m, v) of one clipped AdamW step in FP64 and the bounds on what FP32
    adds to them.  Roundings counted, each at most U relative:
      g^ = (g / n) * coef                 2 operations + coef itself: 3
      m  = b1 m + (1-b1) g^               constants 1, products 1, sum 1: 3, and 3 of g^
      v  = b2 v + (1-b2) g^ g^            the same with two g^ and one product more: 10
      d  = sqrt(v) / root + eps           5 of v's root, root, its constant, division, eps, sum: 10
      u  = step_size (m / d)              m's error, 10 of d, 2 operations, the constant: 13
      p  = p decay - u                    constant, product, sum
    with one rounding of slack each, and the smallest subnormal for products
    that leave the normal range."""
    g, p, m, v = (np.asarray(x, F64) for x in (g, p, m, v))
    on = max_norm > 0 and np.isfinite(max_norm)
    gh = g / n * (min(1.0, max_norm / (norm + 1e-6)) if on else 1.0)
    b1, b2 = hp["beta1"], hp["beta2"]
    m1, m2 = b1 * m, (1 - b1) * gh
    v1 = b2 * v + (1 - b2) * gh * gh
    root = np.sqrt(1 - b2 ** step)
    d = np.sqrt(v1) / root + hp["eps"]
    size = hp["lr"] / (1 - b1 ** step)
    kept = p * ((1 - hp["lr"] * hp["weight_decay"]) if decayed else 1.0)
    with np.errstate(all="ignore"):
        u = size * (m1 + m2) / d
    em = 7 * U * (np.abs(m1) + np.abs(m2)) + 2.0 ** -147
    ev = 11 * U * v1 + 2.0 ** -147
    eu = size / d * em + 14 * U * np.abs(u)
    # a subnormal v1 carries 2^-147, which its root turns into more than U
    ed = np.minimum(np.sqrt(ev), ev / np.maximum(np.sqrt(v1), 2.0 ** -80)) / root
    eu += np.abs(u) * ed / d
    ep = 3 * U * np.abs(kept) + eu + U * np.abs(kept - u)
    return (kept - u, m1 + m2, v1), (ep, em, ev)


def check_step64(got, start, g, n, norm, max_norm, hp, step, decayed, what):
    """got: (p, m, v) after a step on start = (p, m, v) before it, FP32."""
    want, bound = step64(g, n, norm, max_norm, *start, hp, step, decayed)
    for name, x, y, e in zip("pmv", got, want, bound):
        off = np.abs(np.asarray(x, F64) - y)
        assert np.all(off <= e), (what, name, float(np.max(off - e)), int(np.argmax(off - e)))


def check_codes64(codes, scales, exact, bound, first, what):
    """8-bit moments against the 64-bit values they stand for: `first` for m,
    else v.  Half a step of the code (2^-4 of m, 2^-5 of sqrt(v); 2^-18 of the
    block's scale below the codes' normal range, and for the least code of v),
    the FP32 error of the moment itself and of the quotient (2^-22)."""
    dec = (M.decode_m if first else M.decode_v)(codes, scales).astype(F64)
    s = np.repeat(scales.astype(F64), 64)[:codes.size]
    if first:
        x, off = exact, np.abs(dec - exact)
        half = 2.0 ** -4
    else:
        x = np.sqrt(exact)
        off = np.abs(np.sqrt(dec) - x)
        bound = np.minimum(np.sqrt(bound), bound / np.maximum(x, 2.0 ** -80))
        half = 2.0 ** -5
    ok = off <= np.maximum(half * np.abs(x), 2.0 ** -18 * s) + bound + 2.0 ** -22 * np.abs(x) + 2.0 ** -36 * s
    tiny = s < 2.0 ** -99 if first else np.zeros(s.shape, bool)
    ok |= tiny & (np.abs(exact) <= 2.0 ** -99)
    assert ok.all(), (what, int((~ok).sum()), np.flatnonzero(~ok)[:5], off[~ok][:5], x[~ok][:5])
