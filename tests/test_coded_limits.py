"""CPU: what 8-bit moments cannot follow.  Rounding to the nearest code keeps a
moment where it is when a step changes it by less than half a code, so decay
alone does not bring it down: shown for every code, and for a gradient that
falls while its block's largest does not."""
import numpy as np

import oracle.method as M

F32 = np.float32


def decayed(codes, scale, encode, decode, beta):
    """The codes after a step without a gradient, in blocks whose largest
    element, put in front, is held where it is."""
    top = 240 if encode is M.encode_v else 0x78        # the codes of 1.0 and of 256
    blocks = np.full((codes.size, 64), top, np.uint8)
    blocks[:, 1] = codes
    x = decode(blocks.reshape(-1), np.full(codes.size, scale, F32)).reshape(-1, 64)
    x[:, 1] *= F32(beta)
    return encode(x.reshape(-1))[0].reshape(-1, 64)[:, 1]


def test_second_moments_keep_their_code_without_a_gradient():
    """A code's lower border is at least 1/64 below it (1.0 with a finer binade
    underneath), and a step lowers sqrt(v) by 1 - sqrt(beta2): 1/66 at 0.97."""
    codes = np.arange(1, 241, dtype=np.uint8)
    for beta2 in (0.97, 0.99, 0.999, 0.9999):
        assert np.array_equal(decayed(codes, 1.0, M.encode_v, M.decode_v, beta2), codes)
    after = decayed(codes, 1.0, M.encode_v, M.decode_v, 0.93)
    whole = codes >= 16                                 # 1 - sqrt(0.93) = 1/28, more than any border's 1/32 ...
    assert np.all(after[whole] == codes[whole] - 1)
    assert np.array_equal(after[:13], codes[:13])       # ... but the codes of gradual underflow are further apart


def test_first_moments_follow_up_to_a_beta1_of_nine_tenths():
    """Borders at 1/32 to 1/16 below a normal code; code k of gradual underflow
    moves when a tenth of k passes 1/2."""
    codes = np.arange(1, 121, dtype=np.uint8)
    after = decayed(codes, 1.0, M.encode_m, M.decode_m, 0.9)
    assert np.all(after[codes >= 8] < codes[codes >= 8])
    assert np.array_equal(after[:4], codes[:4]) and np.all(after[5:7] < codes[5:7])
    for beta1 in (0.97, 0.99):                          # less than 1/32
        assert np.array_equal(decayed(codes, 1.0, M.encode_m, M.decode_m, beta1), codes)


def test_a_second_moment_stays_when_its_gradient_falls_beside_one_that_does_not():
    """Gradients of +-1, then of +-1/10 for all but the first element of each
    block.  Exactly, sqrt(v) of those goes to 1/10: v = b^n + (1 - b^n) / 100.
    In 8 bits a step lowers sqrt(v) by less than (1 - b) / 2, a twentieth of a
    per cent, of itself, no border is nearer than 1/64, and the scale stays
    1 to within FP32's rounding, so the code never moves."""
    beta2, n = 0.999, 8000
    v = np.ones(128, F32)                               # as a long run of +-1 leaves it
    small = np.arange(128) % 64 != 0
    g2 = np.where(small, F32(0.01), F32(1))
    start = M.encode_v(v)[0]
    for _ in range(n):
        codes, scale = M.encode_v(F32(beta2) * v + F32(1 - beta2) * g2)
        v = M.decode_v(codes, scale)
    assert np.array_equal(codes, start)
    # a step rounds the scale's root, its square, two products, their sum and two constants, under 8 times 2^-24 of v
    # in all, and pulls the difference from 1 back by 1 - b: at most 8000 * 2^-24 in the long run
    assert np.all(np.abs(v - 1) <= 8000 * 2.0 ** -24)
    exact = beta2 ** n + (1 - beta2 ** n) * 0.01
    assert np.all(np.sqrt(v[small] / exact) > 9.8)      # 1 / sqrt(0.01033) = 9.84
