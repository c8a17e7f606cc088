"""CPU: the 8-bit moment formats as the oracle states them -- tied to torch's
e4m3 cast, to FP16's bit layout and to 64-bit arithmetic -- and the host side
of the entry points that use them: tables, sizes and refusals, none of which
reaches a device."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.method as M
from gradient_reduction_optimizer_amd import binding as B
from gradient_reduction_optimizer_amd.buffers import Plan

F32 = np.float32
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


# ------------------------------------------------------------- the formats
def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).float().numpy(), M.e4m3_values().astype(F32))
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(0, 300, 20000), np.exp(rng.uniform(-12, 5.5, 20000)),
                        (M.e4m3_values()[1:] + M.e4m3_values()[:-1]) / 2, M.e4m3_values()]).astype(F32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(M.nearest_code(y, M.e4m3_values()), want)


def test_root_codes_are_bits_6_to_13_of_fp16():
    codes = np.arange(241, dtype=np.uint16)
    assert np.array_equal((codes << 6).view(np.float16).astype(np.float64), M.root_values()[:241])
    assert M.root_values()[240] == 1.0


def values(kind, n, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=n) * np.exp(rng.normal(size=n) * (3.0 if kind == "wide" else 0.5))
    if kind == "zeros":
        x[rng.random(n) < 0.7] = 0.0
    if kind == "tiny":
        x *= 2.0 ** -90
    return x.astype(F32)


@pytest.mark.parametrize("n", [1, 3, 63, 64, 65, 127, 128, 1000, 4099])
@pytest.mark.parametrize("kind", ["plain", "wide", "zeros", "tiny"])
def test_oracle_encodes_to_the_nearest_code(kind, n):
    """Against 64-bit arithmetic.  A quotient carries two FP32 roundings (the
    reciprocal and the product), at most 2^-23 of itself together, so a code
    may be that much further off than half a step."""
    m = values(kind, n, n)
    codes, s = M.encode_m(m)
    scale = np.repeat(s, 64)[:n].astype(np.float64)
    assert s.size == -(-n // 64)
    y = 256 * m.astype(np.float64) / np.where(scale == 0, 1, scale) * (scale > 0)
    got = np.where(codes >= 128, -1, 1) * M.e4m3_values()[codes & 127]
    step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))), 2.0 ** -6) / 8
    assert np.all(np.abs(got - y) <= step / 2 + np.abs(y) * 2.0 ** -22)
    v = (values(kind, n, n + 1).astype(np.float64) ** 2).astype(F32)
    codes, s = M.encode_v(v)
    scale = np.repeat(s, 64)[:n].astype(np.float64)
    y = np.sqrt(v.astype(np.float64)) / np.where(scale == 0, 1, scale)
    got = M.root_values()[codes]
    step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(y, 2.0 ** -14))), 2.0 ** -14) / 16
    floor = np.where(v > 0, 2.0 ** -18, 0.0)
    # the root itself is one more rounding, and below 2^-14 the scaled quotient is rounded to 2^-37
    assert np.all(np.abs(got - np.maximum(y, floor)) <= step / 2 + y * 2.0 ** -21 + 2.0 ** -37)
    assert np.all((codes > 0) == (v > 0)) and codes.max(initial=0) <= 240


@pytest.mark.parametrize("kind", ["plain", "wide", "zeros"])
def test_encoding_what_was_decoded_changes_nothing(kind):
    x = values(kind, 64 * 50 + 17, 5)
    mc, ms = M.encode_m(x)
    vc, vs = M.encode_v(x * x)
    m, v = M.decode_m(mc, ms), M.decode_v(vc, vs)
    for got, want in zip(M.encode_m(m) + M.encode_v(v), (mc, ms, vc, vs)):
        assert np.array_equal(got, want)
    big = np.abs(x[:64 * 50].reshape(-1, 64)).max(axis=1)
    assert np.array_equal(np.abs(m[:64 * 50].reshape(-1, 64)).max(axis=1), big)


def test_edges_of_the_formats():
    z = np.zeros(64, F32)
    for enc, dec in ((M.encode_m, M.decode_m), (M.encode_v, M.decode_v)):
        c, s = enc(z)
        assert not c.any() and not s.any() and not dec(c, s).any()
    m = z.copy()
    m[3], m[40] = 2.0 ** -101, -2.0 ** -120
    c, s = M.encode_m(m)
    assert not s.any() and not np.any(c & 127)              # below the floor: zeros
    m[3] = 2.0 ** -100
    c, s = M.encode_m(m)
    assert s[0] == F32(2.0 ** -100) and M.decode_m(c, s)[3] == m[3]
    v = z.copy()
    v[5], v[6] = np.inf, 1.0
    c, s = M.encode_v(v)
    assert s[0] == M.ROOT_MAX and np.isfinite(M.decode_v(c, s)).all() and c[5] == 240 and c[6] == 1
    v = z.copy()
    v[0], v[1], v[2] = 1.0, 2.0 ** -149, -0.0
    c, s = M.encode_v(v)
    assert c[0] == 240 and c[1] == 1 and c[2] == 0 and s[0] == 1.0
    for bad in (np.nan, -1.0):
        v = np.ones(128, F32)
        v[7] = bad
        c, s = M.encode_v(v)
        d = M.decode_v(c, s)
        assert np.isnan(d[:64]).all() and np.array_equal(d[64:], v[64:])
    for bad in (np.nan, np.inf, -np.inf):
        m = np.ones(128, F32)
        m[7] = bad
        c, s = M.encode_m(m)
        d = M.decode_m(c, s)
        assert np.isnan(d[:64]).all() and np.array_equal(d[64:], m[64:])


# Plausible mistakes in the formats, each of which a check above has to see.
def _truncated(y, values):
    return np.clip(np.searchsorted(values, np.asarray(y, np.float64), side="right") - 1, 0, len(values) - 1)


def _ties_up(y, values):
    y = np.asarray(y, np.float64)
    lo = _truncated(y, values).clip(0, len(values) - 2)
    return np.where(y - values[lo] >= values[lo + 1] - y, lo + 1, lo)


def _no_gradual_underflow():
    c = np.arange(256)
    return np.where(c == 0, 0.0, (1.0 + (c & 15) / 16.0) * 2.0 ** ((c >> 4) - 15.0))


def _codes_that_may_vanish(v, encode=M.encode_v):
    codes, s = encode(v)
    r = np.sqrt(np.asarray(v, np.float64))
    y = r / np.where(s == 0, 1, s).repeat(64)[:r.size]
    return np.where(y < 2.0 ** -19, 0, codes).astype(np.uint8), s


def _scale_of_v(v, encode=M.encode_v):
    codes, s = encode(v)
    return codes, (s * s).astype(F32)


def _scale_to_the_next_power_of_two(m, encode=M.encode_m):
    codes, s = encode(m)
    up = np.where(s > 0, 2.0 ** np.ceil(np.log2(np.where(s > 0, s, 1))), 0).astype(F32)
    return codes, up


MISTAKES = [("nearest_code", _truncated), ("nearest_code", _ties_up), ("root_values", _no_gradual_underflow),
            ("encode_v", _codes_that_may_vanish), ("encode_v", _scale_of_v),
            ("encode_m", _scale_to_the_next_power_of_two)]


@pytest.mark.parametrize("name,wrong", MISTAKES, ids=[w.__name__ for _, w in MISTAKES])
def test_mistakes_in_the_formats_are_seen(monkeypatch, name, wrong):
    monkeypatch.setattr(M, name, wrong)
    checks = [test_e4m3_table_is_torchs, test_root_codes_are_bits_6_to_13_of_fp16, test_edges_of_the_formats,
              lambda: test_oracle_encodes_to_the_nearest_code("wide", 4099),
              lambda: test_encoding_what_was_decoded_changes_nothing("plain")]
    seen = 0
    for check in checks:
        try:
            check()
        except AssertionError:
            seen += 1
    assert seen > 0


# ---------------------------------------------------------------- the host
def code_of(fn):
    with pytest.raises(B.GroError) as e:
        fn()
    return e.value.kind


def test_unbound_plans_and_groups_are_refused():
    plan = Plan([dict(param_id=0, shape=(100,), placement="replicate")], 1, 1 << 20)
    four = [1 << 20, 2 << 20, 3 << 20, 4 << 20]
    assert code_of(lambda: B.gro_clip_adamw_coded(plan.handle, 1 << 20, 1, 1.0, HP, 1, 5 << 20, four)) == "state"
    assert code_of(lambda: B.gro_moments_encode(plan.handle, 1 << 20, 2 << 20, four)) == "state"
    assert code_of(lambda: B.gro_moments_decode(plan.handle, four, 1 << 20, 2 << 20)) == "state"
    for call in (lambda m: B.gro_moments_encode(plan.handle, 1 << 20, 2 << 20, m),):
        with pytest.raises(ValueError):
            call(four[:3])
    h = B.gro_group_create([dict(numel=100)])
    try:
        assert code_of(lambda: B.gro_group_norm(h, [1 << 20])) == "state"
        assert code_of(lambda: B.gro_group_clip_adamw(h, 1.0, HP, 1)) == "state"
        assert code_of(lambda: B.gro_group_get_norm(h)) == "state"
        with pytest.raises(ValueError):
            B.gro_group_norm(h, [])
        with pytest.raises(ValueError):
            B.gro_group_bind(h, [], 256, 1 << 20)
    finally:
        B.gro_group_destroy(h)


def test_group_sizes_and_refused_descriptors():
    for descs, chunks, elems in (([], 0, 0), ([0, 0], 0, 0), ([1], 1, 1), ([4096, 4097, 0, 5], 4, 8198)):
        h = B.gro_group_create([dict(numel=n) for n in descs])
        info = B.gro_group_get_info(h)
        assert (info["n_tensors"], info["n_chunks"], info["n_elems"]) == (len(descs), chunks, elems)
        assert info["workspace_bytes"] > 0 and info["workspace_bytes"] % 256 == 0
        B.gro_group_destroy(h)
    assert code_of(lambda: B.gro_group_create([dict(numel=-1)])) == "invalid"
    assert code_of(lambda: B.gro_group_create([dict(numel=(1 << 46) + 1)])) == "invalid"
    assert code_of(lambda: B.gro_group_create([dict(numel=1 << 37)])) == "invalid"  # too many chunks for a grid
    assert code_of(lambda: B.gro_group_create([dict(numel=1, flags=B.GRO_FROZEN)])) == "placement"
    assert code_of(lambda: B.gro_group_create([dict(numel=1, flags=16)])) == "placement"
    # the flag belongs to groups: a plan holds all of its moments one way
    bad = dict(param_id=0, shape=(4,), placement="replicate", flags=B.GRO_CODED_MOMENTS)
    assert code_of(lambda: B.gro_plan_create([bad], 1, 1 << 20)) == "placement"
    L = B.load()
    row = B.gro_group_desc(4, 0, 1)
    out = ctypes.c_void_p()
    assert L.gro_group_create(ctypes.byref(row), 1, ctypes.byref(out)) == B.GRO_E_PLACEMENT and not out.value
    assert L.gro_group_create(None, 1, ctypes.byref(out)) == B.GRO_E_INVALID
    assert L.gro_group_create(None, -1, ctypes.byref(out)) == B.GRO_E_INVALID
    assert L.gro_group_create(None, 0, None) == B.GRO_E_INVALID
    assert L.gro_group_get_info(None, None) == B.GRO_E_INVALID


def test_group_bind_refusals_before_device_work():
    """Every refused binding is found on the host: no pointer here is one of a
    device."""
    f32 = [(0x10000, 0x20000, 0x30000, 0, 0, 0x40000), (0x50000, 0x60000, 0x70000, 0, 0, 0)]
    coded = [(0x10000, 0x20000, 0x30000, 0x80000, 0x90000, 0), (0x50000, 0x60000, 0x70000, 0xa0000, 0xb0000, 0)]
    for bits8 in (False, True):
        h = B.gro_group_create([dict(numel=1000, coded_moments=bits8)] * 2)
        need = B.gro_group_get_info(h)["workspace_bytes"]
        good = coded if bits8 else f32
        ws = 1 << 24

        def with_(i, j, x):
            rows = [list(r) for r in good]
            rows[i][j] = x
            return rows

        def refused(rows, at=ws, nbytes=need):
            return code_of(lambda: B.gro_group_bind(h, rows, at, nbytes))

        assert refused(good, nbytes=need - 1) == "invalid"
        assert refused(good, at=ws + 16) == "invalid"
        assert refused(good, at=0) == "invalid"
        for j in (0, 1, 2):
            assert refused(with_(0, j, 0)) == "invalid"
        assert refused(with_(0, 0, 0x10002)) == "invalid"
        assert refused(with_(0, 5, 0x40001)) == "invalid"
        if bits8:
            assert refused(with_(1, 3, 0)) == "invalid" and refused(with_(1, 4, 0xb0002)) == "invalid"
            assert refused(with_(1, 4, 0xa0000 + 4 * 15)) == "duplicate"     # 16 scales each
        else:
            assert refused(with_(1, 1, 0x60001)) == "invalid"
        assert refused(with_(1, 0, 0x10000)) == "duplicate"                  # the same tensor twice
        assert refused(with_(1, 0, 0x10000 + 4 * 999)) == "duplicate"        # views that overlap by one element
        assert refused(with_(0, 2, 0x20000)) == "duplicate"                  # m and v in one place
        assert refused(with_(0, 5, 0x10000 + 8)) == "duplicate"              # the copy inside its master
        B.gro_group_destroy(h)
