"""The 8-bit oracle against independent statements of the same rules (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import fp8


def test_decode_is_the_c_oracles():
    c = np.arange(256, dtype=np.uint8)
    fine = (c & 0x7F) != 0x7F
    assert np.array_equal(fp8.decode(c)[fine], oracle.e4m3_decode(c[fine]).astype(np.float64))
    assert np.isnan(fp8.decode(c)[~fine]).all()


def test_encode_is_the_c_oracles():
    rng = np.random.default_rng(1)
    mag = [fp8.decode(np.arange(0x7F, dtype=np.uint8))]
    mag.append((mag[0][1:] + mag[0][:-1]) / 2)  # every tie
    mag.append(np.exp2(rng.uniform(-14, 10, 4000)))
    v = np.concatenate(mag + [-np.concatenate(mag)]).astype(np.float32)
    assert np.array_equal(fp8.encode(v), oracle.e4m3_encode(v))
    assert list(fp8.encode(np.array([np.nan, -0.0, np.inf, -np.inf, 464, 1e30], np.float32))) == \
        [0x7F, 0x80, 0x7E, 0xFE, 0x7E, 0x7E]


@pytest.mark.parametrize("amax,want", [(0.0, 0.0), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
                                       (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (1e-38, 2.0 ** -126)])
def test_page_scale(amax, want):
    s = fp8.page_scale(np.float32(amax))
    assert s == np.float32(want)
    if 0 < amax and want > 2.0 ** -126:
        assert amax / s <= 448 < amax / (s / 2)


def test_block_rules():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((130, 200)).astype(np.float32)
    x[3, 128:] = 0
    codes, scales = fp8.quantize(x, False)
    assert scales.shape == (2, 130) and scales[1, 3] == 0 and not codes[3, 128:].any()
    assert np.array_equal(scales[0], np.abs(x[:, :128]).max(1) / np.float32(448))
    # half an E4M3 step (2^-4 relative, 2^-10 absolute below the normals) of the scaled value, and the quotient's rounding
    back = fp8.values(codes, scales, False)
    s = np.repeat(scales, 128, axis=0)[:200].T.astype(np.float64)
    assert (np.abs(back - x) <= (2.0 ** -4 + 2.0 ** -22) * np.abs(x) + s * 2.0 ** -10).all()
    t, ts = fp8.quantize(x, True)
    assert ts.shape == (2, 2) and ts[0, 1] == np.abs(x[128:, :128]).max() / np.float32(448)
    # tiles commute with the transpose
    u, us = fp8.quantize(np.ascontiguousarray(x.T), True)
    assert np.array_equal(u, t.T) and np.array_equal(us, ts.T)


def test_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(3)
    cache = [fp8.encode(rng.standard_normal((2, 1, 16, 64))) for _ in range(2)]
    cache += [np.full((2, 1), 0.5, np.float32), np.full((2, 1), 0.25, np.float32)]
    q = rng.standard_normal((1, 2, 64)).astype(np.float32)
    o, lse, *_ = fp8.attention(q, cache, np.array([[1]]), np.array([0, 1]), np.array([1]), True, 0.125)
    v = fp8.decode(cache[1][1, 0, 0]) * 0.25
    assert np.allclose(o[0], v) and np.allclose(lse[0], q[0] @ (fp8.decode(cache[0][1, 0, 0]) * 0.5) * 0.125)


def test_append_one_by_one_equals_at_once_but_for_subnormals():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((40, 2, 64)).astype(np.float32) * np.linspace(0.1, 4, 40, dtype=np.float32)[:, None, None]
    empty = lambda: [np.zeros((3, 2, 32, 64), np.uint8) for _ in range(2)] + [np.zeros((3, 2), np.float32) for _ in range(2)]  # noqa: E731
    table = np.array([[2, 0]])
    once = fp8.kv_append(k, -k, empty(), table, np.array([0, 40]), np.array([40]))
    many = empty()
    for t in range(40):
        fp8.kv_append(k[t:t + 1], -k[t:t + 1], many, table, np.array([0, 1]), np.array([t + 1]))
    for i in range(4):
        if i >= 2:
            assert np.array_equal(once[i], many[i])
        else:
            a, b = fp8.decode(once[i]), fp8.decode(many[i])
            assert (np.abs(a - b) <= np.where(np.abs(a) < 2.0 ** -5, 2.0 ** -9, 0)).all()


@pytest.mark.parametrize("tile", [False, True])
def test_a_nan_keeps_its_code_where_the_scale_is_zero(tile):
    """A block without a number other than 0: scale 0, code 0 for the zeros of both signs, the NaN code for NaN."""
    x = np.zeros((130, 200), np.float32)
    x[0] = np.nan
    x[1, 5] = np.nan
    x[2] = -0.0
    x[129, 199] = np.nan
    codes, scales = fp8.quantize(x, tile)
    assert not scales.any() and np.array_equal(codes, np.where(np.isnan(x), 0x7F, 0))
    assert np.array_equal(np.isnan(fp8.values(codes, scales, tile)), np.isnan(x))


def test_append_keeps_the_nan_of_a_page_without_numbers():
    """From a first token of NaN, zeros behind it, and a number that gives the page its scale."""
    k = np.full((1, 1, 64), np.nan, np.float32)
    k[..., :8] = -0.0
    cache = [np.zeros((1, 1, 16, 64), np.uint8) for _ in range(2)] + [np.zeros((1, 1), np.float32) for _ in range(2)]
    table = np.array([[0]])
    first = np.where(np.arange(64) < 8, 0, 0x7F)
    for t, x in enumerate((k, np.zeros_like(k), np.full_like(k, 448.0))):
        fp8.kv_append(x, x, cache, table, np.array([0, 1]), np.array([t + 1]))
        for codes, scale in ((cache[0], cache[2]), (cache[1], cache[3])):
            assert np.array_equal(codes[0, 0, 0], first) and scale[0, 0] == (1 if t == 2 else 0)
    assert not cache[0][0, 0, 1].any() and (cache[0][0, 0, 2] == 0x7E).all()
