"""Pins of the 8-bit cache's and the rotary operator's float64 definitions."""
import math

import numpy as np
import pytest
import torch

from oracle import qcache as Q


def test_e4m3_codes_agree_with_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000), Q.VALUES[:127], -Q.VALUES[:127],
                        (Q.VALUES[:126] + Q.VALUES[1:127]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448.0]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.e4m3_codes(x), want)
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(table, Q.VALUES.astype(np.float32), equal_nan=True)


def test_codes_saturate_and_hold_no_nan():
    assert Q.VALUES[Q.e4m3_codes([1e30, -math.inf, math.nan])].tolist() == [448.0, -448.0, 0.0]


@pytest.mark.parametrize("top", [0.0, 1e-40, 448.0, 449.0, 3.5 * 2.0 ** 40, 1.0, 1.75, 1.7500001])
def test_block_scale_is_the_least_power_of_two(top):
    s = Q.block_scale([top, -top / 3])
    assert math.log2(s) == int(math.log2(s)) and top <= 448 * s
    assert s == 2.0 ** -100 or top > 448 * s / 2


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_complex_product_and_turns_back(layout):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 24))
    pos = np.array([0, 7, 100000])
    f = Q.rope_frequencies(16, 5)
    y = Q.rope(x, pos, f, layout, 16, 1.5)
    i, j = ((np.arange(5), np.arange(5) + 8) if layout == "half" else (2 * np.arange(5), 2 * np.arange(5) + 1))
    z = (x[..., i] + 1j * x[..., j]) * 1.5 * np.exp(1j * pos[:, None, None] * f)
    assert np.allclose(y[..., i], z.real, atol=1e-9) and np.allclose(y[..., j], z.imag, atol=1e-9)
    rest = np.setdiff1d(np.arange(24), np.concatenate([i, j]))
    assert np.array_equal(y[..., rest], x[..., rest])
    back = Q.rope(y, pos, f, layout, 16, 1.0 / 1.5, inverse=True)
    assert np.allclose(back, x, atol=1e-9)


def test_scaled_frequencies():
    g = Q.rope_frequencies(64, 32)
    assert np.allclose(Q.rope_frequencies(64, 32, scaling="linear", factor=4.0), g / 4)
    # raised base: the fastest pair stays, the slowest (j = span/2 - 1) slows by the factor
    r = Q.rope_frequencies(64, 32, scaling="raised", factor=4.0)
    assert r[0] == 1.0 and math.isclose(r[-1], g[-1] / 4)
    p = Q.rope_frequencies(64, 32, scaling="parts", factor=4.0, original=8192)
    turns = 8192 * g / (2 * math.pi)
    assert np.allclose(p[turns >= 32], g[turns >= 32]) and np.allclose(p[turns <= 1], g[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert np.all(p[mid] < g[mid]) and np.all(p[mid] > g[mid] / 4) and mid.any()


def test_append_keeps_the_larger_scale_and_rewrites_the_committed_codes():
    codes = np.zeros((2, 1, 64, 4), dtype=np.uint8)
    scales = np.ones((2, 1, 4), dtype=np.float32)
    Q.append(codes, scales, 16, [1, 0], 0, np.full((10, 1, 4), 448.0))
    assert scales[1, 0, 0] == 1.0 and np.all(codes[1, 0, :10] == Q.e4m3_codes(448.0))
    Q.append(codes, scales, 16, [1, 0], 8, np.full((12, 1, 4), 900.0))     # two rows rolled back
    assert scales[1, 0, 0] == 4.0 and scales[1, 0, 1] == 4.0
    assert np.all(Q.VALUES[codes[1, 0, :8]] * 4 == 448.0)
    assert np.all(Q.VALUES[codes[1, 0, 8:20]] * 4 == 896.0) and not codes[1, 0, 20:].any()
    Q.append(codes, scales, 16, [1, 0], 20, np.full((1, 1, 4), 1.0))       # a smaller row keeps the scale
    assert scales[1, 0, 1] == 4.0


@pytest.mark.parametrize("window", [0, 9])
def test_attention_agrees_with_a_masked_softmax(window):
    rng = np.random.default_rng(2)
    H, G, D, L, n, block = 2, 3, 16, 70, 4, 16
    table = [2, 0]
    pools = [(np.zeros((3, H, 64, D), dtype=np.uint8), np.ones((3, H, 4), dtype=np.float32)) for _ in range(2)]
    x = [rng.normal(size=(L + n, H, D)) for _ in range(2)]
    for (c, s), rows in zip(pools, x):
        Q.append(c, s, block, table, 0, rows)
    q = rng.normal(size=(n, H * G, D))
    out, *_ = Q.attention(q, *pools[0], *pools[1], block, table, L, 0, n, window)
    kv = []
    for c, s in pools:
        j = np.arange(L + n)
        page, slot = np.array(table)[j // 64], j % 64
        kv.append(torch.from_numpy(Q.VALUES[c[page, :, slot]] * s[page, :, slot // block][..., None].astype(float)))
    j, p = torch.arange(L + n), torch.arange(L, L + n)[:, None]
    seen = (j <= p) & ((j > p - window) if window else True)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), *(t.transpose(0, 1).repeat_interleave(G, 0) for t in kv),
        attn_mask=seen).transpose(0, 1).numpy()
    assert np.allclose(out, want, atol=1e-12)


def test_rows_that_see_no_key_are_zero():
    c, s = np.zeros((1, 1, 64, 16), dtype=np.uint8), np.ones((1, 1, 4), dtype=np.float32)
    out, *_ = Q.attention(np.ones((2, 1, 16)), c, s, c, s, 16, [0], 5, 3, 0, 2)   # window ends past the cache
    assert not out.any()
    out, *_ = Q.attention(np.ones((2, 1, 16)), c, s, c, s, 16, [0], 0, 0, 0, 0)   # empty cache
    assert not out.any()
