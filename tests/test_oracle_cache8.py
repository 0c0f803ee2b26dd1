"""The oracle of the 8-bit block-scaled cache against the formats' definitions and closed forms."""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8


def test_e4m3_table_and_rounding_match_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, o8.E4M3_VALUES, equal_nan=True)
    rng = np.random.default_rng(1)
    g = o8.E4M3_VALUES[:127]
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000), g, (g[1:] + g[:-1]) / 2, -(g[1:] + g[:-1]) / 2])
    x = x.astype(np.float32)  # midpoints are exact in fp32
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o8.encode(x, o8.E4M3), want)


@pytest.mark.parametrize("code", [o8.INT8, o8.E4M3])
def test_scale_is_the_least_power_of_two(code):
    top = o8.TOP[code]
    for a in [top, np.nextafter(top, 0), np.nextafter(top, 1e9), 1.0, 3e38, 1e-30, 2.0 ** -126, 2.0 ** -133]:
        s = o8.scale_of(a, code)
        assert np.frexp(s)[0] == 0.5 and a <= top * s
        assert s == 2.0 ** -126 or a > top * s / 2
    assert o8.scale_of(0.0, code) == 2.0 ** -126


@pytest.mark.parametrize("code", [o8.INT8, o8.E4M3])
def test_one_append_rounds_to_half_a_step(code):
    rng = np.random.default_rng(2)
    T, d, tb = 64, 64, 16
    c = np.zeros((1, 2, 1, 1, T, d), np.uint8)
    s = np.zeros((1, 2, 1, 1, T // tb))
    b = np.zeros((1, 1, 1, T // tb, 2, d), np.int8)
    x = rng.standard_normal((1, 2, 1, 1, T, d))
    o8.append(c, s, b, x, [0], None, code, tb)
    sc = np.repeat(s, tb, -1)[..., None]
    y = o8.decode(c, code) * sc
    step = sc if code == o8.INT8 else np.maximum(np.abs(x) * 2.0 ** -3, sc * 2.0 ** -9)
    assert np.all(np.abs(y - x) <= 0.5 * step)
    # the bounds enclose what they bound
    k = o8.decode(c[0, 0, 0, 0], code).reshape(T // tb, tb, d) * (1 if code == o8.INT8 else 127 / 448)
    assert np.all(b[0, 0, 0, :, 0] <= k.min(1) + 1e-12) and np.all(b[0, 0, 0, :, 1] >= k.max(1) - 1e-12)


def test_attention_of_equal_keys_is_the_mean_and_empty_rows_are_zero():
    rng = np.random.default_rng(3)
    T, d, tb = 32, 64, 16
    c = rng.integers(0, 256, (1, 2, 2, 1, T, d)).astype(np.uint8)
    c[0, 0] = 5
    s = np.full((1, 2, 2, 1, T // tb), 0.25)
    q = rng.standard_normal((1, 2, 2, 3, d))
    out, mass, _, _ = o8.attention(q, c, s, [20, 2], o8.INT8, tb, 0.1)
    v = o8.decode(c[0, 1, 0, 0], o8.INT8) * 0.25
    for i in range(3):
        assert np.allclose(out[0, 0, 1, i], v[:18 + i].mean(0))
    assert np.all(out[0, 1, :, 0] == 0) and np.any(out[0, 1, :, 1] != 0)
    assert np.allclose(mass.sum(-1), [[[6.0], [4.0]]])


def test_scores_bound_the_rounded_products_and_ties_go_low():
    rng = np.random.default_rng(4)
    d, tb, nb = 64, 16, 12
    k = rng.integers(-127, 128, (nb, tb, d))
    bounds = np.stack([k.min(1), k.max(1)], 1).astype(np.int8)
    sc = 2.0 ** rng.integers(-3, 3, nb)
    q = rng.standard_normal((3, d))
    got = o8.scores(q, bounds, sc)
    for j in range(3):
        u = o8.scale_of(np.abs(q[j]).max(), o8.INT8)
        assert np.all(got >= (np.rint(q[j] / u) * u * k * sc[:, None, None]).sum(-1).max(1) - 1e-9)
    assert o8._pick(np.array([1.0, 3, 3, 3, 2, 9]), 6, 3, 0, 1) == [1, 2, 5]
