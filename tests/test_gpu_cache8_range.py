"""Attention over the 8-bit cache where scores, value scales, codes and lengths lie far apart, against the fp64 oracle.

Most caches are written by hand: channel 0 of the keys separates the scores, and values and their
scales are set block by block.  The tolerance is that of tests/test_gpu_cache8.py, and half a step of
fp32's subnormals, 2^-150, for each of the three roundings that a subnormal result can meet.

Where weights lie far below their row's largest p s_V, each may be off by 2^-37 of that instead: the
weights' terms are fp16 numbers relative to it, which stands at 2^12 at least, and half a step of
fp16's subnormals is 2^-25 (up to four rows: of the second term, which is times 2^11 there: 2^-48).  A
value code c of such a token turns that into |c| 2^-37 max(p s_V)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache8 as o8
from quantization_cg_encode_b200 import cg
from tests.gpu_util import bf16_np, need_gpu
from tests.test_gpu_cache8 import Cache, _attend, _check_attention, _close, _new

pytestmark = pytest.mark.gpu

# (B, H, T, rows of a KV head): a unit that one CTA takes, one for a cluster, one that equal runs cut
# into many pieces, many units in runs, and runs that cut units into few pieces
SHAPES = [(1, 1, 128, 4), (1, 1, 2048, 4), (1, 1, 24576, 2), (45, 8, 256, 3), (40, 8, 1056, 8), (2, 1, 2048, 16)]


def _byte(v, code):
    return o8.encode(np.asarray(v, np.float64), code)


def _cache(B, H, T, d, code, tb=16):
    """Keys zero, values zero, all scales 1."""
    c = Cache(1, B, H, T, d, code, tb)
    c.codes[:] = 0
    c.scales[:] = 1
    return c


def _queries(B, H, rows, d):
    """1 in channel 0: a token's score is its key's channel 0 times the call's scale."""
    q = torch.zeros((1, B, H * rows, 1, d), dtype=torch.bfloat16)
    q[..., 0] = 1
    return q


def _check(c, q, lens, scale, far=False):
    scale = float(np.float32(scale))
    got = _attend(c, q, lens, scale=scale)
    ref, _, spread, big = o8.attention(bf16_np(q), c.codes, c.scales, lens, c.code, c.tb, scale)
    eps = big[..., None] * (c.dims[4] / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    err, tol = np.abs(got - ref), 2 * eps * spread + 3 * 2.0 ** -150
    if far:  # the rows of a KV head are the same
        n, (_, B, H, T, d) = lens[0], c.dims
        s = o8.decode(c.codes[0, 0, :, :, :n, 0], c.code) * scale
        w = np.exp(s - s.max(-1, keepdims=True))
        largest = (w / w.sum(-1, keepdims=True) * np.repeat(c.scales[0, 1], c.tb, -1)[..., :n]).max(-1)
        low = 2.0 ** (-48 if q.shape[2] // H <= 4 else -37) * largest[..., None] * np.abs(o8.decode(c.codes[0, 1, :, :, :n], c.code)).sum(2)  # [B, H, d]
        tol = tol + np.repeat(low, q.shape[2] // H, 1)[None, :, :, None]
    assert (err <= tol).all(), "worst %.3g of its tolerance" % np.nanmax(err / tol)
    return ref


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,T,rows", SHAPES)
def test_outputs_near_the_least_normal_number(B, H, T, rows, code):
    """Values stored at the least scale give outputs that fp32 holds, whatever the scores are."""
    need_gpu()
    d = 64
    c = _cache(B, H, T, d, code)
    rng = np.random.default_rng(T)
    c.codes[:, 0, ..., 0] = _byte(rng.integers(-8, 9, (B, H, T)), code)
    c.codes[:, 1] = _byte(rng.integers(1, 16, (B, H, T, d)), code)
    c.scales[:, 1] = 2.0 ** -126
    c.up()
    ref = _check(c, _queries(B, H, rows, d), [T - 3] * B, 0.25)
    assert ref.min() > 2.0 ** -126 and ref.max() < 1e-36


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,T,rows", SHAPES)
@pytest.mark.parametrize("gap,light,value", [(95, 0, 0), (110, 100, 0), (95, 120, 96), (120, 110, 0), (140, 120, 1)])
def test_light_tokens_with_the_larger_value_scales_are_the_output(B, H, T, rows, gap, light, value, code):
    """Half of the blocks draw all of the weight and hold values of the least scale, the others have
    weights 2^-gap and the scale 2^light: the output is theirs."""
    need_gpu()
    d = 64
    c = _cache(B, H, T, d, code)
    heavy = np.random.default_rng(T + gap).random((1, B, H, T // 16)) < 0.5
    heavy[..., 0], heavy[..., 1] = True, False
    c.codes[:, 0, ..., 0] = np.where(np.repeat(heavy, 16, -1), _byte(96, code), 0)
    c.codes[:, 1] = np.where(np.repeat(heavy, 16, -1)[..., None], _byte(value, code), _byte(96, code))
    c.scales[:, 1] = np.where(heavy, 2.0 ** -126, 2.0 ** light)
    c.up()
    _check(c, _queries(B, H, rows, d), [T - 3] * B, gap * math.log(2) / 96)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,T,rows", SHAPES)
@pytest.mark.parametrize("ratio", [12, 20, 33, 34, 35, 60])
def test_channels_that_only_blocks_of_small_scales_reach(B, H, T, rows, ratio, code):
    """One value block has a scale 2^ratio times the others' and codes in one channel only: the other
    channels are the other blocks'."""
    need_gpu()
    d = 64
    c = _cache(B, H, T, d, code)
    rng = np.random.default_rng(T + ratio)
    c.codes[:, 0, ..., 0] = _byte(rng.integers(-8, 9, (B, H, T)), code)
    c.codes[:, 1] = _byte(rng.integers(0, 16, (B, H, T, d)), code)
    c.codes[:, 1, :, :, 16:32] = 0
    c.codes[:, 1, :, :, 16:32, 5] = _byte(96, code)
    c.scales[:, 1, :, :, 1] = 2.0 ** ratio
    c.up()
    _check(c, _queries(B, H, rows, d), [T - 3] * B, 0.25, far=True)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,T,rows", SHAPES)
@pytest.mark.parametrize("gap", [12.4, 20.4, 31.4, 33.4, 34.4, 35.4, 60.4])
def test_channels_that_only_light_tokens_reach(B, H, T, rows, gap, code):
    """One token has 2^gap times the others' weights and codes in the even channels only: the odd
    channels are the other tokens', those of its own tile among them."""
    need_gpu()
    d = 64
    c = _cache(B, H, T, d, code)
    rng = np.random.default_rng(T + int(gap))
    c.codes[:, 0, :, :, 21, 0] = _byte(96, code)
    c.codes[:, 1] = _byte(rng.integers(0, 16, (B, H, T, d)), code)
    c.codes[:, 1, :, :, 21, 1::2] = 0
    c.up()
    _check(c, _queries(B, H, rows, d), [T - 3] * B, gap * math.log(2) / 96, far=True)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,rows", [(64, 4), (128, 16)])
def test_queries_with_an_element_far_above_the_others(d, rows, code):
    """One element 2^30, the others down to 1/2, and keys that are zero where it is: exact down to 2^-31
    of the row's largest, so the scores are the others'."""
    need_gpu()
    B, H, T = 2, 2, 256
    c = _cache(B, H, T, d, code)
    rng = np.random.default_rng(d)
    c.codes[:, :, :, :, :, 1:] = _byte(rng.integers(-15, 16, (1, 2, B, H, T, d - 1)), code)
    c.up()
    q = _queries(B, H, rows, d)
    q[..., 0] = 2.0 ** 30
    x = torch.from_numpy(rng.uniform(0.5, 4, q[..., 1:].shape) * rng.choice([-1.0, 1.0], q[..., 1:].shape))
    q[..., 1:] = x.to(torch.bfloat16)
    _check(c, q, [T, T - 39], 2.0 ** -7)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,d,gq,nq,live", [(80, 1, 128, 4, 1, 0), (80, 1, 64, 2, 3, 41), (24, 2, 128, 8, 2, 23), (12, 8, 64, 4, 1, 5)])
def test_one_long_sequence_beside_vacant_slots(B, H, d, gq, nq, live, code):
    """All runs are pieces of its few units, although the batch has many; a short one at the other end."""
    need_gpu()
    T, tb = 8192, 64
    lens = [0] * B
    lens[live], lens[B - 1 - live] = T - 9, 70
    c = Cache(1, B, H, T, d, code, tb)
    rng = np.random.default_rng(B + d)
    for b in (live, B - 1 - live):
        c.codes[0, :, b, :, :lens[b]] = _byte(rng.integers(-60, 61, (2, H, lens[b], d)), code)
        c.scales[0, :, b] = 2.0 ** rng.integers(-9, -5, (2, H, T // tb))
    c.up()
    q = _new(torch.Generator().manual_seed(B), 1, B, H * gq, nq, d)
    ref, want, spread, big = _check_attention(c, q, lens)
    eps = big.max() * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    mass = torch.full((1, B, H, T // tb), 7.0, dtype=torch.float32, device="cuda")
    got = _attend(c, q, lens, mass=mass)
    _close(got, ref, spread, big, d)
    assert np.all(np.abs(mass.cpu().numpy().astype(np.float64) - want) <= 2 * eps * want)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,H,d,gq,nq", [(8, 8, 128, 4, 1), (9, 8, 64, 3, 4), (3, 6, 128, 8, 2), (40, 8, 64, 2, 1)])
def test_short_sequences_in_a_call_for_long_ones(B, H, d, gq, nq, code):
    """The work is laid out for lengths that the sequences do not have."""
    need_gpu()
    T, tb = 20480, 16
    lens = [(1, 16, 40, 0, 17, 33, 5, 130)[b % 8] for b in range(B)]
    c = Cache(1, B, H, T, d, code, tb)
    rng = np.random.default_rng(B + d)
    n = 144
    c.codes[:, :, :, :, :n] = _byte(rng.integers(-60, 61, (1, 2, B, H, n, d)), code)
    c.scales[..., :n // tb] = 2.0 ** rng.integers(-9, -5, (1, 2, B, H, n // tb))
    c.up()
    q = _new(torch.Generator().manual_seed(B), 1, B, H * gq, nq, d)
    ref, want, spread, big = _check_attention(c, q, lens)
    eps = big.max() * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    mass = torch.full((1, B, H, T // tb), 7.0, dtype=torch.float32, device="cuda")
    got = _attend(c, q, lens, mass=mass)
    _close(got, ref, spread, big, d)
    assert np.all(np.abs(mass.cpu().numpy().astype(np.float64) - want) <= 2 * eps * want)
