"""The 8-bit block-scaled KV cache on the GPU against the fp64 oracle (oracle/cache8.py).

Stored bytes, scales, bounds, chosen blocks and moved blocks have to be equal bit for bit: every
step of theirs is exact or one rounding of an exact number.

Attention's tolerance, per output value, with A the largest scale sum_c |q_c k_c| of its row:
  scores    d / 16 + 4 fp32 roundings (the tensor core's sums may be cut off instead of
            rounded: 2^-23 each) of at most A log2(e); to a weight: times ln 2
  weights   2^-22 (ex2.approx, 2 ulp) + 2^-22 (two fp16 terms) + the lazily moved maxima's
            rescaling, one 2^-22 for each of at most 32 moves
so a weight is off by at most eps = A (d / 16 + 4) 2^-23 + 40 2^-22 of itself, numerator and sum
both, and an output by 2 eps sum_t p_t |v_t|; the block weights by 2 eps of themselves."""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8
from quantization_cg_encode_b200 import cg
from tests.gpu_util import bf16_np, need_gpu

pytestmark = pytest.mark.gpu


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Cache:
    """Device buffers of one cache and the oracle's copy of them, filled with whatever was there before."""

    def __init__(self, L, B, H, T, d, code, tb, seed=0):
        rng = np.random.default_rng(seed)
        self.kv, self.c8 = cg.kv_desc(L, B, H, T, d), cg.cache8_desc(code, tb)
        self.code, self.tb, self.dims = code, tb, (L, B, H, T, d)
        nb = T // tb
        # patterns that are NaN as e4m3, scales that are NaN: nothing of it may reach a result
        self.codes = rng.choice(np.array([0x7F, 0xFF, 0x80, 0x55, 0], np.uint8), (L, 2, B, H, T, d))
        self.scales = np.full((L, 2, B, H, nb), np.nan, np.float32)
        self.bounds = rng.integers(-128, 128, (L, B, H, nb, 2, d)).astype(np.int8)
        self.mass = np.zeros((L, B, H, nb), np.float32)
        self.up()

    def up(self):
        self.d_codes, self.d_scales, self.d_bounds, self.d_mass = map(_cuda, (self.codes, self.scales, self.bounds, self.mass))

    def append(self, new, pos, counts=None, layer0=0, bounds=True):
        p = _cuda(np.asarray(pos, np.int32))
        n = None if counts is None else _cuda(np.asarray(counts, np.int32))
        cg.cg_cache8_append(self.kv, self.c8, layer0, new.cuda(), p, n, self.d_codes, self.d_scales, self.d_bounds if bounds else None)
        cg.cg_sync_status()
        o8.append(self.codes, self.scales, self.bounds if bounds else None, bf16_np(new), pos, counts, self.code, self.tb, layer0)

    def same(self):
        assert np.array_equal(self.d_scales.cpu().numpy(), self.scales, equal_nan=True)
        assert np.array_equal(self.d_codes.cpu().numpy(), self.codes)
        assert np.array_equal(self.d_bounds.cpu().numpy(), self.bounds)


def _new(gen, *shape, gain=1.0):
    return (torch.randn(shape, generator=gen) * gain).to(torch.bfloat16)


def _filled(L, B, H, T, d, code, tb, lens, seed=0, spread=0):
    """A cache whose sequence b holds lens[b] tokens; `spread`: scales differ by up to 2^spread."""
    c = Cache(L, B, H, T, d, code, tb, seed)
    gen = torch.Generator().manual_seed(seed)
    n = max(max(lens), 1)
    x = torch.randn((L, 2, B, H, n, d), generator=gen)
    if spread:
        e = torch.randint(-spread // 2, spread // 2 + 1, (L, 1, B, H, -(-n // tb), 1), generator=gen).float()
        x[:, 1:] *= torch.exp2(e).repeat_interleave(tb, 4)[..., :n, :]
    c.append(x.to(torch.bfloat16), [0] * B, lens)
    return c


# ---- append ------------------------------------------------------------------------------------


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,n", [(128, 16, 1), (64, 16, 37), (128, 32, 50), (64, 64, 70), (128, 64, 1), (64, 32, 64)])
def test_append_in_pieces(code, d, tb, n):
    """Pieces at ragged positions, one after another, so that blocks are met empty, partly filled by
    smaller and by larger tokens, and full; untouched bytes stay."""
    need_gpu()
    L, B, H, T = 2, 4, 3, 256
    c = Cache(L, B, H, T, d, code, tb, seed=n)
    gen = torch.Generator().manual_seed(n + d)
    pos = np.array([0, 5, tb, 2 * tb - 1])
    c.append(_new(gen, L, 2, B, H, 2 * tb, d), [0] * B, pos)            # what the sequences hold before
    for step in range(4):
        counts = None if step == 0 else [n, max(0, n - 1), 0, min(n, 3 + step)]
        x = _new(gen, 1, 2, B, H, n, d, gain=2.0 ** (step - 1))
        c.append(x, pos, counts, layer0=1)
        c.same()
        pos = pos + (n if counts is None else np.array(counts))
    assert not np.isnan(c.scales[1, :, 0, :, 0]).any()


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
def test_append_extremes(code):
    """Zeros, the smallest and the largest bf16 numbers, a block that grows by 2^100."""
    need_gpu()
    L, B, H, T, d, tb = 1, 4, 1, 64, 64, 16
    c = Cache(L, B, H, T, d, code, tb)
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((L, 2, B, H, 9, d), generator=gen)
    x[:, :, 0] = 0
    x[:, :, 1] *= 2.0 ** -131
    x[:, :, 2] *= 2.0 ** 124
    x[:, :, 3] *= 2.0 ** -50
    c.append(x.to(torch.bfloat16), [0, 0, 0, 0])
    c.same()
    y = torch.randn((L, 2, B, H, 1, d), generator=gen)
    y[:, :, 3] *= 2.0 ** 50
    c.append(y.to(torch.bfloat16), [9, 9, 9, 9])
    c.same()


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
def test_append_again_after_draft_tokens_are_dropped(code):
    """Positions go back into a block, to its start and into the block before, and are stored again."""
    need_gpu()
    L, B, H, T, d, tb = 1, 4, 2, 128, 64, 32
    c = Cache(L, B, H, T, d, code, tb)
    gen = torch.Generator().manual_seed(8)
    c.append(_new(gen, L, 2, B, H, 70, d), [0] * B)
    c.append(_new(gen, L, 2, B, H, 5, d, gain=8), [69, 64, 60, 33])
    c.append(_new(gen, L, 2, B, H, 5, d, gain=0.25), [66, 64, 32, 34])
    c.same()
    q = _new(gen, L, B, 3 * H, 1, d)
    _check_attention(c, q, [71, 69, 37, 39])


def test_append_off_the_cache_stores_nothing_there():
    need_gpu()
    L, B, H, T, d, tb = 1, 6, 2, 64, 64, 32
    c = Cache(L, B, H, T, d, cg.CACHE8_INT8, tb)
    gen = torch.Generator().manual_seed(6)
    c.append(_new(gen, L, 2, B, H, 40, d), [0] * B)
    x = _new(gen, L, 2, B, H, 20, d, gain=3)
    # negative, at the end, beyond it, across it, a negative and an oversized count
    c.append(x, [-1, T, 2 ** 31 - 1, T - 7, 40, 40], [20, 20, 20, 20, -5, 1000])
    c.same()


def test_append_without_bounds_and_the_last_layers():
    need_gpu()
    c = Cache(3, 2, 2, 64, 128, cg.CACHE8_E4M3, 16)
    gen = torch.Generator().manual_seed(7)
    c.append(_new(gen, 2, 2, 2, 2, 33, 128), [0, 3], layer0=1, bounds=False)
    c.same()


# ---- attention -----------------------------------------------------------------------------------


def _attend(c, q, lens, max_tokens=None, layer0=0, sel=None, mass=None, accumulate=False, scale=None):
    L, B, H, T, d = c.dims
    at = cg.cache8_attn_desc(q.shape[2], max_tokens or T, q_tokens=q.shape[3], layer0=layer0, n_layers=q.shape[0], d_head=d,
                             scale=scale, n_select=0 if sel is None else sel.shape[-1], accumulate=accumulate)
    # the workspace begins as NaN: nothing in it may be read before it is written
    ws = torch.full((cg.cg_cache8_attention_workspace_size(c.kv, c.c8, at, mass is not None),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    cg.cg_cache8_attention(c.kv, c.c8, at, q.cuda(), c.d_codes, c.d_scales, _cuda(np.asarray(lens, np.int32)), out, ws,
                           sel=None if sel is None else _cuda(sel.astype(np.int32)), mass=mass)
    cg.cg_sync_status()
    return out.cpu().numpy().astype(np.float64)


def _close(got, ref, spread, big, d):
    eps = big[..., None] * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    err = np.abs(got - ref)
    ok = err <= 2 * eps * spread
    assert ok.all(), "worst %.3g of its tolerance" % np.nanmax(err / np.maximum(2 * eps * spread, 1e-300))


def _check_attention(c, q, lens, layer0=0, max_tokens=None, sel=None):
    d = c.dims[4]
    got = _attend(c, q, lens, max_tokens, layer0, sel)
    scale = float(np.float32(1.0 / d ** 0.5))
    ref, mass, spread, big = o8.attention(bf16_np(q), c.codes, c.scales, lens, c.code, c.tb, scale, layer0, max_tokens, sel)
    _close(got, ref, spread, big, d)
    return ref, mass, spread, big


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,gq,nq", [(128, 16, 4, 1), (64, 32, 1, 1), (128, 64, 8, 1), (64, 16, 3, 2), (128, 32, 5, 3), (64, 64, 16, 1),
                                        (128, 16, 16, 16), (128, 16, 8, 2), (64, 16, 2, 5)])
def test_attention_lengths_and_groups(code, d, tb, gq, nq):
    """Lengths from none to the capacity, on both sides of tiles and blocks."""
    need_gpu()
    T, H = 512, 2
    lens = [0, 1, 15, 16, 17, tb + 1, 255, T]
    c = _filled(2, len(lens), H, T, d, code, tb, lens, seed=d + gq)
    q = _new(torch.Generator().manual_seed(gq + nq), 1, len(lens), H * gq, nq, d, gain=1.5)
    _check_attention(c, q, lens, layer0=1)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("B,T,gq,nq", [(1, 8192, 4, 1), (3, 2048, 4, 4), (1, 5120, 1, 1), (2, 24576, 3, 1), (3, 17408, 4, 4)])
def test_attention_of_long_sequences(code, B, T, gq, nq):
    """Sequences that the CTAs of a cluster share, or (over 16384 tokens) that equal runs cut into
    many pieces, with value scales 2^40 apart and far tokens that matter."""
    need_gpu()
    lens = [T - 3 - 700 * b for b in range(B)]
    if T > 16384:
        lens[1] = 0                     # a vacant sequence between or behind long ones
    c = _filled(1, B, 1, T, 64, code, 16, lens, seed=T, spread=40)
    q = _new(torch.Generator().manual_seed(2), 1, B, gq, nq, 64, gain=4.0)
    _check_attention(c, q, lens, max_tokens=T - 1)


@pytest.mark.parametrize("d,T,gq,nq", [(128, 40960, 4, 1), (64, 33024, 2, 3), (128, 20480, 8, 2)])
def test_attention_of_one_long_head_cut_into_many_pieces_with_block_weights(d, T, gq, nq):
    """One unit, of which every CTA has a piece: up to 296 of them, merged side by side."""
    need_gpu()
    tb, lens = 64, [T - 5]
    c = _filled(1, 1, 1, T, d, cg.CACHE8_INT8, tb, lens, seed=T, spread=20)
    q = _new(torch.Generator().manual_seed(gq), 1, 1, gq, nq, d, gain=2.0)
    ref, want, spread, big = _check_attention(c, q, lens)
    eps = big.max() * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    mass = torch.full((1, 1, 1, T // tb), 7.0, dtype=torch.float32, device="cuda")
    got = _attend(c, q, lens, mass=mass)
    _close(got, ref, spread, big, d)
    assert np.all(np.abs(mass.cpu().numpy().astype(np.float64) - want) <= 2 * eps * want)


@pytest.mark.parametrize("B,gq,nq", [(4, 8, 2), (8, 4, 1), (17, 3, 1)])
def test_attention_of_units_around_the_number_of_clusters_at_once(B, gq, nq):
    need_gpu()
    T, H, d = 1024, 4, 128
    lens = [T - 60 * b for b in range(B)]
    c = _filled(1, B, H, T, d, cg.CACHE8_E4M3, 32, lens, seed=B)
    q = _new(torch.Generator().manual_seed(B), 1, B, H * gq, nq, d, gain=1.5)
    _check_attention(c, q, lens)


@pytest.mark.parametrize("d,gq,nq", [(128, 2, 1), (64, 3, 4)])
def test_attention_runs_over_many_ragged_sequences_with_block_weights(d, gq, nq):
    """More units than CTAs: a CTA's run holds whole sequences and pieces of two more."""
    need_gpu()
    B, H, T = 45, 8, 256
    lens = [(97 * b) % (T + 1) for b in range(B)]
    c = _filled(1, B, H, T, d, cg.CACHE8_INT8, 32, lens, seed=d)
    q = _new(torch.Generator().manual_seed(d), 1, B, H * gq, nq, d, gain=1.5)
    ref, want, spread, big = _check_attention(c, q, lens)
    eps = big.max() * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    mass = torch.full((1, B, H, T // 32), 7.0, dtype=torch.float32, device="cuda")
    got = _attend(c, q, lens, mass=mass)
    _close(got, ref, spread, big, d)
    assert np.all(np.abs(mass.cpu().numpy().astype(np.float64) - want) <= 2 * eps * want)


def test_attention_batch_of_many_heads_takes_whole_sequences_a_cta():
    need_gpu()
    B, H, T, d = 40, 32, 64, 64
    lens = [(7 * b) % (T + 1) for b in range(B)]
    c = _filled(1, B, H, T, d, cg.CACHE8_INT8, 16, lens, seed=3)
    q = _new(torch.Generator().manual_seed(3), 1, B, H, 1, d)
    _check_attention(c, q, lens)


@pytest.mark.parametrize("gain,spread", [(1e-30, 0), (30.0, 100), (0.0, 0)])
def test_attention_extreme_values(gain, spread):
    """Queries near zero, weights on one token, value blocks 2^100 apart, a block of zeros."""
    need_gpu()
    T, d, lens = 256, 128, [256, 130]
    c = _filled(1, 2, 1, T, d, cg.CACHE8_INT8, 16, lens, seed=11, spread=spread)
    c.append(torch.zeros((1, 2, 2, 1, 16, d), dtype=torch.bfloat16), [32, 32])
    q = _new(torch.Generator().manual_seed(4), 1, 2, 4, 1, d, gain=gain)
    _check_attention(c, q, lens)


def test_attention_lengths_out_of_range_are_clamped():
    need_gpu()
    T, d = 128, 64
    c = _filled(1, 3, 1, T, d, cg.CACHE8_E4M3, 16, [T, T, T], seed=12)
    q = _new(torch.Generator().manual_seed(5), 1, 3, 2, 1, d)
    got = _attend(c, q, [-5, 2 ** 31 - 1, 100], max_tokens=96)
    want = _attend(c, q, [0, 96, 96], max_tokens=96)
    assert np.array_equal(got, want) and np.all(got[0, 0] == 0)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,gq,nq,lens", [(128, 16, 4, 1, [512, 0, 33]), (64, 64, 2, 4, [2, 300, 512]), (128, 32, 8, 3, [70, 511, 1])])
def test_attention_block_weights(code, d, tb, gq, nq, lens):
    need_gpu()
    T, H, L = 512, 2, 2
    c = _filled(L, len(lens), H, T, d, code, tb, lens, seed=d + tb)
    q = _new(torch.Generator().manual_seed(8), 1, len(lens), H * gq, nq, d, gain=2.0)
    _, want, _, big = _check_attention(c, q, lens, layer0=1)
    eps = big.max() * (d / 16 + 4) * 2.0 ** -23 + 40 * 2.0 ** -22
    mass = torch.full((L, len(lens), H, T // tb), 7.0, dtype=torch.float32, device="cuda")
    _attend(c, q, lens, layer0=1, mass=mass)
    got = mass.cpu().numpy().astype(np.float64)
    assert np.all(got[0] == 7.0) and np.all(np.abs(got[1] - want[0]) <= 2 * eps * want[0])
    mass.fill_(7.0)
    _attend(c, q, lens, layer0=1, mass=mass, accumulate=True)
    acc = mass.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(acc[1] - 7.0 - want[0]) <= 2 * eps * want[0] + 2.0 ** -21)
    has = np.arange(T // tb)[None] < -(-np.array(lens) // tb)[:, None]
    assert np.all(np.where(has[:, None], 7.0, acc[1]) == 7.0)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,gq,nq,k", [(128, 16, 4, 1, 9), (64, 32, 3, 3, 1), (128, 64, 16, 2, 8), (64, 16, 8, 1, 32)])
def test_attention_over_listed_blocks(code, d, tb, gq, nq, k):
    """Lists in any order, with absent entries, entries outside the sequence, the same one twice, and none at all."""
    need_gpu()
    T, H = 512, 2
    lens = [0, 1, 200, 331, T]
    c = _filled(1, len(lens), H, T, d, code, tb, lens, seed=k)
    rng = np.random.default_rng(k)
    sel = rng.integers(-1, T // tb, (1, len(lens), H, nq, k)).astype(np.int32)
    sel[0, 2, 0] = -1
    sel[0, 3, 0, 0] = sel[0, 3, 0, 0, 0]
    sel[0, 4, 1, -1, 0] = 2 ** 31 - 1
    sel[0, 4, 0, 0, 0] = -2 ** 31
    q = _new(torch.Generator().manual_seed(k), 1, len(lens), H * gq, nq, d, gain=1.5)
    _check_attention(c, q, lens, sel=sel)


@pytest.mark.parametrize("T,tb,k", [(8192, 16, 300), (32768, 64, 300)])
def test_attention_over_a_long_list(T, tb, k):
    """One list for a cluster, and one (1200 tiles) for equal runs."""
    need_gpu()
    d = 64
    c = _filled(1, 1, 1, T, d, cg.CACHE8_INT8, tb, [T - 5], seed=21)
    sel = np.random.default_rng(1).permutation(T // tb)[:k].reshape(1, 1, 1, 1, k)
    q = _new(torch.Generator().manual_seed(9), 1, 1, 2, 1, d, gain=2.0)
    _check_attention(c, q, [T - 5], sel=sel)


def test_attention_over_lists_of_many_ragged_sequences():
    need_gpu()
    B, H, T, d, tb, k, nq = 30, 4, 512, 64, 16, 9, 3
    lens = [(61 * b) % (T + 1) for b in range(B)]
    c = _filled(1, B, H, T, d, cg.CACHE8_E4M3, tb, lens, seed=22)
    q = _new(torch.Generator().manual_seed(10), 1, B, 2 * H, nq, d)
    sel = _select(c, q, lens, k, 1, 1)
    assert np.array_equal(sel, o8.select(bf16_np(q), c.bounds, c.scales, lens, tb, k, 1, 1, H))
    _check_attention(c, q, lens, sel=sel)


def test_attention_behind_four_gigabytes():
    """A layer whose codes begin above 2^32 bytes gives the bits of the same layer alone."""
    need_gpu()
    L, B, H, T, d, tb = 33, 1, 8, 65536, 128, 64
    one = _filled(1, B, H, 1024, d, cg.CACHE8_INT8, tb, [1000], seed=13)
    kv, c8 = cg.kv_desc(L, B, H, T, d), cg.cache8_desc(cg.CACHE8_INT8, tb)
    codes, scales, bounds, mass = cg.alloc_cache8(kv, c8)
    assert 32 * codes[0].numel() >= 2 ** 32
    codes[32, :, :, :, :1024] = one.d_codes[0]
    scales[32, :, :, :, :16] = one.d_scales[0]
    bounds[32, :, :, :16] = one.d_bounds[0]
    q = _new(torch.Generator().manual_seed(14), 1, B, 4 * H, 1, d).cuda()
    x = _new(torch.Generator().manual_seed(15), 1, 2, B, H, 3, d).cuda()
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    got = []
    for k, cc, ss, bb, l0 in ((one.kv, one.d_codes, one.d_scales, one.d_bounds, 0), (kv, codes, scales, bounds, 32)):
        cg.cg_cache8_append(k, c8, l0, x, lens, None, cc, ss, bb)
        n = lens + 3
        sd = cg.cache8_select_desc(4 * H, 1003, 5, layer0=l0)
        sel = torch.empty((1, B, H, 1, 5), dtype=torch.int32, device="cuda")
        cg.cg_cache8_select(k, c8, sd, q, ss, bb, n, sel, torch.empty(cg.cg_cache8_select_workspace_size(k, c8, sd), dtype=torch.uint8, device="cuda"))
        at = cg.cache8_attn_desc(4 * H, 1003, layer0=l0)
        ws = torch.empty(cg.cg_cache8_attention_workspace_size(k, c8, at), dtype=torch.uint8, device="cuda")
        out = cg.cg_cache8_attention(k, c8, at, q, cc, ss, n, torch.empty(q.shape, dtype=torch.float32, device="cuda"), ws)
        cg.cg_sync_status()
        got.append((sel, out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.equal(codes[32, :, :, :, :1024], one.d_codes[0])
    assert int(codes[:32].max()) == 0 and int(codes[32, :, :, :, 1024:].max()) == 0


# ---- selection -------------------------------------------------------------------------------------


def _select(c, q, lens, k, sink, recent, layer0=0, max_tokens=None):
    H, T = c.dims[2], c.dims[3]
    sd = cg.cache8_select_desc(q.shape[2], max_tokens or T, k, q_tokens=q.shape[3], sink_blocks=sink, recent_blocks=recent,
                               layer0=layer0, n_layers=q.shape[0])
    ws = torch.full((cg.cg_cache8_select_workspace_size(c.kv, c.c8, sd),), 0xFF, dtype=torch.uint8, device="cuda")
    sel = torch.full((q.shape[0], q.shape[1], H, q.shape[3], k), -7, dtype=torch.int32, device="cuda")
    cg.cg_cache8_select(c.kv, c.c8, sd, q.cuda(), c.d_scales, c.d_bounds, _cuda(np.asarray(lens, np.int32)), sel, ws)
    cg.cg_sync_status()
    return sel.cpu().numpy()


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,gq,nq,k,sink,recent", [(128, 16, 4, 1, 8, 1, 1), (64, 16, 1, 3, 5, 0, 0), (128, 32, 8, 2, 7, 3, 4), (64, 64, 16, 16, 4, 1, 0),
                                                      (128, 16, 5, 1, 32, 2, 2), (64, 16, 3, 2, 1, 0, 0)])
def test_select_matches_the_definition(code, d, tb, gq, nq, k, sink, recent):
    need_gpu()
    T, H = 512, 2
    lens = [0, 1, 17, 260, T - 1, T]
    c = _filled(2, len(lens), H, T, d, code, tb, lens, seed=k)
    q = _new(torch.Generator().manual_seed(k), 1, len(lens), H * gq, nq, d)
    got = _select(c, q, lens, k, sink, recent, layer0=1)
    assert np.array_equal(got, o8.select(bf16_np(q), c.bounds, c.scales, lens, tb, k, sink, recent, H, layer0=1))


@pytest.mark.parametrize("T,d,nq,ks", [(32768, 64, 1, (1, 100, 1500, 2047)), (131072, 64, 16, (77,)), (163840, 128, 2, (1, 9000))])
def test_select_among_many_blocks(T, d, nq, ks):
    """Up to 8192 blocks are chosen in one kernel (for 16 query tokens too), more in two."""
    need_gpu()
    tb = 16
    rng = np.random.default_rng(0)
    c = Cache(1, 2, 1, T, d, cg.CACHE8_INT8, tb)
    b = np.sort(rng.integers(-127, 128, c.bounds.shape).astype(np.int8), axis=4)
    c.bounds = np.ascontiguousarray(b)
    c.scales = (2.0 ** rng.integers(-4, 4, c.scales.shape)).astype(np.float32)
    c.up()
    q = _new(torch.Generator().manual_seed(1), 1, 2, 4, nq, d)
    for k in ks:
        lens = [T, T - 4000]
        assert np.array_equal(_select(c, q, lens, k, 0, 1), o8.select(bf16_np(q), c.bounds, c.scales, lens, tb, k, 0, 1, 1))


def test_select_ties_and_zero_queries_go_to_the_lowest_blocks():
    need_gpu()
    T, d, tb = 1024, 128, 16
    c = Cache(1, 1, 1, T, d, cg.CACHE8_INT8, tb)
    c.bounds[:] = np.array([-3, 5], np.int8)[:, None]
    c.scales[:] = 0.5
    c.scales[..., 40:] = 1.0
    c.up()
    q = _new(torch.Generator().manual_seed(1), 1, 1, 2, 1, d)
    assert _select(c, q, [T], 6, 1, 2)[0, 0, 0, 0].tolist() == [0, 40, 41, 42, 62, 63]
    assert _select(c, q * 0, [T], 6, 1, 2)[0, 0, 0, 0].tolist() == [0, 1, 2, 3, 62, 63]


# ---- eviction ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
@pytest.mark.parametrize("d,tb,keep,sink,recent,T2,bounds", [(128, 16, 6, 1, 2, 128, True), (64, 64, 3, 0, 1, 192, True), (64, 16, 20, 4, 16, 320, False),
                                                             (128, 32, 16, 0, 1, 512, True), (64, 32, 1, 0, 1, 32, True)])
def test_evict_matches_the_definition(code, d, tb, keep, sink, recent, T2, bounds):
    need_gpu()
    L, H, T = 3, 2, 512
    lens = [0, 1, tb, 300, 511, T]
    B = len(lens)
    c = _filled(L, B, H, T, d, code, tb, lens, seed=keep)
    rng = np.random.default_rng(keep)
    c.mass = np.exp(2 * rng.standard_normal(c.mass.shape)).astype(np.float32)
    c.mass[..., ::3] = c.mass[..., :1]          # equal ones
    c.mass[1, -1, 0, 3:7] = [np.nan, -1.0, np.inf, -0.0]
    c.up()
    to = Cache(L, B, H, T2, d, code, tb, seed=1)
    to.mass[:] = 9
    to.up()
    tl = np.zeros(B, np.int32)
    d_tl, kept = _cuda(tl), torch.full((2, B, H, keep), -7, dtype=torch.int32, device="cuda")
    ev = cg.cache8_evict_desc(keep, sink_blocks=sink, recent_blocks=recent, layer0=1, n_layers=2)
    cg.cg_cache8_evict(c.kv, c.c8, ev, _cuda(np.array(lens, np.int32)), c.d_codes, c.d_scales, c.d_bounds if bounds else None, c.d_mass,
                       to.kv, to.d_codes, to.d_scales, to.d_bounds if bounds else None, to.d_mass, d_tl, kept)
    cg.cg_sync_status()
    want = o8.evict(c.codes, c.scales, c.bounds if bounds else None, c.mass, lens, (to.codes, to.scales, to.bounds, to.mass, tl), tb,
                    keep, sink, recent, layer0=1, n_layers=2)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(d_tl.cpu().numpy(), tl)
    to.same()
    assert np.array_equal(to.d_mass.cpu().numpy(), to.mass, equal_nan=True)


@pytest.mark.parametrize("T,keep", [(40960, 1000), (163840, 9000)])
def test_evict_from_many_blocks(T, keep):
    need_gpu()
    L, B, H, d, tb = 1, 1, 2, 64, 16
    c = Cache(L, B, H, T, d, cg.CACHE8_INT8, tb)
    rng = np.random.default_rng(3)
    c.scales = np.ones_like(c.scales)
    c.mass = rng.integers(0, 300, c.mass.shape).astype(np.float32)   # many ties
    c.up()
    to = Cache(L, B, H, keep * tb, d, cg.CACHE8_INT8, tb)
    tl = np.zeros(B, np.int32)
    d_tl, kept = _cuda(tl), torch.empty((1, B, H, keep), dtype=torch.int32, device="cuda")
    cg.cg_cache8_evict(c.kv, c.c8, cg.cache8_evict_desc(keep, 3, 5), _cuda(np.array([T - 9], np.int32)), c.d_codes, c.d_scales, c.d_bounds, c.d_mass,
                       to.kv, to.d_codes, to.d_scales, to.d_bounds, to.d_mass, d_tl, kept)
    cg.cg_sync_status()
    want = o8.evict(c.codes, c.scales, c.bounds, c.mass, [T - 9], (to.codes, to.scales, to.bounds, to.mass, tl), tb, keep, 3, 5)
    assert np.array_equal(kept.cpu().numpy(), want) and d_tl.item() == tl[0]
    to.same()


# ---- the binding -----------------------------------------------------------------------------------


def test_binding_refuses_before_a_launch(monkeypatch):
    need_gpu()
    c = _filled(1, 1, 1, 64, 64, cg.CACHE8_INT8, 16, [40])
    at = cg.cache8_attn_desc(2, 64, d_head=64)
    ws = torch.empty(cg.cg_cache8_attention_workspace_size(c.kv, c.c8, at), dtype=torch.uint8, device="cuda")
    q, lens = torch.zeros((1, 1, 2, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 3.0, device="cuda")

    def call(q=q, lens=lens, out=out, ws=ws, codes=c.d_codes, scales=c.d_scales, **more):
        return cg.cg_cache8_attention(c.kv, c.c8, at, q, codes, scales, lens, out, ws, **more)

    for error, bad in ((TypeError, dict(q=q.float())), (TypeError, dict(lens=lens.long())), (TypeError, dict(lens=lens.cpu())),
                       (TypeError, dict(codes=[1])), (ValueError, dict(out=out[..., :32])), (ValueError, dict(q=q[:, :, :, :, ::2])),
                       (ValueError, dict(scales=c.d_scales[..., :2].contiguous())), (cg.CgError, dict(ws=ws[:16])),
                       (cg.CgError, dict(sel=torch.zeros(4, dtype=torch.int32, device="cuda"))), (TypeError, dict(mass=c.d_codes)),
                       (cg.CgError, dict(lens=torch.zeros(8, dtype=torch.int32, device="cuda")[1:]))):
        with pytest.raises(error):
            call(**bad)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)   # the tensors lie on another device
    with pytest.raises(ValueError):
        call()
    monkeypatch.undo()
    cg.cg_sync_status()
    assert bool((out == 3.0).all())
    call()
    cg.cg_sync_status()
    assert not bool((out == 3.0).any())


# ---- together ----------------------------------------------------------------------------------------


def _step_buffers(c, q, k, keep, to):
    L, B, H, T, d = c.dims
    m = dict(at=cg.cache8_attn_desc(q.shape[2], T, q_tokens=1, n_layers=L, d_head=d, accumulate=True),
             sp=cg.cache8_attn_desc(q.shape[2], T, q_tokens=1, n_layers=L, d_head=d, n_select=k),
             sd=cg.cache8_select_desc(q.shape[2], T, k, n_layers=L))
    m["w1"] = torch.empty(cg.cg_cache8_attention_workspace_size(c.kv, c.c8, m["at"], True), dtype=torch.uint8, device="cuda")
    m["w2"] = torch.empty(cg.cg_cache8_attention_workspace_size(c.kv, c.c8, m["sp"]), dtype=torch.uint8, device="cuda")
    m["w3"] = torch.empty(cg.cg_cache8_select_workspace_size(c.kv, c.c8, m["sd"]), dtype=torch.uint8, device="cuda")
    m["sel"] = torch.empty((L, B, H, 1, k), dtype=torch.int32, device="cuda")
    m["out"], m["out2"] = (torch.empty(q.shape, dtype=torch.float32, device="cuda") for _ in range(2))
    m["tl"], m["kept"] = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty((L, B, H, keep), dtype=torch.int32, device="cuda")
    return m


def _step(c, to, m, x, q, lens, after, keep, stream=None):
    """One decode step: store, attend to everything with weights, choose, attend to the chosen, cut."""
    L = c.dims[0]
    cg.cg_cache8_append(c.kv, c.c8, 0, x, lens, None, c.d_codes, c.d_scales, c.d_bounds, stream=stream)
    cg.cg_cache8_attention(c.kv, c.c8, m["at"], q, c.d_codes, c.d_scales, after, m["out"], m["w1"], mass=c.d_mass, stream=stream)
    cg.cg_cache8_select(c.kv, c.c8, m["sd"], q, c.d_scales, c.d_bounds, after, m["sel"], m["w3"], stream=stream)
    cg.cg_cache8_attention(c.kv, c.c8, m["sp"], q, c.d_codes, c.d_scales, after, m["out2"], m["w2"], sel=m["sel"], stream=stream)
    cg.cg_cache8_evict(c.kv, c.c8, cg.cache8_evict_desc(keep, n_layers=L), after, c.d_codes, c.d_scales, c.d_bounds, c.d_mass,
                       to.kv, to.d_codes, to.d_scales, to.d_bounds, to.d_mass, m["tl"], m["kept"], stream=stream)


@pytest.mark.parametrize("code", [cg.CACHE8_INT8, cg.CACHE8_E4M3])
def test_decode_steps_with_all_of_it(code):
    """Steps of a program that uses the operators together, each held to the oracle, then decoding goes
    on in the smaller cache."""
    need_gpu()
    L, B, H, T, d, tb, k, keep = 2, 3, 2, 512, 64, 16, 6, 5
    lens = np.array([200, 0, 95])
    c, to = _filled(L, B, H, T, d, code, tb, list(lens), seed=31), Cache(L, B, H, 128, d, code, tb, seed=32)
    gen = torch.Generator().manual_seed(33)
    q0 = _new(gen, L, B, 4, 1, d)
    m = _step_buffers(c, q0, k, keep, to)
    scale = float(np.float32(1.0 / d ** 0.5))
    mass = np.zeros(c.mass.shape)
    for _ in range(3):
        x, q = _new(gen, L, 2, B, H, 1, d), _new(gen, L, B, 4, 1, d, gain=2)
        _step(c, to, m, x.cuda(), q.cuda(), _cuda(lens.astype(np.int32)), _cuda((lens + 1).astype(np.int32)), keep)
        cg.cg_sync_status()
        o8.append(c.codes, c.scales, c.bounds, bf16_np(x), lens, None, code, tb)
        lens = lens + 1
        c.same()
        ref, w, spread, big = o8.attention(bf16_np(q), c.codes, c.scales, lens, code, tb, scale)
        _close(m["out"].cpu().numpy(), ref, spread, big, d)
        mass += w
        assert np.allclose(c.d_mass.cpu().numpy(), mass, rtol=1e-4, atol=1e-6)
        sel = o8.select(bf16_np(q), c.bounds, c.scales, lens, tb, k, 1, 1, H)
        assert np.array_equal(m["sel"].cpu().numpy(), sel)
        ref, _, spread, big = o8.attention(bf16_np(q), c.codes, c.scales, lens, code, tb, scale, sel=sel)
        _close(m["out2"].cpu().numpy(), ref, spread, big, d)
    tl = np.zeros(B, np.int32)
    want = o8.evict(c.codes, c.scales, c.bounds, c.d_mass.cpu().numpy(), lens, (to.codes, to.scales, to.bounds, to.mass, tl), tb, keep, 1, 1,
                    n_layers=L)
    assert np.array_equal(m["kept"].cpu().numpy(), want) and np.array_equal(m["tl"].cpu().numpy(), tl)
    # (blocks behind the kept ones hold what earlier steps left there)
    x, q = _new(gen, L, 2, B, H, 1, d), _new(gen, L, B, 4, 1, d)
    for b in range(B):
        n = tl[b] // tb * tb + tb
        assert np.array_equal(to.d_codes[:, :, b, :, :n].cpu().numpy()[..., :tl[b], :], to.codes[:, :, b, :, :tl[b]])
    to.codes, to.scales, to.bounds = (v.cpu().numpy() for v in (to.d_codes, to.d_scales, to.d_bounds))
    to.append(x, tl)
    to.same()
    _check_attention(to, q, tl + 1)


def test_captured_steps_replay_on_new_lengths_and_share_workspaces():
    """Two captured graphs with the same workspaces, replayed in turn on lengths and inputs that
    change, give the bits of the same calls made eagerly."""
    need_gpu()
    L, B, H, T, d, tb, k, keep = 2, 4, 2, 1024, 128, 32, 4, 6
    lens = np.array([900, 3, 517, 0], np.int32)
    gen = torch.Generator().manual_seed(41)
    q = _new(gen, L, B, 8, 1, d).cuda()
    x = _new(gen, L, 2, B, H, 1, d).cuda()
    pos, after = _cuda(lens), _cuda(lens + 1)
    pair = [(_filled(L, B, H, T, d, cg.CACHE8_E4M3, tb, list(lens), seed=s), Cache(L, B, H, 256, d, cg.CACHE8_E4M3, tb)) for s in (42, 43)]
    eager = [(_filled(L, B, H, T, d, cg.CACHE8_E4M3, tb, list(lens), seed=s), Cache(L, B, H, 256, d, cg.CACHE8_E4M3, tb)) for s in (42, 43)]
    m, me = _step_buffers(pair[0][0], q, k, keep, pair[0][1]), _step_buffers(pair[0][0], q, k, keep, pair[0][1])
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, to in pair:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            _step(c, to, m, x, q, pos, after, keep)
        graphs.append(g)
    for step in range(3):
        x.copy_(_new(gen, L, 2, B, H, 1, d))
        q.copy_(_new(gen, L, B, 8, 1, d))
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            _step(*eager[i], me, x, q, pos, after, keep)
            cg.cg_sync_status()
            for name in ("out", "out2", "sel", "tl", "kept"):
                assert torch.equal(m[name], me[name]), name
            for a, b in zip(pair[i], eager[i]):
                assert torch.equal(a.d_codes, b.d_codes) and torch.equal(a.d_mass, b.d_mass) and torch.equal(a.d_bounds, b.d_bounds)
                assert torch.equal(a.d_scales.view(torch.int32), b.d_scales.view(torch.int32))
        pos += 1
        after += 1
    del graphs


def test_calls_on_other_streams_at_once():
    """Two streams, each with its own cache and workspaces, give what each gives alone."""
    need_gpu()
    L, B, H, T, d, tb, k, keep = 1, 4, 4, 2048, 64, 16, 9, 20
    lens = np.array([2000, 77, 1024, 0], np.int32)
    gen = torch.Generator().manual_seed(51)
    q, x = _new(gen, L, B, 16, 1, d).cuda(), _new(gen, L, 2, B, H, 1, d).cuda()
    pos, after = _cuda(lens), _cuda(lens + 1)

    def sets():
        r = []
        for s in (52, 53):
            c, to = _filled(L, B, H, T, d, cg.CACHE8_INT8, tb, list(lens), seed=s), Cache(L, B, H, 512, d, cg.CACHE8_INT8, tb)
            r.append((c, to, _step_buffers(c, q, k, keep, to)))
        torch.cuda.synchronize()
        return r

    together, alone = sets(), sets()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for st, (c, to, m) in zip(streams, together):
            _step(c, to, m, x, q, pos, after, keep, stream=st)
    torch.cuda.synchronize()
    for c, to, m in alone:
        for _ in range(5):
            _step(c, to, m, x, q, pos, after, keep)
    cg.cg_sync_status()
    for (c, to, m), (c2, to2, m2) in zip(together, alone):
        assert torch.equal(m["out"], m2["out"]) and torch.equal(m["out2"], m2["out2"]) and torch.equal(m["kept"], m2["kept"])
        assert torch.equal(c.d_codes, c2.d_codes) and torch.equal(to.d_codes, to2.d_codes) and torch.equal(c.d_mass, c2.d_mass)
