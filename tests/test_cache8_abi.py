"""Refusals of the 8-bit block-scaled cache's entry points, before any CUDA call (fake pointers that
are never dereferenced; no GPU needed)."""
import ctypes

import pytest
import torch

from quantization_cg_encode_b200 import cg

KV = cg.kv_desc(2, 3, 2, 512, 128)
C8 = cg.cache8_desc(cg.CACHE8_INT8, 16)


def _p(i):
    return None if i is None else ctypes.c_void_p(i)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def test_sizes_closed_form():
    cb, sc, bb, mc = cg.cg_cache8_sizes_for(KV, C8)
    assert cb == 2 * 2 * 3 * 2 * 512 * 128 and sc == 2 * 2 * 3 * 2 * 32
    assert bb == 2 * 3 * 2 * 32 * 2 * 128 and mc == 2 * 3 * 2 * 32
    codes, scales, bounds, mass = cg.alloc_cache8(KV, cg.cache8_desc(cg.CACHE8_E4M3, 64), device="cpu")
    got = cg.cg_cache8_sizes_for(KV, cg.cache8_desc(cg.CACHE8_E4M3, 64))
    assert (codes.numel(), scales.numel(), bounds.numel(), mass.numel()) == got


@pytest.mark.parametrize("kv,c8,want", [
    (KV, cg.cache8_desc(2, 16), cg.CG_ERR_INVALID), (KV, cg.cache8_desc(-1, 16), cg.CG_ERR_INVALID),
    (KV, cg.cache8_desc(0, 8), cg.CG_ERR_UNSUPPORTED), (KV, cg.cache8_desc(0, 128), cg.CG_ERR_UNSUPPORTED),
    (KV, cg.cache8_desc(0, 0), cg.CG_ERR_UNSUPPORTED), (KV, None, cg.CG_ERR_INVALID), (None, C8, cg.CG_ERR_INVALID),
    (cg.kv_desc(2, 3, 2, 96, 128), cg.cache8_desc(0, 64), cg.CG_ERR_INVALID),    # T is no multiple of the block
    (cg.kv_desc(2, 3, 2, 512, 96), C8, cg.CG_ERR_UNSUPPORTED), (cg.kv_desc(2, 0, 2, 512, 64), C8, cg.CG_ERR_INVALID)])
def test_descriptors(kv, c8, want):
    out = cg.Cache8Sizes()
    assert cg.lib().cg_cache8_sizes_for(_ref(kv), _ref(c8), ctypes.byref(out)) == want


def _append(kv=KV, c8=C8, layer0=0, nl=1, n=4, new=0x1000, pos=0x2000, counts=None, codes=0x3000, scales=0x4000, bounds=None):
    return cg.lib().cg_cache8_append(_ref(kv), _ref(c8), layer0, nl, n, _p(new), _p(pos), _p(counts), _p(codes), _p(scales),
                                     _p(bounds), None)


@pytest.mark.parametrize("bad", [dict(new=0), dict(pos=0), dict(codes=0), dict(scales=0), dict(new=0x1008), dict(pos=0x2004),
                                 dict(counts=0x5004), dict(codes=0x3001), dict(scales=0x4004), dict(bounds=0x6008),
                                 dict(n=-1), dict(n=513), dict(layer0=-1), dict(layer0=2), dict(nl=0), dict(layer0=1, nl=2)])
def test_append_refuses(bad):
    assert _append(**bad) == cg.CG_ERR_INVALID


def test_append_of_nothing_does_nothing():
    assert _append(n=0, new=0) == cg.CG_OK


def _attn(at, kv=KV, c8=C8, q=0x1000, codes=0x2000, scales=0x3000, lens=0x4000, sel=None, out=0x5000, mass=None, ws=0x6000,
          bytes_=1 << 40):
    return cg.lib().cg_cache8_attention(_ref(kv), _ref(c8), _ref(at), _p(q), _p(codes), _p(scales), _p(lens), _p(sel), _p(out),
                                        _p(mass), _p(ws), bytes_, None)


AT = dict(q_heads=8, max_tokens=512)


@pytest.mark.parametrize("over,want", [
    (dict(q_heads=0), cg.CG_ERR_INVALID), (dict(q_heads=7), cg.CG_ERR_INVALID), (dict(q_heads=34), cg.CG_ERR_UNSUPPORTED),
    (dict(q_tokens=0), cg.CG_ERR_INVALID), (dict(q_tokens=17), cg.CG_ERR_UNSUPPORTED),
    (dict(max_tokens=0), cg.CG_ERR_INVALID), (dict(max_tokens=513), cg.CG_ERR_INVALID),
    (dict(layer0=-1), cg.CG_ERR_INVALID), (dict(layer0=1, n_layers=2), cg.CG_ERR_INVALID), (dict(n_layers=0), cg.CG_ERR_INVALID),
    (dict(scale=0.0), cg.CG_ERR_INVALID), (dict(scale=-1.0), cg.CG_ERR_INVALID), (dict(scale=float("nan")), cg.CG_ERR_INVALID),
    (dict(scale=float("inf")), cg.CG_ERR_INVALID), (dict(n_select=-1), cg.CG_ERR_INVALID), (dict(n_select=33), cg.CG_ERR_INVALID)])
def test_attention_descriptor_refusals(over, want):
    at = cg.cache8_attn_desc(**{**AT, **over})
    assert _attn(at, sel=0x7000 if over.get("n_select") else None) == want
    out = ctypes.c_uint64(77)
    assert cg.lib().cg_cache8_attention_workspace_size(_ref(KV), _ref(C8), _ref(at), 0, ctypes.byref(out)) == want
    assert out.value == 77


@pytest.mark.parametrize("bad", [dict(q=0), dict(codes=0), dict(scales=0), dict(lens=0), dict(out=0), dict(ws=0), dict(q=0x1002),
                                 dict(codes=0x2008), dict(scales=0x3004), dict(lens=0x4004), dict(out=0x5008), dict(ws=0x6004),
                                 dict(mass=0x7004), dict(sel=0x7000)])
def test_attention_pointer_refusals(bad):
    assert _attn(cg.cache8_attn_desc(**AT), **bad) == cg.CG_ERR_INVALID


def test_attention_workspace_and_combinations():
    at = cg.cache8_attn_desc(**AT)
    for mass in (False, True):
        need = cg.cg_cache8_attention_workspace_size(KV, C8, at, mass)
        assert _attn(at, mass=0x7000 if mass else None, bytes_=need - 1) == cg.CG_ERR_INVALID
    assert cg.cg_cache8_attention_workspace_size(KV, C8, at, True) > cg.cg_cache8_attention_workspace_size(KV, C8, at, False)
    sparse = cg.cache8_attn_desc(n_select=4, **AT)
    assert _attn(sparse) == cg.CG_ERR_INVALID                                 # a list is wanted
    assert _attn(sparse, sel=0x8004) == cg.CG_ERR_INVALID
    assert _attn(sparse, sel=0x8000, mass=0x7000) == cg.CG_ERR_UNSUPPORTED    # no mass over listed blocks
    bad = cg.cache8_attn_desc(**AT)
    bad.accumulate = 2
    assert _attn(bad) == cg.CG_ERR_INVALID
    assert _attn(None) == cg.CG_ERR_INVALID
    # more than 2^31 - 1 query rows
    huge, out = cg.kv_desc(20000, 4096, 128, 32768, 128), ctypes.c_uint64()
    assert cg.lib().cg_cache8_attention_workspace_size(_ref(huge), _ref(C8), _ref(cg.cache8_attn_desc(128, 32768, n_layers=20000)), 0,
                                                       ctypes.byref(out)) == cg.CG_ERR_TOO_LARGE


def _select(sd, kv=KV, q=0x1000, scales=0x2000, bounds=0x3000, lens=0x4000, sel=0x5000, ws=0x6000, bytes_=1 << 40):
    return cg.lib().cg_cache8_select(_ref(kv), _ref(C8), _ref(sd), _p(q), _p(scales), _p(bounds), _p(lens), _p(sel), _p(ws),
                                     bytes_, None)


@pytest.mark.parametrize("over", [dict(n_select=0), dict(n_select=33), dict(n_select=4, sink_blocks=3, recent_blocks=2),
                                  dict(sink_blocks=-1), dict(recent_blocks=-1), dict(q_heads=3), dict(max_tokens=513),
                                  dict(layer0=2), dict(sink_blocks=2 ** 31 - 1, recent_blocks=2 ** 31 - 1)])
def test_select_refuses(over):
    sd = cg.cache8_select_desc(**{**dict(q_heads=8, max_tokens=512, n_select=8), **over})
    assert _select(sd) == cg.CG_ERR_INVALID


def test_select_pointers_and_workspace():
    sd = cg.cache8_select_desc(8, 500, 8, q_tokens=3)
    need = cg.cg_cache8_select_workspace_size(KV, C8, sd)
    long_kv = cg.kv_desc(1, 3, 2, 1 << 18, 64)                                # scores beyond a CTA's memory
    assert cg.cg_cache8_select_workspace_size(long_kv, C8, cg.cache8_select_desc(8, 1 << 18, 8, q_tokens=3)) == 4 * 3 * 2 * 3 * (1 << 14)
    assert _select(sd, bytes_=need - 1) == cg.CG_ERR_INVALID
    for bad in (dict(q=0), dict(scales=0), dict(bounds=0), dict(lens=0), dict(sel=0), dict(ws=0), dict(bounds=0x3004), dict(sel=0x5004)):
        assert _select(sd, **bad) == cg.CG_ERR_INVALID
    assert _select(None) == cg.CG_ERR_INVALID


TO = cg.kv_desc(2, 3, 2, 256, 128)


def _evict(ev, kv=KV, to=TO, lens=0x1000, codes=0x10000000, scales=0x20000000, bounds=0x30000000, mass=0x40000000, tc=0x50000000,
           ts=0x60000000, tb=0x70000000, tm=0x80000000, tl=0x90000000, kept=0xA0000000):
    return cg.lib().cg_cache8_evict(_ref(kv), _ref(C8), _ref(ev), _p(lens), _p(codes), _p(scales), _p(bounds), _p(mass), _ref(to),
                                    _p(tc), _p(ts), _p(tb), _p(tm), _p(tl), _p(kept), None)


@pytest.mark.parametrize("ev", [dict(keep_blocks=0), dict(keep_blocks=17), dict(keep_blocks=4, recent_blocks=0),
                                dict(keep_blocks=4, sink_blocks=-1), dict(keep_blocks=4, sink_blocks=2, recent_blocks=3),
                                dict(keep_blocks=4, layer0=2), dict(keep_blocks=4, n_layers=0)])
def test_evict_refuses(ev):
    assert _evict(cg.cache8_evict_desc(**ev)) == cg.CG_ERR_INVALID


def test_evict_refuses_caches_that_do_not_go_together():
    ev = cg.cache8_evict_desc(4)
    for to in (cg.kv_desc(1, 3, 2, 256, 128), cg.kv_desc(2, 2, 2, 256, 128), cg.kv_desc(2, 3, 4, 256, 128), cg.kv_desc(2, 3, 2, 256, 64),
               None):
        assert _evict(ev, to=to) == cg.CG_ERR_INVALID
    cb = cg.cg_cache8_sizes_for(KV, C8)[0]
    for bad in (dict(tc=0x10000000), dict(tc=0x10000000 + cb - 16), dict(ts=0x20000000 + 16), dict(tb=0x30000000), dict(tm=0x40000000),
                dict(tl=0x1000), dict(bounds=None), dict(tb=None), dict(kept=0), dict(tl=0), dict(codes=0), dict(mass=0x40000004)):
        assert _evict(ev, **bad) == cg.CG_ERR_INVALID
    assert _evict(None) == cg.CG_ERR_INVALID


def test_binding_checks_tensors():
    kv = cg.kv_desc(1, 1, 1, 32, 64)
    c = cg.alloc_cache8(kv, C8, device="cpu")
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):                                            # host tensors
        cg.cg_cache8_append(kv, C8, 0, torch.zeros(1, 2, 1, 1, 1, 64, dtype=torch.bfloat16), lens, None, c[0], c[1], c[2])
    with pytest.raises(ValueError):                                           # another shape
        cg.cg_cache8_append(kv, C8, 0, torch.zeros(1, 2, 1, 2, 1, 64, dtype=torch.bfloat16), lens, None, c[0], c[1], c[2])
    with pytest.raises(cg.CgError):
        cg.cg_cache8_sizes_for(kv, cg.cache8_desc(0, 48))
