"""Paged cache, without a GPU: the oracle's definitions are pinned, and the
three calls reject bad arguments on the host before anything is enqueued
(every pointer below is fake and never dereferenced).
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import paged as P


def _lib():
    from vla_prefix_lm_b200 import binding, build
    build.build()
    return binding, binding.lib()


# ------------------------------------------------------------------- oracle

def test_e4m3_grid_is_torchs():
    bits = torch.arange(0x7F, dtype=torch.uint8)
    assert np.array_equal(P.e4m3_grid(), bits.view(torch.float8_e4m3fn).double().numpy())


def test_e4m3_rounding_is_torchs():
    g = P.e4m3_grid()
    mid = (g[1:] + g[:-1]) / 2                     # ties
    x = np.concatenate([g, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.linspace(0, 448, 4001)])
    x = np.concatenate([x, -x]).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.to_e4m3(x), ref)


@pytest.mark.parametrize("top", [448.0, 448.0001, 447.9, 1.0, 1.75, 1.7500001, 1e-30, 1e-38, 3e38])
def test_exponent_is_the_smallest(top):
    top = float(np.float32(top))
    e = P.exponent(np.array([0.0, -top]))
    assert top <= 448 * 2.0 ** e
    assert e == -126 or top > 448 * 2.0 ** (e - 1)


def test_mask_is_the_pairwise_rule():
    rng = np.random.default_rng(3)
    for _ in range(60):
        n, Sq = int(rng.integers(0, 12)), int(rng.integers(1, 9))
        ar = rng.integers(0, 2, Sq)
        seg = rng.integers(-1, 3, Sq)
        w, s = int(rng.integers(0, 8)), int(rng.integers(0, 4))
        codes = list(zip(np.cumsum(ar).tolist(), seg.tolist()))
        brute = [[P.visible(n, i, x, codes, w, s) for x in range(n + Sq)] for i in range(Sq)]
        assert np.array_equal(P.mask(n, Sq, codes, w, s), np.array(brute))


def test_attend_is_the_dense_suffix_pass():
    rng = np.random.default_rng(4)
    B, Pn, Sq, Hq, Hkv, d = 2, 7, 5, 4, 2, 8
    q, k, v = (rng.standard_normal((B, Sq, h, d)) for h in (Hq, Hkv, Hkv))
    kc, vc = (rng.standard_normal((B, Pn, Hkv, d)) for _ in range(2))
    ar, seg = np.array([1, 0, 1, 1, 0]), np.array([1, 0, 2, -1, 2])
    ref, _ = oracle.suffix(q, k, v, kc, vc, ar, seg_suf=seg)
    got, lse = P.attend(q, k, v, list(kc), list(vc), ar, seg)
    assert np.abs(got - ref).max() < 1e-12
    assert np.isneginf(lse[:, 3]).all() and np.isfinite(lse[:, :3]).all()


# ----------------------------------------------------------------- refusals

FAKE = ctypes.c_void_p(0x10000)
FAKE2 = ctypes.c_void_p(0x20000)
MIS = ctypes.c_void_p(0x10008)
MIS4 = ctypes.c_void_p(0x10002)


def _desc(b, **kw):
    d = dict(B=2, Sq=16, Hq=8, Hkv=1, d=256, dtype=b.PI_BF16, cache_dtype=b.PI_BF16, page_size=16,
             num_pages=10, max_pages=5, window=0, sinks=0, softmax_scale=1.0, reserved=0,
             mask_batch_stride=0)
    d.update(kw)
    return b.PiPagedDesc(**d)


def _write(L, desc, **kw):
    a = dict(k=FAKE, v=FAKE, mask=None, table=FAKE, lens=FAKE, kp=FAKE, vp=FAKE, ke=None, ve=None,
             lens_out=FAKE2)
    a.update(kw)
    return L.pi_attn_cache_write(None if desc is None else ctypes.byref(desc), a["k"], a["v"],
                                 a["mask"], a["table"], a["lens"], a["kp"], a["vp"], a["ke"],
                                 a["ve"], a["lens_out"], None)


def _read(L, desc, **kw):
    a = dict(kp=FAKE, vp=FAKE, ke=None, ve=None, table=FAKE, lens=FAKE, k=FAKE, v=FAKE, valid=None)
    a.update(kw)
    return L.pi_attn_cache_read(None if desc is None else ctypes.byref(desc), a["kp"], a["vp"],
                                a["ke"], a["ve"], a["table"], a["lens"], a["k"], a["v"],
                                a["valid"], None)


def _attend(L, desc, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ar=FAKE, seg=None, kp=FAKE, vp=FAKE, ke=None, ve=None,
             table=FAKE, lens=FAKE, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return L.pi_attn_paged(None if desc is None else ctypes.byref(desc), a["q"], a["k"], a["v"],
                           a["ar"], a["seg"], a["kp"], a["vp"], a["ke"], a["ve"], a["table"],
                           a["lens"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [_write, _read, _attend])
def test_bad_descriptors(call):
    b, L = _lib()
    assert call(L, None) == b.PI_ERR_ARG
    for kw in (dict(B=-1), dict(Sq=-1), dict(Hkv=0), dict(d=0), dict(num_pages=-1),
               dict(max_pages=-1), dict(page_size=0), dict(reserved=1)):
        assert call(L, _desc(b, **kw)) == b.PI_ERR_ARG, kw
    for kw in (dict(d=48), dict(d=512), dict(page_size=8), dict(page_size=24), dict(page_size=512),
               dict(dtype=b.PI_E4M3, cache_dtype=b.PI_E4M3), dict(cache_dtype=b.PI_F32),
               dict(dtype=b.PI_F32), dict(B=65536),
               dict(page_size=256, num_pages=1 << 23), dict(page_size=256, max_pages=1 << 23)):
        assert call(L, _desc(b, **kw)) == b.PI_ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("call", [_write, _read, _attend])
def test_bad_cache_pointers(call):
    b, L = _lib()
    for kw in (dict(lens=None), dict(table=None), dict(kp=None), dict(vp=None), dict(k=None),
               dict(v=None), dict(ke=FAKE), dict(ve=FAKE)):
        assert call(L, _desc(b), **kw) == b.PI_ERR_ARG, kw
    e4 = _desc(b, cache_dtype=b.PI_E4M3)
    assert call(L, e4) == b.PI_ERR_ARG                        # exponents missing
    assert call(L, e4, ke=FAKE) == b.PI_ERR_ARG
    for kw in (dict(kp=MIS), dict(vp=MIS), dict(k=MIS), dict(v=MIS), dict(lens=MIS4),
               dict(table=MIS4)):
        assert call(L, _desc(b), **kw) == b.PI_ERR_ALIGN, kw


def test_write_and_attention_refusals():
    b, L = _lib()
    assert _write(L, _desc(b), lens_out=FAKE) == b.PI_ERR_ARG      # lens_out is cache_lens
    near = ctypes.c_void_p(FAKE.value + 4)                         # or overlaps it
    assert _write(L, _desc(b, B=2), lens_out=near) == b.PI_ERR_ARG
    assert _write(L, _desc(b), lens_out=ctypes.c_void_p(0x20002)) == b.PI_ERR_ALIGN
    for call in (_write, _attend):
        assert call(L, _desc(b, mask_batch_stride=15)) == b.PI_ERR_ARG
        assert call(L, _desc(b, mask_batch_stride=-16)) == b.PI_ERR_ARG
        assert call(L, _desc(b, Sq=16384)) == b.PI_ERR_UNSUPPORTED
    for kw in (dict(Hq=0), dict(Hq=6, Hkv=4), dict(window=-1), dict(sinks=-1),
               dict(softmax_scale=0.0), dict(softmax_scale=float("inf")),
               dict(softmax_scale=float("nan"))):
        assert _attend(L, _desc(b, **kw)) == b.PI_ERR_ARG, kw
    for kw in (dict(q=None), dict(ar=None), dict(out=None)):
        assert _attend(L, _desc(b), **kw) == b.PI_ERR_ARG, kw
    for kw in (dict(q=MIS), dict(out=MIS), dict(lse=MIS4), dict(seg=MIS4)):
        assert _attend(L, _desc(b), **kw) == b.PI_ERR_ALIGN, kw


def test_workspace_is_checked():
    b, L = _lib()
    for kw in (dict(), dict(Sq=1), dict(Sq=300), dict(cache_dtype=b.PI_E4M3),
               dict(dtype=b.PI_F32, cache_dtype=b.PI_F32), dict(d=64)):
        d = _desc(b, **kw)
        exps = dict(ke=FAKE, ve=FAKE) if kw.get("cache_dtype") == b.PI_E4M3 else {}
        n = L.pi_attn_paged_workspace_bytes(ctypes.byref(d))
        assert n == 0 or n >= 16
        if n > 0:
            assert _attend(L, d, ws=None, **exps) == b.PI_ERR_ARG
            assert _attend(L, d, ws_bytes=n - 1, **exps) == b.PI_ERR_ARG
            assert _attend(L, d, ws=MIS, **exps) == b.PI_ERR_ALIGN
    assert L.pi_attn_paged_workspace_bytes(None) == 0
    assert L.pi_attn_paged_workspace_bytes(ctypes.byref(_desc(b, Hq=0))) == 0


def test_empty_calls_are_noops():
    b, L = _lib()
    none = dict(kp=None, vp=None, table=None, lens=None, k=None, v=None)
    assert _write(L, _desc(b, B=0), lens_out=None, **none) == b.PI_OK
    assert _read(L, _desc(b, Sq=0), **none) == b.PI_OK
    assert _attend(L, _desc(b, Sq=0), q=None, ar=None, out=None, **none) == b.PI_OK
    assert _write(L, _desc(b, Sq=0), lens_out=None, k=None, v=None) == b.PI_OK


def test_binding_rejects_host_tensors_and_mismatches():
    b, _ = _lib()
    k = torch.zeros(1, 1, 1, 256, dtype=torch.bfloat16)
    pages = torch.zeros(2, 16, 1, 256, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ar = torch.ones(1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        b.pi_attn_cache_write(k, k, pages, pages, table, lens)
    with pytest.raises(ValueError):
        b.pi_attn_cache_read(pages, pages, table, lens, 4)
    with pytest.raises(ValueError):
        b.pi_attn_paged(k, k, k, pages, pages, table, lens, ar)
