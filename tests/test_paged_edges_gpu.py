"""Paged cache on the GPU at the edges of what the calls allow: finite values
at the top of the range, infinite scores, hidden positions behind padding,
calls without tokens, calls from several host threads.

Expected values come from the float64 oracle; where a tolerance is needed it
is the one derived in test_paged_gpu.py, whose helpers are used.
"""

import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import paged as P
from test_paged_gpu import BF16, CACHES, E4M3, F32, Cache, _b, _check, _np, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,d", [(1, 32), (3, 32), (1, 256), (2, 256)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_largest_finite_vectors_stay_finite(dtype, Hkv, d):
    """From 248 * 2^120 on, rounding to e4m3 would give 256 * 2^120 = 2^128,
    which no 32-bit float holds; such elements take 240 * 2^120, within 2^-4 of
    them, beside an infinity too."""
    b = _b()
    c = Cache(60, [0], 16, Hkv, d, E4M3, room=16)
    top = torch.finfo(dtype).max
    x = torch.zeros(1, 6, 1, 32, dtype=torch.float64)
    x[0, 0, 0] = torch.linspace(-1, 1, 32, dtype=torch.float64) * top
    x[0, 1, 0, 3] = top
    x[0, 2, 0, 4] = -top
    x[0, 3, 0, :3] = torch.tensor([247.0, 249.0, -255.0], dtype=torch.float64) * 2.0 ** 120
    x[0, 4, 0, :3] = torch.tensor([float("inf"), top, -top], dtype=torch.float64)
    x[0, 5, 0] = 2.0 ** 127
    x = x.to(dtype).repeat(1, 1, Hkv, d // 32).cuda()
    x[0, 5, -1] = 1.0                              # heads of a token differ
    b.pi_attn_cache_write(x, x, *c.args(), **c.exps())
    c.lens += 6
    k, v, _ = b.pi_attn_cache_read(*c.args(), 6, dtype=dtype, **c.exps())
    for y, exps in ((k, c.k_exp), (v, c.v_exp)):
        for t, h in [(t, h) for t in (0, 1, 2, 3, 5) for h in range(Hkv)]:
            x64, y64 = _np(x[0, t, h]), _np(y[0, t, h])
            vals, byte = P.quantise(x64)
            assert exps.view(-1, Hkv)[P.slot(c.table_np, 0, t, 16), h] == byte
            assert np.array_equal(y64, vals * 2.0 ** (byte - 127)), (t, h)
            err, big = np.abs(y64 - x64), np.abs(x64) >= 2.0 ** -13 * np.abs(x64).max()
            assert (err <= 2.0 ** -4 * np.abs(x64))[big].all(), (t, h)
        assert (y[0, 4, :, 0] == float("inf")).all()
        assert (y[0, 4, :, 1] == 240 * 2.0 ** 120).all() and (y[0, 4, :, 2] == -240 * 2.0 ** 120).all()
    assert b.pi_attn_read_status() == b.PI_OK


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,Hq,dtype", [(1, 8, BF16), (1, 1, BF16), (5, 1, BF16), (8, 1, BF16),
                                         (4, 2, BF16), (40, 8, BF16), (150, 8, BF16), (9, 3, BF16),
                                         (6, 2, F32)])
@pytest.mark.parametrize("room", [0, 17000])
def test_a_score_of_minus_infinity_has_no_weight(Sq, Hq, dtype, cache, room):
    """Visible new keys whose scores are -inf, the first one among them, leave
    the other keys' probabilities alone."""
    if dtype == F32 and cache == BF16:
        cache = F32
    b = _b()
    c = Cache(61, [40, 0, 300], 16, 1, 256, cache, room=room)
    rng = c.rng
    q = _rand(rng, (3, Sq, Hq, 256), dtype, 0.25)
    kn, vn = (_rand(rng, (3, Sq, 1, 256), dtype, 0.25) for _ in range(2))
    q[..., 7] = 1.0
    kn[0, ::2, 0, 7] = float("-inf")
    kn[2, ::3, 0, 7] = float("-inf")
    if Sq > 2:                                     # (the query that sees itself alone is left)
        kn[1, 2::3, 0, 7] = float("-inf")
    ar = np.ones(Sq, np.uint8)
    lse = torch.empty(q.shape[:3], device="cuda")
    out = b.pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(ar).cuda(), lse=lse, **c.exps())
    _check(c, q, kn, vn, ar, None, out, lse, 1.0, 0, 0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,Hq,pads", [(3, 2, (1, 2, 0)), (7, 1, (3, 5, 6)), (8, 1, (7, 1, 2)),
                                        (40, 8, (3, 39, 20)), (150, 8, (64, 30, 149)),
                                        (300, 8, (33, 36, 250)), (700, 8, (1, 513, 200))])
@pytest.mark.parametrize("window,sinks", [(37, 0), (37, 4), (200, 130)])
@pytest.mark.parametrize("room", [0, 17000])
def test_positions_hidden_from_all_but_padding_hold_nan(Sq, Hq, pads, window, sinks, cache, room):
    """Padding in front: its tokens see nothing, so a cached position that lies in
    the windows of padding alone is hidden, whatever it holds."""
    b = _b()
    lens = [200, 90, 333]
    c = Cache(62, lens, 16, 1, 256, cache, room=room)
    rng = c.rng
    q = _rand(rng, (3, Sq, Hq, 256), BF16, 0.25)
    kn, vn = (_rand(rng, (3, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    seg = np.zeros((3, Sq), np.int32)
    live = np.zeros((c.k.shape[0], c.k.shape[1]), bool)
    for i, (n, pad) in enumerate(zip(lens, pads)):
        seg[i, :pad] = -1
        first = min(max(0, n + pad - window + 1), n)         # the first real query sees the most
        for x in list(range(min(sinks, n))) + list(range(first, n)):
            live.reshape(-1)[P.slot(c.table_np, i, x, 16)] = True
    dead = torch.from_numpy(~live).cuda()
    for pool, exps in ((c.k, c.k_exp), (c.v, c.v_exp)):
        if cache == E4M3:
            exps[dead] = 255
        else:
            pool[dead] = float("nan")
    ar = np.ones((3, Sq), np.uint8)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    b.pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(ar).cuda(),
                    segment_ids=torch.from_numpy(seg).cuda(), out=out, lse=lse, window=window,
                    sinks=sinks, **c.exps())
    _check(c, q, kn, vn, ar, seg, out, lse, 1.0, window, sinks)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
def test_lengths_after_a_call_without_tokens(cache):
    """Clamped and reported as in a call with tokens."""
    b = _b()
    c = Cache(63, [10, 20, 30], 16, 1, 64, cache)                # room for 32
    empty = torch.empty(3, 0, 1, 64, dtype=F32 if cache == F32 else BF16, device="cuda")
    before = [c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()]
    got = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    b.pi_attn_cache_write(empty, empty, *c.args(), lens_out=got, **c.exps())
    assert got.tolist() == [10, 20, 30] and b.pi_attn_read_status() == b.PI_OK
    for bad, want in ((-7, 0), (33, 32), (2 ** 31 - 1, 32), (-2 ** 31, 0)):
        lens = c.lens.clone()
        lens[1] = bad
        b.pi_attn_cache_write(empty, empty, c.k, c.v, c.table, lens, lens_out=got, **c.exps())
        assert got.tolist() == [10, want, 30]
        assert b.pi_attn_read_status() == b.PI_ERR_ARG
    assert torch.equal(c.k.view(torch.uint8), before[0])
    assert torch.equal(c.v.view(torch.uint8), before[1])


def test_long_chunks_from_several_threads():
    """Calls of two lengths from four host threads: none is refused because
    another thread prepares a shorter one.  (Padding throughout: only the
    launches matter.)"""
    b = _b()
    L = b.lib()
    c = Cache(64, [5], 16, 1, 32, F32)
    jobs = []
    for Sq in (16383, 8300):
        q = torch.zeros(1, Sq, 1, 32, device="cuda")
        out = torch.full_like(q, 3.0)
        ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
        seg = torch.full((Sq,), -1, dtype=torch.int32, device="cuda")
        d = b.PiPagedDesc(1, Sq, 1, 1, 32, b.PI_F32, b.PI_F32, 16, c.k.shape[0], c.table.shape[1],
                          0, 0, 1.0, 0, 0)
        assert L.pi_attn_paged_workspace_bytes(ctypes.byref(d)) == 0
        p = [t.data_ptr() for t in (q, q, q, ar, seg, c.k, c.v)]
        args = (ctypes.byref(d), *p, None, None, c.table.data_ptr(), c.lens.data_ptr(),
                out.data_ptr(), None, None, 0, None)
        jobs.append(((q, ar, seg, out), args))
    bad = []

    def run(i):
        args = jobs[i % 2][-1]
        for _ in range(600):
            rc = L.pi_attn_paged(*args)
            if rc != b.PI_OK:
                bad.append((i % 2, rc))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), bad[:3])
    for tensors, _ in jobs:
        assert (tensors[-1] == 0).all()
    assert b.pi_attn_read_status() == b.PI_OK


def _at(t, shift):
    """t's values at an address `shift` bytes past a multiple of 256."""
    raw = torch.full((t.numel() * t.element_size() + 512,), 0x7F, dtype=torch.uint8, device="cuda")
    raw = raw[shift:shift + t.numel() * t.element_size()]
    assert raw.data_ptr() % 256 == shift
    raw.copy_(t.contiguous().view(torch.uint8).view(-1))
    return raw.view(t.dtype).view(t.shape)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,Hq", [(1, 8), (6, 1), (51, 8), (130, 8), (520, 8), (9, 3)])
def test_the_least_alignment_that_is_asked_for(Sq, Hq, cache):
    """Tensors, pools and workspace at 16 bytes, int32 and fp32 arrays at 4, masks
    and exponents at odd addresses: the same bits as with aligned ones."""
    b = _b()
    c = Cache(65, [333, 0, 1200], 32, 1, 256, cache, room=Sq)
    q = _rand(c.rng, (3, Sq, Hq, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (3, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.from_numpy((c.rng.random((3, Sq)) < 0.3).astype(np.uint8)).cuda()
    seg = torch.from_numpy(c.rng.integers(-1, 3, (3, Sq)).astype(np.int32)).cuda()
    mask = torch.from_numpy((c.rng.random((3, Sq)) < 0.7).astype(np.uint8)).cuda()

    def step(move):
        q_, kn_, vn_, k, v = (move(t, 16 * (i + 1)) for i, t in enumerate((q, kn, vn, c.k, c.v)))
        table, lens, sg = (move(t, 4 * (i + 1)) for i, t in enumerate((c.table, c.lens, seg)))
        ar_, mask_ = move(ar, 1), move(mask, 7)
        exps = {n: move(e, 3) for n, e in c.exps().items() if e is not None}
        out, lse = move(torch.zeros_like(q), 48), move(torch.zeros(q.shape[:3], device="cuda"), 12)
        after = move(torch.zeros_like(c.lens), 4)
        need = b.pi_attn_paged_workspace_bytes(q_, kn_, k, v, table, lens, **exps)
        ws = move(torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda"), 16)
        b.pi_attn_paged(q_, kn_, vn_, k, v, table, lens, ar_, segment_ids=sg, out=out, lse=lse,
                        workspace=ws, **exps)
        b.pi_attn_cache_write(kn_, vn_, k, v, table, lens, token_mask=mask_, lens_out=after, **exps)
        n = int(after.max())
        ko, vo = (move(torch.zeros(3, n, 1, 256, dtype=BF16, device="cuda"), 80) for _ in range(2))
        valid = move(torch.zeros(3, n, dtype=torch.uint8, device="cuda"), 5)
        b.pi_attn_cache_read(k, v, table, after, n, k_out=ko, v_out=vo, valid_out=valid, **exps)
        assert b.pi_attn_read_status() == b.PI_OK
        return [t.contiguous().view(torch.uint8) for t in (out, lse, after, k, v, ko, vo, valid,
                                                           *exps.values())]

    for x, y in zip(step(_at), step(lambda t, shift: t.clone())):
        assert torch.equal(x, y)


@pytest.mark.parametrize("cache", CACHES)
def test_streams_as_objects_and_handles(cache):
    """stream= takes a torch stream or its handle; results of all calls agree."""
    b = _b()
    c = Cache(66, [300, 40], 16, 1, 256, cache, room=60)
    for Sq in (1, 40):
        q = _rand(c.rng, (2, Sq, 8, 256), BF16, 0.25)
        kn, vn = (_rand(c.rng, (2, Sq, 1, 256), BF16, 0.25) for _ in range(2))
        ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
        ref = b.pi_attn_paged(q, kn, vn, *c.args(), ar, **c.exps())
        rows = b.pi_attn_cache_read(*c.args(), 50, **c.exps())
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for stream in (side, side.cuda_stream, torch.cuda.current_stream(), 0):
            out = b.pi_attn_paged(q, kn, vn, *c.args(), ar, stream=stream, **c.exps())
            got = b.pi_attn_cache_read(*c.args(), 50, stream=stream, **c.exps())
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
            assert all(torch.equal(x, y) for x, y in zip(got, rows))
    assert b.pi_attn_read_status() == b.PI_OK


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,Hq,d,dtype", [(1, 8, 256, BF16), (4, 2, 256, BF16), (40, 8, 256, BF16),
                                           (150, 8, 256, BF16), (9, 3, 256, BF16), (9, 4, 64, BF16),
                                           (9, 4, 64, F32)])
@pytest.mark.parametrize("room", [0, 17000])
def test_a_nan_query_stays_in_its_row(Sq, Hq, d, dtype, cache, room):
    """NaN and infinite queries turn their own row and lse to NaN, and no bit of
    another row changes."""
    if dtype == F32 and cache == BF16:
        cache = F32
    b = _b()
    c = Cache(67, [900, 7, 2100], 64, 1, d, cache, room=room)
    q = _rand(c.rng, (3, Sq, Hq, d), dtype, 0.25)
    kn, vn = (_rand(c.rng, (3, Sq, 1, d), dtype, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")

    def call(q):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        b.pi_attn_paged(q, kn, vn, *c.args(), ar, out=out, lse=lse, **c.exps())
        assert b.pi_attn_read_status() == b.PI_OK
        return out, lse

    ref, ref_lse = call(q)
    bad = q.clone()
    hit = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    for i, x in ((0, "nan"), (2, "inf")):
        t, h = Sq // 2, i % Hq
        bad[i, t, h, 5] = float(x)
        hit[i, t, h] = True
    out, lse = call(bad)
    assert torch.equal(out[~hit], ref[~hit]) and torch.equal(lse[~hit], ref_lse[~hit])
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
