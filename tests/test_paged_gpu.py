"""Paged cache on the GPU against the float64 oracle.

Tolerances, from the arithmetic.  The cache's contents are inputs (an e4m3
vector stands for exact values), so the errors are those of the attention:

* scores: fp32 sums of d = 256 products, at most 2^-16 of sum |q_i k_i| <=
  |q| |k|, and as much again for the scale and the exponent;
  delta = 2^-15 * max |q| |k| * scale.  A probability is off by a factor
  1 +- 2 delta.
* bf16: each probability and the result are rounded once, by at most 2^-8;
  weights sum to 1, so out is off by at most (2 * 2^-8 + 2 delta) * max |v|.
* fp32: (2 delta + n * 2^-22) * max |v| for sums over n keys.
* lse: delta, plus n * 2^-22 for its sum and logarithm.
A margin of 2^-14 covers exp2 (2^-22) and the running rescale products.

What is copied or quantised has to be equal bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _b():
    from vla_prefix_lm_b200 import binding
    return binding


def _np(t):
    return t.double().cpu().numpy()


def _table(rng, lens, room, page, spare=3):
    """Scattered pages: [B, max_pages] covering len + room tokens, and the pool size."""
    per = max(1, -(-(max(lens, default=0) + room) // page))
    n = len(lens) * per + spare
    t = rng.permutation(n)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
    return t, n


class Cache:
    """A pool with random vectors in every slot, lengths and a table."""

    def __init__(self, seed, lens, page, Hkv, d, dtype, room=0, std=None):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.d = rng, page, d
        self.table_np, n = _table(rng, lens, room, page)
        shape = (n, page, Hkv, d)
        std = d ** -0.25 if std is None else std
        self.k_exp = self.v_exp = None
        pools = []
        for name in ("k", "v"):
            x = torch.from_numpy(rng.standard_normal(shape) * std).float()
            if dtype == E4M3:
                exps = torch.from_numpy(rng.integers(118, 123, shape[:3])).to(torch.uint8)
                x = (x * 100).clamp(-448, 448).to(E4M3)
                setattr(self, name + "_exp", exps.cuda())
                pools.append(x.cuda())
            else:
                pools.append(x.to(dtype).cuda())
        self.k, self.v = pools
        self.table = torch.from_numpy(self.table_np).cuda()
        self.lens_np = np.array(lens, np.int32)
        self.lens = torch.from_numpy(self.lens_np).cuda()

    def exps(self):
        return dict(k_exp=self.k_exp, v_exp=self.v_exp)

    def args(self):
        return self.k, self.v, self.table, self.lens

    def rows(self, name, b, n=None):
        n = int(self.lens_np[b]) if n is None else n
        pages = self.table_np[b, :-(-n // self.page)]           # only these leave the device
        at = torch.from_numpy(pages.astype(np.int64)).cuda()
        pool, e = getattr(self, name), getattr(self, name + "_exp")
        pool = pool.view(torch.uint8)[at].view(pool.dtype)
        return P.rows(_np(pool), None if e is None else e[at].cpu().numpy(),
                      np.arange(len(pages))[None], 0, n)


def _rand(rng, shape, dtype, std):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(dtype).cuda()


def _check(c, q, kn, vn, ar, seg, out, lse, scale, window, sinks):
    B = q.shape[0]
    keys, vals = [c.rows("k", b) for b in range(B)], [c.rows("v", b) for b in range(B)]
    q64, k64, v64 = _np(q), _np(kn), _np(vn)
    n = max(len(x) for x in keys) + q.shape[1]
    dead = None if seg is None else np.broadcast_to(seg < 0, q.shape[:2])
    if dead is not None:                       # what padding holds has no meaning
        q64, k64, v64 = (np.where(dead[..., None, None], 0, x) for x in (q64, k64, v64))
    ref, ref_lse = P.attend(q64, k64, v64, keys, vals, ar, seg, scale, window, sinks)
    fin = lambda x: np.where(np.isfinite(x), x, 0)   # rows outside every window may hold anything
    norm = lambda xs: max(float(np.sqrt((fin(x) ** 2).sum(-1)).max()) for x in xs if x.size)
    delta = 2.0 ** -15 * norm([q64]) * norm(keys + [k64]) * scale
    vmax = max(float(np.abs(fin(x)).max()) for x in vals + [v64] if x.size)
    rounding = 2 * 2.0 ** -8 if q.dtype == BF16 else n * 2.0 ** -22
    tol = (rounding + 2 * delta + 2.0 ** -14) * vmax
    got = _np(out)
    assert np.isfinite(got).all()
    err = float(np.abs(got - ref).max())
    assert err <= tol, (err, tol)
    none = np.isneginf(ref_lse)
    assert (got[none] == 0).all()
    if lse is not None:
        g = _np(lse)
        assert np.array_equal(np.isneginf(g), none) and not np.isnan(g).any()
        err = float(np.abs(g[~none] - ref_lse[~none]).max()) if (~none).any() else 0.0
        assert err <= delta + n * 2.0 ** -22 + 2.0 ** -14, err
    assert _b().pi_attn_read_status() == _b().PI_OK


def _attend(seed, lens, Sq, cache, page, Hq=8, Hkv=1, d=256, dtype=BF16, mask="causal", window=0,
            sinks=0, scale=1.0, with_lse=True, batch_mask=False, pad=False):
    c = Cache(seed, lens, page, Hkv, d, cache)
    rng, B = c.rng, len(lens)
    q = _rand(rng, (B, Sq, Hq, d), dtype, d ** -0.25)
    kn, vn = (_rand(rng, (B, Sq, Hkv, d), dtype, d ** -0.25) for _ in range(2))
    shape = (B, Sq) if batch_mask else (Sq,)
    if mask == "causal":
        ar = np.ones(shape, np.uint8)
    elif mask == "suffix":
        ar = np.broadcast_to(np.arange(Sq) < 2, shape).astype(np.uint8)
    else:
        ar = (rng.random(shape) < 0.2).astype(np.uint8) * rng.integers(1, 256, shape).astype(np.uint8)
    seg = rng.integers(-1 if pad else 0, 3, shape).astype(np.int32) if mask == "segments" else None
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda") if with_lse else None
    t = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    _b().pi_attn_paged(q, kn, vn, *c.args(), t(ar), segment_ids=t(seg), out=out, lse=lse,
                       softmax_scale=scale, window=window, sinks=sinks, **c.exps())
    _check(c, q, kn, vn, ar, seg, out, lse, scale, window, sinks)


CACHES = [BF16, E4M3]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[0], [1], [15, 16, 17], [880, 0, 401, 127, 128, 129]])
def test_decode(lens, page, cache):
    _attend(1, lens, 1, cache, page)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (4, 1), (16, 1), (8, 2), (8, 8), (32, 2), (6, 2),
                                    (24, 1)])
def test_decode_heads(Hq, Hkv, cache):
    _attend(2, [300, 37], 1, cache, 32, Hq=Hq, Hkv=Hkv)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens,Sq", [([0], 2), ([33, 700], 3), ([816, 0, 130], 51), ([5], 300),
                                     ([200, 3], 700)])
def test_chunk(lens, Sq, page, cache):
    _attend(3, lens, Sq, cache, page, mask="suffix")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (4, 1), (16, 1), (8, 2), (8, 8), (32, 2), (6, 2)])
def test_chunk_heads(Hq, Hkv, cache):
    _attend(4, [200, 37], 45, cache, 16, Hq=Hq, Hkv=Hkv, mask="causal", batch_mask=True)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 4, 33, 200])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (16, 4), (100, 0), (100, 64), (129, 300),
                                          (5000, 3)])
def test_window_and_sinks(Sq, window, sinks, cache):
    _attend(5, [500, 0, 128, 77], Sq, cache, 32, mask="causal", window=window, sinks=sinks)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,window", [(1, 0), (7, 0), (7, 40), (150, 0), (150, 90), (300, 3), (600, 200)])
def test_segments_and_padding(Sq, window, cache):
    _attend(6, [130, 0, 45, 260], Sq, cache, 16, mask="segments", pad=True, batch_mask=True,
            window=window, sinks=2, Hkv=2)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cache", CACHES)
def test_small_head_dims(d, cache):
    _attend(7, [70, 3], 9, cache, 16, d=d, Hkv=2, mask="blocks")


@pytest.mark.parametrize("cache", [F32, E4M3])
@pytest.mark.parametrize("d,Hq,Hkv", [(32, 3, 1), (64, 2, 1), (128, 6, 3), (256, 8, 1)])
@pytest.mark.parametrize("Sq,window", [(1, 0), (9, 0), (40, 21)])
def test_fp32(Sq, window, d, Hq, Hkv, cache):
    _attend(8, [40, 0, 131], Sq, cache, 16, d=d, Hq=Hq, Hkv=Hkv, dtype=F32, mask="segments", pad=True,
            window=window, sinks=3)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 20, 130])
def test_scale_and_no_lse(Sq, cache):
    _attend(9, [222, 31], Sq, cache, 64, scale=0.37, with_lse=False)


@pytest.mark.parametrize("cache", CACHES)
def test_long_ragged(cache):
    _attend(10, [5000, 1, 2500], 1, cache, 64)
    _attend(11, [4100, 17], 70, cache, 128, mask="causal")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 12, 140])
def test_many_sequences(Sq, cache):
    lens = [int(x) for x in np.random.default_rng(12).integers(0, 90, 150 if Sq == 1 else 40)]
    _attend(12, lens, Sq, cache, 16, mask="suffix")


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 12, 140])
def test_sharp_scores(Sq, cache):
    """Large scores (a softmax near one-hot): the running maximum moves often."""
    _attend(13, [600, 250], Sq, cache, 32, scale=6.0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 3, 60, 260])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("room", [40, 17000])
def test_stale_slots_and_padding_hold_nan(Sq, window, cache, room):
    """NaN and infinities in every slot that no query sees, and in padding
    tokens' q, k and v, do not reach the result."""
    lens = [200, 0, 77]
    c = Cache(14, lens, 16, 1, 256, cache, room=room)
    rng, B = c.rng, 3
    q = _rand(rng, (B, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(rng, (B, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    seg = np.zeros((B, Sq), np.int32)
    seg[1, Sq // 2:] = -1
    seg[2, ::3] = -1
    for b in range(B):
        for t in np.nonzero(seg[b] < 0)[0]:
            q[b, t], kn[b, t], vn[b, t] = float("nan"), float("inf"), float("nan")
    live = np.zeros((c.k.shape[0], c.k.shape[1]), bool)
    for b, n in enumerate(lens):
        first = max(0, n - window + 1) if window else 0      # query 0 sees the most
        for x in list(range(min(4, n))) + list(range(first, n)):
            live.reshape(-1)[P.slot(c.table_np, b, x, 16)] = True
    dead = torch.from_numpy(~live).cuda()
    for pool, exps in ((c.k, c.k_exp), (c.v, c.v_exp)):
        if cache == E4M3:
            pool.view(torch.uint8)[dead] = 0x7F
            exps[dead] = 255
        else:
            pool[dead] = float("nan")
            pool.view(-1, 256)[torch.nonzero(dead.view(-1))[::2, 0]] = float("-inf")
    ar = np.ones(Sq, np.uint8)
    arb = np.ascontiguousarray(np.broadcast_to(ar, (B, Sq)))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    _b().pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(arb).cuda(),
                       segment_ids=torch.from_numpy(seg).cuda(), out=out, lse=lse, window=window,
                       sinks=4, **c.exps())
    _check(c, q, kn, vn, arb, seg, out, lse, 1.0, window, 4)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 40, 150])
@pytest.mark.parametrize("room", [0, 17000])
def test_bad_tables_and_lengths_are_reported(Sq, cache, room):
    """Out-of-range page ids and lengths are bounded and recorded; other
    sequences keep their results, and nothing past the buffers is touched."""
    b = _b()
    c = Cache(15, [100, 90, 60], 16, 1, 256, cache, room=room)
    rng = c.rng
    q = _rand(rng, (3, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(rng, (3, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    ref = b.pi_attn_paged(q, kn, vn, *c.args(), ar, **c.exps())
    assert b.pi_attn_read_status() == b.PI_OK
    bad = c.table.clone()
    bad[1, 2], bad[1, 3], bad[1, 4] = -1, 2 ** 31 - 1, c.k.shape[0]
    out = b.pi_attn_paged(q, kn, vn, c.k, c.v, bad, c.lens, ar, **c.exps())
    assert b.pi_attn_read_status() == b.PI_ERR_ARG
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    assert torch.isfinite(out.float()).all()
    lens = c.lens.clone()
    lens[1] = 2 ** 31 - 1
    b.pi_attn_paged(q, kn, vn, c.k, c.v, c.table, lens, ar, **c.exps())
    assert b.pi_attn_read_status() == b.PI_ERR_ARG
    lens[1] = -7
    out = b.pi_attn_paged(q, kn, vn, c.k, c.v, c.table, lens, ar, **c.exps())
    assert b.pi_attn_read_status() == b.PI_ERR_ARG
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    k, v = c.k.clone(), c.v.clone()
    b.pi_attn_cache_write(kn[:, :1].contiguous(), vn[:, :1].contiguous(), c.k, c.v, bad, c.lens,
                          **c.exps())                            # sequence 1's page 5 is fine
    assert b.pi_attn_read_status() == b.PI_OK
    c.k.copy_(k), c.v.copy_(v)
    lens[1] = 40                                                 # its next token's page is not
    b.pi_attn_cache_write(kn[1:2, :1].contiguous(), vn[1:2, :1].contiguous(), c.k, c.v,
                          bad[1:2].contiguous(), lens[1:2].contiguous(), **c.exps())
    assert b.pi_attn_read_status() == b.PI_ERR_ARG
    assert torch.equal(c.k.view(torch.uint8), k.view(torch.uint8))
    assert torch.equal(c.v.view(torch.uint8), v.view(torch.uint8))
    b.pi_attn_cache_read(c.k, c.v, bad, c.lens, 100, **c.exps())
    assert b.pi_attn_read_status() == b.PI_ERR_ARG


# ------------------------------------------------------------- write and read

def _written(c, kn, vn, mask, k0, v0):
    """Pools (as float64) and exponents after the oracle's write, from copies
    of the pools before it."""
    B, S = kn.shape[:2]
    pos = P.positions(c.lens_np, S, mask)
    e4 = c.k.dtype == E4M3
    want = {}
    for name, x, (pool, exps) in (("k", kn, k0), ("v", vn, v0)):
        pool, exps = pool.copy(), None if exps is None else exps.copy()
        flat = pool.reshape(-1, *pool.shape[2:])
        x64 = _np(x)
        for b in range(B):
            for t in range(S):
                if pos[b, t] < 0:
                    continue
                at = P.slot(c.table_np, b, int(pos[b, t]), c.page)
                for h in range(x.shape[2]):
                    if e4:
                        flat[at, h], exps.reshape(-1, exps.shape[2])[at, h] = P.quantise(x64[b, t, h])
                    else:
                        flat[at, h] = x64[b, t, h]
        want[name], want[name + "_exp"] = pool, exps
    return want, c.lens_np + (pos >= 0).sum(1)


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (BF16, E4M3), (F32, F32), (F32, E4M3)])
@pytest.mark.parametrize("B,S,Hkv,d,page,masked", [
    (1, 1, 1, 256, 16, None), (5, 1, 2, 256, 32, None), (3, 50, 1, 256, 16, "batch"),
    (2, 130, 1, 256, 64, "shared"), (2, 33, 3, 64, 16, "batch"), (1, 70, 2, 32, 128, None),
    (2, 9, 1, 128, 256, "batch")])
def test_write_then_read(dtype, cache, B, S, Hkv, d, page, masked):
    b = _b()
    rng = np.random.default_rng(20)
    lens = [int(x) for x in rng.integers(0, 70, B)]
    c = Cache(21, lens, page, Hkv, d, cache, room=S)
    kn, vn = (_rand(rng, (B, S, Hkv, d), dtype, 0.3) for _ in range(2))
    kn *= torch.exp2(torch.from_numpy(rng.integers(-20, 20, (B, S, Hkv, 1))).cuda().to(dtype))
    kn[0, 0, 0] = 0
    mask = None
    if masked:
        mask = (rng.random((B, S) if masked == "batch" else S) < 0.7).astype(np.uint8) * 3
    before = [(_np(p), None if e is None else e.cpu().numpy())
              for p, e in ((c.k, c.k_exp), (c.v, c.v_exp))]
    want, want_lens = _written(c, kn, vn, mask, *before)
    lens_out = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    got = b.pi_attn_cache_write(kn, vn, *c.args(), token_mask=None if mask is None else
                                torch.from_numpy(mask).cuda(), lens_out=lens_out, **c.exps())
    assert got is lens_out and np.array_equal(lens_out.cpu().numpy(), want_lens)
    for name in ("k", "v"):
        assert np.array_equal(_np(getattr(c, name)), want[name])       # untouched slots too
        if cache == E4M3:
            assert np.array_equal(getattr(c, name + "_exp").cpu().numpy(), want[name + "_exp"])
    # read back, some rows past every length
    c.lens_np = want_lens.astype(np.int32)
    c.lens = lens_out
    R = int(want_lens.max()) + 5
    k, v, valid = b.pi_attn_cache_read(*c.args(), R, dtype=dtype, **c.exps())
    for name, x in (("k", k), ("v", v)):
        for i in range(B):
            n = int(want_lens[i])
            ref = torch.from_numpy(c.rows(name, i)).to(dtype).double().numpy()
            assert np.array_equal(_np(x[i, :n]), ref)
            assert (x[i, n:] == 0).all()
    live = np.arange(R)[None] < want_lens[:, None]
    assert np.array_equal(valid.cpu().numpy(), live.astype(np.uint8))
    assert b.pi_attn_read_status() == b.PI_OK


def test_write_special_values():
    """Zero vectors, the scale's borders, subnormals, the largest values, NaN
    and infinities."""
    b = _b()
    c = Cache(22, [0], 32, 1, 32, E4M3, room=32)
    x = torch.zeros(1, 12, 1, 32)
    x[0, 1, 0, 5] = 448.0
    x[0, 2, 0, 5] = float(np.nextafter(np.float32(448), np.float32(1e9)))
    x[0, 3, 0] = torch.linspace(-1, 1, 32) * 3e38
    x[0, 4, 0] = torch.linspace(-1e-39, 1e-39, 32)
    x[0, 5, 0] = 1e-45
    x[0, 6, 0] = torch.linspace(0.9, 1.8, 32)
    x[0, 7, 0, :4] = torch.tensor([1.0, -17.0, 2.0 ** -9, 2.0 ** -14])
    for t in (8, 9):
        x[0, t, 0] = torch.linspace(-2, 2, 32)
    x[0, 8, 0, 3] = float("nan")
    x[0, 9, 0, 3] = float("inf")
    x = x.cuda()
    b.pi_attn_cache_write(x, x, *c.args(), **c.exps())
    flat, exps = _np(c.k).reshape(-1, 32), c.k_exp.cpu().numpy().reshape(-1)
    for t in range(8):
        at = P.slot(c.table_np, 0, t, 32)
        vals, byte = P.quantise(_np(x[0, t, 0]))
        assert exps[at] == byte, t
        assert np.array_equal(flat[at], vals), t
    assert exps[P.slot(c.table_np, 0, 8, 32)] == 255
    c.lens += 12
    k, _, _ = b.pi_attn_cache_read(*c.args(), 12, dtype=F32, **c.exps())
    assert torch.isnan(k[0, 8]).all()
    assert k[0, 9, 0, 3] == float("inf") and (k[0, 9, 0, 4:] == 0).all()


@pytest.mark.parametrize("Sq", [1, 2, 5, 40, 150])
@pytest.mark.parametrize("room", [0, 17000])
def test_cached_values_come_through_exactly(Sq, room):
    """One visible cached key: its probability is 1 and out is its value vector,
    rounded to bf16 only.  Every e4m3 byte and exponents over the range."""
    b = _b()
    c = Cache(24, [32], 32, 1, 256, E4M3, room=room)
    bits = torch.arange(256, dtype=torch.uint8)
    bits[0x7F] = bits[0xFF] = 0
    slot = P.slot(c.table_np, 0, 0, 32)
    c.v.view(torch.uint8).view(-1, 256)[slot] = bits.cuda()
    q = _rand(c.rng, (1, Sq, 8, 256), BF16, 0.25)
    kn = _rand(c.rng, (1, Sq, 1, 256), BF16, 0.25)
    vn = _rand(c.rng, (1, Sq, 1, 256), BF16, 0.25)
    seg = torch.full((Sq,), -1, dtype=torch.int32, device="cuda")
    seg[-1] = 0
    # the last token sees cached key 0 (a sink) and itself; its own key is far
    # below (its score is -2^9 at least), so that its probability underflows
    q[:] = 4.0
    kn[:] = -4.0
    c.k.view(torch.uint8).view(-1, 256)[slot] = 0x38           # 1.0
    c.k_exp.view(-1)[slot] = 127
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    for byte in list(range(0, 250, 7)) + [120, 127, 134, 135, 136, 246, 247]:
        c.v_exp.view(-1)[slot] = byte
        out = b.pi_attn_paged(q, kn, vn, *c.args(), ar, segment_ids=seg, window=1, sinks=1,
                              **c.exps())
        want = bits.view(torch.float8_e4m3fn).double() * 2.0 ** (byte - 127)
        want = want.to(BF16).cuda()
        tiny = want.abs().double() < 2.0 ** -126                # bf16 subnormals may be flushed
        got = out[0, -1]
        ok = (got == want) | (tiny & (got.abs().double() < 2.0 ** -126))
        assert ok.all(), byte


def test_write_past_the_room_is_dropped_and_reported():
    b = _b()
    c = Cache(23, [28], 16, 1, 256, BF16)                  # 2 pages: 4 tokens of room
    kn = _rand(c.rng, (1, 9, 1, 256), BF16, 1.0)
    want = _np(c.k).copy().reshape(-1, 256)
    for t in range(4):
        want[P.slot(c.table_np, 0, 28 + t, 16)] = _np(kn[0, t, 0])
    lens_out = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.pi_attn_cache_write(kn, kn, *c.args(), lens_out=lens_out)
    assert b.pi_attn_read_status() == b.PI_ERR_ARG
    assert int(lens_out) == 32 and np.array_equal(_np(c.k).reshape(-1, 256), want)
    empty = torch.empty(1, 0, 1, 256, dtype=BF16, device="cuda")
    b.pi_attn_cache_write(empty, empty, *c.args(), lens_out=lens_out)
    assert int(lens_out) == 28


# -------------------------------------------------------------- used together

@pytest.mark.parametrize("cache", CACHES)
def test_prefix_then_decoding(cache):
    """A padded prefix enters the cache, then tokens are decoded one by one,
    appended, and a suffix chunk reads it all; the bf16 cache gives what the
    dense entry points give on the read-back rows."""
    b = _b()
    rng = np.random.default_rng(30)
    B, S, Hq, d, page = 3, 60, 8, 256, 16
    c = Cache(31, [0] * B, page, 1, d, cache, room=90)
    for t in (c.k, c.v):                                   # stale slots
        t.view(torch.uint8).fill_(0x7F)
    mask = (rng.random((B, S)) < 0.8).astype(np.uint8)
    lens = [c.lens.clone(), torch.empty_like(c.lens)]
    kn, vn = (_rand(rng, (B, S, 1, d), BF16, 0.25) for _ in range(2))
    b.pi_attn_cache_write(kn, vn, c.k, c.v, c.table, lens[0], torch.from_numpy(mask).cuda(),
                          lens_out=lens[1], **c.exps())
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    for step in range(6):
        lens.reverse()
        q = _rand(rng, (B, 1, Hq, d), BF16, 0.25)
        kn, vn = (_rand(rng, (B, 1, 1, d), BF16, 0.25) for _ in range(2))
        out = b.pi_attn_paged(q, kn, vn, c.k, c.v, c.table, lens[0], one, **c.exps())
        b.pi_attn_cache_write(kn, vn, c.k, c.v, c.table, lens[0], lens_out=lens[1], **c.exps())
        c.lens, c.lens_np = lens[0], lens[0].cpu().numpy().copy()
        _check(c, q, kn, vn, np.ones(1, np.uint8), None, out, None, 1.0, 0, 0)
        assert np.array_equal(lens[1].cpu().numpy(), mask.sum(1) + step + 1)
    c.lens, c.lens_np = lens[1], lens[1].cpu().numpy().copy()
    Sq = 20
    ar = np.array([1, 1] + [0] * (Sq - 2), np.uint8)
    q = _rand(rng, (B, Sq, Hq, d), BF16, 0.25)
    kn, vn = (_rand(rng, (B, Sq, 1, d), BF16, 0.25) for _ in range(2))
    art = torch.from_numpy(ar).cuda()
    out = b.pi_attn_paged(q, kn, vn, *c.args(), art, **c.exps())
    _check(c, q, kn, vn, ar, None, out, None, 1.0, 0, 0)
    kd, vd, valid = b.pi_attn_cache_read(*c.args(), 80, **c.exps())
    dense = b.pi_attn_suffix(q, kn, vn, kd, vd, art, cache_valid=valid)
    vmax = float(torch.maximum(vd.abs().max(), vn.abs().max()))
    # two roundings of probabilities and of the result, each by 2^-8 at most
    assert float((dense.float() - out.float()).abs().max()) <= 4 * 2.0 ** -8 * vmax + 1e-3


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 51, 150])
def test_captured_step_follows_the_lengths(Sq, cache):
    """One captured graph of attention and append, replayed while the lengths
    grow."""
    b = _b()
    rng = np.random.default_rng(32)
    B, Hq, d = 2, 8, 256
    c = Cache(33, [30, 100], 16, 1, d, cache, room=3 * Sq + 40)
    q = _rand(rng, (B, Sq, Hq, d), BF16, 0.25)
    kn, vn = (_rand(rng, (B, Sq, 1, d), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    out, lens_out = torch.empty_like(q), torch.empty_like(c.lens)
    need = b.pi_attn_paged_workspace_bytes(q, kn, *c.args(), **c.exps())
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step():
        b.pi_attn_paged(q, kn, vn, *c.args(), ar, out=out, workspace=ws, **c.exps())
        b.pi_attn_cache_write(kn, vn, *c.args(), lens_out=lens_out, **c.exps())
        c.lens.copy_(lens_out)

    side = torch.cuda.Stream()
    start = [c.lens.clone(), c.k.clone(), c.v.clone()] + [e.clone() for e in (c.k_exp, c.v_exp) if e is not None]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, x in zip([c.lens, c.k, c.v, c.k_exp, c.v_exp], start):
        t.copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        n = c.lens.cpu().numpy().copy()
        for x in (q, kn, vn):
            x.copy_(_rand(rng, tuple(x.shape), BF16, 0.25))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.lens.cpu().numpy(), n + Sq)
        c.lens_np = n
        _check(c, q, kn, vn, np.ones(Sq, np.uint8), None, out, None, 1.0, 0, 0)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 9, 70, 150])
def test_side_stream_and_repeatability(Sq, cache):
    """Calls on two streams at once, each with its own workspace, give the
    same bits as one call after another."""
    b = _b()
    c = Cache(34, [900, 100, 0, 2000], 64, 1, 256, cache)
    q = _rand(c.rng, (4, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (4, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    ref = b.pi_attn_paged(q, kn, vn, *c.args(), ar, **c.exps())
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [b.pi_attn_paged(q, kn, vn, *c.args(), ar, stream=s[i % 2], **c.exps())
            for i in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


@pytest.mark.parametrize("cache", CACHES)
def test_sequences_share_pages(cache):
    """Two sequences with one prefix in the same pages."""
    b = _b()
    c = Cache(35, [64, 64, 80], 16, 1, 256, cache)
    c.table[1, :4] = c.table[0, :4]
    c.table_np = c.table.cpu().numpy()
    for Sq in (1, 30):
        q = _rand(c.rng, (3, Sq, 8, 256), BF16, 0.25)
        kn, vn = (_rand(c.rng, (3, Sq, 1, 256), BF16, 0.25) for _ in range(2))
        ar = np.ones(Sq, np.uint8)
        out = b.pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(ar).cuda(), **c.exps())
        _check(c, q, kn, vn, ar, None, out, None, 1.0, 0, 0)


@pytest.mark.parametrize("cache", CACHES)
def test_offsets_past_32_bits(cache):
    """A pool of more than 2^32 elements, pages at its far end."""
    b = _b()
    page, d, pages = 256, 256, 65536 + 64                  # 2^32 + 2^22 elements
    kp, vp = (torch.zeros(pages, page, 1, d, dtype=torch.uint8, device="cuda").view(E4M3)
              if cache == E4M3 else torch.zeros(pages, page, 1, d, dtype=BF16, device="cuda")
              for _ in range(2))
    exps = {}
    if cache == E4M3:
        exps = {n: torch.full((pages, page, 1), 127, dtype=torch.uint8, device="cuda")
                for n in ("k_exp", "v_exp")}
    rng = np.random.default_rng(36)
    table = torch.tensor([[pages - 1, 3], [pages - 2, pages - 5]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    after = torch.empty_like(lens)
    kn, vn = (_rand(rng, (2, 300, 1, d), BF16, 0.25) for _ in range(2))
    b.pi_attn_cache_write(kn, vn, kp, vp, table, lens, lens_out=after, **exps)
    k, v, _ = b.pi_attn_cache_read(kp, vp, table, after, 300, **exps)
    if cache == BF16:
        assert torch.equal(k, kn) and torch.equal(v, vn)
    else:
        assert float((k.float() - kn.float()).abs().max()) <= 2.0 ** -4 * float(kn.abs().max())
    for Sq in (1, 40):
        q = _rand(rng, (2, Sq, 8, d), BF16, 0.25)
        k1, v1 = (_rand(rng, (2, Sq, 1, d), BF16, 0.25) for _ in range(2))
        ar = np.ones(Sq, np.uint8)
        out = b.pi_attn_paged(q, k1, v1, kp, vp, table, after, torch.from_numpy(ar).cuda(), **exps)
        ref, _ = P.attend(_np(q), _np(k1), _np(v1), list(_np(k)), list(_np(v)), ar)
        assert np.abs(_np(out) - ref).max() <= 3 * 2.0 ** -8 * float(vn.abs().max())
    assert b.pi_attn_read_status() == b.PI_OK


def _guarded(shape, dtype, n=4096):
    size = int(np.prod(shape))
    buf = torch.full((size + 2 * n,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[n:n + size].view(*shape)


def _clean(buf, n=4096):
    return bool((buf[:n] == 7).all()) and bool((buf[-n:] == 7).all())


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,B", [(1, 2), (5, 3), (37, 2), (300, 1)])
def test_nothing_is_written_outside(Sq, B, cache):
    b = _b()
    c = Cache(37, [700, 90, 333][:B], 32, 1, 256, cache)
    q = _rand(c.rng, (B, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (B, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    ob, out = _guarded(q.shape, BF16)
    lb, lse = _guarded(q.shape[:3], F32)
    need = b.pi_attn_paged_workspace_bytes(q, kn, *c.args(), **c.exps())
    wb, ws = _guarded((max(need, 16),), torch.uint8)
    ws.fill_(0xFF)
    pools = [c.k.clone(), c.v.clone()]
    b.pi_attn_paged(q, kn, vn, *c.args(), ar, out=out, lse=lse, workspace=ws, **c.exps())
    assert b.pi_attn_read_status() == b.PI_OK
    assert _clean(ob) and _clean(lb) and _clean(wb)
    assert torch.equal(c.k.view(torch.uint8), pools[0].view(torch.uint8))
    assert torch.equal(c.v.view(torch.uint8), pools[1].view(torch.uint8))
    kb, k = _guarded((B, 71, 1, 256), BF16)
    vb, v = _guarded((B, 71, 1, 256), BF16)
    mb, valid = _guarded((B, 71), torch.uint8)
    b.pi_attn_cache_read(*c.args(), 71, k_out=k, v_out=v, valid_out=valid, **c.exps())
    torch.cuda.synchronize()
    assert _clean(kb) and _clean(vb) and _clean(mb)


def test_binding_checks():
    b = _b()
    c = Cache(38, [10], 16, 1, 256, E4M3)
    q = _rand(c.rng, (1, 1, 8, 256), BF16, 1.0)
    kn = _rand(c.rng, (1, 1, 1, 256), BF16, 1.0)
    ar = torch.ones(1, dtype=torch.uint8, device="cuda")
    ok = dict(c.exps())
    with pytest.raises(ValueError):
        b.pi_attn_paged(q, kn, kn, *c.args(), ar)                      # exponents missing
    with pytest.raises(ValueError):
        b.pi_attn_paged(q, kn, kn, c.k, c.v, c.table, c.lens.long(), ar, **ok)
    with pytest.raises(ValueError):
        b.pi_attn_paged(q, kn, kn, c.k, c.v, torch.zeros(1, 8, dtype=torch.int32, device="cuda")[:, ::2],
                        c.lens, ar, **ok)
    with pytest.raises(ValueError):
        b.pi_attn_paged(q, kn, kn, c.k, c.v[:1], c.table, c.lens, ar, **ok)
    with pytest.raises(ValueError):
        b.pi_attn_paged(q[..., ::2], kn, kn, *c.args(), ar, **ok)
    with pytest.raises(ValueError):
        b.pi_attn_paged(q.float(), kn, kn, *c.args(), ar, **ok)
    with pytest.raises(ValueError):
        b.pi_attn_cache_write(kn, kn, *c.args(), lens_out=torch.zeros(2, dtype=torch.int32, device="cuda"), **ok)
    with pytest.raises(b.PiAttnError):
        b.pi_attn_cache_write(kn, kn, *c.args(), lens_out=c.lens, **ok)
    with pytest.raises(b.PiAttnError):
        b.pi_attn_paged(q, kn, kn, *c.args(), ar, window=-1, **ok)
    with pytest.raises(b.PiAttnError):
        b.pi_attn_paged(q[:, :, :5].contiguous(), kn.expand(1, 1, 1, 256).contiguous(), kn,
                        *c.args(), ar, softmax_scale=0.0, **ok)


# ------------------------------------------------------- the ends of the ranges

@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq,B", [(9, 130), (150, 66), (1, 300)])
def test_more_sequences_than_one_launch_schedules(Sq, B, cache):
    """A last launch of few sequences, one of them long."""
    lens = [int(x) for x in np.random.default_rng(40).integers(0, 120, B)]
    lens[-1], lens[3] = 24000 // B + 801, 700
    _attend(40, lens, Sq, cache, 32, mask="causal")


@pytest.mark.parametrize("Hkv", [1, 2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20), (1, 0)])
def test_chunk_with_a_used_workspace(window, sinks, Hkv):
    """What the workspace held (NaN) does not reach the result."""
    b = _b()
    c = Cache(41, [0, 77, 1000, 513], 64, Hkv, 256, E4M3)
    Sq = 260
    q = _rand(c.rng, (4, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (4, Sq, Hkv, 256), BF16, 0.25) for _ in range(2))
    ar = np.ones(Sq, np.uint8)
    need = b.pi_attn_paged_workspace_bytes(q, kn, *c.args(), window=window, sinks=sinks, **c.exps())
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    b.pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(ar).cuda(), out=out, lse=lse, workspace=ws,
                    window=window, sinks=sinks, **c.exps())
    _check(c, q, kn, vn, ar, None, out, lse, 1.0, window, sinks)


@pytest.mark.parametrize("cache", CACHES)
def test_long_ragged_chunks(cache):
    _attend(42, [5000, 1, 2500], 300, cache, 256, Hkv=2)
    _attend(43, [3000, 2999], 520, cache, 16, mask="segments", pad=True, window=700, sinks=9)


@pytest.mark.parametrize("cache", [F32, E4M3])
@pytest.mark.parametrize("window", [0, 11])
def test_fp32_many_short_rows(cache, window):
    """Enough rows of few keys that each goes to one warp."""
    lens = [int(x) for x in np.random.default_rng(44).integers(0, 90, 70)]
    _attend(44, lens, 16, cache, 16, d=64, Hq=4, Hkv=2, dtype=F32, mask="segments", pad=True,
            window=window, sinks=2)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("Sq", [1, 6, 150])
def test_empty_pool(Sq, d, cache):
    """No page at all, or no column: only the chunk is seen; a length that
    claims cached tokens is clamped and recorded."""
    b = _b()
    rng = np.random.default_rng(45)
    q = _rand(rng, (2, Sq, 8, d), BF16, 0.25)
    kn, vn = (_rand(rng, (2, Sq, 1, d), BF16, 0.25) for _ in range(2))
    ar = np.ones(Sq, np.uint8)
    art = torch.from_numpy(ar).cuda()
    none = [np.zeros((0, 1, d))] * 2
    ref, _ = P.attend(_np(q), _np(kn), _np(vn), none, none, ar)
    for pages, columns in ((0, 0), (0, 2), (2, 0)):
        pool = [torch.zeros(pages, 16, 1, d, device="cuda").to(cache) for _ in range(2)]
        exps = {}
        if cache == E4M3:
            exps = {n: torch.zeros(pages, 16, 1, dtype=torch.uint8, device="cuda")
                    for n in ("k_exp", "v_exp")}
        table = torch.zeros(2, columns, dtype=torch.int32, device="cuda")
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        out = b.pi_attn_paged(q, kn, vn, *pool, table, lens, art, **exps)
        assert b.pi_attn_read_status() == b.PI_OK
        assert np.abs(_np(out) - ref).max() <= 3 * 2.0 ** -8 * float(vn.abs().max())
        k, v, valid = b.pi_attn_cache_read(*pool, table, lens, 3, **exps)
        assert b.pi_attn_read_status() == b.PI_OK
        assert (k == 0).all() and (v == 0).all() and (valid == 0).all()
        out = b.pi_attn_paged(q, kn, vn, *pool, table, lens + 5, art, **exps)
        assert b.pi_attn_read_status() == b.PI_ERR_ARG
        assert torch.isfinite(out.float()).all()
        b.pi_attn_cache_write(kn, vn, *pool, table, lens, **exps)
        assert b.pi_attn_read_status() == b.PI_ERR_ARG


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 64), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_longest_chunk(window, sinks, cache):
    """16383 new tokens: some rows against a float64 sum on the device."""
    b = _b()
    Sq, n = 16383, 1000
    c = Cache(46, [n], 128, 1, 256, cache)
    q = _rand(c.rng, (1, Sq, 2, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (1, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    out = b.pi_attn_paged(q, kn, vn, *c.args(), ar, lse=lse, window=window, sinks=sinks, **c.exps())
    assert b.pi_attn_read_status() == b.PI_OK
    keys = torch.cat([torch.from_numpy(c.rows("k", 0)[:, 0]).cuda(), kn[0, :, 0].double()])
    vals = torch.cat([torch.from_numpy(c.rows("v", 0)[:, 0]).cuda(), vn[0, :, 0].double()])
    x = torch.arange(n + Sq, device="cuda")
    delta = 2.0 ** -15 * float(q.double().norm(dim=-1).max()) * float(keys.norm(dim=-1).max())
    vmax = float(vals.abs().max())
    for i in (0, 1, 127, 128, 5000, 8191, 16000, Sq - 1):
        s = q[0, i].double() @ keys.T
        seen = x <= n + i
        if window:
            seen &= (n + i - x < window) | (x < sinks)
        s[:, ~seen] = float("-inf")
        ref = torch.softmax(s, -1) @ vals
        err = float((out[0, i].double() - ref).abs().max())
        assert err <= (2 * 2.0 ** -8 + 2 * delta + 2.0 ** -14) * vmax, (i, err)
        err = float((lse[0, i].double() - torch.logsumexp(s, -1)).abs().max())
        assert err <= delta + (n + Sq) * 2.0 ** -22 + 2.0 ** -14, (i, err)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 6, 50, 200])
def test_padding_alone(Sq, cache):
    """A batch of padding: zeros and -inf, whatever q, k and v hold."""
    b = _b()
    c = Cache(47, [300, 0, 40], 16, 1, 256, cache)
    q, out = (torch.full((3, Sq, 8, 256), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    kn = torch.full((3, Sq, 1, 256), float("nan"), dtype=BF16, device="cuda")
    lse = torch.zeros(3, Sq, 8, device="cuda")
    seg = torch.full((Sq,), -1, dtype=torch.int32, device="cuda")
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    b.pi_attn_paged(q, kn, kn, *c.args(), ar, segment_ids=seg, out=out, lse=lse, **c.exps())
    assert b.pi_attn_read_status() == b.PI_OK
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 40, 150])
@pytest.mark.parametrize("room", [0, 17000])
def test_two_graphs_at_once(Sq, cache, room):
    """Two captured calls, a workspace each, replayed on two streams together."""
    b = _b()
    c = Cache(48, [900, 100, 0, 2000], 64, 1, 256, cache, room=room)
    kn, vn = (_rand(c.rng, (4, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    qs = [_rand(c.rng, (4, Sq, 8, 256), BF16, 0.25) for _ in range(2)]
    refs = [b.pi_attn_paged(q, kn, vn, *c.args(), ar, **c.exps()) for q in qs]
    need = b.pi_attn_paged_workspace_bytes(qs[0], kn, *c.args(), **c.exps())
    outs = [torch.zeros_like(q) for q in qs]
    spaces = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in qs]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for q, out, ws in zip(qs, outs, spaces):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                b.pi_attn_paged(q, kn, vn, *c.args(), ar, out=out, workspace=ws, **c.exps())
        graphs.append(g)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert b.pi_attn_read_status() == b.PI_OK
    for out, ref in zip(outs, refs):
        assert torch.equal(out, ref)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 30, 150])
def test_one_page_twice_in_a_table(Sq, cache):
    """A page may stand for several places of one sequence when it is read."""
    b = _b()
    c = Cache(49, [96, 64], 16, 1, 256, cache)
    c.table[0, 3], c.table[0, 4], c.table[1, 2] = c.table[0, 0], c.table[0, 0], c.table[0, 5]
    c.table_np = c.table.cpu().numpy()
    q = _rand(c.rng, (2, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (2, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = np.ones(Sq, np.uint8)
    out = b.pi_attn_paged(q, kn, vn, *c.args(), torch.from_numpy(ar).cuda(), **c.exps())
    _check(c, q, kn, vn, ar, None, out, None, 1.0, 0, 0)


def test_binding_checks_of_the_limits():
    b = _b()
    c = Cache(50, [10, 5], 16, 1, 256, BF16)
    q = _rand(c.rng, (2, 1, 8, 256), BF16, 1.0)
    kn = _rand(c.rng, (2, 1, 1, 256), BF16, 1.0)
    ar = torch.ones(1, dtype=torch.uint8, device="cuda")
    for bad in (2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            b.pi_attn_paged(q, kn, kn, *c.args(), ar, window=bad)
        with pytest.raises(ValueError):
            b.pi_attn_paged(q, kn, kn, *c.args(), ar, window=1, sinks=bad)
    with pytest.raises(TypeError):
        b.pi_attn_paged(q, kn, kn, *c.args(), ar, window=2.5)
    lens = torch.tensor([10, 5, 0], dtype=torch.int32, device="cuda")
    with pytest.raises(b.PiAttnError):                   # lens_out overlaps cache_lens
        b.pi_attn_cache_write(kn, kn, c.k, c.v, c.table, lens[:2], lens_out=lens[1:])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window", [0, 5200])
@pytest.mark.parametrize("lens,Sq,Hq,Hkv", [
    ([9000], 1, 8, 1),                         # long for its number of units
    ([12000, 5], 4, 4, 2),
    ([17000] + [3] * 20, 1, 8, 1),
    (list(range(0, 520, 4)), 1, 16, 2),        # more units than half the CTAs
    ([100] * 55, 2, 4, 1),                     # the most units that clusters take
    ([100] * 56, 2, 4, 1),
])
def test_decode_forms(lens, Sq, Hq, Hkv, window, cache):
    """Every way the few-row kernel shares out its work."""
    _attend(51, lens, Sq, cache, 64, Hq=Hq, Hkv=Hkv, mask="segments", pad=True, window=window,
            sinks=7, batch_mask=True)


@pytest.mark.parametrize("d,Hq", [(32, 1), (64, 3)])
def test_fp32_long_chunk(d, Hq):
    """A chunk whose codes take more shared memory than a kernel has by default."""
    b = _b()
    Sq, n = 9001, 21
    c = Cache(52, [n], 16, 1, d, F32)
    q = _rand(c.rng, (1, Sq, Hq, d), F32, d ** -0.25)
    kn, vn = (_rand(c.rng, (1, Sq, 1, d), F32, d ** -0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    out = b.pi_attn_paged(q, kn, vn, *c.args(), ar, lse=lse)
    assert b.pi_attn_read_status() == b.PI_OK
    keys = torch.cat([torch.from_numpy(c.rows("k", 0)[:, 0]).cuda(), kn[0, :, 0].double()])
    vals = torch.cat([torch.from_numpy(c.rows("v", 0)[:, 0]).cuda(), vn[0, :, 0].double()])
    delta = 2.0 ** -15 * float(q.double().norm(dim=-1).max()) * float(keys.norm(dim=-1).max())
    vmax = float(vals.abs().max())
    for i in (0, 3, 4500, Sq - 1):
        s = q[0, i].double() @ keys[:n + i + 1].T
        ref = torch.softmax(s, -1) @ vals[:n + i + 1]
        err = float((out[0, i].double() - ref).abs().max())
        assert err <= (2 * delta + (n + Sq) * 2.0 ** -22 + 2.0 ** -14) * vmax, (i, err)
        err = float((lse[0, i].double() - torch.logsumexp(s, -1)).abs().max())
        assert err <= delta + (n + Sq) * 2.0 ** -22 + 2.0 ** -14, (i, err)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("Sq", [1, 40, 150])
@pytest.mark.parametrize("room", [0, 17000])
def test_out_in_place_of_q(Sq, cache, room):
    """The result may replace the queries."""
    b = _b()
    c = Cache(53, [900, 100, 0, 2000], 64, 1, 256, cache, room=room)
    q = _rand(c.rng, (4, Sq, 8, 256), BF16, 0.25)
    kn, vn = (_rand(c.rng, (4, Sq, 1, 256), BF16, 0.25) for _ in range(2))
    ar = torch.ones(Sq, dtype=torch.uint8, device="cuda")
    ref = b.pi_attn_paged(q, kn, vn, *c.args(), ar, **c.exps())
    for _ in range(3):
        x = q.clone()
        b.pi_attn_paged(x, kn, vn, *c.args(), ar, out=x, **c.exps())
        assert torch.equal(x, ref)
