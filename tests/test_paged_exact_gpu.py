"""Attention over the paged cache, element by element, at long lengths.

A bound of a fraction of the largest value lets much pass where many keys are
averaged: the result shrinks with the square root of their number.  So here

* with q = 0 every visible key has probability 1 / count exactly, and with
  values that are small integers times powers of two every sum is exact in
  fp32: the result is off by one rounding to its type and two fp32 roundings
  (the reciprocal and the product), whatever the length.  One key too few, too
  many or wrong shows.
* with q aimed at one key at a time, the result is that key's value, so a tile,
  page or piece out of place shows wherever it lies.
* with random inputs, element c of a row is off by at most (2^-8 + 2 delta +
  n 2^-22 + 2^-14) * sum_j w_j |v_jc| + 2^-8 |out_c|: each probability is rounded
  to bf16 once (2^-8) and carries its score's error (delta, as in
  test_paged_gpu.py; numerator and denominator), fp32 sums over n keys, a margin
  for exp2; the result is rounded once.  fp32: without the 2^-8 terms, and 2^-24.

The reference is computed on the device in 64 bits from the oracle's mask.
"""

import numpy as np
import pytest
import torch

from oracle import paged as P
from test_paged_gpu import BF16, E4M3, F32, Cache, _b, _rand

pytestmark = pytest.mark.gpu


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Call:
    """One call's inputs over a cache, its result, and per sequence the mask and
    the keys and values in 64 bits."""

    def __init__(self, seed, lens, Sq, cache, page, Hq=8, Hkv=1, d=256, dtype=BF16, mask="causal",
                 window=0, sinks=0, scale=1.0, room=0):
        if dtype == F32 and cache == BF16:
            cache = F32
        self.c = Cache(seed, lens, page, Hkv, d, cache, room=room)
        self.rng, self.B, self.Sq, self.Hq, self.Hkv, self.d = self.c.rng, len(lens), Sq, Hq, Hkv, d
        self.dtype, self.window, self.sinks, self.scale = dtype, window, sinks, scale
        if cache == E4M3:                            # scales of keys alike
            self.c.k_exp.fill_(120)
        rng, B = self.rng, self.B
        self.q = _rand(rng, (B, Sq, Hq, d), dtype, d ** -0.25)
        self.kn, self.vn = (_rand(rng, (B, Sq, Hkv, d), dtype, d ** -0.25) for _ in range(2))
        self.ar = np.ones((B, Sq), np.uint8)
        self.seg = np.zeros((B, Sq), np.int32)
        if mask == "segments":
            self.ar = (rng.random((B, Sq)) < 0.2).astype(np.uint8)
            self.seg = rng.integers(-1, 3, (B, Sq)).astype(np.int32)
        elif mask == "causal segments":
            self.seg = rng.integers(0, 3, (B, Sq)).astype(np.int32)

    def see(self, b):
        codes = list(zip(np.cumsum(self.ar[b] != 0).tolist(), self.seg[b].tolist()))
        return _cuda(P.mask(int(self.c.lens_np[b]), self.Sq, codes, self.window, self.sinks))

    def rows(self, name, b):
        new = (self.kn if name == "k" else self.vn)[b].double()
        return torch.cat([_cuda(self.c.rows(name, b)), new])

    def run(self):
        b = _b()
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:3], float("nan"), device="cuda")
        b.pi_attn_paged(self.q, self.kn, self.vn, *self.c.args(), _cuda(self.ar),
                        segment_ids=_cuda(self.seg), out=out, lse=lse, softmax_scale=self.scale,
                        window=self.window, sinks=self.sinks, **self.c.exps())
        assert b.pi_attn_read_status() == b.PI_OK
        return out.double(), lse.double()

    def reference(self, b, h, see, keys, vals):
        """(out, sum_j w_j |v_j|, lse) of a head; keys, vals of its kv head."""
        x = (self.q[b, :, h].double() @ keys.T) * self.scale
        x = x.masked_fill(~see, float("-inf"))
        lse = torch.logsumexp(x, 1)
        w = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
        return w @ vals, w @ vals.abs(), lse


# (lengths, new tokens, heads, kv heads, d, page, room): what each exercises
FORMS = [
    ([880, 0, 401, 128], 1, 8, 1, 256, 16, 0),        # decoding, a cluster a sequence
    ([2000] * 32, 1, 8, 1, 256, 64, 0),
    ([16384, 5] + [70] * 10, 1, 8, 1, 256, 64, 0),    # (bf16: the longest that clusters take)
    ([5120, 2999, 70], 1, 8, 1, 256, 32, 0),          # (e4m3: the same)
    ([16384, 3, 9001, 12000], 1, 8, 1, 256, 64, 0),
    ([16000, 3, 9001], 1, 8, 1, 256, 32, 0),          # decoding, pieces and a merge
    ([20000, 17], 4, 4, 2, 256, 128, 0),
    (list(range(0, 520, 4)), 1, 16, 2, 256, 16, 0),   # decoding, equal ranges
    ([880, 816, 0, 77], 51, 8, 1, 256, 64, 0),        # chunks, units whole
    ([9000, 31], 70, 8, 1, 256, 16, 0),               # chunks, units cut
    ([5000, 1, 2500], 300, 8, 2, 256, 256, 0),
    ([16000, 15000], 130, 8, 1, 256, 64, 0),          # (e4m3: rows rebuilt once)
    ([700, 3], 200, 16, 1, 256, 32, 0),
    ([120] * 66, 40, 8, 1, 256, 32, 600),             # two launches
    ([0, 40], 2100, 8, 1, 256, 64, 0),                # a long chunk, cut, over an empty cache
    ([300, 5], 70, 6, 2, 64, 16, 0),                  # CUDA cores
    ([3000, 41], 2, 3, 1, 128, 16, 0),
]
CACHES = [BF16, E4M3]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("mask,window,sinks", [("causal", 0, 0), ("segments", 0, 0), ("causal", 700, 20),
                                               ("causal segments", 0, 0), ("segments", 1000, 130)])
@pytest.mark.parametrize("form", FORMS)
def test_equal_weights_are_exact(form, mask, window, sinks, cache):
    lens, Sq, Hq, Hkv, d, page, room = form
    for dtype in ((BF16,) if d == 256 else (BF16, F32)):
        t = Call(70, lens, Sq, cache, page, Hq, Hkv, d, dtype, mask, window, sinks, room=room)
        t.q.zero_()
        c, g = t.c, torch.Generator(device="cuda").manual_seed(1)
        for x in (c.v, t.vn):
            x.copy_(torch.randint(-8, 9, x.shape, generator=g, device="cuda").float().to(x.dtype))
        if c.v_exp is not None:
            c.v_exp.copy_(torch.randint(125, 130, c.v_exp.shape, generator=g, device="cuda"))
        out, lse = t.run()
        half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
        for b in range(t.B):
            see, vals = t.see(b), t.rows("v", b)
            n = see.sum(1)
            for kv in range(Hkv):
                ref = (see.double() @ vals[:, kv]) / n.clamp(min=1)[:, None]
                tol = (half + 2.0 ** -22) * ref.abs()
                if lens[b] >= 32 and mask == "causal" and window == 0:
                    # one 16-key tile read twice instead of its neighbour would show
                    bad = vals[:, kv].clone()
                    bad[:16] = bad[16:32]
                    bad = (see.double() @ bad) / n.clamp(min=1)[:, None]
                    assert ((bad - ref).abs() > 2 * tol).any(1).all()
                for h in range(kv * (Hq // Hkv), (kv + 1) * (Hq // Hkv)):
                    assert ((out[b, :, h] - ref).abs() <= tol).all(), (b, h)
                    assert (torch.isneginf(lse[b, :, h]) == (n == 0)).all()
                    # log2 within 2^-22 of its value, or of 1
                    err = (lse[b, :, h] - torch.log(n.double()))[n > 0].abs()
                    assert (err <= 2.0 ** -18).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 20)])
@pytest.mark.parametrize("form", FORMS)
def test_every_key_is_found_in_its_place(form, window, sinks, cache):
    lens, Sq, Hq, Hkv, d, page, room = form
    # (a target's score is about 16 at least, the others' spread 2 at most)
    t = Call(71, lens, Sq, cache, page, Hq, Hkv, d, window=window, sinks=sinks,
             scale=2.0 * (256 / d) ** 0.5, room=room)
    G = Hq // Hkv
    sees = [t.see(b) for b in range(t.B)]
    keys, vals = ([t.rows(name, b) for b in range(t.B)] for name in ("k", "v"))
    # first and last key of every 16-key tile, and the new keys
    spots = []
    for n in lens:
        x = np.arange(n + Sq)
        spots.append(x[(x % 16 == 0) | (x % 16 == 15) | (x >= n - 1)])
    passes = min(max(-(-len(s) // (Sq * Hq)) for s in spots), 24)
    wrong = 0
    for turn in range(passes):
        aims = []
        for b in range(t.B):
            aim = np.zeros((Sq, Hq), np.int64)
            see = sees[b].cpu().numpy()
            for i in range(Sq):
                may = spots[b][see[i, spots[b]]]
                at = (turn * Sq + i) * Hq + np.arange(Hq)     # evenly over them all
                aim[i] = may[at * len(may) // (passes * Sq * Hq)]
            aim = _cuda(aim)
            aims.append(aim)
            for h in range(Hq):
                t.q[b, :, h] = keys[b][aim[:, h], h // G].to(BF16)
        out, _ = t.run()
        qn = float(t.q.double().norm(dim=-1).max())
        for b in range(t.B):
            delta = 2.0 ** -15 * qn * float(keys[b].norm(dim=-1).max()) * t.scale
            n = len(keys[b])
            for h in range(Hq):
                ref, size, _ = t.reference(b, h, sees[b], keys[b][:, h // G], vals[b][:, h // G])
                tol = (2.0 ** -8 + 2 * delta + n * 2.0 ** -22 + 2.0 ** -14) * size + 2.0 ** -8 * ref.abs()
                assert ((out[b, :, h] - ref).abs() <= tol).all(), (turn, b, h)
                # the next tile's rows in the target's place would be seen
                far = vals[b][(aims[b][:, h] + 16) % n, h // G]
                wrong += int(((out[b, :, h] - far).abs() <= tol).all(1).sum()) if n > 32 else 0
    assert wrong == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("mask,window,sinks", [("causal", 0, 0), ("segments", 1000, 130)])
@pytest.mark.parametrize("form", FORMS)
def test_every_element_within_its_bound(form, mask, window, sinks, cache):
    lens, Sq, Hq, Hkv, d, page, room = form
    for dtype in ((BF16,) if d == 256 else (BF16, F32)):
        t = Call(72, lens, Sq, cache, page, Hq, Hkv, d, dtype, mask, window, sinks, room=room)
        out, lse = t.run()
        qn = float(t.q.double().norm(dim=-1).max())
        p_half, o_half = (2.0 ** -8, 2.0 ** -8) if dtype == BF16 else (0.0, 2.0 ** -24)
        caught = 0
        for b in range(t.B):
            see, keys, vals = t.see(b), t.rows("k", b), t.rows("v", b)
            delta = 2.0 ** -15 * qn * float(keys.norm(dim=-1).max())
            n = len(keys)
            for h in range(Hq):
                k, v = keys[:, h // (Hq // Hkv)], vals[:, h // (Hq // Hkv)]
                ref, size, ref_lse = t.reference(b, h, see, k, v)
                tol = (p_half + 2 * delta + n * 2.0 ** -22 + 2.0 ** -14) * size + o_half * ref.abs()
                assert ((out[b, :, h] - ref).abs() <= tol).all(), (b, h)
                some = see.any(1)
                assert (torch.isneginf(lse[b, :, h]) == ~some).all()
                err = (lse[b, :, h] - ref_lse)[some].abs()
                assert (err <= delta + n * 2.0 ** -22 + 2.0 ** -14).all()
                # a cache whose first 128-key tile holds the second's values
                if h == 0 and 256 <= lens[b] <= 5000 and window == 0:
                    other = v.clone()
                    other[:128], other[128:256] = v[128:256], v[:128]
                    bad, size, _ = t.reference(b, h, see, k, other)
                    caught += int(((out[b, :, h] - bad).abs() > tol).any()) - 1
        assert caught == 0
