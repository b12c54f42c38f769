"""The paged-cache operators of this library, as cases to measure.

Three operators share one paged key/value cache:

* ``write``   new tokens' keys and values go into the pages of their sequences,
              as they are or as e4m3 with one power-of-two scale per vector;
* ``read``    a sequence's cached rows come back as dense tensors;
* ``attend``  a chunk of new tokens (one token in decoding) attends to its
              sequence's cached keys and to the chunk itself under the
              prefix-LM rule, with an optional sliding window and sink tokens.

``own = False`` computes them with elementary torch operations in 32 bits;
``own = True`` makes the library's calls.  Head geometry, batch sizes and
lengths are those of this repository's workloads (8 query heads, 1 key/value
head, head_dim 256; prefixes of 816 and 824 tokens, 51 suffix tokens, decode
caches of 880) and of its largest tests (16000 cached keys).
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}


# ------------------------------------------------------------------ the cases

def _write(name, B, Sq, cache, page, cap, dtype="bf16", Hkv=1, d=256, masked=False):
    return {"name": name, "op": "write", "B": B, "Sq": Sq, "Hkv": Hkv, "d": d, "dtype": dtype,
            "cache": cache, "page": page, "cap": cap, "masked": masked}


def _read(name, B, cap, cache, page, dtype="bf16", Hkv=1, d=256):
    return {"name": name, "op": "read", "B": B, "cap": cap, "Hkv": Hkv, "d": d, "dtype": dtype,
            "cache": cache, "page": page}


def _attend(name, B, Sq, cap, min_len, cache, page, mask, dtype="bf16", Hq=8, Hkv=1, d=256,
            window=0, sinks=0):
    return {"name": name, "op": "attend", "B": B, "Sq": Sq, "cap": cap, "min_len": min_len,
            "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "cache": cache, "page": page,
            "mask": mask, "window": window, "sinks": sinks}


def listed():
    return [
        # one decoded token of each of 32 sequences is appended
        _write("write_token_b32", 32, 1, "e4m3", 16, 880),
        # the prefixes of 32 robots enter the cache, prompts padded to one length
        _write("write_prefix_b32", 32, 824, "e4m3", 64, 880, masked=True),
        # a joint forward's keys and values kept as they are
        _write("write_joint_bf16_b8", 8, 611, "bf16", 32, 1000),
        # cached prefixes handed to the dense entry points
        _read("read_prefix_b32", 32, 880, "e4m3", 16),
        # long sessions read back
        _read("read_long_b4", 4, 16000, "bf16", 64),
        # one robot decodes one token: the smallest call, latency counts
        _attend("decode_b1", 1, 1, 880, 880, "bf16", 16, "causal"),
        # ragged decoding of a batch against an 8-bit cache
        _attend("decode_b32", 32, 1, 880, 400, "e4m3", 16, "causal"),
        # decoding in long sessions
        _attend("decode_long_b16", 16, 1, 16000, 12000, "bf16", 64, "causal"),
        # one Euler step's suffix tokens against ragged prefixes
        _attend("suffix_b32", 32, 51, 816, 700, "bf16", 64, "suffix"),
        # a long prompt's next chunk against an 8-bit cache
        _attend("chunk_long_b4", 4, 512, 16000, 15000, "e4m3", 64, "causal"),
        # a padded batch of observation chunks in a stream: the instruction's
        # tokens stay visible, old observations leave the window
        _attend("stream_window_b8", 8, 256, 16000, 8000, "bf16", 32, "padded", Hq=8, Hkv=2,
                window=2048, sinks=64),
        # the fp32 form at the tiny joint workload's sizes
        _attend("tiny_f32", 1, 9, 40, 40, "f32", 16, "suffix", dtype="f32", Hq=2, d=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 1, 1, 2])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "write":
        Sq = _log(rng, 1, 1000)
        c = _write("", _log(rng, 1, 32), Sq, cache, page, Sq + rng.randint(0, 300), Hkv=Hkv,
                   masked=rng.random() < 0.5)
    elif op == "read":
        B = _log(rng, 1, 32)
        c = _read("", B, _log(rng, 17, min(16000, 64000 // B)), cache, page, Hkv=Hkv)
    else:
        kind = rng.choice(["decode", "decode", "chunk", "chunk", "tiny"])
        if kind == "tiny":
            cap = _log(rng, 1, 100)
            c = _attend("", rng.randint(1, 4), _log(rng, 1, 16), cap, rng.randint(0, cap), "f32",
                        page, rng.choice(["suffix", "causal", "padded"]), dtype="f32",
                        Hq=rng.choice([2, 4]), Hkv=rng.choice([1, 2]), d=64)
        else:
            B = _log(rng, 1, 32)
            Sq = 1 if kind == "decode" else _log(rng, 2, 512)
            # cost at most the long chunk's: 4 * 512 queries of 16000 keys
            cap = _log(rng, 100, min(16000, 256000 // B, max(400, 4 * 512 * 16000 // (B * Sq))))
            mask = "causal" if kind == "decode" else rng.choice(["suffix", "causal", "padded"])
            window, sinks = 0, 0
            if rng.random() < 0.3:
                window, sinks = _log(rng, 64, 4000), rng.choice([0, 4, 64])
            c = _attend("", B, Sq, cap, rng.randint(cap // 2, cap), cache, page, mask,
                        Hq=8, Hkv=Hkv, window=window, sinks=sinks)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _values(g, shape, d, dtype):
    """The repository's distribution of q, k and v: N(0, 1) * d**-0.25."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * d ** -0.25
    return x.to(dtype)


def _table(g, B, cap, page):
    """Every sequence's pages, scattered over the pool."""
    per = -(-cap // page)
    perm = torch.randperm(B * per, generator=g, device=DEV)
    return perm.view(B, per).to(torch.int32)


def _filled(g, c, num_pages):
    """A pool whose every slot holds a vector, in the cache's type."""
    shape = (num_pages, c["page"], c["Hkv"], c["d"])
    x = _values(g, shape, c["d"], torch.float32)
    # token norms differ, as keys' and values' do, so that the scales do too
    x *= torch.exp2(torch.randint(-2, 3, shape[:3], generator=g, device=DEV).float())[..., None]
    if c["cache"] != "e4m3":
        return x.to(DTYPES[c["cache"]]), None
    return _quantised(x)


def prepare(case, seed):
    c = case
    g = _generator(seed)
    B, page, cap = c["B"], c["page"], c["cap"]
    dtype = DTYPES[c["dtype"]]
    s = {"case": c, "page_table": _table(g, B, cap, page)}
    num_pages = s["page_table"].numel()
    if c["op"] == "write":
        Sq = c["Sq"]
        shape = (B, Sq, c["Hkv"], c["d"])
        s["k"], s["v"] = (_values(g, shape, c["d"], dtype) for _ in range(2))
        s["cache_lens"] = torch.randint(0, cap - Sq + 1, (B,), generator=g, device=DEV).int()
        s["token_mask"] = None
        if c["masked"]:
            # images, a prompt padded to its room, then more tokens
            room = min(48, Sq)
            used = torch.randint(room // 2, room + 1, (B, 1), generator=g, device=DEV)
            t = torch.arange(Sq, device=DEV)[None]
            s["token_mask"] = (~((t >= Sq // 2 + used) & (t < Sq // 2 + room))).to(torch.uint8)
        pool = (num_pages, page, c["Hkv"], c["d"])
        s["k_exp"] = s["v_exp"] = None
        if c["cache"] == "e4m3":
            s["k_pages"], s["v_pages"] = (torch.zeros(pool, device=DEV, dtype=torch.uint8).view(E4M3)
                                          for _ in range(2))
            s["k_exp"], s["v_exp"] = (torch.full(pool[:3], 127, device=DEV, dtype=torch.uint8)
                                      for _ in range(2))
        else:
            s["k_pages"], s["v_pages"] = (torch.zeros(pool, device=DEV, dtype=DTYPES[c["cache"]])
                                          for _ in range(2))
        s["lens_out"] = torch.empty(B, device=DEV, dtype=torch.int32)
        return s
    s["k_pages"], s["k_exp"] = _filled(g, c, num_pages)
    s["v_pages"], s["v_exp"] = _filled(g, c, num_pages)
    low = c["cap"] // 2 if c["op"] == "read" else c["min_len"]
    s["cache_lens"] = torch.randint(low, cap + 1, (B,), generator=g, device=DEV).int()
    if c["op"] == "read":
        return s
    Sq, Hq, Hkv, d = c["Sq"], c["Hq"], c["Hkv"], c["d"]
    s["q"] = _values(g, (B, Sq, Hq, d), d, dtype)
    s["k_new"], s["v_new"] = (_values(g, (B, Sq, Hkv, d), d, dtype) for _ in range(2))
    s["segment_ids"] = None
    if c["mask"] == "causal":
        s["ar_mask"] = torch.ones(Sq, device=DEV, dtype=torch.uint8)
    elif c["mask"] == "suffix":
        # one state token, then the action tokens as one block
        s["ar_mask"] = (torch.arange(Sq, device=DEV) < 2).to(torch.uint8)
    else:
        # each sequence's own blocks, its last tokens padding
        u = torch.rand((B, Sq), generator=g, device=DEV)
        s["ar_mask"] = (u < 0.1).to(torch.uint8)
        used = torch.randint((Sq + 1) // 2, Sq + 1, (B, 1), generator=g, device=DEV)
        pad = torch.arange(Sq, device=DEV)[None] >= used
        s["segment_ids"] = -pad.to(torch.int32)
    return s


# -------------------------------------------------------------- the plain form

def _quantised(x):
    """x in e4m3 with the smallest power-of-two scale that keeps every vector's
    largest magnitude at or below 448, as (values, biased exponents)."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(min=-126)
    y = torch.ldexp(x, -e[..., None]).clamp(-448, 448)
    return y.to(E4M3), (e + 127).to(torch.uint8)


def _plain_write(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    B, Sq = k.shape[:2]
    mask = s["token_mask"]
    mask = torch.ones((B, Sq), device=DEV, dtype=torch.bool) if mask is None else mask != 0
    rank = mask.long().cumsum(1) - 1
    at = s["cache_lens"].long()[:, None] + rank
    mask = mask & (at < s["page_table"].shape[1] * c["page"])
    b, t = mask.nonzero(as_tuple=True)
    at = at[b, t]
    slot = s["page_table"].long()[b, at // c["page"]] * c["page"] + at % c["page"]
    for x, pages, exps in ((k, s["k_pages"], s["k_exp"]), (v, s["v_pages"], s["v_exp"])):
        x = x[b, t]
        if exps is None:
            pages.flatten(0, 1)[slot] = x.to(pages.dtype)
        else:
            y, e = _quantised(x)
            pages.view(torch.uint8).flatten(0, 1)[slot] = y.view(torch.uint8)
            exps.flatten(0, 1)[slot] = e
    s["lens_out"].copy_(s["cache_lens"] + mask.sum(1))


def _gathered(s, pages, exps):
    """[B, max_pages * page, Hkv, d] in fp32, rows past the length zero."""
    t = s["page_table"].long()
    if exps is None:
        x = pages[t].float()
    else:
        x = pages.view(torch.uint8)[t].view(E4M3).float()
        x = torch.ldexp(x, exps[t].int()[..., None] - 127)
    x = x.flatten(1, 2)
    live = torch.arange(x.shape[1], device=DEV)[None] < s["cache_lens"][:, None]
    return x * live[..., None, None], live


def _plain_read(s):
    c = s["case"]
    cap, dtype = c["cap"], DTYPES[c["dtype"]]
    k, live = _gathered(s, s["k_pages"], s["k_exp"])
    v, _ = _gathered(s, s["v_pages"], s["v_exp"])
    return {"k": k[:, :cap].to(dtype), "v": v[:, :cap].to(dtype),
            "valid": live[:, :cap].to(torch.uint8)}


def _visible(s, P):
    """[B, Sq, P + Sq]: which cached and which new keys each query sees."""
    c = s["case"]
    Sq = c["Sq"]
    ar = s["ar_mask"].long()
    cs = ar.cumsum(-1).expand(c["B"], Sq)
    new = cs[:, None, :] <= cs[:, :, None]
    lens = s["cache_lens"].long()
    cached = torch.arange(P, device=DEV)[None] < lens[:, None]
    cached = cached[:, None, :].expand(c["B"], Sq, P)
    see = torch.cat([cached, new], 2)
    if s["segment_ids"] is not None:
        ok = s["segment_ids"] >= 0
        see = see & ok[:, :, None]
        see = see & torch.cat([torch.ones((c["B"], P), device=DEV, dtype=torch.bool), ok],
                              1)[:, None, :]
    if c["window"] > 0:
        i = torch.arange(Sq, device=DEV)
        at = lens[:, None] + i[None]
        key = torch.cat([torch.arange(P, device=DEV)[None].expand(c["B"], P), at], 1)
        near = at[:, :, None] - key[:, None, :] < c["window"]
        see = see & (near | (key < c["sinks"])[:, None, :])
    return see


def _plain_attend(s):
    c = s["case"]
    B, Sq, Hq, Hkv, d = c["B"], c["Sq"], c["Hq"], c["Hkv"], c["d"]
    k, _ = _gathered(s, s["k_pages"], s["k_exp"])
    v, _ = _gathered(s, s["v_pages"], s["v_exp"])
    P = k.shape[1]
    k = torch.cat([k, s["k_new"].float()], 1)
    v = torch.cat([v, s["v_new"].float()], 1)
    q = s["q"].float().view(B, Sq, Hkv, Hq // Hkv, d)
    x = torch.einsum("bqhgd,bkhd->bhgqk", q, k)
    x = x.masked_fill(~_visible(s, P)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1)
    out = torch.einsum("bhgqk,bkhd->bqhgd", p, v)
    lq = l.permute(0, 3, 1, 2)[..., None]
    out = torch.where(lq > 0, out / lq, torch.zeros_like(out))
    lse = (m[..., 0] + torch.log(l)).permute(0, 3, 1, 2)
    return {"out": out.reshape(B, Sq, Hq, d).to(s["q"].dtype),
            "lse": lse.reshape(B, Sq, Hq).contiguous()}


def run(state):
    s = state
    c = s["case"]
    if own:
        from vla_prefix_lm_b200 import binding as pi
        if c["op"] == "write":
            pi.pi_attn_cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"],
                                   s["cache_lens"], token_mask=s["token_mask"], k_exp=s["k_exp"],
                                   v_exp=s["v_exp"], lens_out=s["lens_out"])
        elif c["op"] == "read":
            k, v, valid = pi.pi_attn_cache_read(s["k_pages"], s["v_pages"], s["page_table"],
                                                s["cache_lens"], c["cap"],
                                                dtype=DTYPES[c["dtype"]], k_exp=s["k_exp"],
                                                v_exp=s["v_exp"])
            return {"k": k, "v": v, "valid": valid}
        else:
            lse = torch.empty(s["q"].shape[:3], device=DEV, dtype=torch.float32)
            out = pi.pi_attn_paged(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"],
                                   s["page_table"], s["cache_lens"], s["ar_mask"],
                                   segment_ids=s["segment_ids"], k_exp=s["k_exp"],
                                   v_exp=s["v_exp"], lse=lse, window=c["window"],
                                   sinks=c["sinks"])
            return {"out": out, "lse": lse}
    elif c["op"] == "write":
        _plain_write(s)
    elif c["op"] == "read":
        return _plain_read(s)
    else:
        return _plain_attend(s)
    got = {"k": s["k_pages"], "v": s["v_pages"], "lens": s["lens_out"]}
    if s["k_exp"] is not None:
        got.update(k_exp=s["k_exp"], v_exp=s["v_exp"])
    return got


# ------------------------------------------------------- the definition, 64 bits

def _grid_e4m3(x):
    """The e4m3 value nearest each of x (ties to even), |x| <= 448, in 64 bits."""
    a = x.abs()
    # steps: 2^-9 below 2^-6, else 2^(floor(log2 a) - 3)
    _, e = torch.frexp(a)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.sign(x) * torch.round(a / step) * step


def _exact_write(s):
    c = s["case"]
    page, B, Sq = c["page"], c["B"], c["Sq"]
    lens = s["cache_lens"].tolist()
    table = s["page_table"].tolist()
    mask = None if s["token_mask"] is None else s["token_mask"].tolist()
    src, dst, after = [], [], []
    for b in range(B):
        at = lens[b]
        for t in range(Sq):
            if (mask is None or mask[b][t]) and at < len(table[b]) * page:
                src.append(b * Sq + t)
                dst.append(table[b][at // page] * page + at % page)
                at += 1
        after.append(at)
    src = torch.tensor(src, device=DEV, dtype=torch.long)
    dst = torch.tensor(dst, device=DEV, dtype=torch.long)
    got = {"lens": torch.tensor(after, device=DEV, dtype=torch.int32)}
    for name in ("k", "v"):
        x = s[name].double().flatten(0, 1)[src]
        pool = torch.zeros_like(s[name + "_pages"], dtype=torch.float64)
        if c["cache"] == "e4m3":
            top = x.abs().amax(-1)
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126, max=120)
            # the logarithm is rounded: settle the exponent by comparing
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
            e = torch.where(top == 0, torch.zeros_like(e), e)
            pool.flatten(0, 1)[dst] = _grid_e4m3(x / torch.exp2(e)[..., None])
            exps = torch.full(pool.shape[:3], 127, device=DEV, dtype=torch.uint8)
            exps.flatten(0, 1)[dst] = (e + 127).to(torch.uint8)
            got[name + "_exp"] = exps
        else:
            pool.flatten(0, 1)[dst] = x
        got[name] = pool
    return got


def _rows64(s, name, b, n):
    """Sequence b's first n cached rows in 64 bits, page by page."""
    page = s["case"]["page"]
    pages = s["page_table"][b, :-(-n // page)].long() if n else s["page_table"][b, :0].long()
    raw, exps = s[name + "_pages"], s[name + "_exp"]
    if exps is None:
        x = raw.index_select(0, pages).double()
    else:
        x = raw.view(torch.uint8).index_select(0, pages).view(E4M3).double()
        x = x * torch.exp2(exps.index_select(0, pages).double() - 127.0)[..., None]
    return x.reshape(-1, *raw.shape[2:])[:n]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "write":
        return _exact_write(s)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    lens = s["cache_lens"].tolist()
    if c["op"] == "read":
        got = {"valid": torch.zeros((B, c["cap"]), device=DEV, dtype=torch.uint8)}
        for name in ("k", "v"):
            got[name] = torch.zeros((B, c["cap"], Hkv, d), device=DEV, dtype=torch.float64)
            for b in range(B):
                got[name][b, :lens[b]] = _rows64(s, name, b, lens[b])
                got["valid"][b, :lens[b]] = 1
        return got
    Sq, Hq = c["Sq"], c["Hq"]
    G = Hq // Hkv
    out = torch.zeros((B, Sq, Hq, d), device=DEV, dtype=torch.float64)
    lse = torch.full((B, Sq, Hq), -math.inf, device=DEV, dtype=torch.float64)
    i = torch.arange(Sq, device=DEV)
    for b in range(B):
        n = lens[b]
        ar = s["ar_mask"] if s["ar_mask"].dim() == 1 else s["ar_mask"][b]
        block = torch.cumsum(ar.long(), 0)
        pos = torch.arange(n + Sq, device=DEV)
        see = torch.ones((Sq, n + Sq), device=DEV, dtype=torch.bool)
        see[:, n:] = block[None, :] <= block[:, None]
        if s["segment_ids"] is not None:
            pad = s["segment_ids"][b] < 0
            see[pad] = False
            see[:, n:][:, pad] = False
        if c["window"] > 0:
            far = (n + i)[:, None] - pos[None, :] >= c["window"]
            see &= ~(far & (pos >= c["sinks"])[None, :])
        keys = torch.cat([_rows64(s, "k", b, n), s["k_new"][b].double()])
        vals = torch.cat([_rows64(s, "v", b, n), s["v_new"][b].double()])
        for h in range(Hq):
            x = s["q"][b, :, h].double() @ keys[:, h // G].T
            x[~see] = -math.inf
            z = torch.logsumexp(x, 1)
            some = see.any(1)
            lse[b, :, h] = z
            w = torch.exp(x - torch.where(some, z, torch.zeros_like(z))[:, None])
            out[b, :, h] = w @ vals[:, h // G]
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------- the work

def _row_bytes(c):
    """One cached vector: its values, and its exponent where it has one."""
    return c["d"] + 1 if c["cache"] == "e4m3" else c["d"] * (2 if c["cache"] == "bf16" else 4)


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "write":
        n = B * c["Sq"] * Hkv * 2
        return {"bytes": n * (d * size + _row_bytes(c)) + 12 * B, "flops": 0}
    if c["op"] == "read":
        n = B * 0.75 * c["cap"] * Hkv * 2
        return {"bytes": n * _row_bytes(c) + B * c["cap"] * (Hkv * 2 * d * size + 1), "flops": 0}
    Sq, Hq = c["Sq"], c["Hq"]
    mean = 0.5 * (c["min_len"] + c["cap"])
    # keys a query sees, and cached rows that some query of the chunk sees
    seen = rows = mean
    new = Sq if c["mask"] == "suffix" else (Sq + 1) / 2
    live = 1.0 if c["mask"] != "padded" else 0.75
    if c["window"] > 0:
        seen = min(mean, c["window"] + c["sinks"])
        rows = min(mean, c["window"] + c["sinks"] + Sq)
        new = min(new, c["window"])
    return {"bytes": B * (2 * rows * Hkv * _row_bytes(c) + 2 * Sq * Hkv * d * size
                          + 2 * Sq * Hq * d * size + 4 * Sq * Hq),
            "flops": 4.0 * B * Sq * live * Hq * d * (seen + new)}
