"""What is measured of the operators that make a KV cache smaller: appending to a
cache held in 4 bits (e2m1 codes; keys with a scale for every 32 channels, values
with one for each token and head), decode attention over it, the attention weight
that every key of a bf16 cache has gathered, and eviction of the keys that gathered
least.

A case is a dict of plain values.  `run` computes a case in elementary torch
operations in 32 bits (angles in 64), or, where `own` is true, calls the
framework.  `exact` is the operators' definition in 64 bits, written apart.

Shapes are those of the framework's own workloads (32 query heads on 8 KV heads
of 128 channels, pages of 128) and generic ones around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # the e2m1 numbers; codes 8 to 15 are negative
KMIN, KMAX = -60, 125                               # exponents of the appended scales
MOST_SCORES = 600_000_000                           # of a drawn batch, padded


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    app = dict(op="append4", hq=32, hkv=8, rot=128, interleaved=False, norm=False, ctx=1024,
               page=128, head_major=True, lens=2)
    dec = dict(op="decode4", hq=32, hkv=8, q_rows=1, sink=False, page=128, head_major=True, lens=2)
    wei = dict(op="weights", hq=32, hkv=8, dim=128, q_rows=1, causal=True, decay=1.0, page=128,
               head_major=False, lens=2)
    evi = dict(op="evict", hkv=8, dim=128, page=128, first=4, recent=128, head_major=False, lens=2)
    return [
        # a decode step of 64 sequences
        dict(app, name="append4_b64", batch=64, q_rows=1),
        # ragged prompts mixed with decoding sequences, heads normed; the prompts' own attention
        # reads the values that come back
        dict(app, name="append4_prompts", batch=16, q_rows=4096, ctx=512, norm=True,
             head_major=False, lens=5),
        # two short sequences: latency
        dict(dec, name="decode4_short", batch=2, hq=4, hkv=1, len_lo=37, len_hi=100, page=64, lens=1),
        # a decode step of 64 ragged sequences
        dict(dec, name="decode4_b64", batch=64, len_lo=512, len_hi=8192),
        # one sequence of 131072 tokens, with sinks
        dict(dec, name="decode4_long", batch=1, len_lo=131072, len_hi=131072, sink=True, lens=3),
        # draft rows being verified, a token's heads side by side
        dict(dec, name="decode4_draft", batch=64, q_rows=4, len_lo=512, len_hi=4096,
             head_major=False, lens=6),
        # after a decode step of 64 sequences: the weight of its row on every key
        dict(wei, name="weights_b64", batch=64, len_lo=512, len_hi=8192),
        # after ragged prompts: the weight of all their rows
        dict(wei, name="weights_prompts", batch=4, q_rows=4096, len_lo=1024, len_hi=4096, lens=5),
        # draft rows of one long sequence, earlier weights fading
        dict(wei, name="weights_long", batch=1, q_rows=3, len_lo=131072, len_hi=131072, decay=0.98,
             lens=7),
        # two short sequences: latency
        dict(evi, name="evict_short", batch=2, hkv=1, len_lo=150, len_hi=300, keep=0.5, page=64,
             first=1, recent=16, lens=1),
        # prompts cut to a quarter before decoding starts
        dict(evi, name="evict_prompts", batch=16, len_lo=1024, len_hi=8192, keep=0.25),
        # one long sequence cut to an eighth
        dict(evi, name="evict_long", batch=1, len_lo=131072, len_hi=131072, keep=0.125, lens=3),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append4", "decode4", "decode4", "weights", "weights", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hkv=hkv, page=rng.choice([16, 32, 64, 128, 256]),
             head_major=rng.random() < 0.5, lens=rng.randrange(1, 1 << 20),
             batch=_log(rng, 1, 64))
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op == "append4":
        c.update(hq=hq, rot=rng.choice([128, 64, 32]), interleaved=rng.random() < 0.5,
                 norm=rng.random() < 0.5, ctx=_log(rng, 1, 1024))
        c["q_rows"] = rng.choice([1, rng.randint(2, 8), _log(rng, 1, max(1, 16384 // c["batch"]))])
        return c
    if op == "decode4":
        hi = _log(rng, 1, max(1, min(131072, 64 * 4096 // c["batch"])))
        c.update(hq=hq, q_rows=rng.choice([1, 1, rng.randint(1, 16 * hkv // hq)]),
                 sink=rng.random() < 0.5)
    elif op == "weights":
        hi = _log(rng, 1, max(1, min(131072, 64 * 4096 // c["batch"])))
        most = max(1, min(hi, MOST_SCORES // (c["batch"] * hq * hi), 4096))
        c.update(hq=hq, dim=rng.choice([64, 128]), causal=rng.random() < 0.8,
                 decay=rng.choice([1.0, 0.9]),
                 q_rows=rng.choice([1, min(most, rng.randint(1, 16)), _log(rng, 1, most)]))
    else:
        dim = rng.choice([64, 128, 256])
        hi = _log(rng, 1, max(1, min(131072, (1 << 26) // (c["batch"] * hkv * dim))))
        c.update(dim=dim, first=rng.choice([0, 1, 4]),
                 recent=_log(rng, 1, 256), keep=rng.choice([0.125, 0.25, 0.5, 0.9]))
    c.update(len_lo=max(1, hi // rng.choice([1, 2, 16])), len_hi=hi)
    return c


def _lengths(case):
    """(query rows, keys) per sequence: from the case alone."""
    rng = random.Random(case["lens"])
    b, n = case["batch"], case.get("q_rows", 1)
    if case["op"] == "append4":     # long runs are mixed with single rows
        rows = [1 if n == 1 or (n > 8 and i % 2) else rng.randint(max(1, n // 8), n)
                for i in range(b)]
        return rows, [r + rng.randint(0, case["ctx"]) for r in rows]
    keys = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(b)]
    if n > 16:      # prompts: all of a sequence's rows, up to q_rows
        return [min(n, k) for k in keys], keys
    rows = [1 if n == 1 else rng.randint(1, n) for _ in range(b)]
    return rows, [max(r, k) for r, k in zip(rows, keys)]


def _kept(case):
    return [max(1, int(k * case["keep"])) for k in _lengths(case)[1]]


def work(case):
    rows, keys = _lengths(case)
    op, hkv, n, tokens = case["op"], case["hkv"], sum(rows), sum(keys)
    if op == "append4":
        hq = case["hq"]
        # q in and out, k and v in, their values out, codes and scales
        return {"bytes": n * (512 * hq + hkv * (4 * 256 + 2 * 64 + 8)),
                "flops": 10 * n * (hq + 2 * hkv) * 128}
    if op == "decode4":
        pairs = sum(r * k for r, k in zip(rows, keys))
        return {"bytes": tokens * hkv * (2 * 64 + 8) + n * case["hq"] * (4 * 128 + 4),
                "flops": 4 * pairs * case["hq"] * 128}
    if op == "weights":
        seen = sum(r * k - (r * (r - 1) // 2 if case["causal"] else 0) for r, k in zip(rows, keys))
        return {"bytes": tokens * hkv * (2 * case["dim"] + 4) +
                (tokens - n) * hkv * 4 + n * case["hq"] * (2 * case["dim"] + 4),
                "flops": (2 * case["dim"] + 4) * seen * case["hq"]}
    kept = sum(_kept(case))
    return {"bytes": 4 * tokens * hkv + kept * hkv * (8 * case["dim"] + 4 + 4),
            "flops": 4 * tokens * hkv}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _table(pages, host):
    order = list(range(sum(pages)))
    host.shuffle(order)
    table = torch.zeros((len(pages), max(pages)), dtype=torch.int32)
    at = 0
    for i, m in enumerate(pages):
        table[i, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return table.to(DEV)


def _in_layout(x, case):
    """[pages, page, heads, ...] with a head's tokens side by side, where the case wants it."""
    return x.transpose(1, 2).contiguous().transpose(1, 2) if case["head_major"] else x


def _exponent(amax):
    """The least e with amax <= 6 * 2^e (6 is the largest e2m1 number, 0.75 * 2^3)."""
    m, e = torch.frexp(amax)
    k = e - 3 + (m > 0.75).to(e.dtype)
    return torch.where(amax > 0, k, KMIN).clamp(KMIN, KMAX)


def _codes(x):
    """The codes of e2m1 numbers nearest to x (ties to even codes)."""
    a = x.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() +
         (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return torch.where(x < 0, c + 8, c)


def _numbers(codes, dtype=torch.float32):
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=dtype, device=codes.device)
    return grid[codes.long()]


def _held(x, groups):
    """x [..., 128] in 4 bits: codes, exponents of `groups` scales, and the values they stand for."""
    y = x.unflatten(-1, (groups, 128 // groups))
    e = _exponent(y.abs().amax(-1))
    s = torch.exp2(e.float())[..., None]
    c = _codes(y / s)
    return c.flatten(-2), e, (_numbers(c) * s).flatten(-2)


def _packed(codes):
    """Two codes to a byte, the even channel in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def _unpacked(codes, dtype=torch.float32):
    return _numbers(torch.stack([codes & 15, codes >> 4], -1).flatten(-2), dtype)


def _caches4(case, pages, g, st):
    shape = (pages, case["page"], case["hkv"], 128)
    for name in ("kc", "vc"):
        x = torch.randn(shape, generator=g, device=DEV)
        if name == "kc":        # a few channels of keys are far larger than the rest
            x *= 1 + 7 * (torch.rand((1, 1, case["hkv"], 128), generator=g, device=DEV) < 0.03)
        codes, e, _ = _held(x, 4 if name == "kc" else 1)
        st[name] = _in_layout(_packed(codes), case)
        s = (e + 127).to(torch.uint8) if name == "kc" else torch.exp2(e[..., 0].float())
        s = _in_layout(s, case)
        st[name + "_s"] = s.view(torch.float8_e8m0fnu) if name == "kc" else s
        del x, codes


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    host = random.Random(seed)
    op, hkv, page = case["op"], case["hkv"], case["page"]
    rows, keys = _lengths(case)
    n = sum(rows)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)   # noqa: E731
    pages = [-(-k // page) for k in keys]
    st = {"case": case, "table": _table(pages, host), "max_kv": max(keys), "max_q": max(rows),
          "kv_len": torch.tensor(keys, dtype=torch.int32, device=DEV), "offs": None}
    if case.get("q_rows", 1) > 1:
        st["offs"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)],
                                  dtype=torch.int32, device=DEV)
    if op == "append4":
        hq = case["hq"]
        # the projection's output: q, k and v of a row side by side
        packed = randn(n, hq + 2 * hkv, 128).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
        st["q_norm"] = (1 + 0.1 * randn(128)).to(torch.bfloat16) if case["norm"] else None
        st["k_norm"] = (1 + 0.1 * randn(128)).to(torch.bfloat16) if case["norm"] else None
        freq = [500000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        # the same as a fraction of a turn per position, in units of 2^-64
        t = [int(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
        st["turns"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in t], dtype=torch.int64,
                                   device=DEV)
        empty = lambda h: torch.empty((n, h, 128), dtype=torch.bfloat16, device=DEV)   # noqa: E731
        st["q_out"], st["k_out"], st["v_out"] = empty(hq), empty(hkv), empty(hkv)
        _caches4(case, sum(pages), g, st)
        return st
    if op == "decode4":
        st["q"] = randn(n, case["hq"], 128).to(torch.bfloat16)
        st["scale"] = float(torch.tensor(1 / math.sqrt(128), dtype=torch.float32))
        st["sink"] = randn(case["hq"]) if case["sink"] else None
        _caches4(case, sum(pages), g, st)
        return st
    dim = case["dim"]
    st["kc"] = _in_layout(randn(sum(pages), page, hkv, dim).to(torch.bfloat16), case)
    # what earlier steps gathered: a few keys hold most of the weight, some weigh the same
    w = torch.exp(2 * randn(sum(pages), page, hkv))
    w = torch.where(w < 0.2, torch.round(w * 64) / 64, w)
    st["w"] = _in_layout(w, case)
    if op == "weights":
        st["q"] = randn(n, case["hq"], dim).to(torch.bfloat16)
        st["scale"] = float(torch.tensor(1 / math.sqrt(dim), dtype=torch.float32))
        st["lse"] = torch.empty((n, case["hq"]), device=DEV)       # as the attention before leaves it
        r0 = 0
        for b, (r, L) in enumerate(zip(rows, keys)):
            kb = st["kc"][st["table"][b, :pages[b]].long()].flatten(0, 1)[:L].float()
            q = st["q"][r0:r0 + r].float().view(r, hkv, -1, dim)
            s = torch.einsum("rhgd,thd->hgrt", q, kb) * st["scale"]
            if case["causal"]:
                s.masked_fill_(torch.ones((r, L), dtype=torch.bool, device=DEV).triu(L - r + 1),
                               -math.inf)
            st["lse"][r0:r0 + r] = torch.logsumexp(s, -1).permute(2, 0, 1).flatten(1)
            r0 += r
            del s
        return st
    st["vc"] = _in_layout(randn(sum(pages), page, hkv, dim).to(torch.bfloat16), case)
    kept = _kept(case)
    to = [-(-k // page) for k in kept]
    st["to"], st["max_keep"] = _table(to, host), max(kept)
    st["keep"] = torch.tensor(kept, dtype=torch.int32, device=DEV)
    for name in ("kc", "vc"):
        st[name + "_to"] = _in_layout(torch.zeros((sum(to), page, hkv, dim), dtype=torch.bfloat16,
                                                  device=DEV), case)
    st["w_to"] = _in_layout(torch.zeros((sum(to), page, hkv), device=DEV), case)
    st["kept"] = torch.zeros(len(keys), dtype=torch.int32, device=DEV)
    st["index"] = torch.full((len(keys), hkv, max(kept)), -1, dtype=torch.int32, device=DEV)
    return st


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _turned(x, norm, pos, st):
    """Norm and rotation of x [rows, heads, 128] in 32 bits."""
    c, y = st["case"], x.float()
    if norm is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * norm.float()
    r = c["rot"]
    angle = pos.double()[:, None, None] * st["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    z = y[..., :r]
    if c["interleaved"]:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = z[..., :r // 2], z[..., r // 2:]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([z, y[..., r:]], -1)


def _places(st):
    """(sequence, token) of every row."""
    n, L = st["q"].shape[0], st["kv_len"].long()
    r = torch.arange(n, device=DEV)
    if st["offs"] is None:
        return r, L - 1
    offs = st["offs"].long()
    b = torch.searchsorted(offs, r, right=True) - 1
    return b, L[b] - (offs[b + 1] - r)


def _padded_rows(st):
    """Rows of every sequence [batch, most], and which there are."""
    n, L = st["q"].shape[0], st["kv_len"]
    offs = torch.arange(n + 1, device=DEV) if st["offs"] is None else st["offs"].long()
    i = torch.arange(st["max_q"], device=DEV)
    count = offs[1:] - offs[:-1]
    return (offs[:-1, None] + i).clamp_max(n - 1), i < count[:, None], count, L.long(), i


def _scores(st, keys, causal):
    """Scaled scores [batch, hkv, rows, group, tokens]; -inf where a row does not see a key."""
    c = st["case"]
    at, live, count, L, i = _padded_rows(st)
    T = st["max_kv"]
    q = st["q"].float()[at].view(len(L), len(i), c["hkv"], c["hq"] // c["hkv"], -1)
    s = torch.einsum("brhgd,bthd->bhrgt", q, keys) * st["scale"]
    end = (L[:, None] - count[:, None] + i + 1).clamp_max(L[:, None]) if causal else L[:, None] + 0 * i
    seen = (torch.arange(T, device=DEV) < end[:, :, None]) & live[:, :, None]
    return s.masked_fill_(~seen[:, None, :, None], -math.inf)


def _plain_decode4(st):
    c = st["case"]
    hkv, T = c["hkv"], st["max_kv"]
    tab = st["table"].long()

    def whole(name):
        x = _unpacked(st[name][tab])
        if name == "kc":
            e = st["kc_s"].view(torch.uint8)[tab].float() - 127
            x = x.unflatten(-1, (4, 32)) * torch.exp2(e)[..., None]
            x = x.flatten(-2)
        else:
            x = x * st["vc_s"][tab][..., None]
        return x.flatten(1, 2)[:, :T]

    s = _scores(st, whole("kc"), True)
    m = s.amax(-1, keepdim=True)
    sink = (st["sink"].view(1, hkv, 1, -1, 1) if st["sink"] is not None
            else torch.full_like(m, -math.inf))
    m = torch.maximum(m, sink).clamp_min(-1e30)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True) + torch.exp(sink - m)
    lse = (m + torch.log(z))[..., 0]
    out = torch.einsum("bhrgt,bthd->bhrgd", p / z, whole("vc"))
    live = _padded_rows(st)[1]
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[live]
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 2, 1, 3).flatten(2)[live]}


def _plain_append4(st):
    b, t = _places(st)
    st["q_out"].copy_(_turned(st["q"], st["q_norm"], t, st))
    page = st["case"]["page"]
    at = (st["table"][b, t // page].long(), t % page)
    for name, x in (("k", _turned(st["k"], st["k_norm"], t, st)), ("v", st["v"].float())):
        codes, e, value = _held(x, 4 if name == "k" else 1)
        st[name + "c"][at] = _packed(codes)
        if name == "k":
            st["kc_s"].view(torch.uint8)[at] = (e + 127).to(torch.uint8)
        else:
            st["vc_s"][at] = torch.exp2(e[..., 0].float())
        st[name + "_out"].copy_(value)


def _plain_weights(st):
    c = st["case"]
    tab, page, T = st["table"].long(), c["page"], st["max_kv"]
    at, live, count, L, i = _padded_rows(st)
    p = _scores(st, st["kc"].float()[tab].flatten(1, 2)[:, :T], c["causal"])
    p -= st["lse"][at].view(len(L), len(i), c["hkv"], -1).permute(0, 2, 1, 3)[..., None]
    new = p.exp_().sum((2, 3)).transpose(1, 2)                       # [batch, tokens, hkv]
    b, t = (torch.arange(T, device=DEV) < L[:, None]).nonzero(as_tuple=True)
    to = (tab[b, t // page], t % page)
    held = torch.where((t < L[b] - count[b])[:, None], st["w"][to] * c["decay"],
                       torch.zeros((), device=DEV))
    st["w"][to] = held + new[b, t]


def _plain_evict(st):
    c = st["case"]
    tab, page, T, most = st["table"].long(), c["page"], st["max_kv"], st["max_keep"]
    L = st["kv_len"].long()[:, None]
    n = torch.minimum(L, st["keep"].long()[:, None])
    r = n.clamp_max(c["recent"])
    f = (n - r).clamp_max(c["first"])
    t = torch.arange(T, device=DEV)
    w = st["w"][tab].flatten(1, 2)[:, :T]                            # [batch, tokens, hkv]
    always = ((t < f) | (t >= L - r))[..., None]
    rank = torch.where(always, math.inf, w).masked_fill((t >= L)[..., None], -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    order = order.masked_fill((t >= n)[..., None], T)
    index = torch.sort(order, dim=1).values[:, :most]                # ascending; T: none
    b, j, h = (index < T).nonzero(as_tuple=True)
    src = index[b, j, h]
    src = (tab[b, src // page], src % page, h)
    dst = (st["to"].long()[b, j // page], j % page, h)
    for name in ("kc", "vc", "w"):
        st[name + "_to"][dst] = st[name][src]
    st["index"][b, h, j] = index[b, j, h].int()
    st["kept"].copy_(n[:, 0])


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from split_flash_decoding_gb300 import attn
        kw = dict(max_kv_len=st["max_kv"], page_table=st["table"])
        if op == "append4":
            attn.attn_append_kv_fp4(
                st["k"], st["v"], st["kc"], st["vc"], st["kc_s"], st["vc_s"], st["kv_len"],
                q=st["q"], q_out=st["q_out"], k_out=st["k_out"], v_out=st["v_out"],
                q_row_offsets=st["offs"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS,
                rope=attn.Rope(st["turns"], interleaved=c["interleaved"]), **kw)
        elif op == "decode4":
            out, lse = attn.attn_decode_fp4(
                st["q"], st["kc"], st["vc"], st["kc_s"], st["vc_s"], st["kv_len"],
                group=c["hq"] // c["hkv"], scale=st["scale"], sink=st["sink"],
                q_row_offsets=st["offs"], max_q_len=st["max_q"], causal=True, **kw)
            return {"out": out, "lse": lse}
        elif op == "weights":
            attn.attn_key_weights(
                st["q"], st["kc"], st["lse"], st["kv_len"], st["w"], group=c["hq"] // c["hkv"],
                scale=st["scale"], q_row_offsets=st["offs"], max_q_len=st["max_q"],
                causal=c["causal"], decay=c["decay"], **kw)
        else:
            attn.attn_evict_kv(
                st["kc"], st["vc"], st["w"], st["kv_len"], st["keep"], st["kc_to"], st["vc_to"],
                st["w_to"], max_keep=st["max_keep"], first=c["first"], recent=c["recent"],
                out_page_table=st["to"], kept_len=st["kept"], indices=st["index"], **kw)
    elif op == "append4":
        _plain_append4(st)
    elif op == "decode4":
        return _plain_decode4(st)
    elif op == "weights":
        _plain_weights(st)
    else:
        _plain_evict(st)
    return _state(st)


def _state(st):
    """What a call left in the caller's buffers; a 4-bit cache's new rows as the values they
    stand for."""
    if st["case"]["op"] == "append4":
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"], "k_scale": st["kc_s"],
                "v_scale": st["vc_s"]}
    if st["case"]["op"] == "weights":
        return {"w": st["w"]}
    return {"kc": st["kc_to"], "vc": st["vc_to"], "w": st["w_to"], "kept": st["kept"],
            "index": st["index"]}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def _rotated64(x, norm, pos, st):
    c = st["case"]
    y = x.double().clone()
    if norm is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / 128 + EPS) * norm.double()
    half = c["rot"] // 2
    i = torch.arange(half, device=x.device)
    lo = 2 * i if c["interleaved"] else i
    hi = lo + (1 if c["interleaved"] else half)
    z = torch.polar(torch.ones((len(pos), 1, half), dtype=torch.float64, device=x.device),
                    (pos.double()[:, None] * st["freq"])[:, None])
    z = torch.complex(y[..., lo], y[..., hi]) * z
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _nearest64(y, e):
    """The numbers code * 2^e nearest to y (ties to the even code)."""
    a = (y / torch.exp2(e)).abs().clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    # (round() takes ties to even multiples of the step: those are the even codes here)
    return torch.round(a / step) * step * torch.sign(y) * torch.exp2(e)


def _exponent64(top):
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -300) / 6)).clamp(KMIN, KMAX)
    return torch.where(top > 6 * torch.exp2(e), e + 1, e)


def _exact_append4(st, rows, keys, page):
    token = torch.cat([torch.arange(L - n, L) for n, L in zip(rows, keys)]).to(DEV)
    seq = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows)).to(DEV)
    at = (st["table"].long()[seq, token // page], token % page)
    got = {"q": _rotated64(st["q"], st["q_norm"], token, st)}
    k = _rotated64(st["k"], st["k_norm"], token, st).unflatten(-1, (4, 32))
    e = _exponent64(k.abs().amax(-1))
    got["k"] = _nearest64(k, e[..., None]).flatten(-2)
    got["k_scale"] = torch.exp2(st["kc_s"].view(torch.uint8).double() - 127)
    got["k_scale"][at] = torch.exp2(e)
    v = st["v"].double()
    e = _exponent64(v.abs().amax(-1))
    got["v"] = _nearest64(v, e[..., None])
    got["v_scale"] = st["vc_s"].double()
    got["v_scale"][at] = torch.exp2(e)
    return got


def _exact_decode4(st, rows, keys, page):
    c, hkv, r0 = st["case"], st["case"]["hkv"], 0
    outs, lses = [], []
    for b, (n, L) in enumerate(zip(rows, keys)):
        own_pages = st["table"].long()[b, :-(-L // page)]

        def cached(name):
            x = _unpacked(st[name][own_pages], torch.float64)
            if name == "kc":
                s = torch.exp2(st["kc_s"].view(torch.uint8)[own_pages].double() - 127)
                x = x * s.repeat_interleave(32, -1)
            else:
                x = x * st["vc_s"][own_pages].double()[..., None]
            return x.reshape(-1, hkv, 128)[:L].transpose(0, 1)
        q = st["q"][r0:r0 + n].double().view(n, hkv, -1, 128).permute(1, 0, 2, 3)
        s = torch.matmul(q.flatten(1, 2), cached("kc").transpose(1, 2)).view(hkv, n, -1, L)
        late = torch.arange(L, device=DEV) > (L - n + torch.arange(n, device=DEV))[:, None]
        s = (s * st["scale"]).masked_fill(late[None, :, None], -math.inf)
        if c["sink"]:
            extra = st["sink"].double().view(hkv, 1, -1, 1).expand(hkv, n, -1, 1)
            lse = torch.logsumexp(torch.cat([s, extra], -1), -1)
        else:
            lse = torch.logsumexp(s, -1)
        o = torch.matmul(torch.exp(s - lse[..., None]).flatten(1, 2), cached("vc"))
        outs.append(o.view(hkv, n, -1, 128).permute(1, 0, 2, 3).reshape(n, -1, 128))
        lses.append(lse.permute(1, 0, 2).reshape(n, -1))
        r0 += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_weights(st, rows, keys, page):
    c, r0 = st["case"], 0
    got = st["w"].double()
    group = c["hq"] // c["hkv"]
    for b, (n, L) in enumerate(zip(rows, keys)):
        pg = st["table"].long()[b, :-(-L // page)]
        t = torch.arange(L, device=DEV)
        late = t > (L - n + torch.arange(n, device=DEV))[:, None]
        for h in range(c["hkv"]):
            k = st["kc"][pg, :, h].double().flatten(0, 1)[:L]
            total = torch.zeros(L, dtype=torch.float64, device=DEV)
            for hq in range(h * group, (h + 1) * group):
                s = torch.matmul(st["q"][r0:r0 + n, hq].double(), k.T) * st["scale"]
                p = torch.exp(s - st["lse"][r0:r0 + n, hq].double()[:, None])
                total += (p.masked_fill(late, 0.0) if c["causal"] else p).sum(0)
            total[:L - n] += got[pg[t // page], t % page, h][:L - n] * c["decay"]
            got[pg[t // page], t % page, h] = total
        r0 += n
    return {"w": got}


def _exact_evict(st, rows, keys, page):
    c = st["case"]
    got = {"kc": st["kc_to"].double(), "vc": st["vc_to"].double(), "w": st["w_to"].double(),
           "kept": st["kept"].clone(), "index": st["index"].clone()}
    for b, (L, keep) in enumerate(zip(keys, _kept(c))):
        n = min(L, keep)
        r = min(n, c["recent"])
        f = min(n - r, c["first"])
        got["kept"][b] = n
        old = torch.arange(L, device=DEV)
        old = (st["table"].long()[b, old // page], old % page)
        for h in range(c["hkv"]):
            w = st["w"][old][:, h].cpu().tolist()
            best = sorted(range(f, L - r), key=lambda i: (-w[i], i))[:n - r - f]
            mine = sorted(list(range(f)) + best + list(range(L - r, L)))
            i = torch.tensor(mine, device=DEV)
            j = torch.arange(n, device=DEV)
            src, dst = (old[0][i], old[1][i], h), (st["to"].long()[b, j // page], j % page, h)
            for name in ("kc", "vc", "w"):
                got[name][dst] = st[name][src].double()
            got["index"][b, h, :n] = i.int()
    return got


def exact(case, seed):
    st = prepare(case, seed)
    form = {"append4": _exact_append4, "decode4": _exact_decode4, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]]
    return form(st, *_lengths(case), case["page"])
