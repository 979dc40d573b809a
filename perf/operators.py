"""What is measured of the operators that fill and read a KV cache: the norm and
rotation of query and key heads, appending to a bf16 cache, appending to a cache
held in 8 bits (e4m3) with a scale for each block of tokens and KV head, and
decode attention over that cache.

A case is a dict of plain values.  `run` computes a case in elementary torch
operations in 32 bits (angles in 64), or, where `own` is true, calls the
framework.  `exact` is the operators' definition in 64 bits, written apart.

Shapes are those of the framework's own workloads (32 query heads on 8 KV heads
of 128 channels, pages of 128; latent rows of 576 channels, pages of 64) and
generic ones around them.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
FP8 = torch.float8_e4m3fn
KMIN, KMAX = -60, 120   # exponents of the appended blocks' scales


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    qk = dict(op="qk", hq=32, hkv=8, dim=128, rot=128, start=0, interleaved=False, norm=False,
              scaling="none")
    app = dict(op="append", hq=32, hkv=8, dim=128, rot=128, start=0, interleaved=False, norm=False,
               scaling="none", latent=False, lens=2)
    app8 = dict(app, op="append8")
    dec = dict(op="decode8", hq=32, hkv=8, q_rows=1, sink=False, page=128, block=64, lens=2)
    return [
        # one decoded token: latency
        dict(qk, name="qk_one_token", rows=1),
        # a long prompt, heads normed, adjacent channels rotated, scaled for a long context
        dict(qk, name="qk_norm_prompt", rows=8191, interleaved=True, norm=True, scaling="ramp"),
        # a decode step of 64 sequences
        dict(app, name="append_b64", batch=64, q_rows=1, ctx=1024, page=128),
        # ragged prompts mixed with decoding sequences, heads normed
        dict(app, name="append_mixed", batch=16, q_rows=4096, ctx=512, page=128, norm=True,
             lens=5, scaling="bands"),
        # draft rows of a latent cache: 512 normed channels and 64 rotated ones
        dict(app, name="append_latent_draft", batch=32, q_rows=2, ctx=1024, page=64, hq=128,
             hkv=1, dim=576, rot=64, start=512, interleaved=True, norm=True, latent=True, lens=4),
        # a decode step into the 8-bit cache: a block's scale may have to grow
        dict(app8, name="append8_b64", batch=64, q_rows=1, ctx=1024, page=128, block=64),
        # ragged prompts into the 8-bit cache
        dict(app8, name="append8_mixed", batch=16, q_rows=4096, ctx=512, page=128, block=128,
             norm=True, lens=5),
        # draft rows, one scale per token
        dict(app8, name="append8_draft", batch=37, q_rows=4, ctx=700, page=64, block=1, rot=64,
             lens=6),
        # two short sequences: latency
        dict(dec, name="decode8_short", batch=2, hq=4, hkv=1, len_lo=37, len_hi=100, page=64,
             block=16, lens=1),
        # a decode step of 64 ragged sequences
        dict(dec, name="decode8_b64", batch=64, len_lo=512, len_hi=8192),
        # one sequence of 131072 tokens, with sinks
        dict(dec, name="decode8_long", batch=1, len_lo=131072, len_hi=131072, sink=True, block=128,
             lens=3),
        # draft rows being verified, one scale per token
        dict(dec, name="decode8_draft", batch=64, q_rows=4, len_lo=512, len_hi=4096, block=1,
             lens=6),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "append", "append8", "decode8", "decode8"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    seed = rng.randrange(1, 1 << 20)
    if op == "decode8":
        group = hq // hkv
        q_rows = rng.choice([1, 1, rng.randint(1, 16 // group)])
        page = rng.choice([16, 32, 64, 128, 256])
        block = 1 << rng.randint(0, page.bit_length() - 1)
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(131072, 64 * 4096 // batch)))
        return dict(op=op, hq=hq, hkv=hkv, q_rows=q_rows, sink=rng.random() < 0.5, page=page,
                    block=block, lens=seed, batch=batch, len_lo=max(1, hi // rng.choice([1, 2, 16])),
                    len_hi=hi)
    scaling = rng.choice(["none", "linear", "ramp", "bands"])
    inter, norm = rng.random() < 0.5, rng.random() < 0.5
    if op == "qk":
        dim = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([dim, dim // 2, 32])
        return dict(op=op, hq=hq, hkv=hkv, dim=dim, rot=rot, start=rng.choice([0, dim - rot]),
                    interleaved=inter, norm=norm, scaling=scaling, rows=_log(rng, 1, 8191), lens=seed)
    page = rng.choice([16, 32, 64, 128, 256])
    c = dict(op=op, hq=hq, hkv=hkv, dim=128, rot=rng.choice([128, 64, 32]), start=0,
             interleaved=inter, norm=norm, scaling=scaling, latent=False, lens=seed,
             batch=_log(rng, 1, 64), page=page, ctx=_log(rng, 1, 1024))
    c["q_rows"] = rng.choice([1, rng.randint(2, 8), _log(rng, 1, max(1, 16384 // c["batch"]))])
    if op == "append8":
        c["block"] = 1 << rng.randint(0, min(7, page.bit_length() - 1))
    return c


def _lengths(case):
    """(query rows, keys) per sequence: from the case alone."""
    rng = random.Random(case["lens"])
    b, n = case["batch"], case["q_rows"]
    if case["op"] == "decode8":
        rows = [1 if n == 1 else rng.randint(1, n) for _ in range(b)]
        keys = [max(r, rng.randint(case["len_lo"], case["len_hi"])) for r in rows]
        return rows, keys
    # appends: long runs are mixed with single rows, as prompts with decoding sequences
    rows = [1 if n == 1 or (n > 8 and i % 2) else rng.randint(max(1, n // 8), n) for i in range(b)]
    return rows, [r + rng.randint(0, case["ctx"]) for r in rows]


def work(case):
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    if op == "qk":
        n = case["rows"] * (hq + hkv) * case["dim"]
        return {"bytes": 4 * n, "flops": 10 * n}
    rows, keys = _lengths(case)
    if op == "decode8":
        tokens = sum(keys)
        pairs = sum(r * k for r, k in zip(rows, keys))
        scales = 2 * 4 * hkv * sum(-(-k // case["block"]) for k in keys)
        return {"bytes": tokens * hkv * 128 * 2 + scales + sum(rows) * hq * (4 * 128 + 4),
                "flops": 4 * pairs * hq * 128}
    kv = hkv * case["dim"] * (1 if case["latent"] else 2)
    n = sum(rows)
    per = n * (4 * hq * case["dim"] + (3 if op == "append8" else 4) * kv)
    return {"bytes": per, "flops": 10 * n * (hq * case["dim"] + kv)}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _frequencies(case):
    """Radians per position and the factor of cos and sin, for the case's scaling."""
    rot, base, factor, orig = case["rot"], 500000.0, 8.0, 8192
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "ramp":       # by parts: from plain to stretched between two wavelengths
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32))), min(rot - 1, math.ceil(at(1)))
        part = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
        return [x * (1 - p) + x / factor * p for x, p in zip(f, part)], 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":      # by wavelength: kept, stretched, smooth in between
        def band(x):
            n = orig * x / (2 * math.pi)
            s = min(1.0, max(0.0, (n - 1.0) / (4.0 - 1.0)))
            return (1 - s) * x / factor + s * x
        return [band(x) for x in f], 1.0
    return f, 1.0


def _quantised(x, block):
    """x [pages, page, heads, 128] -> e4m3 codes and fp32 scales [pages, page / block, heads]."""
    p, n, h, d = x.shape
    y = x.view(p, n // block, block, h, d)
    s = (y.abs().amax(dim=(2, 4)) / 448.0).clamp_min(2.0 ** -20)
    return (y / s[:, :, None, :, None]).to(FP8).view(p, n, h, d), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    host = random.Random(seed)
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)   # noqa: E731
    st = {"case": case}
    if op != "decode8":
        dim = case["dim"]
        rows = [case["rows"]] if op == "qk" else _lengths(case)[0]
        n = sum(rows)
        # the projection's output: q, k and v of a row side by side
        heads = hq + hkv * (1 if op == "qk" or case["latent"] else 2)
        packed = randn(n, heads, dim).to(torch.bfloat16)
        st["q"], st["k"] = packed[:, :hq], packed[:, hq:hq + hkv]
        st["v"] = packed[:, hq + hkv:] if heads > hq + hkv else None
        nd = case["start"] if case.get("latent") else dim
        st["k_norm"] = (1 + 0.1 * randn(nd)).to(torch.bfloat16) if case["norm"] else None
        st["q_norm"] = ((1 + 0.1 * randn(nd)).to(torch.bfloat16)
                        if case["norm"] and not case.get("latent") else None)
        freq, st["mscale"] = _frequencies(case)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        # the same as a fraction of a turn per position, in units of 2^-64
        t = [int(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
        st["turns"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in t], dtype=torch.int64,
                                   device=DEV)
        st["q_out"] = torch.empty((n, hq, dim), dtype=torch.bfloat16, device=DEV)
        if op == "qk":
            first = host.randrange(0, 100000)
            st["pos"] = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
            st["k_out"] = torch.empty((n, hkv, dim), dtype=torch.bfloat16, device=DEV)
            return st
    else:
        rows = _lengths(case)[0]
        dim = 128
        st["q"] = randn(sum(rows), hq, dim).to(torch.bfloat16)
        st["scale"] = float(torch.tensor(1 / math.sqrt(dim), dtype=torch.float32))
        st["sink"] = randn(hq) if case["sink"] else None
    keys, page, b = _lengths(case)[1], case["page"], case["batch"]
    pages = [-(-k // page) for k in keys]
    order = list(range(sum(pages)))
    host.shuffle(order)
    table = torch.zeros((b, max(pages)), dtype=torch.int32)
    at = 0
    for i, m in enumerate(pages):
        table[i, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    st["table"] = table.to(DEV)
    st["kv_len"] = torch.tensor(keys, dtype=torch.int32, device=DEV)
    st["offs"] = None
    if case["q_rows"] > 1:
        st["offs"] = torch.tensor([sum(rows[:i]) for i in range(b + 1)], dtype=torch.int32,
                                  device=DEV)
    st["max_kv"], st["max_q"] = max(keys), max(rows)
    caches = ["kc"] if case.get("latent") else ["kc", "vc"]
    for name in caches:
        x = randn(len(order), page, hkv, dim)
        if op == "append":
            st[name] = x.to(torch.bfloat16)
        elif op == "append8":
            blk = case["block"]
            # what earlier appends left: scales are powers of two, some blocks far smaller
            x *= 2.0 ** torch.randint(-6, 1, (len(order), page // blk, 1, hkv, 1), generator=g,
                                      device=DEV).float().repeat_interleave(blk, 1).view(
                                          len(order), page, hkv, 1)
            y = x.view(len(order), page // blk, blk, hkv, dim)
            s = torch.exp2(_exponent(y.abs().amax(dim=(2, 4))))
            st[name] = (y / s[:, :, None, :, None]).to(FP8).view_as(x)
            st[name + "_s"] = s
        else:
            st[name], st[name + "_s"] = _quantised(x, case["block"])
        del x
    return st


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _exponent(amax):
    """The least k with amax <= 448 * 2^k (448 is the largest e4m3 number, 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    k = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, k, KMIN).clamp(KMIN, KMAX).float()


def _turned(x, norm, pos, st):
    """Norm and rotation of x [rows, heads, dim] in 32 bits."""
    c = st["case"]
    y = x.float()
    if norm is not None:
        nd = norm.numel()
        z = y[..., :nd]
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * norm.float()
        y = torch.cat([z, y[..., nd:]], -1)
    s, r = c["start"], c["rot"]
    angle = pos.double()[:, None, None] * st["freq"]
    cos, sin = (angle.cos() * st["mscale"]).float(), (angle.sin() * st["mscale"]).float()
    z = y[..., s:s + r]
    if c["interleaved"]:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = z[..., :r // 2], z[..., r // 2:]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y[..., :s], z, y[..., s + r:]], -1)


def _places(st):
    """(sequence, token) of every row."""
    n, L = st["q"].shape[0], st["kv_len"].long()
    r = torch.arange(n, device=DEV)
    if st["offs"] is None:
        return r, L - 1
    offs = st["offs"].long()
    b = torch.searchsorted(offs, r, right=True) - 1
    return b, L[b] - (offs[b + 1] - r)


def _append8(x, codes, scales, b, t, st):
    """Appends the rows x [rows, heads, 128] (32 bits) to one 8-bit cache."""
    page, blk = st["case"]["page"], st["case"]["block"]
    pg = st["table"][b, t // page].long()
    slot = t % page
    nb = page // blk
    unit = pg * nb + slot // blk                           # the row's block
    flat = scales.view(-1, scales.shape[-1])
    need = torch.full_like(flat, -1e9)
    need.index_reduce_(0, unit, _exponent(x.abs().amax(-1)), "amax")
    # tokens before the first new row are held already; slots after the last stay as they are
    first = torch.full_like(flat[:, 0], blk).index_reduce_(0, unit, (slot % blk).float(), "amin")
    touched = torch.unique(unit)
    old = flat[touched]
    new = torch.exp2(need[touched])
    new = torch.where(first[touched][:, None] == 0, new, torch.maximum(old, new))
    body = codes.view(torch.uint8).view(-1, blk, *codes.shape[2:])
    held = body[touched]
    scaled = (held.view(FP8).float() * (old / new)[:, None, :, None]).to(FP8).view(torch.uint8)
    before = torch.arange(blk, device=DEV) < first[touched][:, None]
    body[touched] = torch.where(before[:, :, None, None], scaled, held)
    flat[touched] = new
    rows = (x / flat[unit][..., None]).to(FP8).view(torch.uint8)
    body[unit, slot % blk] = rows


def _decode8(st):
    c = st["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    L = st["kv_len"].long()
    T, R, n = st["max_kv"], st["max_q"], st["q"].shape[0]
    offs = torch.arange(n + 1, device=DEV) if st["offs"] is None else st["offs"].long()
    count = offs[1:] - offs[:-1]
    i = torch.arange(R, device=DEV)
    at = (offs[:-1, None] + i).clamp_max(n - 1)
    q = st["q"].float()[at].view(len(L), R, hkv, hq // hkv, 128)

    def whole(codes, s):
        x = codes[st["table"].long()].float().view(len(L), -1, page // s.shape[1], hkv, 128)
        x *= s[st["table"].long()].view(len(L), -1, 1, hkv, 1)
        return x.view(len(L), -1, hkv, 128)[:, :T]

    t = torch.arange(T, device=DEV)
    seen = t < (L[:, None] - count[:, None] + i + 1)[:, :, None]          # causal, [b, row, key]
    scores = torch.einsum("brhgd,bthd->bhrgt", q, whole(st["kc"], st["kc_s"])) * st["scale"]
    scores = scores.masked_fill(~seen[:, None, :, None], -math.inf)
    m = scores.amax(-1, keepdim=True)
    sink = (st["sink"].view(1, hkv, 1, -1, 1) if st["sink"] is not None
            else torch.full_like(m, -math.inf))
    m = torch.maximum(m, sink)
    p = torch.exp(scores - m)
    z = p.sum(-1, keepdim=True) + torch.exp(sink - m)
    lse = (m + torch.log(z))[..., 0]
    out = torch.einsum("bhrgt,bthd->bhrgd", p / z, whole(st["vc"], st["vc_s"]))
    live = i < count[:, None]
    out = out.permute(0, 2, 1, 3, 4).reshape(len(L), R, hq, 128)[live]
    lse = lse.permute(0, 2, 1, 3).reshape(len(L), R, hq)[live]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _held(st):
    """The 8-bit caches: the codes (as numbers, in units of their block's scale) and the scales."""
    return {"q": st["q_out"], "kc": st["kc"], "vc": st["vc"], "kc_s": st["kc_s"],
            "vc_s": st["vc_s"]}


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from split_flash_decoding_gb300 import attn
        if op == "decode8":
            out, lse = attn.attn_decode_fp8(
                st["q"], st["kc"], st["vc"], st["kc_s"], st["vc_s"], st["kv_len"],
                group=c["hq"] // c["hkv"], scale=st["scale"], max_kv_len=st["max_kv"],
                page_table=st["table"], sink=st["sink"], q_row_offsets=st["offs"],
                max_q_len=st["max_q"], causal=True)
            return {"out": out, "lse": lse}
        rope = attn.Rope(st["turns"], interleaved=c["interleaved"], mscale=st["mscale"],
                         start=c["start"])
        if op == "qk":
            attn.attn_qk_norm_rope(st["q"], st["k"], st["pos"], rope=rope, q_norm=st["q_norm"],
                                   k_norm=st["k_norm"], eps=EPS, q_out=st["q_out"],
                                   k_out=st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        kw = dict(q=st["q"], q_out=st["q_out"], max_kv_len=st["max_kv"], page_table=st["table"],
                  q_row_offsets=st["offs"], rope=rope, q_norm=st["q_norm"], k_norm=st["k_norm"],
                  eps=EPS)
        if op == "append":
            attn.attn_append_kv(st["k"], st["v"], st["kc"], st.get("vc"), st["kv_len"], **kw)
            return {"q": st["q_out"], "kc": st["kc"], "vc": st.get("vc")}
        attn.attn_append_kv_fp8(st["k"], st["v"], st["kc"], st["vc"], st["kc_s"], st["vc_s"],
                                st["kv_len"], max_q_len=st["max_q"], **kw)
        return _held(st)
    if op == "decode8":
        return _decode8(st)
    if op == "qk":
        st["q_out"].copy_(_turned(st["q"], st["q_norm"], st["pos"], st))
        st["k_out"].copy_(_turned(st["k"], st["k_norm"], st["pos"], st))
        return {"q": st["q_out"], "k": st["k_out"]}
    b, t = _places(st)
    st["q_out"].copy_(_turned(st["q"], st["q_norm"], t, st))
    k = _turned(st["k"], st["k_norm"], t, st)
    if op == "append":
        page = c["page"]
        at = (st["table"][b, t // page].long(), t % page)
        st["kc"][at] = k.to(torch.bfloat16)
        if st["v"] is not None:
            st["vc"][at] = st["v"]
        return {"q": st["q_out"], "kc": st["kc"], "vc": st.get("vc")}
    _append8(k, st["kc"], st["kc_s"], b, t, st)
    _append8(st["v"].float(), st["vc"], st["vc_s"], b, t, st)
    return _held(st)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def _nearest_code(x):
    """The e4m3 number nearest to x (ties to even), |x| <= 448, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -300))).clamp_min(-6)
    e = e - (torch.exp2(e) > x.abs().clamp_min(2.0 ** -6)).double()      # a log2 rounded up
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _rotated64(x, norm, pos, st):
    c = st["case"]
    y = x.double().clone()
    if norm is not None:
        nd = norm.numel()
        rms = torch.sqrt((y[..., :nd] ** 2).sum(-1, keepdim=True) / nd + EPS)
        y[..., :nd] = y[..., :nd] / rms * norm.double()
    half = c["rot"] // 2
    i = torch.arange(half, device=x.device)
    lo = c["start"] + (2 * i if c["interleaved"] else i)
    hi = lo + (1 if c["interleaved"] else half)
    z = torch.polar(torch.full((len(pos), 1, half), st["mscale"], dtype=torch.float64,
                               device=x.device), (pos.double()[:, None] * st["freq"])[:, None])
    z = torch.complex(y[..., lo], y[..., hi]) * z
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return {"q": _rotated64(st["q"], st["q_norm"], st["pos"], st),
                "k": _rotated64(st["k"], st["k_norm"], st["pos"], st)}
    rows, keys = _lengths(case)
    page, hkv = case["page"], case["hkv"]
    table = st["table"].long()
    if case["op"] == "decode8":
        G = case["hq"] // hkv
        outs, lses, r0 = [], [], 0
        for b, (n, L) in enumerate(zip(rows, keys)):
            def cached(name):
                s = st[name + "_s"].double()[table[b, :-(-L // page)]]
                x = st[name][table[b, :-(-L // page)]].double()
                x = x * s.repeat_interleave(page // s.shape[1], 1)[..., None]
                return x.reshape(-1, hkv, 128)[:L].transpose(0, 1)
            q = st["q"][r0:r0 + n].double().view(n, hkv, G, 128)
            s = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, n * G, 128),
                             cached("kc").transpose(1, 2)).view(hkv, n, G, L) * st["scale"]
            late = torch.arange(L, device=DEV) > (L - n + torch.arange(n, device=DEV))[:, None]
            s = s.masked_fill(late[None, :, None], -math.inf)
            if case["sink"]:
                extra = st["sink"].double().view(hkv, 1, G, 1).expand(hkv, n, G, 1)
                lse = torch.logsumexp(torch.cat([s, extra], -1), -1)
            else:
                lse = torch.logsumexp(s, -1)
            o = torch.matmul(torch.exp(s - lse[..., None]).view(hkv, n * G, L), cached("vc"))
            outs.append(o.view(hkv, n, G, 128).permute(1, 0, 2, 3).reshape(n, -1, 128))
            lses.append(lse.permute(1, 0, 2).reshape(n, -1))
            r0 += n
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    token = torch.cat([torch.arange(L - n, L) for n, L in zip(rows, keys)]).to(DEV)
    seq = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows)).to(DEV)
    got = {"q": _rotated64(st["q"], st["q_norm"], token, st)}
    new = {"kc": _rotated64(st["k"], st["k_norm"], token, st)}
    if st["v"] is not None:
        new["vc"] = st["v"].double()
    pg, slot = table[seq, token // page], token % page
    for name, x in new.items():
        if case["op"] == "append":
            y = st[name].double()
            y[pg, slot] = x
            got[name] = y
            continue
        blk = case["block"]
        s = st[name + "_s"].double()
        y = st[name].double().view(-1, page // blk, blk, hkv, 128)
        value = y * s[:, :, None, :, None]
        is_new = torch.zeros(y.shape[:3], dtype=torch.bool, device=DEV)
        is_new[pg, slot // blk, slot % blk] = True
        value[pg, slot // blk, slot % blk] = x
        top = (value.abs().amax(-1) * is_new[..., None]).amax(2)          # of the new tokens
        k = torch.ceil(torch.log2(top.clamp_min(2.0 ** -300) / 448)).clamp(KMIN, KMAX)
        k = torch.where(top > 448 * torch.exp2(k), k + 1, k)
        grown = torch.where(is_new[:, :, 0, None], torch.exp2(k),
                            torch.maximum(torch.exp2(k), s))
        s = torch.where(is_new.any(2)[..., None], grown, s)[:, :, None, :, None]
        live = is_new | ((is_new.cumsum(2) == 0) & is_new.any(2, keepdim=True))
        y = torch.where(live[..., None, None], _nearest_code(value / s), y)
        got[name] = y.view(-1, page, hkv, 128)
        got[name + "_s"] = s[:, :, 0, :, 0]
    return got
