"""The cache held in 4 bits: its append against the 64-bit norm, rotation and rounding, its
decode attention against a 64-bit reference.

Append.  A value y is off its exact one by at most err (tests/cache_ref.py).  The scale
is that of a largest value within err of the exact one, and the code's number is one of the
two e2m1 numbers around y or the nearest: |code 2^e - y| <= half a step of the grid at y
2^-e (0.25 below 2, 0.5 to 4, 1 to 6) times 2^e + err.  Keys that are neither normed nor
rotated, and values, have no err: their codes and scales are exact, ties to the even code.

Decode attends over code * scale in 64 bits.  What the kernel may differ by:

* weights: p_j 2^(e_j), e_j the exponent of the key's value scale, is rounded to f16 (2^-11 of
  itself at most; the exponential before that errs by 2^-22) and enters the product as four
  e5m2 terms of 3 bits each, which hold all 11 bits down to 2^-16 in units in which the
  largest, u, is 2^11 at least: what is cut off is less than 2^-27 u.  So out misses at most
  2^-11 sum_j w_j |v_j| + 2^-27 u sum_j 2^(-e_j) |v_j| by this, with w_j the normalised weights
  and u the largest w_j 2^(e_j).  (The random codes of these tests make rows in which one key
  has all but 2^-25 of the weight and a value of 0: there out is small weights alone.)
* scores: the queries' two terms miss at most 2^-21 of the row's largest channel, and that
  only in channels below 2^-13 of it; a score is a sum of 2 x 4 blocks of 32 exact products
  and four products with powers of two, each step rounded in fp32.  rho = 2^-16 max_j sum_c
  |q_c k_jc| scale + 2^-20 bounds it as for the 8-bit cache; it moves every weight and the
  normaliser by a factor of at most 1 + 2 rho.
* half a bf16 step of out, 2^-8 |out|.

So |out - exact| <= 2^-8 |exact| + 1.01 (2^-11 + 2^-20 + 4 rho) sum_j w_j |v_j| + 2^-27 u sum_j
2^(-e_j) |v_j|, and |lse - exact| <= rho + 2^-20 max(1, |exact|).
"""
import math

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module")
def attn():
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn as a
    a.attn_device_error_flags(clear=True)
    yield a
    assert a.attn_device_error_flags(clear=True) == 0


def i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)


def numbers(codes):
    """Bytes [..., 64] to the numbers of their codes [..., 128]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return torch.cat([GRID, -GRID])[c]


def exponent(top):
    """Least e with top <= 6 * 2^e, clamped."""
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -300) / 6))
    e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e)
    return torch.where(top > 0, e, -60.0).clamp(-60, 125)


def nearest(x):
    """The nearest e2m1 numbers (ties to the even code), |x| clamped to 6."""
    d = (x.abs().clamp_max(6)[..., None] - GRID).abs()
    best = d.min(-1, keepdim=True).values
    # of two at the same distance the one with the even code
    pick = torch.where(d == best, torch.arange(8) % 2, 9).argmin(-1)
    return GRID[pick] * torch.where(x < 0, -1.0, 1.0)


def half_step(x):
    a = x.abs()
    return torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)).double()


class Pool:
    """Places of sequences in a paged or contiguous cache."""

    def __init__(self, lens, page, seed, contiguous=False, max_len=None):
        self.page = max(max_len or max(lens), 1) if contiguous else page
        self.lens = lens
        if contiguous:
            self.pages, self.table = len(lens), None
            return
        need = [max(1, -(-x // page)) for x in lens]
        g = torch.Generator().manual_seed(seed)
        self.pages = sum(need) + 2
        perm = torch.randperm(self.pages, generator=g)
        self.table, at = torch.full((len(lens), max(need)), -1, dtype=torch.int32), 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n

    def place(self, b, t):
        if self.table is None:
            return b, t
        return int(self.table[b, t // self.page]), t % self.page

    def gpu_table(self):
        return None if self.table is None else self.table.to(DEV)


def layout(x, head_major):
    return x.transpose(1, 2).contiguous().transpose(1, 2) if head_major else x


class Cache:
    """Codes and scales of K and V."""

    def __init__(self, pool, hkv, seed, head_major=False, random=True):
        g = torch.Generator().manual_seed(seed)
        shape = (pool.pages, pool.page, hkv)
        byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)   # noqa: E731
        self.k, self.v = byte(*shape, 64), byte(*shape, 64)
        self.ks = torch.randint(122, 131, (*shape, 4), generator=g, dtype=torch.uint8)
        self.vs = torch.exp2(torch.randint(-4, 3, shape, generator=g).float())
        self.head_major = head_major

    def gpu(self):
        k, v, ks, vs = (layout(x.to(DEV), self.head_major) for x in (self.k, self.v, self.ks, self.vs))
        return [k, v, ks.view(torch.float8_e8m0fnu), vs]

    def read(self, got):
        """A GPU cache's four tensors on the CPU (scales of keys as bytes)."""
        k, v, ks, vs = got
        return k.cpu(), v.cpu(), ks.view(torch.uint8).cpu(), vs.cpu()

    @staticmethod
    def values(k, v, ks, vs):
        """What codes and scales stand for, in 64 bits."""
        s = torch.exp2(ks.double() - 127)
        s = torch.where(ks == 255, math.nan, s).repeat_interleave(32, -1)
        return numbers(k) * s, numbers(v) * vs.double()[..., None]


# ---- appending --------------------------------------------------------------------------

def check_append(attn, lens, q_lens, *, hq=4, hkv=2, page=16, rot=128, start=0, interleaved=False,
                 norm=False, head_major=False, contiguous=False, outs=True, seed=0, scale=1.0,
                 q_dim=128, positions=None, in_place=False, behind=2):
    g = torch.Generator().manual_seed(seed)
    rows_of = q_lens or [1] * len(lens)
    rows = sum(rows_of)
    n = rows + (behind if q_lens else 0)
    pool = Pool(lens, page, seed, contiguous)
    x = (torch.randn(n, 2 * hkv, 128, generator=g) * scale).to(torch.bfloat16)
    k, v = x[:, :hkv], x[:, hkv:]
    q = torch.randn(n, hq, q_dim, generator=g).to(torch.bfloat16)
    kn = (1 + 0.1 * torch.randn(128, generator=g)).to(torch.bfloat16) if norm else None
    cache = Cache(pool, hkv, seed + 1, head_major)
    got = cache.gpu()
    rope = turns = None
    if rot:
        turns, mscale = attn.rope_turns(rot, 10000.0)
        rope = attn.Rope(turns.to(DEV), interleaved=interleaved, mscale=mscale, start=start)
    offs = None if q_lens is None else [sum(q_lens[:i]) for i in range(len(lens) + 1)]
    token = torch.cat([torch.arange(L - m, L) for L, m in zip(lens, rows_of)])
    where = positions if positions is not None else token.clamp_min(0)
    xg, qg = x.to(DEV), q.to(DEV)
    fill = lambda h, d: torch.full((n, h, d), -9.0, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    ko, vo, qo = fill(hkv, 128), fill(hkv, 128), fill(hq, q_dim)
    if in_place:
        ko, vo = xg[:, :hkv], xg[:, hkv:]
    more = dict(k_out=ko, v_out=vo) if outs else {}
    ret = attn.attn_append_kv_fp4(
        xg[:, :hkv], xg[:, hkv:], *got, i32(lens), max_kv_len=max(max(lens), 1),
        page_table=pool.gpu_table(), q=qg, q_out=qo, q_row_offsets=i32(offs), rope=rope,
        k_norm=None if kn is None else kn.to(DEV),
        positions=None if positions is None else
        torch.cat([positions, torch.zeros(n - rows, dtype=torch.int64)]).to(torch.int32).to(DEV),
        **more)
    torch.cuda.synchronize()
    assert ret is qo
    # (a token below 0 is reported)
    short = any(0 < L < m for L, m in zip(lens, rows_of))
    assert attn.attn_device_error_flags(clear=True) == (4 if short else 0)
    kc, vc, ks, vs = cache.read(got)
    exact, err = R.head_rows(k[:rows], turns, where, norm=kn, start=start, interleaved=interleaved)
    want_v = v[:rows].double()
    ev = exponent(want_v.abs().amax(-1))
    codes_v = nearest(want_v / torch.exp2(ev)[..., None]) * torch.exp2(ev)[..., None]
    y = exact.unflatten(-1, (4, 32))
    top, etop = y.abs().amax(-1), err.unflatten(-1, (4, 32)).amax(-1)
    lo, hi = exponent((top - etop).clamp_min(0)), exponent(top + etop)
    held_k, held_v = Cache.values(kc, vc, ks, vs)
    r = 0
    left = torch.ones(pool.pages, pool.page, dtype=torch.bool)
    for b, m in enumerate(rows_of):
        for i in range(m):
            t = lens[b] - m + i
            if t >= 0:
                at = pool.place(b, t)
                left[at] = False
                e = ks[at].double() - 127
                assert ((e == lo[r]) | (e == hi[r])).all(), f"row {r}: a key's scale"
                s = torch.exp2(e)[..., None]
                z = held_k[at].unflatten(-1, (4, 32))
                off = (z - y[r]).abs() - half_step(y[r] / s) * s * (1 + 1e-9) - \
                    err[r].unflatten(-1, (4, 32))
                assert off.max() <= 0, f"row {r}: a key's codes, {off.max():.3g}"
                if not rot and not norm:
                    assert torch.equal(z, nearest(y[r] / s) * s)
                assert torch.equal(vs[at].double(), torch.exp2(ev[r])), f"row {r}: a value's scale"
                assert torch.equal(held_v[at], codes_v[r]), f"row {r}: a value's codes"
                if outs:
                    assert torch.equal(ko[r].cpu().double(), held_k[at])
                    assert torch.equal(vo[r].cpu().double(), held_v[at])
            r += 1
    # nothing else changed
    for a, b in ((kc, cache.k), (vc, cache.v), (ks, cache.ks), (vs, cache.vs)):
        assert torch.equal(a[left], b[left])
    if not in_place:
        assert (ko[rows:] == -9).all() and (qo[rows:] == -9).all()
    eq, qerr = R.head_rows(q[:rows], turns, where, start=start, interleaved=interleaved)
    R.assert_bf16(qo[:rows], eq, qerr, "q")


CASES = [
    ([1], None, {}),
    ([1, 64, 65, 128, 700, 0, 33], None, dict(page=64, norm=True)),
    ([5, 300, 17], [5, 130, 1], dict(norm=True, interleaved=True)),
    ([40, 200, 9, 64], [1, 200, 9, 3], dict(contiguous=True, head_major=True)),
    ([1000, 1, 8, 513], [600, 0, 8, 2], dict(page=128, hq=8, hkv=4)),
    ([30, 9], [40, 9], dict(page=8)),                     # more rows than tokens
]


@pytest.mark.parametrize("lens,q_lens,kw", CASES)
@pytest.mark.parametrize("outs", [False, True])
def test_append(attn, lens, q_lens, kw, outs):
    check_append(attn, lens, q_lens, outs=outs, seed=len(lens), **kw)


@pytest.mark.parametrize("rot,start,interleaved", [
    (0, 0, False), (128, 0, True), (64, 0, False), (64, 0, True), (64, 64, False), (64, 32, True),
    (32, 0, False), (32, 96, False), (16, 8, False), (32, 40, True), (96, 0, False), (8, 0, False),
    (6, 0, True), (20, 64, False)])
@pytest.mark.parametrize("q_lens", [None, [3, 40]])
def test_append_rotations(attn, rot, start, interleaved, q_lens):
    check_append(attn, [30, 60], q_lens, rot=rot, start=start, interleaved=interleaved,
                 norm=rot % 32 == 0 and rot > 0, seed=rot + start)


@pytest.mark.parametrize("scale", [1e-30, 1e-17, 1e-3, 1e4, 1e30])
def test_append_sizes_of_values(attn, scale):
    check_append(attn, [30, 9], [20, 3], rot=0, scale=scale, seed=3)
    check_append(attn, [30, 9], [20, 3], rot=64, scale=scale, seed=4)


def test_append_many_rows(attn):
    lens, q_lens = [2600, 700, 5, 1300], [2600, 600, 1, 1300]
    check_append(attn, lens, q_lens, hq=8, hkv=2, page=128, norm=True, head_major=True, seed=8)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 7), (32, 8), (5, 3)])
def test_append_heads(attn, hq, hkv):
    check_append(attn, [30, 9, 200], [4, 1, 33], hq=hq, hkv=hkv, seed=hq)
    check_append(attn, [30, 9, 200], None, hq=hq, hkv=hkv, seed=hq)


@pytest.mark.parametrize("q_dim,rot,start", [(64, 64, 0), (256, 64, 32), (576, 64, 64), (200, 0, 0)])
def test_append_queries_of_other_sizes(attn, q_dim, rot, start):
    if q_dim == 64:
        start = 0
    check_append(attn, [30, 9, 200], [4, 1, 33], q_dim=q_dim, rot=rot, start=start, seed=q_dim)


def test_append_given_positions_and_in_place(attn):
    pos = torch.tensor([5, 0, 1 << 20, 77, 3, 9, 123456])
    check_append(attn, [30, 9, 20], [4, 1, 2], positions=pos, in_place=True, seed=2)


def test_append_ties_and_extremes(attn):
    """Ties go to the even code; a zero vector, infinities and NaN."""
    v = torch.zeros(8, 1, 128, dtype=torch.bfloat16)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    v[1, 0, :8], v[1, 0, 8:16] = ties, -ties
    v[2, 0, 3] = math.inf
    v[3, 0, 100] = math.nan
    v[4] = 3.38e38
    v[5, 0, 7] = 2.0 ** -62
    v[6, 0, 7] = 1e-40
    v[7, 0, 40] = 6.0
    pool = Pool([8], 16, 0)
    cache = Cache(pool, 1, 3)
    got = cache.gpu()
    out = [torch.empty(8, 1, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    attn.attn_append_kv_fp4(v.to(DEV), v.to(DEV), *got, i32([8]), max_kv_len=8,
                            page_table=pool.gpu_table(), q_row_offsets=i32([0, 8]), k_out=out[0],
                            v_out=out[1])
    kc, vc, ks, vs = cache.read(got)
    pg = int(pool.table[0, 0])
    e = ks[pg, :8, 0].int() - 127
    assert e[0].tolist() == [-60] * 4 and vs[pg, 0, 0] == 2.0 ** -60
    want = torch.tensor([0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0])
    for o in out:
        assert torch.equal(o[1, 0, :8].cpu().float(), want)
        assert torch.equal(o[1, 0, 8:16].cpu().float(), -want)
    assert e[2].tolist() == [128, -60, -60, -60] and e[3].tolist() == [-60, -60, -60, 128]
    assert torch.isnan(vs[pg, 2:4, 0]).all()
    assert torch.isnan(out[1][2:4]).all() and torch.isnan(out[0][2, 0, :32]).all()
    assert torch.equal(out[0][2, 0, 32:].cpu().float(), torch.zeros(96))
    assert e[4].tolist() == [125] * 4 and (out[1][4].cpu().double() == 6 * 2.0 ** 125).all()
    assert e[5].tolist() == [-60] * 4 and (out[0][5] == 0).all()
    assert e[6].tolist() == [-60] * 4 and (out[0][6] == 0).all()
    assert e[7].tolist() == [-60, 0, -60, -60] and out[0][7, 0, 40] == 6


def test_append_bad_pages_and_lengths(attn):
    pool = Pool([30, 9], 16, 5)
    x = torch.randn(5, 4, 128).to(torch.bfloat16).to(DEV)
    for table, max_len, flag in (("bad", 30, 2), ("good", 29, 4)):
        cache = Cache(pool, 2, 3)
        got = cache.gpu()
        t = pool.table.clone()
        if table == "bad":
            t[0, 1] = 999
        outs = [torch.full((5, 2, 128), -9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        attn.attn_append_kv_fp4(x[:, :2], x[:, 2:], *got, i32([30, 9]), max_kv_len=max_len,
                                page_table=t.to(DEV), q_row_offsets=i32([0, 3, 5]), k_out=outs[0],
                                v_out=outs[1])
        assert attn.attn_device_error_flags(clear=True) == flag
        kc, _, ks, vs = cache.read(got)
        rows = {pool.place(0, t) for t in ((27, 28) if flag == 4 else ())}
        rows |= {pool.place(1, t) for t in (7, 8)}
        changed = {(p, s) for p in range(pool.pages) for s in range(16)
                   if not torch.equal(kc[p, s], cache.k[p, s])}
        assert changed == rows
        assert (outs[0] != -9).any(-1).all()              # the values of every row are given


# ---- decode -----------------------------------------------------------------------------

class Case:
    def __init__(self, lens, q_lens=None, *, hq=8, hkv=2, page=64, seed=0, sink=False, causal=True,
                 contiguous=False, head_major=False, scale=None, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.q_lens, self.causal, self.group = lens, q_lens, causal, hq // hkv
        rows = sum(q_lens) if q_lens else len(lens)
        self.q = (torch.randn(rows, hq, 128, generator=g) * size).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(128) / 2 if scale is None else scale
        self.sink = torch.randn(hq, generator=g) if sink else None
        self.pool = Pool(lens, page, seed, contiguous)
        self.cache = Cache(self.pool, hkv, seed + 1, head_major)
        self.offsets = None if q_lens is None else [sum(q_lens[:i]) for i in range(len(lens) + 1)]
        # scales of what no token owns must not be used
        dead = torch.ones(self.pool.pages, self.pool.page, dtype=torch.bool)
        for b, L in enumerate(lens):
            for t in range(L):
                dead[self.pool.place(b, t)] = False
        self.cache.ks[dead] = 255
        self.cache.vs[dead] = float("nan")

    def run(self, attn, **kw):
        args = dict(group=self.group, scale=self.scale, max_kv_len=max(max(self.lens), 1),
                    page_table=self.pool.gpu_table(),
                    sink=None if self.sink is None else self.sink.to(DEV),
                    q_row_offsets=i32(self.offsets),
                    max_q_len=max(self.q_lens) if self.q_lens else 1, causal=self.causal)
        args.update(kw)
        out = attn.attn_decode_fp4(self.q.to(DEV), *self.cache.gpu(), i32(self.lens), **args)
        torch.cuda.synchronize()
        return out

    def sequences(self):
        c = self.cache
        seqs = []
        for x in Cache.values(c.k, c.v, c.ks, c.vs):
            if self.pool.table is None:
                seqs.append([x[b, :L] for b, L in enumerate(self.lens)])
            else:
                seqs.append([x[self.pool.table[b, :max(1, -(-L // self.pool.page))].long()]
                             .flatten(0, 1)[:L] for b, L in enumerate(self.lens)])
        return seqs

    def small_weights(self):
        """2^-27 u sum_j 2^(-e_j) |v_j| of every row and head."""
        K, V = self.sequences()
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        for b, L in enumerate(self.lens):
            r0, r1 = (b, b + 1) if self.offsets is None else self.offsets[b:b + 2]
            e = torch.stack([self.cache.vs[self.pool.place(b, t)] for t in range(L)]) if L else None
            for r in range(r0, r1):
                lim = min(L, L - r1 + r + 1) if self.causal else L
                if lim <= 0:
                    continue
                for h in range(self.q.shape[1]):
                    g = h // self.group
                    s = (K[b][:lim, g] @ self.q[r, h].double()) * self.scale
                    m = max(s.max().item(), -math.inf if self.sink is None else float(self.sink[h]))
                    p = torch.exp(s - m)
                    z = p.sum() + (0 if self.sink is None else math.exp(float(self.sink[h]) - m))
                    x = e[:lim, g].double()
                    f = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -126))))
                    u = (p / z * f).max()
                    out[r, h] = 2.0 ** -27 * u * (V[b][:lim, g].abs() / f[:, None]).sum(0)
        return out

    def reference(self):
        seqs = self.sequences()
        return R.decode_reference(self.q, seqs[0], seqs[1], self.lens, group=self.group,
                                  scale=self.scale, offsets=self.offsets, causal=self.causal,
                                  sink=self.sink)

    def check(self, attn, what="", **kw):
        self.compare(*self.run(attn, **kw), what)

    def compare(self, out, lse, what=""):
        o, l = out.cpu().double(), lse.cpu().double()
        eo, el, mass, big = self.reference()
        n = eo.shape[0]
        o, l = o[:n], l[:n]
        rho = (2.0 ** -16 * big + 2.0 ** -20)[..., None]
        bound = (R.BF16_HALF * eo.abs() + 1.01 * (2.0 ** -11 + 2.0 ** -20 + 4 * rho) * mass +
                 self.small_weights()[:n] + 2.0 ** -130)
        worst = ((o - eo).abs() / bound).max().item()
        assert bool(torch.isfinite(o).all()) and worst <= 1, f"{what}: {worst:.3g} times the bound"
        none = el.isneginf()
        assert torch.equal(none, l.isneginf()), f"{what}: -inf lse"
        d = ((l - el).abs() - rho[..., 0] - 2.0 ** -20 * el.abs().clamp_min(1))[~none]
        assert d.numel() == 0 or d.max() <= 0, f"{what}: lse {d.max():.3g} above the bound"


@pytest.mark.parametrize("lens", [[1], [2, 127, 128, 129], [0, 5], [1000, 1, 0, 300, 256, 255, 257],
                                  [37, 100]])
@pytest.mark.parametrize("sink", [False, True])
def test_lengths(attn, lens, sink):
    Case(lens, seed=len(lens), sink=sink).check(attn, f"lens {lens}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 3), (12, 4), (4, 1), (5, 1), (14, 2), (8, 1),
                                    (16, 1), (24, 2), (11, 1)])
def test_groups(attn, hq, hkv):
    Case([300, 5, 129], hq=hq, hkv=hkv, seed=hq).check(attn, f"{hq} on {hkv}")


@pytest.mark.parametrize("page", [8, 16, 32, 128, 256, 1024])
@pytest.mark.parametrize("head_major", [False, True])
def test_pages_and_layouts(attn, page, head_major):
    Case([300, 700, 9], page=page, seed=page, head_major=head_major).check(attn, f"page {page}")


def test_contiguous(attn):
    Case([300, 700, 9], contiguous=True, seed=3, sink=True).check(attn)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,q_lens", [(8, 2, [4, 1, 3, 2]), (2, 2, [16, 3, 0, 9]),
                                           (8, 1, [2, 0, 0, 1]), (4, 2, [5, 8, 1, 2])])
def test_draft_rows(attn, causal, hq, hkv, q_lens):
    Case([300, 3, 129, 1000], q_lens, hq=hq, hkv=hkv, seed=7, causal=causal).check(attn)


def test_row_that_sees_nothing(attn):
    Case([2, 300], [4, 3], seed=5).check(attn)
    Case([0, 300], [2, 3], seed=5, sink=True).check(attn)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.7])
def test_score_scales(attn, scale):
    Case([300, 40], seed=9, scale=scale).check(attn)


@pytest.mark.parametrize("size", [1e-20, 1e-3, 1e3])
def test_sizes_of_queries(attn, size):
    Case([300, 40], seed=9, size=size, scale=0.05 / size).check(attn)


def test_query_channels_of_far_sizes(attn):
    c = Case([300, 40], seed=9, scale=0.01)
    c.q = (c.q.float() * torch.exp2(-torch.arange(128).float() / 8)).to(torch.bfloat16)
    c.check(attn)


def test_scales_of_far_sizes(attn):
    """Groups of channels 2^20 apart in one key, values 2^40 apart."""
    c = Case([300, 200], seed=10, scale=2.0 ** -14)
    live = c.cache.ks != 255
    c.cache.ks = torch.where(live, torch.randint(110, 131, c.cache.ks.shape, dtype=torch.uint8,
                                                 generator=torch.Generator().manual_seed(1)),
                             c.cache.ks)
    vs = torch.exp2(torch.randint(-40, 1, c.cache.vs.shape,
                                  generator=torch.Generator().manual_seed(2)).float()) * 1.37
    c.cache.vs = torch.where(torch.isnan(c.cache.vs), c.cache.vs, vs)
    c.check(attn)


def test_zero_codes_and_scales(attn):
    c = Case([300, 40], seed=4)
    c.cache.k[:, :, 0] = 0
    c.cache.v[:, :, 1] = 0x88                             # -0
    c.cache.vs[:, :8] = torch.where(torch.isnan(c.cache.vs[:, :8]), c.cache.vs[:, :8], 0.0)
    c.check(attn)


def test_many_sequences_cut_and_whole(attn):
    g = torch.Generator().manual_seed(1)
    Case(torch.randint(0, 900, (150,), generator=g).tolist(), hq=4, hkv=1, page=16, seed=2).check(attn)


@pytest.mark.parametrize("batch", [388, 2048])
def test_more_sequences_than_leave_room_for_three_stages(attn, batch):
    g = torch.Generator().manual_seed(batch)
    Case(torch.randint(0, 600 if batch < 1000 else 200, (batch,), generator=g).tolist(), hq=4, hkv=1,
         page=16, seed=2).check(attn)


def test_long_sequence(attn):
    Case([20000], hq=4, hkv=1, page=128, seed=2, sink=True).check(attn)


def test_nan_scales_reach_only_the_rows_that_see_them(attn):
    for kind in ("k", "v"):
        for hq in (4, 8):
            c = Case([300, 200], [4, 2], hq=hq, hkv=2, seed=6)
            clean = c.reference()
            at = c.pool.place(0, 298)                     # the third of four rows' token
            if kind == "k":
                c.cache.ks[at][0, 1] = 255
            else:
                c.cache.vs[at][0] = float("nan")
            out, lse = c.run(attn)
            g = hq // 2
            assert torch.isnan(out[2:4, :g]).all()
            ok = torch.ones(6, hq, dtype=torch.bool)
            ok[2:4, :g] = False
            d = (out.cpu().double() - clean[0]).abs()[ok]
            assert torch.isfinite(out.cpu()[ok]).all() and d.max() < 0.1


def test_rows_of_no_sequence_are_left(attn):
    c = Case([300, 40], [3, 2], seed=5)
    c.q = torch.cat([c.q, torch.full((2, *c.q.shape[1:]), float("nan"), dtype=torch.bfloat16)])
    out = torch.full(c.q.shape, -5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(c.q.shape[:2], -5.0, device=DEV)
    c.run(attn, out=out, lse=lse)
    assert (out[5:] == -5).all() and (lse[5:] == -5).all()
    c.q = c.q[:5]
    c.compare(out[:5], lse[:5])


def test_sequences_that_share_pages(attn):
    c = Case([300, 300, 128], seed=11)
    c.pool.table[1] = c.pool.table[0]
    c.pool.table[2, :2] = c.pool.table[0, :2]
    c.cache = Cache(c.pool, 2, 3)
    c.check(attn)


def test_calls_on_two_streams_at_once(attn):
    cases = [Case([3000], hq=4, hkv=1, seed=1), Case([500, 900, 20], [2, 4, 1], seed=2)]
    torch.cuda.synchronize()
    got = [c.run(attn, stream=torch.cuda.Stream()) for c in cases]
    torch.cuda.synchronize()
    for c, o in zip(cases, got):
        c.compare(*o)


def test_captured_and_replayed_with_other_lengths(attn):
    big = Case([900, 500, 300], [4, 2, 3], seed=12)
    q, cache, lens = big.q.to(DEV), big.cache.gpu(), i32(big.lens)
    args = dict(group=4, scale=big.scale, max_kv_len=900, page_table=big.pool.gpu_table(),
                q_row_offsets=i32(big.offsets), max_q_len=4, causal=True)
    attn.attn_decode_fp4(q, *cache, lens, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attn.attn_decode_fp4(q, *cache, lens, **args)
    for new in ([900, 500, 300], [130, 2, 0], [1, 400, 256]):
        c = Case([900, 500, 300], [4, 2, 3], seed=12)
        c.lens = new
        lens.copy_(torch.tensor(new))
        graph.replay()
        torch.cuda.synchronize()
        c.compare(out, lse, f"replay {new}")


def test_bad_page_and_length_are_reported(attn):
    c = Case([300, 100], seed=3)
    bad = c.pool.gpu_table()
    bad[0, 1] = 1 << 20
    c.run(attn, page_table=bad)
    assert attn.attn_device_error_flags(clear=True) == 2
    c.run(attn, max_kv_len=299)
    assert attn.attn_device_error_flags(clear=True) == 4
    c = Case([300, 100], [5, 1], seed=3)
    c.run(attn, max_q_len=4)
    assert attn.attn_device_error_flags(clear=True) & 4


def test_offsets_beyond_32_bits(attn):
    """Pages past 4 GB of codes."""
    pages, page = (1 << 26) // 64 + 8, 64                  # 4 GB and a bit of codes each
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    c = Case([300], hq=4, hkv=1, page=64, seed=5)
    small = c.cache.gpu()
    k, v = (torch.empty((pages, page, 1, 64), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks = torch.empty((pages, page, 1, 4), dtype=torch.uint8, device=DEV)
    vs = torch.empty((pages, page, 1), device=DEV)
    far = pages - c.pool.pages
    for big, x in zip((k, v, ks, vs), small):
        big[far:] = x.view(torch.uint8) if x.dtype == torch.float8_e8m0fnu else x
    table = c.pool.gpu_table() + far
    out, lse = attn.attn_decode_fp4(c.q.to(DEV), k, v, ks.view(torch.float8_e8m0fnu), vs, i32([300]),
                                    group=4, scale=c.scale, max_kv_len=300, page_table=table)
    c.compare(out, lse)


def test_append_beyond_32_bits(attn):
    """A prompt into pages past 4 GB of codes: what it leaves near the base."""
    pages = (1 << 20) + 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")

    def caches(n):
        k, v = (torch.zeros((n, 64, 1, 64), dtype=torch.uint8, device=DEV) for _ in range(2))
        ks = torch.zeros((n, 64, 1, 4), dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        return k, v, ks, torch.zeros((n, 64, 1), device=DEV)

    x = torch.randn(300, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    table = i32([[3, 0, 7, 2, 5]])
    near, far = caches(8), caches(pages)
    for cache, at in ((near, 0), (far, pages - 8)):
        attn.attn_append_kv_fp4(x[:, :1], x[:, 1:], *cache, i32([300]), max_kv_len=320,
                                page_table=table + at, q_row_offsets=i32([0, 300]))
    for a, b in zip(near, far):
        a, b = (t.view(torch.uint8) for t in (a, b))
        assert torch.equal(a, b[pages - 8:]) and bool(a.any()) and not bool(b[:8].any())


@pytest.mark.parametrize("capacity,padded", [(703, 704), (702, 702), (701, 703)])
@pytest.mark.parametrize("hkv", [1, 2])
def test_scales_on_any_boundary(attn, capacity, padded, hkv):
    """Contiguous caches whose scales end inside four tokens, begin on 16 bytes or do not."""
    c = Case([capacity, 650], hq=4 * hkv, hkv=hkv, contiguous=True, head_major=True, seed=capacity)
    assert c.cache.k.shape[1] == capacity
    k, v, ks, vs = c.cache.gpu()
    wide = [torch.zeros(2, hkv, padded, 4, dtype=torch.uint8, device=DEV),
            torch.full((2, hkv, padded), math.nan, device=DEV)]
    wide[0].fill_(255)
    e, s = wide[0][:, :, :capacity].transpose(1, 2), wide[1][:, :, :capacity].transpose(1, 2)
    e.copy_(ks.view(torch.uint8))
    s.copy_(vs)
    e = wide[0].view(torch.float8_e8m0fnu)[:, :, :capacity].transpose(1, 2)
    out, lse = attn.attn_decode_fp4(c.q.to(DEV), k, v, e, s, i32(c.lens), group=4, scale=c.scale,
                                    max_kv_len=capacity)
    c.compare(out, lse)


# ---- together ---------------------------------------------------------------------------

@pytest.mark.parametrize("q_lens", [None, [3, 1, 2]])
def test_append_then_decode(attn, q_lens):
    """A step: new tokens appended, then attended to with all before; the rows that are read
    are those the codes stand for."""
    c = Case([300, 64, 129], q_lens, seed=14)
    rows = c.q.shape[0]
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    cache = c.cache.gpu()
    q = attn.attn_append_kv_fp4(x[:, :2], x[:, 2:], *cache, i32(c.lens), max_kv_len=300,
                                page_table=c.pool.gpu_table(), q=c.q.to(DEV),
                                q_row_offsets=i32(c.offsets))
    assert torch.equal(q.cpu(), c.q)                      # neither normed nor rotated
    c.cache.k, c.cache.v, c.cache.ks, c.cache.vs = c.cache.read(cache)
    c.check(attn)


def test_a_prompt_cut_to_its_heaviest_keys(attn):
    """The whole run: a prompt attended to in bf16, the weight of its keys, the heaviest kept,
    held in 4 bits, and decoding over them with new tokens at their positions."""
    torch.manual_seed(3)
    lens, hq, hkv, page, keep = [700, 260], 8, 2, 64, 128
    rows = sum(lens)
    offs = i32([0, lens[0], rows])
    x = torch.randn(rows, hq + 2 * hkv, 128, device=DEV).to(torch.bfloat16)
    turns, _ = attn.rope_turns(128, 10000.0, device=DEV)
    rope = attn.Rope(turns)
    table = i32([list(range(11)), list(range(11, 16)) + [0] * 6])
    kc, vc = (torch.zeros(16, page, hkv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kv_len = i32(lens)
    kw = dict(max_kv_len=700, page_table=table)
    q = attn.attn_append_kv(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, kv_len, q=x[:, :hq],
                            q_row_offsets=offs, rope=rope, **kw)
    _, lse = attn.attn_decode(q, kc, vc, kv_len, group=4, scale=0.1, q_row_offsets=offs,
                              max_q_len=700, causal=True, **kw)
    w = torch.full((16, page, hkv), float("nan"), device=DEV)
    attn.attn_key_weights(q, kc, lse, kv_len, w, group=4, scale=0.1, q_row_offsets=offs,
                          max_q_len=700, causal=True, **kw)
    # every row's weights sum to 1
    got = w[table[0, :11].long()].flatten(0, 1)[:700].sum(0)
    assert torch.allclose(got, torch.full((2,), 700.0 * 4, device=DEV), rtol=1e-3)
    small = [torch.zeros(2, keep, hkv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    w2 = torch.zeros(2, keep, hkv, device=DEV)
    kept, index = attn.attn_evict_kv(kc, vc, w, kv_len, i32([keep, keep]), *small, w2, first=4,
                                     recent=32, max_keep=keep, **kw)
    assert kept.tolist() == [keep, keep]
    # into a cache in 4 bits, the keys rotated already
    pool = Pool([keep + 3, keep + 1], page, 4)
    cache = Cache(pool, hkv, 5).gpu()
    attn.attn_append_kv_fp4(small[0].flatten(0, 1), small[1].flatten(0, 1), *cache, kept,
                            max_kv_len=keep, page_table=pool.gpu_table(),
                            q_row_offsets=i32([0, keep, 2 * keep]))
    # new tokens behind them, at their positions in the text
    y = torch.randn(4, hq + 2 * hkv, 128, device=DEV).to(torch.bfloat16)
    new, offs2 = i32([keep + 3, keep + 1]), i32([0, 3, 4])
    q2 = attn.attn_append_kv_fp4(y[:, hq:hq + hkv], y[:, hq + hkv:], *cache, new,
                                 max_kv_len=keep + 3, page_table=pool.gpu_table(), q=y[:, :hq],
                                 q_row_offsets=offs2, rope=rope,
                                 positions=i32([700, 701, 702, 260]))
    c = Case([keep + 3, keep + 1], [3, 1], hq=hq, hkv=hkv, page=page, seed=1, scale=0.1)
    c.pool, c.q = pool, q2.cpu()
    c.cache.k, c.cache.v, c.cache.ks, c.cache.vs = c.cache.read(cache)
    c.compare(*attn.attn_decode_fp4(q2, *cache, new, group=4, scale=0.1, max_kv_len=keep + 3,
                                    page_table=pool.gpu_table(), q_row_offsets=offs2, max_q_len=3,
                                    causal=True))
