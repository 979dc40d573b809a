"""Filling a KV cache on the GPU: norm and rotation of head rows, appending to a
bf16 cache and to a cache held in 8 bits, against 64-bit references."""
import math

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def attn():
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn as a
    a.attn_device_error_flags(clear=True)
    yield a
    assert a.attn_device_error_flags(clear=True) == 0


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def rope_of(attn, rot, *, theta=500000.0, start=0, interleaved=False, **scaling):
    turns, mscale = attn.rope_turns(rot, theta, **scaling)
    return turns, attn.Rope(turns.to(DEV), interleaved=interleaved, mscale=mscale, start=start)


# ---- norm and rotation ------------------------------------------------------

# dim, rotated channels, first rotated channel, normed channels
SHAPES = [(128, 128, 0, 128), (128, 64, 0, 0), (128, 32, 96, 128), (64, 64, 0, 64),
          (96, 96, 0, 96), (96, 32, 64, 0), (192, 64, 128, 0), (256, 128, 0, 256),
          (576, 64, 512, 512), (8, 8, 0, 8), (128, 20, 8, 128), (128, 2, 0, 0),
          (1024, 1024, 0, 1024), (128, 0, 0, 128), (80, 40, 40, 80), (128, 16, 16, 64),
          (128, 128, 0, 64), (128, 24, 16, 128), (640, 512, 64, 640), (40, 8, 8, 40)]


@pytest.mark.parametrize("dim,rot,start,nd", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation(attn, dim, rot, start, nd, interleaved):
    rows, hq, hkv = 37, 6, 2
    q, k = randn(dim + rot, rows, hq, dim), randn(dim + rot + 1, rows, hkv, dim, scale=30.0)
    qn = (1 + randn(3, nd, scale=0.2)).to(torch.bfloat16) if nd else None
    kn = (1 + randn(4, nd, scale=0.2)).to(torch.bfloat16) if nd else None
    pos = torch.randint(0, 1 << 20, (rows,), generator=torch.Generator().manual_seed(rot),
                        dtype=torch.int32)
    pos[:4] = torch.tensor([0, 1, 2 ** 31 - 1, -5], dtype=torch.int32)
    turns, rope = rope_of(attn, rot, start=start, interleaved=interleaved, scaling="yarn",
                          factor=4.0, original_len=4096) if rot else (None, None)
    cu = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    qo, ko = attn.attn_qk_norm_rope(cu(q), cu(k), cu(pos), rope=rope, q_norm=cu(qn),
                                    k_norm=cu(kn), eps=1e-5)
    m = 1.0 if rope is None else rope.struct.mscale
    for got, x, w, name in ((qo, q, qn, "q"), (ko, k, kn, "k")):
        exact, err = R.head_rows(x, turns, pos, norm=w, eps=1e-5, start=start,
                                 interleaved=interleaved, mscale=m)
        R.assert_bf16(got, exact, err, f"{name} dim {dim} rot {rot}+{start} norm {nd}")


@pytest.mark.parametrize("rows,hq,hkv", [(1, 32, 8), (1, 1, 0), (3, 128, 1), (300, 5, 3),
                                         (4099, 32, 8)])
def test_rows_and_heads(attn, rows, hq, hkv):
    """From one head of one row to many rows, out of a packed projection."""
    packed = randn(rows, rows, hq + 2 * hkv, 128).to(DEV)
    q = packed[:, :hq]
    k = packed[:, hq:hq + hkv] if hkv else None
    pos = torch.arange(rows, dtype=torch.int32) + 131000
    turns, rope = rope_of(attn, 128)
    qo, ko = attn.attn_qk_norm_rope(q, k, pos.to(DEV), rope=rope)
    assert (ko is None) == (k is None)
    pick = torch.tensor(sorted({0, rows // 2, rows - 1}))
    for got, x in ((qo, q), (ko, k)):
        if x is not None:
            exact, err = R.head_rows(x.cpu()[pick], turns, pos[pick])
            R.assert_bf16(got.cpu()[pick], exact, err, f"rows {rows}")
    # the other rows: each as if it came alone
    one, _ = attn.attn_qk_norm_rope(q[rows - 1:], None, pos[rows - 1:].to(DEV), rope=rope)
    assert torch.equal(one[0], qo[rows - 1])


def test_in_place_and_strided(attn):
    base = randn(5, 50, 48, 160).to(DEV)
    turns, rope = rope_of(attn, 128, interleaved=True)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    x = base[:, 8:40, 16:144]                       # channels contiguous, wide strides
    want, _ = attn.attn_qk_norm_rope(x, None, pos, rope=rope)
    keep = base.clone()
    attn.attn_qk_norm_rope(x, None, pos, rope=rope, q_out=x)
    assert torch.equal(x, want)
    keep[:, 8:40, 16:144] = want
    assert torch.equal(base, keep)                  # nothing beside the heads


def test_norm_without_rotation_of_extreme_rows(attn):
    """A row of zeros, huge and tiny rows; fp32 sums of squares must not overflow below 1e19."""
    x = torch.zeros(5, 1, 128, dtype=torch.bfloat16)
    x[1] = 1e18
    x[2] = 1e-18
    x[3, 0, 7] = 3.0
    x[4] = -1.0
    got, _ = attn.attn_qk_norm_rope(x.to(DEV), q_norm=torch.ones(128, dtype=torch.bfloat16,
                                                                   device=DEV), eps=1e-6)
    exact, err = R.head_rows(x, None, None, norm=torch.ones(128), eps=1e-6)
    R.assert_bf16(got, exact, err, "extreme rows")


def test_no_rows(attn):
    q = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    out, _ = attn.attn_qk_norm_rope(q, None, torch.empty(0, dtype=torch.int32, device=DEV),
                                    rope=rope_of(attn, 128)[1])
    assert out.shape == (0, 4, 128)


# ---- appending --------------------------------------------------------------

class Pool:
    """A paged (or contiguous) cache layout with a table of scattered pages."""

    def __init__(self, lens, page, seed, spare=2, contiguous=False):
        self.lens, self.page, self.contiguous = lens, page, contiguous
        if contiguous:
            self.pages, self.table = len(lens), None
            return
        need = [max(1, -(-x // page)) for x in lens]
        g = torch.Generator().manual_seed(seed)
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=g)
        self.table = torch.zeros(len(lens), max(need), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n

    def place(self, b, t):
        if self.contiguous:
            return b, t
        return int(self.table[b, t // self.page]), t % self.page


def rows_of(lens, q_lens):
    """(row, sequence, token) of every row."""
    r = 0
    for b, n in enumerate(q_lens):
        for i in range(n):
            yield r, b, lens[b] - n + i
            r += 1


CASES = [
    # lens, rows per sequence (None: one each), page, contiguous
    ([1], None, 64, False),
    ([1, 64, 65, 128, 700, 0, 33], None, 64, False),
    ([5, 300, 17], [5, 130, 1], 16, False),
    ([40, 200, 9, 64], [1, 200, 9, 3], 32, True),
    ([1000, 1, 8, 513], [600, 0, 8, 2], 128, False),
]


@pytest.mark.parametrize("lens,q_lens,page,contiguous", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_bf16(attn, lens, q_lens, page, contiguous, interleaved):
    hq, hkv, dim = 6, 3, 128
    rows = sum(q_lens) if q_lens else len(lens)
    counts = q_lens or [1] * len(lens)
    pool = Pool(lens, 256 if contiguous else page, 3, contiguous=contiguous)
    size = 1 + rows + 2                                       # rows behind the last sequence
    packed = randn(rows, size if q_lens else rows, hq + 2 * hkv, dim)
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    kc = randn(1, pool.pages, pool.page, hkv, dim)
    vc = randn(2, pool.pages, pool.page, hkv, dim)
    kn = (1 + randn(4, dim, scale=0.2)).to(torch.bfloat16)
    turns, rope = rope_of(attn, 64, start=32, interleaved=interleaved)
    kg, vg = kc.to(DEV), vc.to(DEV)
    pg = packed.to(DEV)
    qo = torch.full((pg.shape[0], hq, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    offs = None
    if q_lens:
        offs = torch.tensor([sum(q_lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    attn.attn_append_kv(pg[:, hq:hq + hkv], pg[:, hq + hkv:], kg, vg,
                        torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=max(lens),
                        page_table=None if contiguous else pool.table.to(DEV), q=pg[:, :hq],
                        q_out=qo, q_row_offsets=None if offs is None else offs.to(DEV), rope=rope,
                        k_norm=kn.to(DEV))
    torch.cuda.synchronize()
    places = [(r, b, t) for r, b, t in rows_of(lens, counts)]
    tokens = torch.tensor([max(t, 0) for _, _, t in places], dtype=torch.int64)
    ke, kerr = R.head_rows(k[:rows], turns, tokens, norm=kn, start=32, interleaved=interleaved)
    qe, qerr = R.head_rows(q[:rows], turns, tokens, start=32, interleaved=interleaved)
    R.assert_bf16(qo[:rows], qe, qerr, "q")
    assert (qo[rows:] == 7.0).all()
    kh, vh = kg.cpu(), vg.cpu()
    for r, b, t in places:
        if t < 0:
            continue
        pg_, slot = pool.place(b, t)
        R.assert_bf16(kh[pg_, slot], ke[r], kerr[r], f"k of row {r}")
        assert torch.equal(vh[pg_, slot], v[r])
        kh[pg_, slot], vh[pg_, slot] = kc[pg_, slot], vc[pg_, slot]
    assert torch.equal(kh, kc) and torch.equal(vh, vc)        # nothing else was written


def test_append_latent_rows(attn):
    """Rows of 576 channels, 512 normed and 64 rotated, without a V cache."""
    lens, q_lens = [70, 3, 200], [2, 1, 4]
    pool = Pool(lens, 64, 9)
    k, q = randn(1, 7, 1, 576), randn(2, 7, 16, 576)
    kn = (1 + randn(4, 512, scale=0.2)).to(torch.bfloat16)
    turns, rope = rope_of(attn, 64, start=512, interleaved=True)
    cache = torch.zeros(pool.pages, 64, 1, 576, dtype=torch.bfloat16, device=DEV)
    qo = attn.attn_append_kv(k.to(DEV), None, cache, None,
                             torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=200,
                             page_table=pool.table.to(DEV), q=q.to(DEV),
                             q_row_offsets=torch.tensor([0, 2, 3, 7], dtype=torch.int32,
                                                        device=DEV), rope=rope,
                             k_norm=kn.to(DEV))
    places = list(rows_of(lens, q_lens))
    tokens = torch.tensor([t for _, _, t in places])
    ke, kerr = R.head_rows(k, turns, tokens, norm=kn, start=512, interleaved=True)
    qe, qerr = R.head_rows(q, turns, tokens, start=512, interleaved=True)
    R.assert_bf16(qo, qe, qerr, "q")
    ch = cache.cpu()
    for r, b, t in places:
        R.assert_bf16(ch[pool.place(b, t)], ke[r], kerr[r], f"row {r}")
    assert int((ch.abs().sum((1, 2, 3)) > 0).sum()) <= 5


def test_append_positions_and_bad_rows(attn):
    """Given positions replace the tokens'; a length above the bound and a page outside the pool
    are reported, not stored."""
    kc = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = randn(1, 4, 1, 128).to(DEV), randn(2, 4, 1, 128).to(DEV)
    table = torch.tensor([[0, 1], [9, 9], [2, 2], [3, 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([17, 3, 33, 1], dtype=torch.int32, device=DEV)
    turns, rope = rope_of(attn, 128)
    pos = torch.tensor([100000, 5, 6, 7], dtype=torch.int32)
    attn.attn_append_kv(k, v, kc, vc, lens, max_kv_len=32, page_table=table, rope=rope,
                        positions=pos.to(DEV))
    assert attn.attn_device_error_flags(clear=True) == 6
    exact, err = R.head_rows(k.cpu(), turns, pos)
    R.assert_bf16(kc[1, 0], exact[0], err[0], "row 0")
    R.assert_bf16(kc[3, 0], exact[3], err[3], "row 3")
    assert torch.equal(vc[1, 0], v[0]) and torch.equal(vc[3, 0], v[3])
    assert int((vc != 0).any(-1).sum()) == 2


# ---- appending to the 8-bit cache -------------------------------------------

def check_fp8(attn, lens, q_lens, page, block, seed, *, contiguous=False, magnitude=0.0, hkv=2,
              rope_kw=None):
    dim, hq = 128, 4
    counts = q_lens or [1] * len(lens)
    rows = sum(counts)
    pool = Pool(lens, page, seed, contiguous=contiguous)
    g = torch.Generator().manual_seed(seed)
    scale = torch.exp2(torch.randn(rows, 1, 1, generator=g) * magnitude)
    packed = (torch.randn(rows, hq + 2 * hkv, dim, generator=g) * scale).to(torch.bfloat16)
    old = {}
    for name in "kv":
        e = torch.randint(-8, 3, (pool.pages, page // block, hkv), generator=g).float()
        codes = (torch.randn(pool.pages, page, hkv, dim, generator=g) * 100).clamp(-448, 448)
        old[name] = (codes.to(FP8), torch.exp2(e))
    turns, rope = rope_of(attn, 128, **(rope_kw or {}))
    kn = (1 + randn(4, dim, scale=0.2)).to(torch.bfloat16)
    new = {n: (old[n][0].to(DEV), old[n][1].to(DEV)) for n in "kv"}
    offs = None
    if q_lens:
        offs = torch.tensor([sum(q_lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    pg = packed.to(DEV)
    qo = attn.attn_append_kv_fp8(
        pg[:, hq:hq + hkv], pg[:, hq + hkv:], new["k"][0], new["v"][0], new["k"][1], new["v"][1],
        torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=max(lens),
        max_q_len=max(counts), page_table=None if contiguous else pool.table.to(DEV),
        q=pg[:, :hq], q_row_offsets=None if offs is None else offs.to(DEV), rope=rope,
        k_norm=kn.to(DEV))
    torch.cuda.synchronize()
    places = list(rows_of(lens, counts))
    tokens = torch.tensor([max(t, 0) for _, _, t in places], dtype=torch.int64)
    inter = bool(rope.struct.interleaved)
    qe, qerr = R.head_rows(packed[:, :hq], turns, tokens, interleaved=inter)
    R.assert_bf16(qo, qe, qerr, "q")
    ke, kerr = R.head_rows(packed[:, hq:hq + hkv], turns, tokens, norm=kn, interleaved=inter)
    rows64 = {"k": (ke, kerr), "v": (packed[:, hq + hkv:].double(),
                                     torch.zeros(rows, hkv, dim, dtype=torch.float64))}
    for name, (x, err) in rows64.items():
        codes = new[name][0].cpu().float().double()
        scales = new[name][1].cpu().double()
        c0, s0 = old[name][0].float().double(), old[name][1].double()
        want_codes, want_scales = c0.clone(), s0.clone()
        blocks = {}
        for r, b, t in places:
            if t >= 0:
                blocks.setdefault((b, t // block), []).append((r, t))
        for (b, _), members in blocks.items():
            r0, t0 = members[0]
            pgi, slot = pool.place(b, t0)
            blk, held = slot // block, t0 % block
            ids = [r for r, _ in members]
            amax = x[ids].abs().amax((0, 2))
            slack = err[ids].amax((0, 2))
            lo, hi = R.scale_exponents(amax - slack), R.scale_exponents(amax + slack)
            got = torch.log2(scales[pgi, blk])
            if held:
                lo = torch.maximum(lo, torch.log2(s0[pgi, blk]))
                hi = torch.maximum(hi, torch.log2(s0[pgi, blk]))
            assert ((got >= lo) & (got <= hi)).all(), f"{name} scale of block {blk}: {got} {lo} {hi}"
            want_scales[pgi, blk] = scales[pgi, blk]
            s = scales[pgi, blk][:, None]
            if held:
                first = slot - held
                exact = c0[pgi, first:slot] * (s0[pgi, blk][:, None] / s)
                d = (codes[pgi, first:slot] - exact).abs()
                assert (d <= R.half_step(exact)).all(), f"{name}: a held code"
                want_codes[pgi, first:slot] = codes[pgi, first:slot]
            for r, t in members:
                p2, slot2 = pool.place(b, t)
                d = (codes[p2, slot2] - x[r] / s).abs()
                bound = R.half_step(x[r] / s) + err[r] / s * (1 + 2.0 ** -3)
                assert (d <= bound).all(), f"{name}: row {r}, {(d - bound).max():.3g} above"
                want_codes[p2, slot2] = codes[p2, slot2]
        assert torch.equal(codes, want_codes), f"{name}: a code elsewhere changed"
        assert torch.equal(scales, want_scales), f"{name}: a scale elsewhere changed"


@pytest.mark.parametrize("block", [1, 2, 8, 16, 64])
def test_append_fp8_single_rows(attn, block):
    check_fp8(attn, [1, 64, 65, 128, 700, 0, 33, 16, 17, 2], None, 64, block, 100 + block,
              magnitude=4.0)


@pytest.mark.parametrize("page,block,q_lens", [
    (16, 16, [5, 130, 1]), (128, 128, [600, 1, 8]), (64, 4, [3, 0, 200]), (32, 1, [40, 40, 40]),
    (256, 256, [700, 300, 2]), (8, 8, [9, 17, 33]), (1024, 512, [600, 3, 200]),
    # tiles of a few rows in calls with long runs, blocks of every size
    (128, 16, [140, 5, 129, 33]), (128, 64, [150, 20, 131]), (32, 1, [50, 7, 130, 1]),
    (128, 128, [40, 100, 3])])
def test_append_fp8_ragged(attn, page, block, q_lens):
    lens = [n + x for n, x in zip(q_lens, (7, 130, 70, 126))]
    check_fp8(attn, lens, q_lens, page, block, page + block, magnitude=2.0,
              rope_kw=dict(interleaved=True))


def test_append_fp8_contiguous(attn):
    check_fp8(attn, [40, 200, 9, 255], [1, 200, 9, 3], 256, 32, 5, contiguous=True, hkv=8)


@pytest.mark.parametrize("block", [1, 64])
def test_append_fp8_extreme_values(attn, block):
    """Zeros, values at the borders of a scale, the largest and least bf16 numbers, infinities and
    NaN (which become NaN and leave the scale to the finite values)."""
    x = torch.zeros(8, 1, 128, dtype=torch.bfloat16)
    x[1, 0, 5] = 448.0
    x[2, 0, 5] = 450.0
    x[3] = 3.3e38
    x[4, 0, 1] = 1e-38
    x[5, 0, 3], x[5, 0, 4], x[5, 0, 5] = float("inf"), float("nan"), 2.0
    x[6, 0, 9] = -448.0 * 2.0 ** -20
    x[7] = float("nan")
    cache = [torch.zeros(8, 64, 1, 128, dtype=FP8, device=DEV) for _ in range(2)]
    scales = [torch.ones(8, 64 // block, 1, device=DEV) for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device=DEV)[:, None].contiguous()
    attn.attn_append_kv_fp8(x.to(DEV), x.to(DEV), *cache, *scales,
                            torch.ones(8, dtype=torch.int32, device=DEV), max_kv_len=64,
                            page_table=table)
    for c, s in zip(cache, scales):
        codes, e = c.cpu().float()[:, 0, 0], torch.log2(s.cpu()[:, 0, 0])
        assert e.tolist()[:5] == [-60, 0, 1, 120, -60]
        assert e[5] == -7 and e[6] == -20 and e[7] == -60
        assert codes[0].abs().max() == 0 and codes[1, 5] == 448 and codes[2, 5] == 224
        assert (codes[3] - 3.3e38 / 2.0 ** 120).abs().max() <= 16
        assert codes[4].abs().max() == 0
        assert codes[5, 3:5].isnan().all() and codes[5, 5] == 256 and not codes[5, 6:].any()
        assert codes[6, 9] == -448 and codes[7].isnan().all()


def test_append_fp8_again_changes_nothing(attn):
    """The same rows appended twice: the second call finds the scales grown and the codes placed."""
    lens, q_lens = [70, 33, 64], [3, 1, 20]
    pool = Pool(lens, 64, 1)
    k, v = randn(1, 24, 2, 128, scale=9.0).to(DEV), randn(2, 24, 2, 128).to(DEV)
    cache = [(torch.randn(pool.pages, 64, 2, 128, device=DEV) * 50).to(FP8) for _ in range(2)]
    scales = [torch.full((pool.pages, 2, 2), 2.0 ** -9, device=DEV) for _ in range(2)]

    def go():
        attn.attn_append_kv_fp8(k, v, *cache, *scales,
                                torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=70,
                                max_q_len=20, page_table=pool.table.to(DEV),
                                q_row_offsets=torch.tensor([0, 3, 4, 24], dtype=torch.int32,
                                                           device=DEV))
        return [c.view(torch.uint8).clone() for c in cache] + [s.clone() for s in scales]

    for a, b in zip(go(), go()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("runs", [[1, 1, 1, 1], [40, 2, 50, 1]])
def test_append_fp8_bad_pages_and_lengths(attn, runs):
    """A page outside the pool, a length above the bound and rows before token 0 are reported;
    their queries are written, their keys are not, and the others' are as alone."""
    page, hkv = 16, 2
    lens = [max(runs[0], 17), 3, max(runs[2], 1) if runs[2] > 1 else 33, 1]
    if runs[2] > 1:
        lens[2] = 49                                     # 50 rows: the first has token -1
    cap = 48
    table = torch.tensor([[0, 1, 2, 3], [99, 99, 99, 99], [4, 5, 6, 7], [8, 8, 8, 8]],
                         dtype=torch.int32, device=DEV)
    rows = sum(runs)
    x = randn(21, rows, 4 + 2 * hkv, 128).to(DEV)
    offs = torch.tensor([sum(runs[:i]) for i in range(5)], dtype=torch.int32, device=DEV)
    turns, rope = rope_of(attn, 128)

    def go(which, lens, table, runs, offs, x):
        c = [torch.zeros(9, page, hkv, 128, dtype=FP8, device=DEV) for _ in range(2)]
        s = [torch.ones(9, 2, hkv, device=DEV) for _ in range(2)]
        q = attn.attn_append_kv_fp8(
            x[:, 4:4 + hkv], x[:, 4 + hkv:], *c, *s,
            torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=cap,
            max_q_len=max(runs), page_table=table, q=x[:, :4],
            q_row_offsets=offs if max(runs) > 1 else None, rope=rope)
        return q, c, s

    q, c, s = go("all", lens, table, runs, offs, x)
    # (single rows: every length within the bound)
    assert attn.attn_device_error_flags(clear=True) == (6 if max(runs) > 1 else 2)
    n0 = runs[0]
    tokens = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, runs)]).clamp_min(0)
    exact, err = R.head_rows(x[:, :4].cpu(), turns, tokens)
    R.assert_bf16(q, exact, err, "q")
    # the first sequence alone gives the same pages
    o1 = torch.tensor([0, n0], dtype=torch.int32, device=DEV)
    _, c1, s1 = go("one", lens[:1], table[:1].contiguous(), runs[:1], o1, x[:n0])
    assert attn.attn_device_error_flags(clear=True) == 0
    for a, b in zip(c + s, c1 + s1):
        a, b = (t.view(torch.uint8) if t.dtype == FP8 else t for t in (a, b))
        assert torch.equal(a[:4], b[:4])
    live = c[1].float().abs().sum((2, 3)) > 0            # [page, slot] with values
    assert int(live[:4].sum()) == min(n0, cap) and int(live[8].sum()) == 1
    assert int(live[4:8].sum()) == (min(lens[2], cap) if runs[2] > 1 else 1)


@pytest.mark.parametrize("dim,inter", [(256, False), (256, True), (200, False), (64, True)])
def test_append_bf16_many_rows(attn, dim, inter):
    """Enough rows for CTAs of several heads and 16 rows, in sequences of every length."""
    lens = [700, 3000, 1, 900, 640]
    q_lens = [650, 2999, 1, 900, 577]
    rows, page = sum(q_lens), 64
    pool = Pool(lens, page, 8)
    rot = 64
    x = randn(5, rows, 5, dim)
    turns, rope = rope_of(attn, rot, interleaved=inter)
    kn = (1 + randn(6, dim, scale=0.2)).to(torch.bfloat16)
    offs = torch.tensor([sum(q_lens[:i]) for i in range(6)], dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros(pool.pages, page, 1, dim, dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    g = x.to(DEV)
    qo = attn.attn_append_kv(g[:, 3:4], g[:, 4:], kc, vc,
                             torch.tensor(lens, dtype=torch.int32, device=DEV), max_kv_len=3000,
                             page_table=pool.table.to(DEV), q=g[:, :3], q_row_offsets=offs,
                             rope=rope, k_norm=kn.to(DEV))
    places = list(rows_of(lens, q_lens))
    tokens = torch.tensor([t for _, _, t in places])
    qe, qerr = R.head_rows(x[:, :3], turns, tokens, interleaved=inter)
    R.assert_bf16(qo, qe, qerr, "q")
    at = torch.tensor([pool.place(b, t) for _, b, t in places])
    ke, kerr = R.head_rows(x[:, 3:4], turns, tokens, norm=kn, interleaved=inter)
    R.assert_bf16(kc.cpu()[at[:, 0], at[:, 1]], ke, kerr, "k")
    assert torch.equal(vc.cpu()[at[:, 0], at[:, 1]], x[:, 4:])
    assert int((vc != 0).any(-1).sum()) <= rows


@pytest.mark.parametrize("dim,rot,start", [(64, 0, 0), (192, 0, 0), (256, 0, 0), (256, 64, 32),
                                           (576, 64, 512), (40, 0, 0)])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [4, 1, 2], [40, 3, 130]])
def test_append_fp8_query_heads_of_other_sizes(attn, dim, rot, start, q_lens):
    """Queries need not have the keys' 128 channels."""
    lens = [200, 77, 140]
    pool = Pool(lens, 64, 3)
    rows = sum(q_lens)
    k, v, q = randn(1, rows, 2, 128), randn(2, rows, 2, 128), randn(3, rows, 6, dim)
    qn = (1 + randn(4, dim, scale=0.2)).to(torch.bfloat16)
    turns, rope = rope_of(attn, rot, start=start) if rot else (None, None)
    offs = torch.tensor([sum(q_lens[:i]) for i in range(4)], dtype=torch.int32, device=DEV)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tokens = torch.tensor([t for _, _, t in rows_of(lens, q_lens)])
    # (the rotation's place is the queries': keys rotated alike only where they fit)
    if rot and start + rot > 128:
        with pytest.raises(attn.AttnError):
            attn.attn_append_kv_fp8(k.to(DEV), v.to(DEV), *fresh8(pool), L, max_kv_len=200,
                                    max_q_len=max(q_lens), page_table=pool.table.to(DEV),
                                    q=q.to(DEV), q_row_offsets=offs, rope=rope)
        return
    with_q, without = fresh8(pool), fresh8(pool)
    kw = dict(max_kv_len=200, max_q_len=max(q_lens), page_table=pool.table.to(DEV),
              q_row_offsets=offs, rope=rope)
    qo = attn.attn_append_kv_fp8(k.to(DEV), v.to(DEV), *with_q, L, q=q.to(DEV), q_norm=qn.to(DEV),
                                 **kw)
    attn.attn_append_kv_fp8(k.to(DEV), v.to(DEV), *without, L, **kw)
    exact, err = R.head_rows(q, turns, tokens, norm=qn, start=start)
    R.assert_bf16(qo, exact, err, "q")
    for a, b in zip(with_q, without):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert a.float().abs().sum() > 0


def fresh8(pool):
    return ([torch.zeros(pool.pages, 64, 2, 128, dtype=FP8, device=DEV) for _ in range(2)] +
            [torch.ones(pool.pages, 4, 2, device=DEV) for _ in range(2)])


@pytest.mark.parametrize("kind", ["bf16", "latent", "odd", "fp8", "fp8 odd"])
def test_rows_of_no_sequence_are_left(attn, kind):
    """Rows before the first offset and behind the last: neither stored nor written."""
    lens, q_lens, pad = [70, 3, 200], [2, 1, 60], 5
    pool = Pool(lens, 64, 9)
    dim = 576 if kind == "latent" else 128
    hkv = 1 if kind == "latent" else 2
    rows = sum(q_lens)
    odd = "odd" in kind
    rot = 20 if odd else 64                       # 20: pairs that cross 16-byte vectors
    turns, rope = rope_of(attn, rot, start=8 if odd else 0)
    x = [randn(i, rows + 2 * pad, h, dim).to(DEV) for i, h in ((1, hkv), (2, hkv), (3, 4))]
    offs = torch.tensor([pad, pad + 2, pad + 3, pad + 63], dtype=torch.int32, device=DEV)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def go(k, v, q, offs):
        qo = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device=DEV)
        kw = dict(max_kv_len=200, page_table=pool.table.to(DEV), q=q, q_out=qo,
                  q_row_offsets=offs, rope=rope)
        if "fp8" in kind:
            cache = fresh8(pool)
            attn.attn_append_kv_fp8(k, v, *cache, L, max_q_len=60, **kw)
        else:
            cache = [torch.zeros(pool.pages, 64, hkv, dim, dtype=torch.bfloat16, device=DEV)
                     for _ in range(1 if kind == "latent" else 2)]
            vs = (None, None) if kind == "latent" else (v, cache[1])
            attn.attn_append_kv(k, vs[0], cache[0], vs[1], L, **kw)
        return qo, cache

    qo, cache = go(*x, offs)
    q1, cache1 = go(*[t[pad:-pad] for t in x], offs - pad)
    assert (qo[:pad] == 3.0).all() and (qo[-pad:] == 3.0).all()
    assert torch.equal(qo[pad:-pad], q1)
    for a, b in zip(cache, cache1):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert a.float().abs().sum() > 0


def test_offsets_beyond_32_bits(attn):
    """Pages whose first byte is behind 2^32, in both caches, appended to and read."""
    pages, page, hkv = 70000, 64, 8
    last = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    k, v, q = (randn(i, 100, h, 128).to(DEV) for i, h in ((1, hkv), (2, hkv), (3, 8)))
    turns, rope = rope_of(attn, 128)
    L = torch.tensor([100], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 100], dtype=torch.int32, device=DEV)

    def caches(n, dtype):
        return [torch.zeros(n, page, hkv, 128, dtype=dtype, device=DEV) for _ in range(2)]

    def go(n, table):
        kw = dict(max_kv_len=100, page_table=table, q=q, q_row_offsets=offs, rope=rope)
        c16, c8 = caches(n, torch.bfloat16), caches(n, FP8)
        s8 = [torch.ones(n, 4, hkv, device=DEV) for _ in range(2)]
        q16 = attn.attn_append_kv(k, v, *c16, L, **kw)
        q8 = attn.attn_append_kv_fp8(k, v, *c8, *s8, L, max_q_len=100, **kw)
        kw = dict(group=1, scale=0.05, max_kv_len=100, page_table=table)
        a, _ = attn.attn_decode(q16[-1:], *c16, L, **kw)
        b, _ = attn.attn_decode_fp8(q8[-1:], *c8, *s8, L, **kw)
        return a, b

    near = go(2, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV))
    far = go(pages, last)
    for a, b in zip(near, far):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_append_then_attend_bf16(attn):
    """A prompt and then single tokens: attention over the cache against attention over the rows."""
    hq, hkv, page = 8, 2, 64
    table = torch.tensor([[3, 1], [0, 5]], dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros(6, page, hkv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    turns, rope = rope_of(attn, 128)
    lens, history = [70, 31], [[], []]
    for step in range(4):
        n = lens if step == 0 else [1, 1]
        if step:
            lens = [x + 1 for x in lens]
        x = randn(step, sum(n), hq + 2 * hkv, 128).to(DEV)
        L = torch.tensor(lens, dtype=torch.int32, device=DEV)
        offs = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32, device=DEV)
        q = attn.attn_append_kv(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, L, max_kv_len=128,
                                page_table=table, q=x[:, :hq],
                                q_row_offsets=offs if step == 0 else None, rope=rope)
        tokens = [torch.arange(a - b, a) for a, b in zip(lens, n)]
        ke, _ = R.head_rows(x[:, hq:hq + hkv].cpu(), turns, torch.cat(tokens))
        at = 0
        for b in range(2):
            history[b].append((ke[at:at + n[b]], x[at:at + n[b], hq + hkv:].cpu().double()))
            at += n[b]
        if step == 0:
            continue
        out, _ = attn.attn_decode(q, kc, vc, L, group=4, scale=0.05, max_kv_len=128,
                                  page_table=table)
        for b in range(2):
            K, V = (torch.cat([h[i] for h in history[b]]).repeat_interleave(4, 1) for i in (0, 1))
            s = torch.einsum("hd,thd->ht", q[b].cpu().double(), K) * 0.05
            want = torch.einsum("ht,thd->hd", torch.softmax(s, 1), V)
            # keys off by half a step of bf16 move a score by at most 2^-8 sum |q k| scale = d,
            # a weight by a factor of at most e^(2 d); weights and output round to bf16 once
            d = (torch.einsum("hd,thd->ht", q[b].cpu().double().abs(), K.abs()) * 0.05 *
                 R.BF16_HALF).amax(1)
            bound = (torch.expm1(2 * d)[:, None] + 2 * R.BF16_HALF) * V.abs().amax()
            assert ((out[b].cpu().double() - want).abs() <= bound).all()


def test_append_then_attend_latent(attn):
    """Latent rows appended token by token, against the same rows written at once."""
    hq, page, steps = 128, 64, 70
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    turns, rope = rope_of(attn, 64, start=512, interleaved=True)
    k, q = randn(1, steps, 1, 576).to(DEV), randn(2, steps, hq, 576).to(DEV)
    one, all_ = (torch.zeros(3, page, 1, 576, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    outs = []
    for t in range(steps):
        L = torch.tensor([t + 1], dtype=torch.int32, device=DEV)
        qt = attn.attn_append_kv(k[t:t + 1], None, one, None, L, max_kv_len=128,
                                 page_table=table, q=q[t:t + 1], rope=rope)
    L = torch.tensor([steps], dtype=torch.int32, device=DEV)
    qa = attn.attn_append_kv(k, None, all_, None, L, max_kv_len=128, page_table=table, q=q,
                             q_row_offsets=torch.tensor([0, steps], dtype=torch.int32, device=DEV),
                             rope=rope)
    assert torch.equal(one, all_) and torch.equal(qt[0], qa[-1])
    for c in (one, all_):
        outs.append(attn.attn_mla_decode(qt, c, L, scale=0.04, max_kv_len=128,
                                         page_table=table)[0])
    assert torch.equal(*outs) and outs[0].abs().sum() > 0


@pytest.mark.parametrize("fp8", [False, True])
def test_append_is_captured_and_replayed(attn, fp8):
    """A captured append replayed with other lengths and rows, on another stream."""
    lens = torch.tensor([5, 64, 17], dtype=torch.int32, device=DEV)
    pool = Pool([128, 128, 128], 64, 1)
    k, v = randn(1, 3, 2, 128).to(DEV), randn(2, 3, 2, 128).to(DEV)
    dt = FP8 if fp8 else torch.bfloat16
    turns, rope = rope_of(attn, 128)
    table = pool.table.to(DEV)

    def make():
        c = [torch.zeros(pool.pages, 64, 2, 128, dtype=dt, device=DEV) for _ in range(2)]
        return c + ([torch.ones(pool.pages, 4, 2, device=DEV) for _ in range(2)] if fp8 else [])

    def go(c):
        f = attn.attn_append_kv_fp8 if fp8 else attn.attn_append_kv
        f(k, v, *c, lens, max_kv_len=128, page_table=table, rope=rope)

    c1, c2 = make(), make()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        go(make())
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            go(c1)
    torch.cuda.synchronize()
    for step in range(3):
        lens += 1
        k.copy_(randn(10 + step, 3, 2, 128))
        graph.replay()
        go(c2)
        torch.cuda.synchronize()
    for a, b in zip(c1, c2):
        assert torch.equal(a.view(torch.uint8) if a.dtype == FP8 else a,
                           b.view(torch.uint8) if b.dtype == FP8 else b)


@pytest.mark.parametrize("qd,kd,rot,start", [(64, 128, 64, 0), (192, 128, 32, 64), (576, 192, 64, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_query_and_key_heads_of_unequal_dims(attn, qd, kd, rot, start, interleaved):
    q, k = randn(1, 70, 5, qd), randn(2, 70, 3, kd)
    qn, kn = ((1 + randn(i, d, scale=0.2)).to(torch.bfloat16) for i, d in ((3, qd), (4, kd)))
    pos = torch.arange(70, dtype=torch.int32) * 977
    turns, rope = rope_of(attn, rot, start=start, interleaved=interleaved)
    got = attn.attn_qk_norm_rope(q.to(DEV), k.to(DEV), pos.to(DEV), rope=rope, q_norm=qn.to(DEV),
                                 k_norm=kn.to(DEV))
    for y, x, n in zip(got, (q, k), (qn, kn)):
        exact, err = R.head_rows(x, turns, pos, norm=n, start=start, interleaved=interleaved)
        R.assert_bf16(y, exact, err, f"dim {x.shape[2]}")


def test_append_fp8_many_heads(attn):
    check_fp8(attn, [70, 200], [40, 150], 64, 16, 9, hkv=40, magnitude=2.0)


@pytest.mark.parametrize("q_lens", [[3, 1], [50, 2]])
def test_append_fp8_given_positions_and_in_place(attn, q_lens):
    """Positions of the tokens given: the same result; queries in place of themselves."""
    lens = [60, 140]
    pool = Pool(lens, 64, 2)
    rows = sum(q_lens)
    x = randn(7, rows, 8, 128).to(DEV)
    turns, rope = rope_of(attn, 128)
    offs = torch.tensor([0, q_lens[0], rows], dtype=torch.int32, device=DEV)
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tokens = torch.tensor([t for _, _, t in rows_of(lens, q_lens)], dtype=torch.int32)

    def go(x, shift=None, in_place=False):
        c = fresh8(pool)
        q = x[:, :4]
        pos = None if shift is None else (tokens + shift).to(DEV)
        out = attn.attn_append_kv_fp8(x[:, 4:6], x[:, 6:], *c, L, max_kv_len=140,
                                      max_q_len=max(q_lens), page_table=pool.table.to(DEV), q=q,
                                      q_out=q if in_place else None, q_row_offsets=offs, rope=rope,
                                      positions=pos)
        return [out.clone()] + [t.view(torch.uint8) if t.dtype == FP8 else t for t in c]

    want = go(x)
    for a, b in zip(want, go(x, 0)):
        assert torch.equal(a, b)
    y = x.clone()
    for a, b in zip(want, go(y, in_place=True)):
        assert torch.equal(a, b)
    assert torch.equal(y[:, 4:], x[:, 4:])
    far = go(x, 1 << 30)
    exact, err = R.head_rows(x[:, :4].cpu(), turns, tokens + (1 << 30))
    R.assert_bf16(far[0], exact, err, "far positions")
    assert not torch.equal(far[1], want[1]) and torch.equal(far[2], want[2])


def test_long_append_and_decode_in_one_graph(attn):
    """A prompt's append (two overlapping launches) and the decode behind it, captured together
    and replayed with other rows and lengths."""
    lens = torch.tensor([300, 70], dtype=torch.int32, device=DEV)
    runs = torch.tensor([0, 260, 300], dtype=torch.int32, device=DEV)
    pool = Pool([384, 384], 64, 4)
    table = pool.table.to(DEV)
    x = randn(1, 300, 8 + 4, 128).to(DEV)
    turns, rope = rope_of(attn, 128)

    def go(c):
        q = attn.attn_append_kv_fp8(x[:, 8:10], x[:, 10:], *c, lens, max_kv_len=384,
                                    max_q_len=260, page_table=table, q=x[:, :8],
                                    q_row_offsets=runs, rope=rope)
        last = q[259::40].contiguous()                   # the last row of each
        return attn.attn_decode_fp8(last, *c, lens, group=4, scale=0.09, max_kv_len=384,
                                    page_table=table)

    c1, c2 = fresh8(pool), fresh8(pool)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(fresh8(pool))
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out, lse = go(c1)
    torch.cuda.synchronize()
    for step in range(4):
        lens += torch.tensor([11, 40], dtype=torch.int32, device=DEV)
        x.copy_(randn(20 + step, 300, 12, 128))
        graph.replay()
        want, wl = go(c2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert torch.isfinite(out).all()
    for a, b in zip(c1, c2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_fp8_more_rows_than_said(attn):
    pool = Pool([100], 64, 1)
    c = fresh8(pool)
    k = randn(1, 40, 2, 128).to(DEV)
    attn.attn_append_kv_fp8(k, k, *c, torch.tensor([100], dtype=torch.int32, device=DEV),
                            max_kv_len=100, max_q_len=4, page_table=pool.table.to(DEV),
                            q_row_offsets=torch.tensor([0, 40], dtype=torch.int32, device=DEV))
    assert attn.attn_device_error_flags(clear=True) == 4


@pytest.mark.parametrize("kind", ["rows", "short", "runs", "large_blocks"])
def test_lengths_past_31_bits(attn, kind):
    """Lengths that no cache has (left-over memory, a -1): reported, nothing of theirs is read
    from the page table or stored, and the sequence between them is as alone."""
    n = 3 if kind == "short" else 70
    lens = [-1, 100, -2 ** 31 + 5, 2 ** 31 - 1, -2 ** 31 + n // 2]     # as 32-bit patterns
    table = torch.tensor([[5, 6], [2, 0], [7, 3], [8, 1], [4, 4]], dtype=torch.int32, device=DEV)
    x = randn(31, 5 * n, 4, 128).to(DEV)
    _, rope = rope_of(attn, 128)
    block = 256 if kind == "large_blocks" else 16
    page = max(64, block)

    def go(seqs):
        dt = torch.bfloat16 if kind == "rows" else FP8
        c = [torch.zeros(9, page, 2, 128, dtype=dt, device=DEV) for _ in range(2)]
        if kind != "rows":
            c += [torch.ones(9, page // block, 2, device=DEV) for _ in range(2)]
        append = attn.attn_append_kv if kind == "rows" else attn.attn_append_kv_fp8
        rows = torch.cat([x[b * n:(b + 1) * n] for b in seqs])
        append(rows[:, :2], rows[:, 2:], *c,
               torch.tensor([lens[b] for b in seqs], dtype=torch.int32, device=DEV), max_kv_len=128,
               page_table=table[torch.tensor(seqs, device=DEV)].contiguous(), rope=rope,
               q_row_offsets=torch.arange(0, n * len(seqs) + 1, n, dtype=torch.int32, device=DEV),
               **({} if kind == "rows" else {"max_q_len": n}))
        torch.cuda.synchronize()
        return c

    got = go([0, 1, 2, 3, 4])
    assert attn.attn_device_error_flags(clear=True) == 4
    for a, b in zip(got, go([1])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert got[0].view(torch.uint8).any() and attn.attn_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("q_lens", [[40, 1, 7], [1, 1, 1], [20, 1, 20]])
def test_append_fp8_rows_without_a_bound(attn, q_lens):
    """q_row_offsets without max_q_len: every row is stored."""
    lens = [100, 1, 50]
    pool = Pool(lens, 64, 1)
    rows = sum(q_lens)
    k, v = randn(2, rows, 2, 128).to(DEV), randn(3, rows, 2, 128).to(DEV)
    offs = torch.tensor([sum(q_lens[:i]) for i in range(4)], dtype=torch.int32, device=DEV)

    def go(**kw):
        c = fresh8(pool)
        attn.attn_append_kv_fp8(k, v, *c, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                max_kv_len=100, page_table=pool.table.to(DEV), q_row_offsets=offs,
                                **kw)
        return c

    for a, b in zip(go(), go(max_q_len=max(q_lens))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert attn.attn_device_error_flags(clear=True) == 0
