"""Decode attention over a cache held in 8 bits against a 64-bit reference.

The reference attends over code * scale in 64 bits.  The kernel may differ by
its own roundings only, per output element:

* half a bf16 step of the output, 2^-8 |out|;
* weights: each p v_scale enters the product to a relative 2^-11 (four e4m3
  terms leave at most 2^-13, the approximate exp2 2^-22) and the sums are fp32;
  a weight of less than 2^-16 of its piece's largest may miss 2^-29 of that
  instead, which the keys of these tests (20000 at most) keep below the rest
  of the bound (test_one_key_far_above_the_rest is about it);
* scores: q as two e4m3 terms misses at most 2^-18 of the row's largest
  channel, and the sum of 128 products, the scale and the exponent round in
  fp32 (16 steps): a score errs by at most rho = 2^-16 max_j sum_c |q_c k_jc|
  scale + 2^-20, which moves every weight by a factor of at most 1 + 2 rho and
  the normaliser as well.

So |out - exact| <= 2^-8 |exact| + (2^-11 + 4 rho) sum_j w_j |v_j| (times 1.01
for second order), and |lse - exact| <= rho + 2^-20 max(1, |exact|).
"""
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


class Case:
    def __init__(self, lens, q_lens=None, *, hq=8, hkv=2, page=64, block=16, seed=0, sink=False,
                 causal=True, contiguous=False, spread=0.0, scale=None, garbage=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.q_lens, self.causal = lens, q_lens, causal
        self.group = hq // hkv
        rows = sum(q_lens) if q_lens else len(lens)
        self.q = torch.randn(rows, hq, 128, generator=g).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(128) if scale is None else scale
        self.sink = torch.randn(hq, generator=g) if sink else None
        need = [max(1, -(-x // page)) for x in lens]
        if contiguous:
            page = max(block, -(-max(max(lens), 1) // block) * block)
            self.pages, self.table = len(lens), None
        else:
            self.pages = sum(need) + 1
            perm = torch.randperm(self.pages, generator=g)
            self.table = torch.zeros(len(lens), max(need), dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = perm[at:at + n].to(torch.int32)
                at += n
        self.page, self.block = page, block
        self.caches = []
        for _ in range(2):
            x = torch.randn(self.pages, page, hkv, 128, generator=g)
            f = torch.exp2(torch.randn(self.pages, page // block, hkv, generator=g) * spread)
            s = x.view(self.pages, page // block, block, hkv, 128).abs().amax((2, 4)) / 448.0
            codes = (x.view(self.pages, page // block, block, hkv, 128) /
                     s[:, :, None, :, None]).to(FP8).view(self.pages, page, hkv, 128)
            self.caches.append([codes, s * f])
        self.offsets = None if q_lens is None else [sum(q_lens[:i]) for i in range(len(lens) + 1)]
        if garbage:
            # what no token owns: NaN codes and scales that must not be used
            live = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, L in enumerate(lens):
                for t in range(L):
                    live[self.place(b, t)] = True
            for c in self.caches:
                c[0].view(torch.uint8)[~live] = 0x7f
                dead = ~live.view(self.pages, page // block, block).any(2)
                c[1][dead] = float("nan")

    def place(self, b, t):
        if self.table is None:
            return b, t
        return int(self.table[b, t // self.page]), t % self.page

    def run(self, attn, **kw):
        cu = lambda t: None if t is None else t.to(DEV)   # noqa: E731
        (kc, ks), (vc, vs) = self.caches
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        args = dict(group=self.group, scale=self.scale, max_kv_len=max(self.lens),
                    page_table=cu(self.table), sink=cu(self.sink), q_row_offsets=i32(self.offsets),
                    max_q_len=max(self.q_lens) if self.q_lens else 1, causal=self.causal)
        args.update(kw)
        out, lse = attn.attn_decode_fp8(cu(self.q), cu(kc), cu(vc), cu(ks), cu(vs),
                                        i32(self.lens), **args)
        torch.cuda.synchronize()
        return out, lse

    def reference(self):
        seqs = []
        for codes, s in self.caches:
            x = codes.float().double() * s.double().repeat_interleave(self.block, 1)[..., None]
            if self.table is None:
                seqs.append([x[b, :L] for b, L in enumerate(self.lens)])
            else:
                seqs.append([x[self.table[b].long()].reshape(-1, *x.shape[2:])[:L]
                             for b, L in enumerate(self.lens)])
        return R.decode_reference(self.q, seqs[0], seqs[1], self.lens, group=self.group,
                                  scale=self.scale, offsets=self.offsets, causal=self.causal,
                                  sink=self.sink)

    def check(self, attn, what="", **kw):
        out, lse = self.run(attn, **kw)
        o, l = out.cpu().double(), lse.cpu().double()
        eo, el, mass, big = self.reference()
        rho = (2.0 ** -16 * big + 2.0 ** -20)[..., None]
        bound = R.BF16_HALF * eo.abs() + 1.01 * (2.0 ** -11 + 4 * rho) * mass + 2.0 ** -130
        worst = ((o - eo).abs() / bound).max().item()
        assert torch.isfinite(o).all() and worst <= 1, f"{what}: {worst:.3g} times the bound"
        none = el.isneginf()
        assert torch.equal(none, l.isneginf()), f"{what}: -inf lse"
        d = ((l - el).abs() - rho[..., 0] - 2.0 ** -20 * el.abs().clamp_min(1))[~none]
        assert d.numel() == 0 or d.max() <= 0, f"{what}: lse {d.max():.3g} above the bound"
        return out, lse


@pytest.mark.parametrize("lens", [[1], [2, 127, 128, 129], [0, 5], [1000, 1, 0, 300, 256, 255, 257],
                                  [37, 100]])
@pytest.mark.parametrize("sink", [False, True])
def test_lengths(attn, lens, sink):
    Case(lens, seed=len(lens), sink=sink).check(attn, f"lens {lens}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 3), (12, 4), (4, 1), (5, 1), (6, 1), (14, 2),
                                    (8, 1), (16, 1), (24, 2), (11, 1)])
def test_groups(attn, hq, hkv):
    Case([300, 77, 513], hq=hq, hkv=hkv, seed=hq, sink=True).check(attn, f"heads {hq}/{hkv}")


@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 4), (32, 32), (64, 1), (128, 128),
                                        (256, 64), (512, 256), (1024, 2)])
def test_pages_and_blocks(attn, page, block):
    Case([700, 129, 8, 9], page=page, block=block, seed=page + block).check(
        attn, f"page {page} block {block}")


def test_contiguous(attn):
    Case([130, 400, 0, 33], contiguous=True, block=16, seed=4).check(attn, "contiguous")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,q_lens", [(8, 2, [4, 1, 3, 2]), (2, 2, [16, 3, 0, 9]),
                                           (8, 1, [2, 1, 2, 2]), (5, 1, [3, 3, 1, 2]),
                                           (16, 1, [1, 1, 1, 1])])
def test_draft_rows(attn, causal, hq, hkv, q_lens):
    lens = [500, 3, 130, 16]
    lens = [max(a, b) for a, b in zip(lens, q_lens)]
    Case(lens, q_lens, hq=hq, hkv=hkv, causal=causal, seed=hq + hkv, sink=hkv == 2).check(
        attn, f"draft rows {q_lens}")


@pytest.mark.parametrize("hq,hkv,q_lens,lens", [
    (4, 1, [1, 4], [32000, 6900]), (32, 8, [1, 4], [2944, 768]), (4, 1, [4, 1], [2560, 35840]),
    (8, 2, [4, 1, 1, 1], [4096] * 4)])
def test_draft_rows_of_unequal_cost(attn, hq, hkv, q_lens, lens):
    """About as many tiles as CTAs, some dearer than others.  The merge reads what the
    partition kernel wrote and nothing else: the partial slots are NaN before the call
    (the table of slots behind them, 8 bytes a sequence and KV head, is 0)."""
    n = attn.attn_decode_fp8_workspace(len(lens), hq, hq // hkv)
    ws = torch.full((n // 4,), float("nan"), device=DEV)
    ws[n // 4 - 64 * -(-len(lens) * hkv * 8 // 256):] = 0
    Case(lens, q_lens, hq=hq, hkv=hkv, page=128, block=64, seed=21, garbage=False).check(
        attn, f"rows {q_lens} of {lens}", workspace=ws)


def weight_error(w):
    """Bound of |four e4m3 terms of w - w|, w = 16 at a weight of 1 with V scale mantissa 1
    (tests/test_fp8_weight_terms.py)."""
    return torch.maximum(2.0 ** -13 * w, torch.minimum(torch.full_like(w, 2.0 ** -25),
                                                       (2.0 ** -4 * w).clamp_min(2.0 ** -35)))


@pytest.mark.parametrize("n,batch", [(128, 1), (1000, 3), (4096, 304), (131072, 1), (131072, 304)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("spread", [0, 6])
def test_one_key_far_above_the_rest(attn, n, batch, where, spread):
    """A key 10 to 20 nats above the others whose V is 0: the output is what the small weights
    leave.  304 sequences (of one set of pages) on one KV head: a piece holds a whole one.

    Beside the roundings at the top of this file, per key: the weight's terms (weight_error,
    relative to the largest p_i 2^(e_i), e_i the exponent of the key's V scale), and the
    accumulator's roundings, one step 2^-23 of what it holds for each of n / 32 products."""
    g = torch.Generator(device=DEV).manual_seed(n + spread)
    page, block, hq = 128, 64, 4
    pages = -(-n // page)
    k = torch.zeros(pages, page, 1, 128, device=DEV)
    k[..., 0] = torch.randint(-4, 5, (pages, page, 1), generator=g, device=DEV) / 16.0
    v = torch.rand(pages, page, 1, 128, generator=g, device=DEV) * 400 + 40
    at = {"first": 0, "middle": n // 2, "last": n - 1}[where]
    k.view(-1, 128)[at, 0] = 20.0
    v.view(-1, 128)[at] = 0.0
    kc, vc = k.to(FP8), v.to(FP8)
    ks = torch.ones(pages, page // block, 1, device=DEV)
    vs = 1.3 * torch.exp2(-torch.randint(0, spread + 1, ks.shape, generator=g, device=DEV).float())
    q = torch.zeros(batch, hq, 128, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = torch.tensor([0.5, 0.625, 0.75, 1.0])                # 10 to 20 nats
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(batch, pages).contiguous()
    lens = torch.full((batch,), n, dtype=torch.int32, device=DEV)
    out, lse = attn.attn_decode_fp8(q, kc, vc, ks, vs, lens, group=hq, scale=1.0, max_kv_len=n,
                                    page_table=table)
    codes = vc.double().view(-1, 128)[:n]
    vscale = vs.double().repeat_interleave(block, 1).view(-1)[:n]
    scores = q[0, :, :1].double() * kc.double().view(-1, 128)[:n, 0]   # [heads, n]
    el = torch.logsumexp(scores, -1)
    p = torch.exp(scores - el[:, None])
    exact = (p * vscale) @ codes
    rho = 2.0 ** -16 * 20 + 2.0 ** -20
    e2 = torch.exp2(torch.floor(torch.log2(vscale)))                  # 2^(e_j)
    unit = (p * e2).amax(-1, keepdim=True) / 16                       # of w
    terms = (weight_error(p * vscale / unit) * unit) @ codes
    bound = R.BF16_HALF * exact + 1.01 * (terms + (2.0 ** -20 + 4 * rho + n / 32 * 2.0 ** -23) *
                                          exact)
    worst = ((out.double() - exact).abs() / bound).max().item()
    assert worst <= 1, f"{worst:.3g} times the bound"
    assert (lse.double() - el).abs().max() <= rho + 2.0 ** -20 * 20


def test_row_that_sees_nothing(attn):
    """Two rows of a sequence with one key, bottom aligned: the first sees none."""
    c = Case([1, 300], [2, 2], seed=8)
    out, lse = c.check(attn, "no key")
    assert not out[0].any() and lse[0].isneginf().all()


@pytest.mark.parametrize("spread", [3.0, 8.0])
def test_scales_of_far_sizes(attn, spread):
    """Block scales many powers of two apart, in K (scores far apart) and V."""
    c = Case([600, 200], block=16, seed=int(spread), spread=spread, scale=0.01)
    c.check(attn, f"spread {spread}")


def test_v_scales_at_the_ends_of_the_range(attn):
    for e in (-64, 0, 64):
        c = Case([300, 129], block=32, seed=3, sink=True, garbage=False)
        c.caches[1][1] = torch.full_like(c.caches[1][1], 2.0 ** e)
        c.check(attn, f"2^{e}")
    c = Case([300, 129], block=32, seed=3, garbage=False)
    c.caches[1][1][:] = 0.0                                   # V is 0
    out, _ = c.check(attn, "zero")
    assert not out.any()


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.7])
def test_score_scales(attn, scale):
    Case([400, 33], seed=2, scale=scale, sink=True).check(attn, f"scale {scale}")


def test_large_and_tiny_queries(attn):
    c = Case([200, 200, 200], seed=5)
    c.q[0] *= 2.0 ** -100
    c.q[1] = 0
    c.q[2, 0, 3] = 300.0                     # one channel far above the others
    c.scale = 0.002
    c.check(attn, "q magnitudes")


def test_many_sequences_cut_and_whole(attn):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 900, (70,), generator=g).tolist() + [5000]
    Case(lens, hq=4, hkv=2, page=128, block=128, seed=6, sink=True).check(attn, "71 sequences")


def test_long_sequence(attn):
    Case([20000], hq=8, hkv=2, page=128, block=64, seed=7, garbage=False).check(attn, "20000 keys")


def test_nan_in_a_visible_token_only(attn):
    """NaN in K or V of a later draft token reaches the rows that see it and no others."""
    for which in (0, 1):
        c = Case([300, 300], [3, 1], hq=4, hkv=1, seed=9)
        clean, _ = c.run(attn)
        pg, slot = c.place(0, 298)                            # seen by rows 1 and 2
        c.caches[which][0].view(torch.uint8)[pg, slot, 0, 17] = 0x7f
        out, _ = c.run(attn)
        assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
        assert out[1:3].isnan().any(-1).all()


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 1, 2]])
def test_rows_of_no_sequence_are_left(attn, q_lens):
    """A padded batch: more rows than the offsets give out."""
    c = Case([300, 77, 1000], q_lens, seed=14)
    n = c.q.shape[0]
    c.q = torch.cat([c.q, torch.full((3, 8, 128), float("nan"), dtype=torch.bfloat16)])
    out = torch.full((n + 3, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n + 3, 8), 5.0, device=DEV)
    c.run(attn, out=out, lse=lse)
    assert (out[n:] == 3.0).all() and (lse[n:] == 5.0).all()
    c.q = c.q[:n]
    want, wl = c.check(attn, "rows")
    assert torch.equal(out[:n], want) and torch.equal(lse[:n], wl)


def test_sequences_that_share_pages(attn):
    """A common prefix: two sequences' tables name the same pages."""
    c = Case([256, 256], page=64, seed=15, garbage=False)
    c.table[1] = c.table[0]
    c.check(attn, "shared pages")


def test_calls_on_two_streams_at_once(attn):
    a, b = Case([3000, 77], seed=16), Case([900, 1], seed=17)
    want = [x.run(attn)[0] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = []
    for x in (a, b):
        (kc, ks), (vc, vs) = [[t.to(DEV) for t in y] for y in x.caches]
        data.append((x.q.to(DEV), kc, vc, ks, vs,
                     torch.tensor(x.lens, dtype=torch.int32, device=DEV), x.table.to(DEV)))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, x, d in zip(streams, (a, b), data):
            with torch.cuda.stream(s):
                got.append(attn.attn_decode_fp8(*d[:6], group=x.group, scale=x.scale,
                                                max_kv_len=max(x.lens), page_table=d[6],
                                                causal=True)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


@pytest.mark.parametrize("hq", [4, 8])
def test_v_scale_past_the_range_of_a_later_token(attn, hq):
    """It counts as NaN for the rows that see its token and for no others."""
    c = Case([300, 300], [2, 1], hq=hq, hkv=1, block=1, seed=22)
    clean, _ = c.run(attn)
    pg, slot = c.place(0, 299)                                # seen by row 1
    c.caches[1][1][pg, slot] = 2.0 ** 66
    out, _ = c.run(attn)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert out[1].isnan().all()


def test_v_scale_past_the_range_is_not_silent(attn):
    c = Case([200], seed=18, garbage=False, block=64)
    c.caches[1][1][int(c.table[0, 1])] = 2.0 ** 66
    out, _ = c.run(attn)
    assert out.isnan().all()


def test_outputs_given_and_workspace_shared_in_order(attn):
    c = Case([300, 77, 1000], seed=10)
    ws = torch.empty(attn.attn_decode_fp8_workspace(3, 8, c.group) + 512, dtype=torch.uint8,
                     device=DEV)
    out = torch.full((3, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    a, lse = c.run(attn, workspace=ws, out=out, return_lse=False)
    assert lse is None and a is out
    b, _ = c.run(attn)
    assert torch.equal(a, b)


def test_captured_and_replayed_with_other_lengths(attn):
    c = Case([900, 900], seed=11, garbage=False)
    lens = torch.tensor([900, 900], dtype=torch.int32, device=DEV)
    q = c.q.to(DEV)
    (kc, ks), (vc, vs) = [[t.to(DEV) for t in x] for x in c.caches]
    ws = torch.empty(attn.attn_decode_fp8_workspace(2, 8, c.group), dtype=torch.uint8, device=DEV)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 8, device=DEV)
    table = c.table.to(DEV)

    def go():
        attn.attn_decode_fp8(q, kc, vc, ks, vs, lens, group=c.group, scale=c.scale, max_kv_len=900,
                             page_table=table, workspace=ws, out=out, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        go()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            go()
    torch.cuda.synchronize()
    for n in ([900, 900], [1, 640], [0, 129]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        c.lens = n
        want, _ = c.run(attn, max_kv_len=900)
        assert torch.equal(got, want), n


def test_bad_page_and_length_are_reported(attn):
    c = Case([300, 40], page=64, seed=12)
    c.table[0, 1] = c.pages + 7
    c.run(attn)
    assert attn.attn_device_error_flags(clear=True) & 2
    c = Case([300, 40], page=64, seed=12)
    c.run(attn, max_kv_len=256)
    assert attn.attn_device_error_flags(clear=True) & 4


def test_more_rows_than_said(attn):
    c = Case([300, 40], [6, 1], seed=19)
    c.run(attn, max_q_len=1)
    assert attn.attn_device_error_flags(clear=True) == 4


@pytest.mark.parametrize("hq,hkv,q_lens", [(8, 2, [4, 1, 3]), (16, 1, [1, 1, 1]), (2, 2, [16, 2, 1])])
def test_rows_without_a_bound(attn, hq, hkv, q_lens):
    """q_row_offsets without max_q_len: all rows all the same."""
    c = Case([300, 40, 77], q_lens, hq=hq, hkv=hkv, seed=23)
    want = c.check(attn, "bound given")
    got = c.check(attn, "no bound", max_q_len=None)
    if hq // hkv * max(q_lens) > 8:                # the same kernel
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_append_then_decode(attn):
    """A prompt and then single tokens, appended and attended to: against attention over the
    values that the cache holds, step by step."""
    hq, hkv, page, block, steps = 8, 2, 64, 32, 5
    start = [70, 31]
    pool = 6
    table = torch.tensor([[3, 1], [0, 5]], dtype=torch.int32, device=DEV)
    kc = torch.zeros(pool, page, hkv, 128, dtype=FP8, device=DEV)
    vc = torch.zeros_like(kc)
    ks = torch.ones(pool, page // block, hkv, device=DEV)
    vs = torch.ones_like(ks)
    turns, m = attn.rope_turns(128, 500000.0, device=DEV)
    rope = attn.Rope(turns, mscale=m)
    g = torch.Generator().manual_seed(0)
    lens = list(start)
    for step in range(steps + 1):
        n = start if step == 0 else [1, 1]
        if step:
            lens = [x + 1 for x in lens]
        x = (torch.randn(sum(n), hq + 2 * hkv, 128, generator=g) * (1 + step)).to(torch.bfloat16)
        x = x.to(DEV)
        L = torch.tensor(lens, dtype=torch.int32, device=DEV)
        offs = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32, device=DEV)
        q = attn.attn_append_kv_fp8(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, ks, vs, L,
                                    max_kv_len=128, max_q_len=max(n), page_table=table,
                                    q=x[:, :hq], q_row_offsets=offs if step == 0 else None,
                                    rope=rope)
        if step == 0:
            continue
        out, lse = attn.attn_decode_fp8(q, kc, vc, ks, vs, L, group=4, scale=0.05, max_kv_len=128,
                                        page_table=table)
        c = Case.__new__(Case)
        c.lens, c.q_lens, c.offsets, c.causal, c.group = lens, None, None, False, 4
        c.scale, c.sink, c.page, c.block, c.table = 0.05, None, page, block, table.cpu()
        c.q, c.caches = q.cpu(), [[kc.cpu(), ks.cpu()], [vc.cpu(), vs.cpu()]]
        c.check(attn, f"step {step}")
