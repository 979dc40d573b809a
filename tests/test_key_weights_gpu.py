"""The attention weight that keys gather (attn_key_weights) against a 64-bit reference.

w_t = [t < L - n] decay w_t + sum over rows that see t and heads of e^x, x = scale q.k - lse.
What the kernel may differ by, per term p = e^x:

* the score is an fp32 MMA sum of d exact products in steps of 16, one rounding a step
  and two more: rho = (d / 16 + 2) 2^-23 scale sum_c |q_c k_c|;
* with many rows the exponent is one multiply-add of fl(scale log2 e) and fl(lse log2 e), each
  rounded once and the product not: 2^-23 (|scale q.k| + |lse|) of x, which the bound takes for
  all calls;
* otherwise x itself is rounded once (2^-24 |x|), then multiplied by log2 e (2^-24 for the product
  and 2^-25 for the constant), and e^x taken to 2^-22: together 2^-22 (|x| + 1);
* the sum of N positive terms in four running fp32 sums: (N / 4 + 8) 2^-24 of the sum;
* weights below 2^-126 count as 0: N 2^-126.

The earlier weight enters in one fused multiply-add: 2^-24 of the result.  scale and decay
are fp32 numbers at the entry point: the reference takes those numbers (fl(0.98) = 0.98 (1 +
d) with d up to 2^-24, as much as the bound of a weight that is only multiplied by decay).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def attn():
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn as a
    a.attn_device_error_flags(clear=True)
    yield a
    assert a.attn_device_error_flags(clear=True) == 0


class Case:
    def __init__(self, lens, q_lens=None, *, hq=8, hkv=2, dim=128, page=64, seed=0, causal=True,
                 contiguous=False, decay=1.0, scale=None, head_major=False, size=1.0):
        g = torch.Generator().manual_seed(seed)
        in32 = lambda x: float(torch.tensor(x, dtype=torch.float32))   # noqa: E731
        self.lens, self.q_lens, self.causal, self.decay = lens, q_lens, causal, in32(decay)
        self.group, self.hkv, self.dim, self.page = hq // hkv, hkv, dim, page
        self.rows_of = q_lens or [1] * len(lens)
        rows = sum(self.rows_of)
        self.q = (torch.randn(rows, hq, dim, generator=g) * size).to(torch.bfloat16)
        self.scale = in32(1 / math.sqrt(dim) if scale is None else scale)
        need = [max(1, -(-x // page)) for x in lens]
        if contiguous:
            self.page = max(max(lens), 1)
            self.pages, self.table = len(lens), None
        else:
            self.pages = sum(need) + 1
            perm = torch.randperm(self.pages, generator=g)
            self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = perm[at:at + n].to(torch.int32)
                at += n
        self.k = torch.randn(self.pages, self.page, hkv, dim, generator=g).to(torch.bfloat16)
        self.w = torch.rand(self.pages, self.page, hkv, generator=g)
        self.offsets = None if q_lens is None else [sum(q_lens[:i]) for i in range(len(lens) + 1)]
        # what no token owns: never read, never written; a fresh token's weight: never read
        owned = torch.zeros(self.pages, self.page, dtype=torch.bool)
        self.fresh = []
        for b, L in enumerate(lens):
            for t in range(L):
                owned[self.place(b, t)] = True
                if t >= L - self.rows_of[b]:
                    self.fresh.append(self.place(b, t))
        self.k[~owned] = float("nan")
        self.w[~owned] = 17.0
        for p in self.fresh:
            self.w[p] = float("nan")
        self.owned, self.head_major = owned, head_major
        self.lse = self.reference_lse()

    def place(self, b, t):
        if self.table is None:
            return b, t
        return int(self.table[b, t // self.page]), t % self.page

    def keys(self, b):
        L = self.lens[b]
        if self.table is None:
            return self.k[b, :L].double()
        n = -(-L // self.page)
        return self.k[self.table[b, :n].long()].reshape(-1, self.hkv, self.dim)[:L].double()

    def scores(self, b):
        """[n, hq, L] scaled scores, -inf where a row does not see a key; and the same of
        magnitudes."""
        n, L, r0 = self.rows_of[b], self.lens[b], sum(self.rows_of[:b])
        q = self.q[r0:r0 + n].double().view(n, self.hkv, self.group, self.dim)
        k = self.keys(b)
        s = torch.einsum("nhgd,thd->nhgt", q, k) * self.scale
        a = torch.einsum("nhgd,thd->nhgt", q.abs(), k.abs()) * abs(self.scale)
        if self.causal:
            late = torch.arange(L) > (L - n + torch.arange(n))[:, None]
            s = s.masked_fill(late[:, None, None], -math.inf)
        return s, a

    def reference_lse(self):
        out = []
        for b in range(len(self.lens)):
            if self.rows_of[b]:
                s, _ = self.scores(b)
                out.append(torch.logsumexp(s, -1).reshape(self.rows_of[b], -1))
        return torch.cat(out).float() if out else torch.zeros(0, self.q.shape[1])

    def reference(self):
        """The new weights and how far the kernel's may be off."""
        want, err = self.w.double().clone(), torch.zeros_like(self.w, dtype=torch.float64)
        for b, L in enumerate(self.lens):
            n, r0 = self.rows_of[b], sum(self.rows_of[:b])
            total, off = torch.zeros(L, self.hkv).double(), torch.zeros(L, self.hkv).double()
            if n and L:
                s, a = self.scores(b)
                lse = self.lse[r0:r0 + n].double().view(n, self.hkv, self.group, 1)
                x = torch.where(s == -math.inf, s, s - lse)
                p = torch.exp(x)
                rel = ((self.dim / 16 + 2) * 2.0 ** -23 * a +
                       2.0 ** -23 * (s.abs() + lse.abs()).clamp_max(1e4) +
                       2.0 ** -22 * (x.abs().clamp_max(1e4) + 1))
                N = n * self.group
                total = p.sum((0, 2)).T
                off = (p * rel).sum((0, 2)).T + (N / 4 + 8) * 2.0 ** -24 * total + N * 2.0 ** -126
            for t in range(L):
                at = self.place(b, t)
                old = self.w[at].double() * self.decay if t < L - n else 0.0
                want[at] = old + total[t]
                err[at] = 1.01 * off[t] + 2.0 ** -24 * want[at].abs()
        return want, err

    def to_gpu(self, x):
        if x is None:
            return None
        if self.head_major and x.dim() >= 3:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        return x.to(DEV)

    def args(self, **kw):
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        args = dict(group=self.group, scale=self.scale, max_kv_len=max(max(self.lens), 1),
                    page_table=None if self.table is None else self.table.to(DEV),
                    q_row_offsets=i32(self.offsets), max_q_len=max(max(self.rows_of), 1),
                    causal=self.causal, decay=self.decay)
        args.update(kw)
        return (self.q.to(DEV), self.to_gpu(self.k), self.lse.to(DEV), i32(self.lens)), args

    def check(self, attn, what="", **kw):
        pos, args = self.args(**kw)
        w = self.to_gpu(self.w)
        got = attn.attn_key_weights(*pos, w, **args)
        torch.cuda.synchronize()
        assert got is w
        self.compare(w, what)
        return w

    def compare(self, w, what):
        want, err = self.reference()
        w = w.cpu()
        left = ~self.owned
        assert torch.equal(w[left], self.w[left]), f"{what}: slots of no token changed"
        d = (w.double() - want).abs()[self.owned] - err[self.owned]
        worst = d.max().item() if d.numel() else -1.0
        finite = bool(torch.isfinite(w[self.owned]).all())
        assert finite and worst <= 0, f"{what}: {worst:.3g} above the bound"


@pytest.mark.parametrize("lens", [[1], [2, 127, 128, 129], [0, 5], [1000, 1, 0, 300, 256, 255, 257],
                                  [37, 100], [0]])
@pytest.mark.parametrize("dim", [64, 128])
def test_single_rows(attn, lens, dim):
    Case(lens, dim=dim, seed=len(lens), decay=0.9).check(attn, f"lens {lens}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 3), (4, 1), (5, 1), (14, 2), (16, 1),
                                    (17, 1), (40, 2), (128, 1)])
def test_groups(attn, hq, hkv):
    Case([300, 5, 129], hq=hq, hkv=hkv, seed=hq).check(attn, f"{hq} on {hkv}")
    Case([300, 5, 129], [40, 5, 129], hq=hq, hkv=hkv, seed=hq + 1).check(attn, f"rows, {hq} on {hkv}")


@pytest.mark.parametrize("page", [8, 16, 32, 128, 256, 1024])
@pytest.mark.parametrize("head_major", [False, True])
def test_pages_and_layouts(attn, page, head_major):
    Case([300, 700, 9], page=page, seed=page, head_major=head_major).check(attn, f"page {page}")
    Case([300, 700, 9], [300, 4, 9], page=page, seed=page, head_major=head_major,
         decay=0.5).check(attn, f"page {page}, rows")


@pytest.mark.parametrize("q_lens", [None, [3, 1, 2], [290, 50, 7]])
def test_contiguous(attn, q_lens):
    Case([300, 50, 7], q_lens, contiguous=True, seed=3).check(attn)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,q_lens", [(8, 2, [4, 1, 3, 2]), (2, 2, [16, 3, 0, 9]),
                                           (8, 1, [2, 0, 0, 1])])
def test_draft_rows(attn, causal, hq, hkv, q_lens):
    Case([300, 3, 129, 40], q_lens, hq=hq, hkv=hkv, seed=7, causal=causal, decay=0.98).check(attn)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,q_lens", [
    ([513], [513]), ([700, 33, 260], [700, 33, 256]), ([900, 10, 400], [130, 10, 1]),
    ([256, 255, 257, 1], [256, 255, 257, 1]), ([600, 0, 80], [31, 0, 33])])
def test_prompts(attn, causal, dim, lens, q_lens):
    Case(lens, q_lens, dim=dim, seed=11, causal=causal, decay=0.75).check(attn, f"{lens} {q_lens}")


def test_more_rows_than_keys(attn):
    # rows before the first token see nothing; their lse is -inf
    Case([3, 200], [10, 230], seed=5).check(attn)
    Case([3, 20], [5, 21], hq=2, seed=5).check(attn)


@pytest.mark.parametrize("max_q_len", [1, 2, 1000])
def test_any_bound_of_the_rows(attn, max_q_len):
    # the bound picks the kernel; more rows than it says are taken as well
    Case([300, 40], [70, 3], seed=9).check(attn, max_q_len=max_q_len)


@pytest.mark.parametrize("q_lens", [None, [3, 40, 1]])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 4)])
def test_decay_of_zero_reads_no_weights(attn, q_lens, hq, hkv):
    """As over memory that nothing was written to."""
    c = Case([300, 64, 129], q_lens, hq=hq, hkv=hkv, decay=0.0, seed=6)
    zeros = torch.where(c.owned[..., None], torch.zeros_like(c.w), c.w)
    w = c.to_gpu(torch.where(c.owned[..., None], torch.full_like(c.w, math.nan), c.w))
    pos, args = c.args()
    attn.attn_key_weights(*pos, w, **args)
    c.w = zeros
    c.compare(w, "decay 0")


def test_rows_of_no_sequence_are_not_read(attn):
    c = Case([300, 40], [30, 3], seed=9)
    c.q = torch.cat([c.q, torch.full((5, *c.q.shape[1:]), float("nan"), dtype=torch.bfloat16)])
    c.lse = torch.cat([c.lse, torch.full((5, c.lse.shape[1]), float("nan"))])
    c.check(attn)
    c = Case([300, 40], [3, 2], seed=9)
    c.q = torch.cat([c.q, torch.full((5, *c.q.shape[1:]), float("nan"), dtype=torch.bfloat16)])
    c.lse = torch.cat([c.lse, torch.full((5, c.lse.shape[1]), float("nan"))])
    c.check(attn)


def test_no_rows_at_all(attn):
    c = Case([300, 40], [0, 0], seed=9, decay=0.5)
    c.check(attn)


def test_nan_key_stays_with_its_own_weight(attn):
    for q_lens in (None, [200, 30]):
        c = Case([300, 40], q_lens, seed=4)
        want, err = c.reference()
        at = c.place(0, 20)
        c.k[at][0, 5] = float("nan")
        pos, args = c.args()
        w = c.to_gpu(c.w)
        attn.attn_key_weights(*pos, w, **args)
        w = w.cpu()
        assert torch.isnan(w[at][0])
        c.owned[at] = False
        d = (w.double() - want).abs()[c.owned] - err[c.owned]
        assert d.max() <= 0


def test_large_scores(attn):
    Case([400, 60], [100, 1], seed=6, size=6.0).check(attn)
    Case([400, 60], seed=6, size=6.0).check(attn)


def test_equal_calls_give_equal_weights(attn):
    c = Case([700, 300, 20], [700, 40, 20], seed=8)
    first = c.check(attn).clone()
    for _ in range(3):
        assert torch.equal(c.check(attn), first)


def test_many_sequences(attn):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 400, (301,), generator=g).tolist()
    Case(lens, hq=2, hkv=1, page=16, seed=2).check(attn)
    Case(lens, [min(x, 30) for x in lens], hq=2, hkv=1, page=16, seed=2).check(attn)


@pytest.mark.parametrize("q_lens", [None, [40]])
def test_offsets_beyond_32_bits(attn, q_lens):
    """Pages past 4 GB of keys, and weights past 4 GB of their base."""
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("not enough memory")
    c = Case([300], q_lens, hq=4, hkv=1, dim=64, seed=5)
    pages = (1 << 20) + 8
    k = torch.empty((pages, 64, 1, 64), dtype=torch.bfloat16, device=DEV)        # 8 GB
    w = torch.empty((pages, 64, 1, 16), device=DEV)[..., 3]                      # of 4 GB
    far = pages - c.pages
    k[far:], w[far:] = c.k.to(DEV), c.w.to(DEV)
    (q, _, lse, lens), args = c.args()
    args["page_table"] = args["page_table"] + far
    attn.attn_key_weights(q, k, lse, lens, w, **args)
    c.compare(w[far:], "far pages")


def test_captured_and_replayed_with_other_lengths(attn):
    for q_lens in (None, [60, 8, 40]):
        big = Case([500, 300, 260], q_lens, seed=12)
        pos, args = big.args()
        w = big.to_gpu(big.w)
        attn.attn_key_weights(*pos, w, **args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.attn_key_weights(*pos, w, **args)
        for lens in ([500, 300, 260], [61, 300, 129], [400, 9, 70]):
            c = Case(lens, q_lens, seed=13)
            # the same pages, other lengths, keys and weights
            c.table, c.pages = big.table, big.pages
            gen = torch.Generator().manual_seed(lens[0])
            c.k = torch.randn(big.k.shape, generator=gen).to(torch.bfloat16)
            c.w = torch.rand(big.w.shape, generator=gen)
            c.owned = torch.zeros(big.pages, big.page, dtype=torch.bool)
            for b, L in enumerate(lens):
                for t in range(L):
                    c.owned[c.place(b, t)] = True
            c.lse = c.reference_lse()
            pos[0].copy_(c.q)
            pos[1].copy_(c.k)
            pos[2].copy_(c.lse)
            pos[3].copy_(torch.tensor(lens))
            w.copy_(c.w)
            graph.replay()
            torch.cuda.synchronize()
            c.compare(w, f"replay {lens}")


def test_two_streams_at_once(attn):
    cases = [Case([900, 500], [200, 100], seed=1), Case([700, 20, 300], seed=2)]
    streams = [torch.cuda.Stream() for _ in cases]
    work = [(c.args(), c.to_gpu(c.w)) for c in cases]
    torch.cuda.synchronize()
    for s, ((pos, args), w) in zip(streams, work):
        attn.attn_key_weights(*pos, w, stream=s, **args)
    torch.cuda.synchronize()
    for c, (_, w) in zip(cases, work):
        c.compare(w, "streams")


def test_bad_page_and_length_are_reported(attn):
    for q_lens in (None, [130, 4]):
        c = Case([300, 100], q_lens, seed=3)
        pos, args = c.args()
        w = c.to_gpu(c.w)
        bad = args["page_table"].clone()
        bad[0, 1] = c.pages                       # tokens 64 to 127 of sequence 0
        attn.attn_key_weights(*pos, w, **{**args, "page_table": bad})
        assert attn.attn_device_error_flags(clear=True) == 2
        at = c.place(0, 64)
        assert torch.equal(w.cpu()[at[0]].nan_to_num(-1), c.w[at[0]].nan_to_num(-1))
        attn.attn_key_weights(*pos, c.to_gpu(c.w), **{**args, "max_kv_len": 299})
        assert attn.attn_device_error_flags(clear=True) == 4


def test_weights_of_decode_sum_to_its_rows(attn):
    # with the lse that attn_decode returns: every row gives weight 1 in all, and a sink takes
    # its part
    torch.manual_seed(0)
    lens = [1000, 333, 1]
    c = Case(lens, hq=32, hkv=8, page=128, seed=5)
    pos, args = c.args()
    q, k, _, kv_len = pos
    k = torch.nan_to_num(k)
    v = torch.randn_like(k)
    for sink in (None, torch.randn(32, device=DEV)):
        _, lse = attn.attn_decode(q, k, v, kv_len, group=4, scale=c.scale,
                                  max_kv_len=args["max_kv_len"], page_table=args["page_table"],
                                  sink=sink)
        w = torch.zeros(c.w.shape, device=DEV)
        attn.attn_key_weights(q, k, lse, kv_len, w, **args)
        part = 1 - (torch.exp(sink - lse) if sink is not None else torch.zeros_like(lse))
        for b in range(3):
            got = w[args["page_table"][b, :-(-lens[b] // 128)].long()].flatten(0, 1)[:lens[b]].sum(0)
            assert torch.allclose(got, part[b].view(8, 4).sum(1), atol=1e-3)
