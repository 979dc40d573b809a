"""Eviction of the keys that gathered least (attn_evict_kv) against lists in Python: whole
numbers and moved rows, all of them equal."""
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


def choice(w, L, keep, first, recent):
    """The kept tokens of one head: w a list of L floats."""
    n = min(L, max(keep, 0))
    r = min(recent, n)
    f = min(first, n - r)
    value = lambda i: -math.inf if math.isnan(w[i]) else w[i]   # noqa: E731
    best = sorted(range(f, L - r), key=lambda i: (-value(i), i))[:n - r - f]
    return sorted(list(range(f)) + best + list(range(L - r, L)))


def tables(lens, page, g):
    need = [max(1, -(-x // page)) for x in lens]
    pages = sum(need) + 1
    perm = torch.randperm(pages, generator=g)
    table, at = torch.full((len(lens), max(need)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return table, pages


class Case:
    def __init__(self, lens, keep, *, hkv=2, dim=64, dim_v=None, page=16, to_page=None, first=1,
                 recent=3, seed=0, values="heavy", contiguous=False, head_major=False, latent=False,
                 max_keep=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.keep, self.first, self.recent, self.hkv = lens, keep, first, recent, hkv
        self.kept = [min(L, max(k, 0)) for L, k in zip(lens, keep)]
        self.max_keep = max(max(keep), 0) if max_keep is None else max_keep
        to_page = to_page or page
        if contiguous:
            page, to_page = max(max(lens), 1), max(self.max_keep, 1)
            self.table = self.to = None
            pages = to_pages = len(lens)
        else:
            self.table, pages = tables(lens, page, g)
            self.to, to_pages = tables([self.max_keep] * len(lens), to_page, g)
        self.page, self.to_page = page, to_page
        shape = (pages, page, hkv)
        rnd = lambda d: torch.randn(*shape, d, generator=g).to(torch.bfloat16)   # noqa: E731
        self.k = rnd(dim)
        self.v = None if latent else rnd(dim_v or dim)
        if values == "heavy":
            self.w = torch.exp(3 * torch.randn(shape, generator=g))
        elif values == "ties":
            self.w = torch.randint(0, 4, shape, generator=g).float() * 0.25
        elif values == "equal":
            self.w = torch.full(shape, 0.125)
        elif values == "near":      # differ in the last bits only
            self.w = (torch.randint(0, 64, shape, generator=g) + 0x3f800000).to(torch.int32).view(torch.float32)
        else:                       # of both signs, infinite, NaN, zeros of both signs
            some = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, -1.5, 2.0, 1e-42])
            self.w = some[torch.randint(0, 8, shape, generator=g)]
        self.out = [torch.full((to_pages, to_page, hkv, x.shape[3]), -7.0, dtype=torch.bfloat16)
                    if x is not None else None for x in (self.k, self.v)]
        self.w_out = torch.full((to_pages, to_page, hkv), -7.0)
        self.head_major = head_major

    def place(self, b, t, to=False):
        table, page = (self.to, self.to_page) if to else (self.table, self.page)
        return (b, t) if table is None else (int(table[b, t // page]), t % page)

    def gpu(self, x):
        if x is None:
            return None
        if self.head_major and x.dim() >= 3:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        return x.to(DEV)

    def inputs(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
        kw = dict(max_kv_len=max(self.lens), max_keep=self.max_keep, first=self.first,
                  recent=self.recent,
                  page_table=None if self.table is None else self.table.to(DEV),
                  out_page_table=None if self.to is None else self.to.to(DEV),
                  indices=torch.full((len(self.lens), self.hkv, self.max_keep), -1,
                                     dtype=torch.int32, device=DEV))
        return [self.gpu(self.k), self.gpu(self.v), self.gpu(self.w), i32(self.lens),
                i32(self.keep), self.gpu(self.out[0]), self.gpu(self.out[1]), self.gpu(self.w_out)], kw

    def check(self, attn, **more):
        pos, kw = self.inputs()
        kw.update(more)
        kept, indices = attn.attn_evict_kv(*pos, **kw)
        torch.cuda.synchronize()
        self.compare(kept, indices, pos[5:])

    def compare(self, kept, indices, outs):
        assert kept.cpu().tolist() == self.kept
        want = [None if x is None else x.clone() for x in self.out] + [self.w_out.clone()]
        index = torch.full((len(self.lens), self.hkv, self.max_keep), -1, dtype=torch.int32)
        for b, L in enumerate(self.lens):
            old = [self.place(b, t) for t in range(L)]
            new = [self.place(b, j, True) for j in range(self.kept[b])]
            for h in range(self.hkv):
                tokens = choice([float(self.w[p][h]) for p in old], L, self.keep[b], self.first,
                                self.recent)
                assert len(tokens) == self.kept[b]
                index[b, h, :len(tokens)] = torch.tensor(tokens, dtype=torch.int32)
                for j, t in enumerate(tokens):
                    for x, y in zip((self.k, self.v, self.w), want):
                        if x is not None:
                            y[new[j]][h] = x[old[t]][h]
        assert torch.equal(indices.cpu(), index)
        for got, y in zip(outs, want):
            if y is not None:
                a, b = got.cpu().contiguous(), y.contiguous()
                bits = torch.int32 if a.dtype == torch.float32 else torch.int16
                assert torch.equal(a.view(bits), b.view(bits))


@pytest.mark.parametrize("values", ["heavy", "ties", "equal", "near", "odd"])
@pytest.mark.parametrize("lens,keep", [([40], [10]), ([1, 0, 7, 33], [1, 1, 3, 32]),
                                       ([600, 511, 513, 512], [100, 512, 512, 1])])
def test_choice(attn, values, lens, keep):
    Case(lens, keep, values=values, seed=len(lens)).check(attn)


@pytest.mark.parametrize("first,recent", [(0, 0), (0, 5), (4, 0), (4, 200), (200, 4), (100, 100)])
def test_tokens_that_always_stay(attn, first, recent):
    Case([150, 90, 3, 301], [60, 90, 2, 100], first=first, recent=recent, seed=first + recent).check(attn)


def test_nothing_or_everything(attn):
    Case([30, 40, 0], [0, -3, 0], seed=1, max_keep=4).check(attn)
    Case([30, 40, 0], [0, 0, 0], seed=1).check(attn)
    Case([30, 40, 1], [30, 99, 1], seed=1).check(attn)


@pytest.mark.parametrize("page,to_page", [(8, 64), (64, 8), (256, 16), (32, 32)])
@pytest.mark.parametrize("head_major", [False, True])
def test_pages_and_layouts(attn, page, to_page, head_major):
    Case([100, 300, 9], [50, 120, 9], page=page, to_page=to_page, head_major=head_major,
         seed=page).check(attn)


def test_contiguous(attn):
    Case([100, 300, 9], [50, 120, 9], contiguous=True, seed=2).check(attn)


@pytest.mark.parametrize("hkv,dim,dim_v", [(1, 8, 8), (3, 72, 128), (8, 128, 128), (16, 256, 64),
                                           (5, 1024, 8)])
def test_heads_and_dims(attn, hkv, dim, dim_v):
    Case([70, 41], [20, 40], hkv=hkv, dim=dim, dim_v=dim_v, seed=dim).check(attn)


def test_latent_rows(attn):
    Case([200, 90], [64, 64], hkv=1, dim=576, latent=True, seed=4).check(attn)


@pytest.mark.parametrize("values", ["heavy", "ties", "equal"])
@pytest.mark.parametrize("L,keep", [(5000, 700), (20000, 19000), (40000, 4096)])
def test_long_sequences_over_a_cluster(attn, values, L, keep):
    Case([L, 100], [keep, 30], hkv=1, dim=8, page=256, values=values, first=4, recent=64,
         seed=L).check(attn)


def test_longer_than_a_cluster_holds(attn):
    # the weights no longer fit the CTAs' shared memory and are read again for every digit
    L = 8 * 32768 + 1000
    Case([L], [3000], hkv=1, dim=8, page=1024, values="heavy", seed=3).check(attn)


def test_many_sequences(attn):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 60, (300,), generator=g).tolist()
    Case(lens, [x // 2 for x in lens], hkv=2, dim=8, page=8, seed=2).check(attn)


def test_without_weights_out_and_given_outputs(attn):
    c = Case([100, 30], [20, 20], seed=6)
    pos, kw = c.inputs()
    del kw["indices"]
    pos[7] = None
    kept, indices = attn.attn_evict_kv(*pos, **kw)
    for b in range(2):
        for h in range(2):
            w = [float(c.w[c.place(b, t)][h]) for t in range(c.lens[b])]
            assert indices[b, h, :int(kept[b])].tolist() == choice(w, c.lens[b], c.keep[b], 1, 3)


def test_into_other_pages_of_the_same_pool(attn):
    g = torch.Generator().manual_seed(3)
    pool = torch.randn(12, 16, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    v = torch.randn(12, 16, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand(12, 16, 2, generator=g).to(DEV)
    before = pool.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    kept, index = attn.attn_evict_kv(pool, v, w, i32([60]), i32([20]), pool, v, w, max_kv_len=60,
                                     max_keep=20, page_table=i32([[3, 1, 7, 9]]),
                                     out_page_table=i32([[0, 5]]))
    src = before[[3, 1, 7, 9]].reshape(64, 2, 64)
    dst = pool[[0, 5]].reshape(32, 2, 64)
    for h in range(2):
        assert torch.equal(dst[:20, h], src[index[0, h].long(), h])
    same = [1, 2, 3, 4, 6, 7, 8, 9, 10, 11]
    assert torch.equal(pool[same], before[same])


def test_lengths_are_there_where_no_token_stays(attn):
    """What follows a call that moves nothing: the lengths are 0, whatever they were."""
    c = Case([3000, 200, 0], [0, -5, 7], seed=2)
    pos, kw = c.inputs()
    want = torch.zeros(3, dtype=torch.int32, device=DEV)
    seen = []
    for _ in range(20):
        kept = torch.full((3,), 77, dtype=torch.int32, device=DEV)
        attn.attn_evict_kv(*pos, **kw, kept_len=kept)
        seen.append(kept.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in seen)


def test_offsets_beyond_32_bits(attn):
    # pages far apart in one large pool: 3 G elements of keys, as much of values
    pages, page, dim = 1 << 15, 64, 1024
    free = torch.cuda.mem_get_info()[0]
    if free < 20 << 30:
        pytest.skip("not enough memory")
    pool = torch.empty((pages, page, 1, dim), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((pages, page, 1), device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    table = i32([[pages - 1, 2, pages - 3]])
    for p in (pages - 1, 2, pages - 3):
        pool[p].normal_()
        w[p].uniform_()
    kept, index = attn.attn_evict_kv(pool, None, w, i32([150]), i32([64]), pool, None, None,
                                     max_kv_len=150, max_keep=64, page_table=table,
                                     out_page_table=i32([[pages - 2]]))
    src = pool[table[0].long()].reshape(-1, dim)
    assert torch.equal(pool[pages - 2, :, 0], src[index[0, 0].long()])


def test_captured_and_replayed_with_other_lengths(attn):
    big = Case([300, 200], [80, 80], seed=8)
    pos, kw = big.inputs()
    kept = torch.zeros(2, dtype=torch.int32, device=DEV)
    attn.attn_evict_kv(*pos, kept_len=kept, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attn_evict_kv(*pos, kept_len=kept, **kw)
    for lens, keep in (([300, 200], [80, 80]), ([50, 7], [13, 80]), ([0, 200], [5, 0])):
        c = Case([300, 200], [80, 80], seed=8)
        c.w = torch.rand(c.w.shape, generator=torch.Generator().manual_seed(lens[1]))
        c.lens, c.keep = lens, keep
        c.kept = [min(a, b) for a, b in zip(lens, keep)]
        pos[2].copy_(c.w)
        pos[3].copy_(torch.tensor(lens))
        pos[4].copy_(torch.tensor(keep))
        for i, x in zip((5, 6, 7), (*c.out, c.w_out)):
            pos[i].copy_(x)
        kw["indices"].fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        c.compare(kept, kw["indices"], pos[5:])


def test_two_streams_at_once(attn):
    cases = [Case([3000], [700], hkv=1, seed=1), Case([500, 90], [100, 90], seed=2)]
    streams = [torch.cuda.Stream() for _ in cases]
    work = [c.inputs() for c in cases]
    torch.cuda.synchronize()
    got = [attn.attn_evict_kv(*pos, stream=s, **kw) for s, (pos, kw) in zip(streams, work)]
    torch.cuda.synchronize()
    for c, (pos, _), (kept, index) in zip(cases, work, got):
        c.compare(kept, index, pos[5:])


def test_bad_pages_and_bounds_are_reported(attn):
    c = Case([100, 50], [40, 20], seed=5)
    pos, kw = c.inputs()
    for name, flag in (("page_table", 2), ("out_page_table", 2)):
        bad = kw[name].clone()
        bad[0, 1] = 1 << 20
        attn.attn_evict_kv(*pos, **{**kw, name: bad})
        assert attn.attn_device_error_flags(clear=True) == flag
    attn.attn_evict_kv(*pos, **{**kw, "max_kv_len": 99})
    assert attn.attn_device_error_flags(clear=True) == 4
    attn.attn_evict_kv(*pos, **{**kw, "max_keep": 39, "indices": None})
    assert attn.attn_device_error_flags(clear=True) == 4
