"""Calls on a given stream of the entry points of a 4-bit cache, of key weights and of eviction:
what they allocate is the call's stream's, and what the current stream allocates and writes
meanwhile is other memory; and the same calls captured twice over shared inputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def codes(attn, x, table, lens, offs):
    """A 4-bit cache of rows x, head-major."""
    k, v = [torch.zeros(20, 2, 64, 64, dtype=torch.uint8, device=DEV).transpose(1, 2)
            for _ in range(2)]
    ke = torch.zeros(20, 2, 64, 4, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    ke, vs = ke.transpose(1, 2), torch.zeros(20, 2, 64, device=DEV).transpose(1, 2)
    attn.attn_append_kv_fp4(x[:, :2], x[:, 2:], k, v, ke, vs, lens, max_kv_len=640,
                            page_table=table, q_row_offsets=offs)
    return k, v, ke, vs


@pytest.fixture(scope="module")
def calls():
    """name -> a call with the stream it is given, its inputs ready; returns its outputs."""
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10).contiguous()
    to_table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3).contiguous()
    lens = torch.tensor([600, 640], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 600, 1240], dtype=torch.int32, device=DEV)
    x, q = rand(1240, 4, 128), rand(2, 8, 128)
    cache = codes(attn, x, table, lens, offs)
    again = [torch.empty_strided(t.shape, t.stride(), dtype=torch.uint8, device=DEV).zero_()
             .view(t.dtype) if t.dtype != torch.float32 else torch.zeros_like(t) for t in cache]
    k, v = rand(20, 64, 2, 128), rand(20, 64, 2, 128)
    lse = attn.attn_decode(q, k, v, lens, group=4, scale=0.1, max_kv_len=640, page_table=table)[1]
    w = torch.rand(20, 64, 2, generator=g).to(DEV)
    added = torch.zeros_like(w)
    keep = torch.tensor([150, 170], dtype=torch.int32, device=DEV)
    ko, vo = [torch.zeros(6, 64, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kw = dict(max_kv_len=640, page_table=table)

    def append(s):
        return (attn.attn_append_kv_fp4(x[:, :2], x[:, 2:], *again, lens, q=x, q_row_offsets=offs,
                                        stream=s, **kw),)

    def weights(s):
        attn.attn_key_weights(q, k, lse, lens, added, group=4, scale=0.1, decay=0.0, stream=s, **kw)
        return (added,)

    torch.cuda.synchronize()
    yield {
        "append_fp4": append,
        "decode_fp4": lambda s: attn.attn_decode_fp4(q, *cache, lens, group=4, scale=0.1, stream=s,
                                                     **kw),
        "key_weights": weights,
        "evict": lambda s: (*attn.attn_evict_kv(k, v, w, lens, keep, ko, vo, max_keep=170, recent=8,
                                                out_page_table=to_table, stream=s, **kw), ko, vo),
    }
    assert attn.attn_device_error_flags(clear=True) == 0


def filled(name, outs):
    """The parts of outs that a call writes (an eviction's indices only up to what it keeps)."""
    if name != "evict":
        return [t.clone() for t in outs]
    kept, indices = outs[:2]
    keep = kept.long()
    return [kept.clone()] + [indices[b, :, :keep[b]].clone() for b in range(2)] + [
        t.clone() for t in outs[2:]]


NAMES = ["append_fp4", "decode_fp4", "key_weights", "evict"]


@pytest.mark.parametrize("name", NAMES)
def test_other_stream_and_allocations_meanwhile(calls, name):
    call = calls[name]
    outs = call(None)
    want = filled(name, outs)
    sizes = [t.numel() * t.element_size() for t in outs] + [1 << n for n in range(12, 27)]
    del outs
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    with torch.cuda.stream(side):
        for _ in range(20):
            busy @ busy
    got = call(side)
    held = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    for t in held:
        t.fill_(0xff)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(filled(name, got), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_of_a_call(calls, name):
    """Captured twice and replayed in turns and side by side: the same each time."""
    call = calls[name]
    want = filled(name, call(None))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(None))
        graphs.append(g)
    for g in (*graphs, *graphs):
        g.replay()
    torch.cuda.synchronize()
    if name in ("append_fp4", "decode_fp4"):         # (the others write what both are given)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(filled(name, o), want):
            assert torch.equal(a, b)
