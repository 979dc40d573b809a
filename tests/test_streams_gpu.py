"""Calls on a given stream (stream=) that allocate their outputs and workspace:
what the current stream allocates and writes meanwhile is other memory."""
import contextlib
import math

import pytest
import torch

from split_flash_decoding_gb300 import workloads as W

DEV = "cuda:0"
FP8 = torch.float8_e4m3fn


def test_memory_of_a_call_on_another_stream(monkeypatch):
    """Without a GPU: taken on the call's stream, returned tensors also known to the current one."""
    from split_flash_decoding_gb300 import attn
    log = []

    class Stream:
        def __init__(self, n):
            self.cuda_stream = n

    class Memory:
        numel = element_size = lambda self: 4

        def record_stream(self, s):
            log.append(("record", s.cuda_stream))

    @contextlib.contextmanager
    def on(s):
        log.append(("enter", s.cuda_stream))
        yield
        log.append(("leave", s.cuda_stream))

    def empty(*a, **k):
        log.append("empty")
        return Memory()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream(1))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    dev = torch.device("cuda", 0)
    took = ["empty"], [("enter", 2), "empty", ("leave", 2)]
    for s, want in ((None, took[0]), (Stream(1), took[0]), (Stream(2), took[1] + [("record", 1)])):
        log.clear()
        attn._empty((3, 4), torch.float32, dev, s)
        assert log == want
    log.clear()
    attn._workspace(4, dev, None, Stream(2))
    assert log == took[1]


@pytest.fixture(scope="module")
def calls():
    """name -> a call with the stream it is given, its inputs ready; returns its outputs."""
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    w = W.make_workload("gqa", batch=3, num_q_heads=32, num_kv_heads=8, dim_qk=128,
                        kv_lens=[3000, 700, 2000], page_size=64, seed=1, device=DEV)
    m = W.make_workload("mla", batch=3, num_q_heads=128, num_kv_heads=1, dim_qk=576, dim_v=512,
                        mla=True, kv_lens=[3000, 700, 2000], page_size=64, seed=2, device=DEV,
                        scale=1.0 / math.sqrt(192.0))
    x = rand(500, 12, 128)
    k8, v8 = [rand(20, 64, 2, 128).to(FP8) for _ in range(2)]
    s8 = torch.full((20, 4, 2), 0.01, device=DEV)
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10).contiguous()
    lens = torch.tensor([600, 640], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 200, 500], dtype=torch.int32, device=DEV)
    kb, vb = [torch.zeros(20, 64, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ka, va = torch.zeros_like(k8), torch.zeros_like(v8)
    sa, sb = torch.ones_like(s8), torch.ones_like(s8)
    turns, mscale = attn.rope_turns(128, 500000.0, device=DEV)
    rope = attn.Rope(turns, mscale=mscale)
    pos = torch.arange(500, dtype=torch.int32, device=DEV)
    part = [torch.randn(4, 30, 8, 128, generator=g).to(DEV)] + [
        torch.rand(4, 30, 8, generator=g).to(DEV) + 1 for _ in range(2)]
    q2 = x[:2, :8].contiguous()
    app = dict(max_kv_len=640, page_table=table, q_row_offsets=offs, rope=rope, q=x[:, :8])
    torch.cuda.synchronize()
    yield {
        "qk_norm_rope": lambda s: attn.attn_qk_norm_rope(x[:, :8], x[:, 8:], pos, rope=rope, stream=s),
        "append_kv": lambda s: (attn.attn_append_kv(x[:, 8:10], x[:, 10:], kb, vb, lens, stream=s,
                                                    **app),),
        "append_kv_fp8": lambda s: (attn.attn_append_kv_fp8(x[:, 8:10], x[:, 10:], ka, va, sa, sb,
                                                            lens, max_q_len=300, stream=s, **app),),
        "decode_fp8": lambda s: attn.attn_decode_fp8(q2, k8, v8, s8, s8, lens, group=4,
                                                     scale=0.1, max_kv_len=640, page_table=table,
                                                     stream=s),
        "decode": lambda s: attn.attn_decode(w.q, w.k_cache, w.v_cache, w.kv_len, group=4,
                                             scale=w.scale, max_kv_len=3000,
                                             page_table=w.page_table, stream=s),
        "mla_decode": lambda s: attn.attn_mla_decode(m.q, m.k_cache, m.kv_len, scale=m.scale,
                                                     max_kv_len=3000, page_table=m.page_table,
                                                     stream=s),
        "splitk_reduce": lambda s: attn.attn_splitk_reduce(*part, stream=s),
    }
    assert attn.attn_device_error_flags(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["qk_norm_rope", "append_kv", "append_kv_fp8", "decode_fp8", "decode",
                                  "mla_decode", "splitk_reduce"])
def test_other_stream_and_allocations_meanwhile(calls, name):
    call = calls[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + [1 << n for n in range(12, 27)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def scribble():
        """Blocks of many sizes from the current stream's memory, written there."""
        held = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        for t in held:
            t.fill_(0xff)

    # the call is still to come on its stream while the current one allocates and writes
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = call(side)
    scribble()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # writes to freed blocks are still to come on the current stream while the call runs
    torch.cuda._sleep(20_000_000)
    scribble()
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
