"""Calls from host threads of the user's: the first that a thread makes, and calls of two threads
at once whose kernels need unlike amounts of shared memory (a kernel's limit is the process's,
so no call may set it to its own bytes)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CALLS = 5000                # of each thread


@pytest.fixture(scope="module")
def attn():
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn as a
    a.attn_device_error_flags(clear=True)
    yield a
    assert a.attn_device_error_flags(clear=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bf16(*shape):
    return torch.randn(*shape, device=DEV).to(torch.bfloat16)


def small_tables(batch):
    """Sequences of 1 token, all of page 0."""
    return i32([1] * batch), torch.zeros(batch, 1, dtype=torch.int32, device=DEV)


def decode(attn, batch, s, dim):
    k, v, q = bf16(1, 16, 1, dim), bf16(1, 16, 1, dim), bf16(batch, 1, dim)
    lens, table = small_tables(batch)
    return lambda: attn.attn_decode(q, k, v, lens, group=1, scale=0.1, max_kv_len=16,
                                    page_table=table, stream=s)


def decode_fp4(attn, batch, s):
    k, v = (torch.zeros(1, 16, 1, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    e = torch.full((1, 16, 1, 4), 127, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    vs, q = torch.ones(1, 16, 1, device=DEV), bf16(batch, 1, 128)
    lens, table = small_tables(batch)
    return lambda: attn.attn_decode_fp4(q, k, v, e, vs, lens, group=1, scale=0.1, max_kv_len=16,
                                        page_table=table, stream=s)


def decode_fp8(attn, batch, s):
    k, v = (torch.zeros(1, 16, 1, 128, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs, q = torch.ones(1, 1, 1, device=DEV), torch.ones(1, 1, 1, device=DEV), bf16(batch, 1, 128)
    lens, table = small_tables(batch)
    return lambda: attn.attn_decode_fp8(q, k, v, ks, vs, lens, group=1, scale=0.1, max_kv_len=16,
                                        page_table=table, stream=s)


def key_weights(attn, batch, s):
    k, w, q = bf16(batch, 16, 1, 64), torch.ones(batch, 16, 1, device=DEV), bf16(batch, 1, 64)
    lse = torch.zeros(batch, 1, device=DEV)
    lens = small_tables(batch)[0]
    return lambda: attn.attn_key_weights(q, k, lse, lens, w, group=1, scale=0.1, max_kv_len=16,
                                         decay=0.0, stream=s)


def evict(attn, tokens, s):
    # (one sequence over 8 CTAs, whose keys are in shared memory: its length is the size)
    k, out = bf16(1, tokens, 1, 8), bf16(1, 8, 1, 8)
    w = torch.rand(1, tokens, 1, device=DEV)
    lens, keep = i32([100]), i32([8])
    return lambda: attn.attn_evict_kv(k, None, w, lens, keep, out, None, max_kv_len=tokens,
                                      max_keep=8, stream=s)


def append(attn, rows, s):
    # (all heads of a row in one CTA, and tiles of 8 or 16 rows)
    x = bf16(rows, 48, 256)
    k, v = (torch.zeros(1, rows, 8, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    turns, _ = attn.rope_turns(256, 10000.0, device=DEV)
    lens, offs = i32([rows]), i32([0, rows])
    return lambda: attn.attn_append_kv(x[:, 32:40], x[:, 40:], k, v, lens, max_kv_len=rows,
                                       q=x[:, :32], rope=attn.Rope(turns), q_row_offsets=offs,
                                       stream=s)


def append_fp8(attn, rot, s):
    x = bf16(300, 4, 128)
    k, v = (torch.zeros(1, 512, 2, 128, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(1, 4, 2, device=DEV) for _ in range(2))
    rope = attn.Rope(attn.rope_turns(128, 10000.0, device=DEV)[0]) if rot else None
    lens, offs = i32([300]), i32([0, 300])
    return lambda: attn.attn_append_kv_fp8(x[:, :2], x[:, 2:], k, v, ks, vs, lens, max_kv_len=512,
                                           rope=rope, q_row_offsets=offs, stream=s)


def attend(attn, s, q_lens, **kw):
    """Rows of two sequences: by tiles where there are many."""
    rows = sum(q_lens)
    k, v, q = bf16(8, 64, 2, 128), bf16(8, 64, 2, 128), bf16(rows, 8, 128)
    lens, table = i32([200, 130]), torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    offs = i32([0, q_lens[0], rows])
    return lambda: attn.attn_decode(q, k, v, lens, group=4, scale=0.1, max_kv_len=256,
                                    q_row_offsets=offs, max_q_len=max(q_lens), causal=True,
                                    page_table=table, stream=s, **kw)


def mla(attn, s, sparse):
    cache, q = bf16(8, 64, 1, 576), bf16(2, 128, 576)
    lens, table = i32([200, 130]), torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    if sparse:
        some = i32([200, 130])
        index = torch.arange(400, dtype=torch.int32, device=DEV).view(2, 200).contiguous()
        return lambda: attn.attn_mla_decode_sparse(q, cache, index, some, scale=0.1, stream=s)
    return lambda: attn.attn_mla_decode(q, cache, lens, scale=0.1, max_kv_len=256, page_table=table,
                                        stream=s)


FIRST = {
    "decode of 64 channels": lambda a, s: decode(a, 3, s, 64),
    "decode of 128 channels": lambda a, s: decode(a, 3, s, 128),
    "few rows": lambda a, s: attend(a, s, [3, 2]),
    "prompt rows": lambda a, s: attend(a, s, [200, 100]),
    "prompt rows, tile pairs": lambda a, s: attend(a, s, [200, 100],
                                                   num_partitions=a.ATTN_PARTITIONS_TILE_PAIR),
    "mla": lambda a, s: mla(a, s, False),
    "mla, sparse": lambda a, s: mla(a, s, True),
    "decode in 8 bits": lambda a, s: decode_fp8(a, 3, s),
    "decode in 4 bits": lambda a, s: decode_fp4(a, 3, s),
    "append": lambda a, s: append(a, 40, s),
    "append in 8 bits": lambda a, s: append_fp8(a, True, s),
    "key weights": lambda a, s: key_weights(a, 3, s),
    "eviction": lambda a, s: evict(a, 300, s),
}


def flat(x):
    return [x] if torch.is_tensor(x) else [y for y in x or () if y is not None]


@pytest.mark.parametrize("name", list(FIRST))
def test_first_call_of_a_thread(attn, name):
    stream = torch.cuda.Stream()
    run = FIRST[name](attn, stream)
    torch.cuda.synchronize()
    want, got, failed = flat(run()), [], []

    def work():
        try:
            got.extend(flat(run()))
        except Exception as e:      # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for a, b in zip(got, want):
        if a.dtype == torch.int32 and a.dim() == 3:      # (kept tokens: eight of them are there)
            a, b = a[..., :8], b[..., :8]
        assert torch.equal(a, b)


PAIRS = {
    "decode of 64 channels": (lambda a, s: decode(a, 1, s, 64), lambda a, s: decode(a, 2048, s, 64)),
    "decode of 128 channels": (lambda a, s: decode(a, 1, s, 128),
                               lambda a, s: decode(a, 2048, s, 128)),
    "decode in 4 bits": (lambda a, s: decode_fp4(a, 400, s), lambda a, s: decode_fp4(a, 2048, s)),
    "decode in 8 bits": (lambda a, s: decode_fp8(a, 1, s), lambda a, s: decode_fp8(a, 2048, s)),
    "key weights": (lambda a, s: key_weights(a, 1, s), lambda a, s: key_weights(a, 2048, s)),
    "eviction": (lambda a, s: evict(a, 140000, s), lambda a, s: evict(a, 262144, s)),
    "append": (lambda a, s: append(a, 4000, s), lambda a, s: append(a, 5000, s)),
    "append in 8 bits": (lambda a, s: append_fp8(a, False, s), lambda a, s: append_fp8(a, True, s)),
}


class Recorder:
    """In place of the library: what a call of the binding gives it, and nothing runs."""

    def __init__(self, attn):
        self.lib, self.calls = attn.lib(), []

    def __getattr__(self, name):
        if name.endswith("_workspace") or name == "attn_plan_partitions":
            return getattr(self.lib, name)
        return lambda *args: self.calls.append((getattr(self.lib, name), args)) or 0


@pytest.mark.parametrize("name", list(PAIRS))
def test_two_threads_at_once(attn, monkeypatch, name):
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [make(attn, s) for make, s in zip(PAIRS[name], streams)]
    outs, calls = [], []
    with monkeypatch.context() as m:
        for run in runs:
            recorder = Recorder(attn)
            m.setattr(attn, "lib", lambda: recorder)
            outs.append(run())                           # (held: the calls write them)
            calls.append(recorder.calls[0])
            m.undo()
    torch.cuda.synchronize()
    start, codes = threading.Barrier(2), [0, 0]

    def work(me):
        fn, args = calls[me]
        start.wait(60)
        for i in range(CALLS):
            code = fn(*args)
            if code != 0:
                codes[me] = code
                break
            if i % 100 == 99:
                streams[me].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [attn.ATTN_OK, attn.ATTN_OK]
