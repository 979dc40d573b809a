"""Every way that attn_evict_kv's choice is cut: CTAs of a (sequence, head) by how many of them
there are and how long the longest may be, weights of a thread by what falls to it, and past
its registers in shared memory or read again for every digit.

Most sequences are short, so that many units cost little; the long ones end off every
boundary.  The reference is a stable sort of the weights."""
import pytest
import torch

from .test_evict_gpu import attn  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def weights(kind, n, g):
    if kind == "heavy":
        return torch.exp(3 * torch.randn(n, generator=g, device=DEV))
    if kind == "ties":
        return torch.randint(0, 4, (n,), generator=g, device=DEV).float() * 0.25
    if kind == "near":                       # differ in the last bits only
        return (torch.randint(0, 64, (n,), generator=g, device=DEV) + 0x3f800000).to(
            torch.int32).view(torch.float32)
    return torch.full((n,), 0.125, device=DEV)


def kept_tokens(w, keep, first, recent):
    L = w.numel()
    n = min(L, keep)
    r = min(recent, n)
    f = min(first, n - r)
    order = torch.sort(w[f:L - r], descending=True, stable=True).indices[:n - r - f] + f
    t = torch.arange(L, device=DEV)
    return torch.cat([t[:f], order.sort().values, t[L - r:]])


def check(attn, units, longest, lens, kind, first=4, recent=33):  # noqa: F811
    """units sequences of one head, the first of them lens, the others short."""
    g = torch.Generator(device=DEV).manual_seed(longest + len(kind))
    lens = lens + [7 + i % 60 for i in range(units - len(lens))]
    page = 64
    need = [-(-n // page) for n in lens]
    table = torch.full((units, -(-longest // page)), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pages = sum(need)
    k = torch.randint(-99, 100, (pages, page, 1, 8), generator=g, device=DEV).to(torch.bfloat16)
    w = weights(kind, pages * page, g).view(pages, page, 1)
    keep = [max(1, n // 3) for n in lens]
    most = max(keep)
    out = torch.zeros(units, most, 1, 8, dtype=torch.bfloat16, device=DEV)
    w_out = torch.zeros(units, most, 1, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    kept, index = attn.attn_evict_kv(k, None, w, i32(lens), i32(keep), out, None, w_out,
                                     max_kv_len=longest, max_keep=most, first=first, recent=recent,
                                     page_table=table)
    assert kept.tolist() == keep
    for b, n in enumerate(lens):
        mine = table[b, :need[b]].long()
        values = w[mine].flatten()[:n]
        tokens = kept_tokens(values, keep[b], first, recent)
        assert torch.equal(index[b, 0, :keep[b]].long(), tokens), b
        assert torch.equal(out[b, :keep[b], 0], k[mine].flatten(0, 2)[:n][tokens]), b
        assert torch.equal(w_out[b, :keep[b], 0], values[tokens]), b


# On 152 SMs: 80 units have a CTA each, 40 two, 30 four and 10 eight, unless the longest may be
# longer than those hold in registers (16 weights of 1024 threads).
@pytest.mark.parametrize("kind", ["heavy", "ties", "near", "equal"])
@pytest.mark.parametrize("units,longest", [
    (80, 1000), (80, 1024), (80, 1025), (80, 2048), (80, 4096), (80, 4097), (80, 8192), (80, 8193),
    (80, 16384), (80, 16385), (80, 32769),
    (40, 2049), (40, 8192), (40, 8193), (40, 16385), (40, 32768),
    (30, 4097), (30, 16384), (30, 16385), (30, 32769), (30, 65536), (30, 65537),
    (10, 8193), (10, 32768), (10, 32769), (10, 65537), (10, 131072)])
def test_weights_in_registers(attn, kind, units, longest):  # noqa: F811
    check(attn, units, longest, [longest, longest - 1, longest // 2 + 5, longest // 8, 1], kind)


@pytest.mark.parametrize("kind", ["heavy", "ties", "near", "equal"])
@pytest.mark.parametrize("longest", [131073, 140000, 262143, 262144, 262145, 300001])
def test_weights_in_shared_memory_or_read_again(attn, kind, longest):  # noqa: F811
    check(attn, 3, longest, [longest, 131072, 90], kind)
    check(attn, 1, longest, [longest - 70000], kind)


@pytest.mark.parametrize("longest", [1000, 5000, 20000, 140000, 263000])
def test_all_or_none_chosen_among(attn, longest):  # noqa: F811
    """Where what stays anyway is all there is."""
    check(attn, 2, longest, [longest, 300], "heavy", first=0, recent=longest)
    check(attn, 2, longest, [longest, 300], "heavy", first=longest, recent=0)
    check(attn, 2, longest, [longest, 300], "ties", first=0, recent=0)
