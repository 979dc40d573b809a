"""Decode over a 4-bit cache where nearly all the weight lies on keys that have no value in most
channels: the others' values are all there is of those.

Every sixteenth key has a score of `nats`, the others of 0 (q and all keys are in one channel, so
both scores are exact).  A heavy key's value is in channel 0 alone, the light ones' in channels 1
to 127.  Then out there is sum_j v_j / (heavy e^nats + light), and a light key's
weight may be off by 2^-34 of a heavy one's, relative to its own 2^-34 e^nats, or by 2^-12."""
import math

import pytest
import torch

from .test_fp4_cache_gpu import attn, i32  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
L = 20000
# Half a bf16 step: 8 bits, so a step is 2^-7 of the power of two below a value.  (And a bit for
# the products of the bound's terms.)
BF16_HALF = 2.0 ** -8 * (1 + 2.0 ** -6)


@pytest.mark.parametrize("rows,hq", [(1, 1), (1, 4), (2, 4), (4, 4)])
@pytest.mark.parametrize("nats", [10, 15, 17, 19, 20, 21])
def test_light_keys(attn, nats, rows, hq):  # noqa: F811
    g = torch.Generator().manual_seed(nats)
    k = torch.zeros(1, L, 1, 64, dtype=torch.uint8)
    k[:, ::16, :, 0] = 2                                  # code of 1, channel 0
    heavy = torch.zeros(L, dtype=torch.bool)
    heavy[::16] = True
    codes = torch.randint(1, 8, (L, 128), generator=g, dtype=torch.uint8)
    codes[:, 0] = 0
    codes[heavy] = 0
    codes[heavy, 0] = 7
    v = (codes[:, 0::2] | (codes[:, 1::2] << 4)).view(1, L, 1, 64)
    e = torch.full((1, L, 1, 4), 127, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    vs = torch.ones(1, L, 1)
    q = torch.zeros(rows, hq, 128, dtype=torch.bfloat16)
    q[..., 0] = nats
    q[..., 1] = 1.0                                       # (no key has it)
    out, lse = attn.attn_decode_fp4(q.to(DEV), k.to(DEV), v.to(DEV), e.to(DEV), vs.to(DEV), i32([L]),
                                    group=hq, scale=1.0, max_kv_len=L,
                                    q_row_offsets=i32([0, rows]), max_q_len=rows)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    z = int(heavy.sum()) * math.exp(nats) + int((~heavy).sum())
    want = grid[codes[~heavy].long()].sum(0) / z
    rel = BF16_HALF + max(2.0 ** -12, 2.0 ** -34 * math.exp(nats)) + 2.0 ** -18   # (2^-18: e^nats)
    got = out.cpu().double()
    assert ((got[..., 1:] - want[1:]).abs() <= rel * want[1:]).all(), (got[0, 0, 1:] / want[1:])
    assert ((lse.cpu().double() - math.log(z)).abs() <= 2.0 ** -20 * nats).all()
    first = 6 * int(heavy.sum()) * math.exp(nats) / z
    assert ((got[..., 0] - first).abs() <= rel * first).all()
