"""The two kernels of the append into a 4-bit cache round alike: a rotation whose pairs cut
16-byte vectors has a kernel of its own, and the same rotation with pairs behind it that do not
turn has the tiles'.  Equal values, so equal codes and scales."""
import pytest
import torch

from .test_fp4_cache_gpu import attn, i32  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def appended(attn, x, turns, k_norm=None):  # noqa: F811
    """Codes and scales of keys x, interleaved pairs turned."""
    rows, heads = x.shape[:2]
    k, v = (torch.zeros(1, rows, heads, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    e = torch.zeros(1, rows, heads, 4, dtype=torch.uint8, device=DEV)
    attn.attn_append_kv_fp4(x, x, k, v, e.view(torch.float8_e8m0fnu),
                            torch.zeros(1, rows, heads, device=DEV), i32([rows]), max_kv_len=rows,
                            rope=attn.Rope(turns, interleaved=True), k_norm=k_norm,
                            q_row_offsets=i32([0, rows]))
    return k, e


def wide(turns, pairs):
    """Turns and pairs behind them that stay."""
    return torch.cat([turns, turns.new_zeros(pairs)])


def test_rotation(attn):  # noqa: F811
    """100 million codes: a different rounding of the products shows in about one in ten million."""
    turns, _ = attn.rope_turns(124, 10000.0, device=DEV)
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn(50000, 4, 128, generator=g, device=DEV).to(torch.bfloat16)
        (k, e), (k2, e2) = appended(attn, x, turns), appended(attn, x, wide(turns, 2))
        assert torch.equal(e, e2), (e != e2).sum()
        assert torch.equal(k, k2), (k != k2).sum()


def test_norm(attn):  # noqa: F811
    """Values whose squares add up exactly, in any order: the factor is the same."""
    still = torch.zeros(2, dtype=torch.int64, device=DEV)
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = (torch.randint(-31, 32, (50000, 4, 128), generator=g, device=DEV) / 8).to(torch.bfloat16)
        norm = (1 + 0.1 * torch.randn(128, generator=g, device=DEV)).to(torch.bfloat16)
        (k, e), (k2, e2) = appended(attn, x, still, norm), appended(attn, x, wide(still, 2), norm)
        assert torch.equal(e, e2), (e != e2).sum()
        assert torch.equal(k, k2), (k != k2).sum()
