"""What attn_evict_kv writes beside the caches shares no memory with what it reads: refused
before anything is launched (every CTA of both kernels reads the lengths for itself)."""
import pytest

from .test_cache_abi import P, attn, kv  # noqa: F401
from .test_fp4_evict_abi import call_evict

BATCH, HEADS, KEEP, PAGES = 4, 8, 200, 8
LENS, LIST, TABLE = 4 * BATCH, 4 * BATCH * HEADS * KEEP, 4 * BATCH * PAGES
# apart from one another: kv_len, keep, kept_len, indices, the two page tables
AT = dict(lens=P, keep=2 * P, kept=3 * P, idx=4 * P, table=8 * P, to_table=9 * P)


def call(attn, **over):  # noqa: F811
    at = {**AT, **over}
    src = lambda: kv(attn, page_table=at["table"])   # noqa: E731
    dst = lambda: kv(attn, page_table=at["to_table"])   # noqa: E731
    return call_evict(attn, k=src(), v=src(), ko=dst(), vo=dst(),
                      **{x: at[x] for x in ("lens", "keep", "kept", "idx")})


@pytest.mark.parametrize("out,n", [("kept", LENS), ("idx", LIST)])
@pytest.mark.parametrize("name,m", [("lens", LENS), ("keep", LENS), ("table", TABLE),
                                    ("to_table", TABLE)])
def test_outputs_over_inputs(attn, out, n, name, m):  # noqa: F811
    at = AT[name]
    for where in (at, at + 4, at + m - 4, at - n + 4):
        assert call(attn, **{out: where}) == attn.ATTN_ERR_INVALID_ARG, where - at


def test_outputs_over_one_another(attn):  # noqa: F811
    assert call(attn, kept=AT["idx"]) == attn.ATTN_ERR_INVALID_ARG
    assert call(attn, kept=AT["idx"] + LIST - 4) == attn.ATTN_ERR_INVALID_ARG
