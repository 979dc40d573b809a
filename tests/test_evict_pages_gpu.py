"""Pages outside the pool under any token that attn_evict_kv weighs, keeps or writes: reported,
and the rest moved as ever."""
import pytest
import torch

from .test_evict_gpu import Case, attn, choice  # noqa: F401

pytestmark = pytest.mark.gpu
PAGE = 16


# Of sequence 0, 100 tokens in 7 pages: the bad page, what is kept, first and recent tokens.
@pytest.mark.parametrize("page,keep,first,recent", [
    (0, 40, 16, 8),          # the first tokens
    (6, 40, 1, 20),          # the last ones
    (6, 3, 1, 20),           # the last ones, and no others stay
    (0, 100, 0, 0), (3, 100, 0, 0), (6, 100, 4, 8),      # everything stays
    (3, 40, 1, 3)])          # tokens that are chosen among
@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_bad_source_page(attn, page, keep, first, recent, entry):  # noqa: F811
    c = Case([100, 50], [keep, 20], page=PAGE, first=first, recent=recent, seed=page)
    pos, kw = c.inputs()
    bad = kw["page_table"].clone()
    bad[0, page] = entry
    before = [x.clone() for x in pos[5:]]
    kept, indices = attn.attn_evict_kv(*pos, **{**kw, "page_table": bad})
    assert attn.attn_device_error_flags(clear=True) == 2
    assert kept.cpu().tolist() == c.kept
    for h in range(c.hkv):
        w = [float(c.w[c.place(0, t)][h]) for t in range(100)]
        w = [float("-inf") if t // PAGE == page else x for t, x in enumerate(w)]
        tokens = choice(w, 100, keep, first, recent)
        assert indices[0, h, :c.kept[0]].tolist() == tokens
        for j, t in enumerate(tokens):
            for x, was, out in zip((c.k, c.v, c.w), before, pos[5:]):
                at = c.place(0, j, True)
                want = was[at][h].cpu() if t // PAGE == page else x[c.place(0, t)][h]
                assert torch.equal(out[at][h].cpu(), want), (h, j, t)


def test_pages_of_tokens_that_nobody_reads(attn):  # noqa: F811
    """Only the last tokens stay: the others are neither weighed nor moved."""
    c = Case([100, 50], [5, 5], page=PAGE, first=0, recent=5, seed=1)
    pos, kw = c.inputs()
    bad = kw["page_table"].clone()
    bad[0, :5] = -1                                       # tokens 0 to 79; 95 to 99 stay
    kept, indices = attn.attn_evict_kv(*pos, **{**kw, "page_table": bad})
    assert attn.attn_device_error_flags(clear=True) == 0
    c.compare(kept, indices, pos[5:])
