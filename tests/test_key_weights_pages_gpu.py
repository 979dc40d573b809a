"""Pages outside the pool under any token of attn_key_weights, whatever rows its sequence has:
reported, their weights left, the others as ever."""
import pytest
import torch

from .test_key_weights_gpu import Case, attn  # noqa: F401

pytestmark = pytest.mark.gpu


# Of sequence 0, 300 tokens in 5 pages of 64; the rows of the two sequences.
@pytest.mark.parametrize("q_lens", [[0, 3], [0, 60], [0, 0], [2, 1], [70, 0], [300, 100], None])
@pytest.mark.parametrize("page", [0, 2, 4])
@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_bad_page(attn, q_lens, page, entry):  # noqa: F811
    c = Case([300, 100], q_lens, seed=page, decay=0.5)
    pos, args = c.args()
    bad = args["page_table"].clone()
    bad[0, page] = entry
    w = c.to_gpu(c.w)
    attn.attn_key_weights(*pos, w, **{**args, "page_table": bad})
    assert attn.attn_device_error_flags(clear=True) == 2
    lost = int(c.table[0, page])
    assert torch.equal(w.cpu()[lost].nan_to_num(-1), c.w[lost].nan_to_num(-1))
    c.owned[lost] = False
    left = torch.ones(c.pages, dtype=torch.bool)
    left[lost] = False
    want, err = c.reference()
    got = w.cpu().double()
    here = c.owned & left[:, None]
    assert ((got - want).abs()[here] <= err[here]).all()
    rest = ~c.owned & left[:, None]
    assert torch.equal(got[rest], c.w.double()[rest])
