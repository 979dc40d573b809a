"""Key weights of 17 to 128 columns (rows x heads of a group), by both kernels: the one that the
bound of rows picks, and each one asked for by a bound that is not the rows' (more rows than it
says are taken as well)."""
import pytest

from .test_key_weights_gpu import Case, attn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_q_len", [None, 1, 1 << 20])
@pytest.mark.parametrize("group,q_lens", [
    (1, [33, 128, 0, 17]), (2, [9, 64, 40, 1]), (3, [6, 40, 11, 33]), (4, [5, 8, 32, 0]),
    (5, [7, 20, 1, 4]), (7, [3, 18, 5, 2]), (8, [3, 4, 16, 9]), (11, [2, 11, 4, 3]),
    (16, [2, 3, 8, 1])])
@pytest.mark.parametrize("causal", [True, False])
def test_columns(attn, max_q_len, group, q_lens, causal):  # noqa: F811
    c = Case([300, 129, 1000, 40], q_lens, hq=5 * group, hkv=5, seed=group, causal=causal, decay=0.9)
    c.check(attn, **({} if max_q_len is None else dict(max_q_len=max_q_len)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch", [3, 30, 130])
def test_amounts_of_work(attn, dim, batch):  # noqa: F811
    """The limit goes by the items of a call: less than a round of them over the GPU, a few, more."""
    lens = [200 + 7 * (i % 50) for i in range(batch)]
    for q_lens in ([4] * batch, [7 + i % 2 for i in range(batch)], [16] * batch, [17] * batch):
        Case(lens, q_lens, hq=16, hkv=4, dim=dim, seed=batch, page=128).check(attn)
