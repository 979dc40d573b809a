"""Outputs of attn_evict_kv right beside its inputs, in one buffer: apart, so they are taken."""
import pytest
import torch

from .test_evict_gpu import Case, attn  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_beside_inputs(attn):  # noqa: F811
    c = Case([100, 50], [40, 20], seed=5)
    pos, kw = c.inputs()
    n = 2 * c.hkv * c.max_keep
    buf = torch.zeros(6 + n, dtype=torch.int32, device="cuda:0")
    buf[2:4], buf[4 + n:] = pos[3], pos[4]
    pos[3], pos[4] = buf[2:4], buf[4 + n:]                # kept_len, kv_len, indices, keep
    indices = buf[4:4 + n].view(2, c.hkv, c.max_keep)
    indices.fill_(-1)
    kw["indices"] = indices
    kept, indices = attn.attn_evict_kv(*pos, **kw, kept_len=buf[:2])
    torch.cuda.synchronize()
    c.compare(kept, indices, pos[5:])
    for name, at in (("kept_len", buf[2:4]), ("kept_len", buf[1:3]), ("kept_len", buf[4 + n:]),
                     ("kept_len", buf[4:6]), ("indices", buf[3:3 + n].view(indices.shape)),
                     ("indices", buf[5:5 + n].view(indices.shape))):
        with pytest.raises(attn.AttnError):
            attn.attn_evict_kv(*pos, **{**kw, name: at})
