"""The entry points that fill a KV cache and read one held in 8 bits, without a
GPU: refusals before anything is launched, and the host-side frequencies."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

P = 0x10000      # a 256-byte aligned address that is never read


@pytest.fixture(scope="module")
def attn():
    from split_flash_decoding_gb300 import build
    build.build()
    from split_flash_decoding_gb300 import attn as a
    return a


def struct(cls, base, over):
    d = cls()
    for k, v in {**base, **over}.items():
        setattr(d, k, v)
    return d


def heads(attn, **over):
    return struct(attn.attn_head_rows_t,
                  dict(in_=P, in_row_stride=48 * 128, in_head_stride=128, out=P,
                       out_row_stride=32 * 128, out_head_stride=128, norm_weight=P, norm_eps=1e-6,
                       norm_dim=128, num_heads=32, dim=128), over)


def kv(attn, **over):
    return struct(attn.attn_kv_t,
                  dict(base=P, page_stride=64 * 8 * 128, token_stride=8 * 128, head_stride=128,
                       page_size=64, num_pages=10, page_table=P, max_pages=8), over)


def rope(attn, **over):
    return struct(attn.attn_rope_t, dict(turns=P, rot_dim=128, mscale=1.0), over)


def scales(attn, **over):
    return struct(attn.attn_kv_scale_t,
                  dict(base=P, page_stride=32, block_stride=8, head_stride=1, block_tokens=16), over)


def ref(x):
    return None if x is None else ctypes.byref(x)


def call_qk(attn, q=0, k=0, r=0, pos=P, rows=4):
    q = heads(attn) if q == 0 else q
    k = heads(attn, num_heads=8) if k == 0 else k
    r = rope(attn) if r == 0 else r
    return attn.lib().attn_qk_norm_rope(ref(q), ref(k), ref(r), pos, rows, None)


def test_struct_layouts(attn):
    assert ctypes.sizeof(attn.attn_rope_t) == 24
    assert ctypes.sizeof(attn.attn_head_rows_t) == 80
    assert ctypes.sizeof(attn.attn_kv_scale_t) == 40


def test_qk_norm_rope_refusals(attn):
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    H = lambda **o: heads(attn, **o)   # noqa: E731
    assert call_qk(attn, q=None) == INV
    assert call_qk(attn, rows=-1) == INV
    assert call_qk(attn, pos=None) == INV
    assert call_qk(attn, pos=P + 2) == INV
    for over in (dict(in_=None), dict(out=None), dict(in_=P + 8), dict(out=P + 2),
                 dict(norm_weight=P + 8), dict(in_row_stride=100), dict(in_head_stride=4),
                 dict(out_row_stride=100), dict(out_head_stride=129), dict(num_heads=0),
                 dict(num_heads=-1), dict(dim=0), dict(norm_dim=136), dict(norm_dim=-8),
                 dict(rot_start=-8), dict(rot_start=8), dict(reserved=1),
                 dict(norm_eps=float("nan")), dict(norm_eps=-1.0)):
        assert call_qk(attn, q=H(**over)) == INV, over
        assert call_qk(attn, k=H(**over)) == INV, over
    for over in (dict(dim=132, norm_dim=0), dict(dim=1032, norm_dim=0), dict(norm_dim=12),
                 dict(rot_start=4)):
        assert call_qk(attn, q=H(**over)) == UNS, over
    for over in (dict(rot_dim=-2), dict(rot_dim=7), dict(rot_dim=130), dict(turns=None),
                 dict(turns=P + 4), dict(mscale=float("nan")), dict(reserved=1)):
        assert call_qk(attn, r=rope(attn, **over)) == INV, over
    # nothing to do: nothing is launched, bad arguments are refused all the same
    assert call_qk(attn, rows=0) == attn.ATTN_OK
    assert call_qk(attn, rows=0, q=H(reserved=1)) == INV


def call_append(attn, fp8=False, q=0, k=0, v=0, r=0, pos=None, kc=0, vc=0, ks=0, vs=0, lens=P,
                offs=None, batch=4, rows=4, max_q=1, max_kv=500):
    q = heads(attn) if q == 0 else q
    k = heads(attn, num_heads=8, out=None) if k == 0 else k
    v = heads(attn, num_heads=8, out=None, norm_dim=0, norm_weight=None) if v == 0 else v
    r = rope(attn) if r == 0 else r
    kc = kv(attn) if kc == 0 else kc
    vc = kv(attn) if vc == 0 else vc
    ks = scales(attn) if ks == 0 else ks
    vs = scales(attn) if vs == 0 else vs
    head = (ref(q), ref(k), ref(v), ref(r), pos, ref(kc), ref(vc))
    if fp8:
        return attn.lib().attn_append_kv_fp8(*head, ref(ks), ref(vs), lens, offs, batch, rows,
                                             max_q, max_kv, None)
    return attn.lib().attn_append_kv(*head, lens, offs, batch, rows, max_kv, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(attn, fp8):
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    call = lambda **o: call_append(attn, fp8, **o)   # noqa: E731
    K = lambda **o: heads(attn, **{**dict(num_heads=8, out=None), **o})   # noqa: E731
    V = lambda **o: K(**{**dict(norm_dim=0, norm_weight=None), **o})      # noqa: E731
    assert call(k=None) == INV
    assert call(lens=None) == INV
    assert call(lens=P + 2) == INV
    assert call(pos=P + 1) == INV
    assert call(offs=P + 2) == INV
    assert call(batch=-1) == INV
    assert call(rows=5) == INV                        # without offsets: one row per sequence
    assert call(max_kv=-1) == INV
    assert call(max_kv=513) == INV                    # 8 pages of 64
    assert call(v=None) == INV and call(vc=None) == INV
    assert call(k=K(out=P)) == INV                    # keys go to the cache
    assert call(q=heads(attn, out=None)) == INV
    assert call(v=V(norm_dim=128)) == INV             # values are stored unchanged
    assert call(v=V(num_heads=4)) == INV
    for over in (dict(base=None), dict(base=P + 8), dict(reserved=1), dict(page_size=0),
                 dict(num_pages=0), dict(token_stride=1028), dict(head_stride=0),
                 dict(token_stride=64), dict(head_stride=64), dict(max_pages=0),
                 dict(page_table=None, page_size=400), dict(page_table=None, page_size=512,
                                                             num_pages=3)):
        assert call(kc=kv(attn, **over)) == INV, over
    assert call(kc=kv(attn, page_size=48)) == UNS
    assert call(kc=kv(attn, page_size=4, max_pages=200)) == UNS
    assert call(vc=kv(attn, page_table=2 * P)) == UNS
    assert call(k=K(dim=132, norm_dim=0)) == UNS
    # nothing to do
    assert call(batch=0, rows=0) == attn.ATTN_OK
    assert call(offs=P, rows=0) == attn.ATTN_OK


def test_append_fp8_refusals(attn):
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    call = lambda **o: call_append(attn, True, **o)   # noqa: E731
    for name in ("ks", "vs"):
        assert call(**{name: None}) == INV
        for over in (dict(base=None), dict(base=P + 2), dict(reserved=2), dict(block_tokens=0),
                     dict(block_tokens=12), dict(block_tokens=128), dict(block_stride=0),
                     dict(page_stride=-1), dict(head_stride=0)):
            assert call(**{name: scales(attn, **over)}) == INV, over
    assert call(vs=scales(attn, block_tokens=32)) == UNS
    assert call(max_q=0) == INV and call(max_q=2) == INV
    assert call(kc=kv(attn, token_stride=1032)) == INV          # strides of 16 bytes
    k = heads(attn, num_heads=8, out=None, dim=64, norm_dim=0)
    assert call(k=k, r=rope(attn, rot_dim=64)) == UNS
    assert call(v=None, vc=None) == INV


def call_decode(attn, k=0, v=0, ks=0, vs=0, **over):
    a = dict(q=P, lens=P, offs=None, batch=4, rows=None, hq=32, group=4, d=128, max_q=1,
             max_kv=500, scale=0.1, causal=0, ws=P, ws_bytes=1 << 40, out=P, lse=None)
    a.update(over)
    a["rows"] = a["batch"] if a["rows"] is None else a["rows"]
    k = kv(attn) if k == 0 else k
    v = kv(attn) if v == 0 else v
    ks = scales(attn) if ks == 0 else ks
    vs = scales(attn) if vs == 0 else vs
    return attn.lib().attn_decode_fp8(a["q"], ref(k), ref(v), ref(ks), ref(vs), a["lens"],
                                      a["offs"], a["batch"], a["rows"], a["hq"], a["group"],
                                      a["d"], a["max_q"], a["max_kv"], a["scale"], None,
                                      a["causal"], a["ws"], a["ws_bytes"], a["out"], a["lse"],
                                      None)


def test_decode_fp8_refusals(attn):
    INV, UNS, WS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_WORKSPACE
    call = lambda **o: call_decode(attn, **o)   # noqa: E731
    assert call(q=None) == INV and call(out=None) == INV and call(lens=None) == INV
    assert call(q=P + 8) == INV and call(out=P + 8) == INV
    assert call(group=0) == INV and call(hq=30) == INV and call(scale=float("nan")) == INV
    assert call(max_kv=-1) == INV and call(max_q=0) == INV and call(batch=-1) == INV
    assert call(rows=5) == INV and call(max_q=2) == INV
    assert call(d=64) == UNS and call(hq=34, group=17) == UNS
    assert call(offs=P, rows=20, max_q=5) == UNS                # 5 rows x 4 heads > 16
    assert call(batch=2049) == UNS
    assert call(max_kv=2 ** 31 - 1) == UNS                      # token numbers in ints
    assert call(batch=2048, rows=2048, hq=4 * 65535) == UNS     # costs of the split in ints
    assert call(max_kv=513) == INV
    for over in (dict(base=None), dict(base=P + 8), dict(token_stride=1032), dict(page_size=0)):
        assert call(k=kv(attn, **over)) == INV and call(v=kv(attn, **over)) == INV, over
    assert call(k=kv(attn, page_size=48)) == UNS
    assert call(v=kv(attn, page_table=2 * P)) == UNS
    assert call(ks=None) == INV and call(vs=None) == INV
    assert call(vs=scales(attn, block_tokens=32)) == UNS
    assert call(ks=scales(attn, block_tokens=24)) == INV
    assert call(ws=None) == WS and call(ws=P + 16) == WS
    assert call(batch=0) == attn.ATTN_OK


def test_decode_fp8_workspace(attn):
    small = attn.attn_decode_fp8_workspace(1, 32, 4, num_sms=152)
    assert small >= 8 * 16 * 128 * 4 and small % 256 == 0
    assert attn.attn_decode_fp8_workspace(64, 32, 4, num_sms=152) > small
    assert attn.attn_decode_fp8_workspace(0, 32, 4, num_sms=152) == small
    for bad in ((-1, 32, 4), (1, 0, 1), (1, 32, 0), (1, 30, 4)):
        with pytest.raises(attn.AttnError):
            attn.attn_decode_fp8_workspace(*bad, num_sms=152)


# ---- frequencies ------------------------------------------------------------

def turns_of(attn, rot, theta, **kw):
    t, m = attn.rope_turns(rot, theta, **kw)
    return [int(x) % (1 << 64) for x in t.tolist()], m


def near(turns, radians):
    """The double that was held differs from the radians' by a few 2^-52."""
    for t, f in zip(turns, radians):
        exact = Fraction(f) / Fraction(2 * math.pi) * (1 << 64)
        assert abs(t - exact) <= abs(exact) * Fraction(1, 1 << 49) + 1


def test_plain_linear_and_ntk_frequencies(attn):
    base = [10000.0 ** (-2 * i / 64) for i in range(32)]
    near(turns_of(attn, 64, 10000.0)[0], base)
    near(turns_of(attn, 64, 10000.0, scaling="linear", factor=4.0)[0], [f / 4 for f in base])
    t, m = turns_of(attn, 64, 10000.0, scaling="ntk", factor=8.0)
    theta = 10000.0 * 8 ** (64 / 62)
    near(t, [theta ** (-2 * i / 64) for i in range(32)])
    assert m == 1.0
    assert turns_of(attn, 2, 10000.0)[0] == turns_of(attn, 2, 7.0)[0]      # one radian


def test_scaling_by_parts_keeps_the_fast_and_stretches_the_slow(attn):
    rot, theta, factor, n0 = 128, 500000.0, 8.0, 8192
    base = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    for scaling, low, high in (("yarn", 1.0, 32.0), ("bands", 1.0, 4.0)):
        t, m = turns_of(attn, rot, theta, scaling=scaling, factor=factor, original_len=n0)
        got = [x / 2.0 ** 64 * 2 * math.pi for x in t]
        ratio = [g / f for g, f in zip(got, base)]
        assert all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))     # never rises
        assert ratio[0] == pytest.approx(1, rel=1e-12)
        assert ratio[-1] == pytest.approx(1 / factor, rel=1e-12)
        for f, r in zip(base, ratio):
            if n0 * f / (2 * math.pi) > 2 * high:
                assert r == pytest.approx(1, rel=1e-12)
            if n0 * f / (2 * math.pi) < low / 2:
                assert r == pytest.approx(1 / factor, rel=1e-12)
        assert m == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)
    # bands: halfway between the two wavelengths the blend is half and half
    f = 2.5 * 2 * math.pi / n0
    i = -math.log(f) / math.log(theta) * rot / 2
    t, _ = turns_of(attn, rot, theta, scaling="bands", factor=factor, original_len=n0)
    lo, hi = math.floor(i), math.ceil(i)
    ratio = [t[j] / 2.0 ** 64 * 2 * math.pi / base[j] for j in (lo, hi)]
    assert ratio[0] >= 0.5 + 0.5 / factor >= ratio[1]


def test_frequency_refusals(attn):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(theta=0.0), dict(theta=-1.0),
               dict(theta=float("inf")), dict(scaling="linear", factor=0.0),
               dict(scaling="yarn", factor=2.0), dict(scaling="bands", factor=2.0,
                                                      original_len=100.0, low=4.0, high=4.0),
               dict(scaling="ntk", factor=float("nan"))):
        a = {**dict(rot_dim=64, theta=10000.0), **kw}
        with pytest.raises(attn.AttnError):
            attn.rope_turns(a.pop("rot_dim"), a.pop("theta"), **a)
    with pytest.raises(ValueError):
        attn.rope_turns(64, 10000.0, scaling="other")


def test_frequencies_that_are_no_numbers_are_refused(attn):
    """Finite arguments whose quotients or powers overflow."""
    for kw in (dict(scaling="linear", factor=1e-320), dict(scaling="ntk", factor=1e-320, rot_dim=4),
               dict(scaling="yarn", factor=1e-320, original_len=4096.0),
               dict(scaling="bands", factor=1e-320, original_len=4096.0), dict(theta=5e-324,
                                                                               rot_dim=4096)):
        a = {**dict(rot_dim=64, theta=10000.0), **kw}
        with pytest.raises(attn.AttnError):
            attn.rope_turns(a.pop("rot_dim"), a.pop("theta"), **a)
    # a base that overflows leaves frequencies of 0: positions that far apart never turn
    t, _ = turns_of(attn, 4, 10000.0, scaling="ntk", factor=1e300)
    assert t[1] == 0


# ---- the binding's own checks -----------------------------------------------

def test_binding_refuses_wrong_tensors(attn):
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    t = torch.zeros(64, dtype=torch.int64)
    with pytest.raises(ValueError):
        attn.Rope(t.to(torch.int32))
    with pytest.raises(ValueError):
        attn.Rope(torch.zeros(128, dtype=torch.int64)[::2])
    with pytest.raises(TypeError):
        attn.attn_qk_norm_rope(x.float())
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(x.transpose(1, 2))
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(x, x[:2])
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(x, q_out=x[:, :2])
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(x, q_norm=torch.ones(128))
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(x, None, torch.zeros(2, dtype=torch.int32), rope=attn.Rope(t))
    with pytest.raises(ValueError):                       # a CPU tensor
        attn.attn_qk_norm_rope(x)
    cache = torch.zeros(2, 64, 4, 128, dtype=torch.bfloat16)
    lens = torch.ones(3, dtype=torch.int32)
    table = torch.zeros(3, 1, dtype=torch.int32)
    for bad in (dict(k=x[:, :2]), dict(v=None), dict(k_cache=cache.float()), dict(lens=lens.long()),
                dict(table=table[:2])):
        a = {**dict(k=x, v=x, k_cache=cache, v_cache=cache, lens=lens, table=table), **bad}
        with pytest.raises((ValueError, TypeError)):
            attn.attn_append_kv(a["k"], a["v"], a["k_cache"], a["v_cache"], a["lens"],
                                max_kv_len=64, page_table=a["table"])
    s = torch.ones(2, 4, 4)
    c8 = cache.to(torch.float8_e4m3fn)
    for scale in (s.half(), s[:, :3], s[:1], s[:, :, :2], s[0]):
        with pytest.raises(ValueError):
            attn.scale_descriptor(scale, c8)
    assert attn.scale_descriptor(s, c8).block_tokens == 16
    with pytest.raises(TypeError):
        attn.attn_decode_fp8(x, cache, cache, s, s, lens, group=1, scale=1.0, max_kv_len=64,
                             page_table=table, workspace=torch.zeros(8, dtype=torch.uint8))


def test_decode_fp8_refuses_caches_of_other_channels(attn):
    """Heads of 64 channels, or views of the first 128 of 256: not read as heads of 128."""
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    lens = torch.ones(2, dtype=torch.int32)
    s = torch.ones(2, 4, 1)
    for dim, base in ((64, 64), (64, 128), (256, 256)):
        c = torch.zeros(2, 64, 1, base, dtype=torch.bfloat16).to(torch.float8_e4m3fn)[..., :dim]
        with pytest.raises(ValueError, match="do not fit caches"):
            attn.attn_decode_fp8(q, c, c, s, s, lens, group=4, scale=1.0, max_kv_len=64)


def test_packed_descriptors_are_the_structures(attn):
    """The binding packs descriptors; their bytes are those of the C structures."""
    n = [0x1111111111111000 + 16 * i for i in range(8)]
    pairs = [(attn._pack_head_rows, attn.attn_head_rows_t,
              (n[0], -8, 16, n[1], 24, 32, n[2], 0.5, 64, 5, 128, 8, 0)),
             (attn._pack_kv, attn.attn_kv_t, (n[0], n[1], 16, 32, 64, 7, n[2], 9, 0)),
             (attn._pack_kv_scale, attn.attn_kv_scale_t, (n[0], n[1], 2, 3, 16, 0))]
    for pack, struct, fields in pairs:
        assert pack(*fields) == bytes(struct(*fields))
