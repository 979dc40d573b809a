"""The entry points of a cache held in 4 bits, of key weights and of eviction, without a GPU:
what they refuse before anything is launched."""
import pytest
import torch

from .test_cache_abi import P, attn, heads, kv, ref, rope, scales  # noqa: F401

NAN = float("nan")


def kv4(attn, **over):
    """Rows of 64 bytes."""
    return kv(attn, **{**dict(page_stride=64 * 8 * 64, token_stride=8 * 64, head_stride=64), **over})


def sc4(attn, **over):
    return scales(attn, **{**dict(page_stride=512, block_tokens=1), **over})


def call_append(attn, q=0, k=0, v=0, r=0, pos=None, kc=0, vc=0, ks=0, vs=0, lens=P, offs=None,
                batch=4, rows=4, max_kv=500):
    q = heads(attn) if q == 0 else q
    k = heads(attn, num_heads=8) if k == 0 else k
    v = heads(attn, num_heads=8, norm_dim=0, norm_weight=None) if v == 0 else v
    r = rope(attn) if r == 0 else r
    kc, vc = [kv4(attn) if c == 0 else c for c in (kc, vc)]
    ks, vs = [sc4(attn) if s == 0 else s for s in (ks, vs)]
    return attn.lib().attn_append_kv_fp4(ref(q), ref(k), ref(v), ref(r), pos, ref(kc), ref(vc),
                                         ref(ks), ref(vs), lens, offs, batch, rows, max_kv, None)


def test_append_fp4_refusals(attn):  # noqa: F811
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    call = lambda **o: call_append(attn, **o)   # noqa: E731
    K = lambda **o: heads(attn, **{**dict(num_heads=8), **o})                      # noqa: E731
    V = lambda **o: K(**{**dict(norm_dim=0, norm_weight=None), **o})               # noqa: E731
    for over in (dict(k=None), dict(lens=None), dict(lens=P + 2), dict(pos=P + 1), dict(offs=P + 2),
                 dict(batch=-1), dict(rows=5), dict(max_kv=-1), dict(max_kv=513), dict(v=None),
                 dict(vc=None), dict(v=None, vc=None), dict(q=heads(attn, out=None)),
                 dict(v=V(norm_dim=128)), dict(v=V(num_heads=4)), dict(k=K(out=P + 8)),
                 dict(k=K(out_row_stride=1028)), dict(v=V(in_row_stride=1028))):
        assert call(**over) == INV, over
    for over in (dict(base=None), dict(base=P + 16), dict(reserved=1), dict(page_size=0),
                 dict(num_pages=0), dict(token_stride=8 * 64 + 16), dict(head_stride=48),
                 dict(head_stride=0), dict(token_stride=32), dict(page_stride=64 * 8 * 64 + 16),
                 dict(max_pages=0), dict(page_table=None, page_size=400)):
        assert call(kc=kv4(attn, **over)) == INV, over
        assert call(vc=kv4(attn, **over)) == INV, over
    for over in (dict(base=None), dict(base=P + 2), dict(reserved=2), dict(block_tokens=0),
                 dict(block_tokens=16), dict(block_stride=0), dict(page_stride=-1),
                 dict(head_stride=0)):
        assert call(ks=sc4(attn, **over)) == INV, over
        assert call(vs=sc4(attn, **over)) == INV, over
    assert call(ks=None) == INV and call(vs=None) == INV
    assert call(kc=kv4(attn, page_size=48)) == UNS
    assert call(vc=kv4(attn, page_table=2 * P)) == UNS
    assert call(k=K(dim=64, norm_dim=0), r=rope(attn, rot_dim=64)) == UNS
    assert call(v=V(dim=64)) == UNS
    wide = 1 << 26
    assert call(kc=kv4(attn, max_pages=wide), vc=kv4(attn, max_pages=wide),
                max_kv=2 ** 31 - 8192) == UNS
    assert call(batch=0, rows=0) == attn.ATTN_OK
    assert call(offs=P, rows=0) == attn.ATTN_OK


def call_decode(attn, k=0, v=0, ks=0, vs=0, **over):
    a = dict(q=P, lens=P, offs=None, batch=4, rows=None, hq=32, group=4, d=128, max_q=1,
             max_kv=500, scale=0.1, causal=0, ws=P, ws_bytes=1 << 40, out=P, lse=None)
    a.update(over)
    a["rows"] = a["batch"] if a["rows"] is None else a["rows"]
    k, v = [kv4(attn) if c == 0 else c for c in (k, v)]
    ks, vs = [sc4(attn) if s == 0 else s for s in (ks, vs)]
    return attn.lib().attn_decode_fp4(a["q"], ref(k), ref(v), ref(ks), ref(vs), a["lens"], a["offs"],
                                      a["batch"], a["rows"], a["hq"], a["group"], a["d"], a["max_q"],
                                      a["max_kv"], a["scale"], None, a["causal"], a["ws"],
                                      a["ws_bytes"], a["out"], a["lse"], None)


def test_decode_fp4_refusals(attn):  # noqa: F811
    INV, UNS, WS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_WORKSPACE
    call = lambda **o: call_decode(attn, **o)   # noqa: E731
    for over in (dict(q=None), dict(out=None), dict(lens=None), dict(q=P + 8), dict(out=P + 8),
                 dict(group=0), dict(hq=30), dict(scale=NAN), dict(max_kv=-1), dict(max_q=0),
                 dict(batch=-1), dict(rows=5), dict(max_q=2), dict(max_kv=513), dict(ks=None),
                 dict(vs=None), dict(ks=sc4(attn, block_tokens=16)),
                 dict(vs=sc4(attn, block_tokens=16)), dict(vs=sc4(attn, base=P + 1))):
        assert call(**over) == INV, over
    for over in (dict(base=None), dict(base=P + 16), dict(token_stride=8 * 64 + 16),
                 dict(page_size=0), dict(head_stride=48), dict(token_stride=32)):
        assert call(k=kv4(attn, **over)) == INV and call(v=kv4(attn, **over)) == INV, over
    for over in (dict(d=64), dict(d=256), dict(hq=34, group=17), dict(offs=P, rows=20, max_q=5),
                 dict(batch=2049), dict(max_kv=2 ** 31 - 1),
                 dict(batch=2048, rows=2048, hq=4 * 65535), dict(k=kv4(attn, page_size=48)),
                 dict(v=kv4(attn, page_table=2 * P))):
        assert call(**over) == UNS, over
    assert call(ws=None) == WS and call(ws=P + 16) == WS
    assert call(batch=0) == attn.ATTN_OK
    n = attn.attn_decode_fp4_workspace(64, 32, 4, num_sms=152)
    assert n == attn.attn_decode_fp8_workspace(64, 32, 4, num_sms=152)
    with pytest.raises(attn.AttnError):
        attn.attn_decode_fp4_workspace(1, 30, 4, num_sms=152)


def call_weights(attn, k=0, w=0, **over):
    a = dict(q=P, lse=P, lens=P, offs=None, batch=4, rows=None, hq=32, group=4, d=128, max_q=1,
             max_kv=500, scale=0.1, causal=0, decay=1.0)
    a.update(over)
    a["rows"] = a["batch"] if a["rows"] is None else a["rows"]
    k = kv(attn) if k == 0 else k
    w = sc4(attn) if w == 0 else w
    return attn.lib().attn_key_weights(a["q"], ref(k), a["lse"], a["lens"], a["offs"], a["batch"],
                                       a["rows"], a["hq"], a["group"], a["d"], a["max_q"],
                                       a["max_kv"], a["scale"], a["causal"], a["decay"], ref(w),
                                       None)


def test_key_weights_refusals(attn):  # noqa: F811
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    call = lambda **o: call_weights(attn, **o)   # noqa: E731
    for over in (dict(q=None), dict(lse=None), dict(lens=None), dict(q=P + 8), dict(lse=P + 2),
                 dict(lens=P + 1), dict(offs=P + 2), dict(group=0), dict(hq=0), dict(hq=30),
                 dict(scale=NAN), dict(decay=NAN), dict(max_kv=-1), dict(max_q=0), dict(batch=-1),
                 dict(rows=5), dict(rows=-1, offs=P), dict(max_q=2), dict(max_kv=513), dict(k=None),
                 dict(w=None)):
        assert call(**over) == INV, over
    for over in (dict(base=None), dict(base=P + 8), dict(reserved=1), dict(page_size=0),
                 dict(num_pages=0), dict(token_stride=1028), dict(token_stride=64),
                 dict(head_stride=64), dict(head_stride=0), dict(page_stride=0), dict(max_pages=0),
                 dict(page_table=None, page_size=400),
                 dict(page_table=None, page_size=512, num_pages=3)):
        assert call(k=kv(attn, **over)) == INV, over
    for over in (dict(base=None), dict(base=P + 2), dict(reserved=1), dict(block_tokens=16),
                 dict(block_tokens=0), dict(page_stride=0), dict(block_stride=-1),
                 dict(head_stride=0)):
        assert call(w=sc4(attn, **over)) == INV, over
    for over in (dict(d=256), dict(d=96), dict(hq=129, group=129), dict(batch=2049),
                 dict(max_kv=2 ** 31 - 1), dict(k=kv(attn, page_size=48)),
                 dict(k=kv(attn, page_size=4, max_pages=200))):
        assert call(**over) == UNS, over
    assert call(batch=2048, hq=1 << 20, group=1, max_kv=512) == UNS   # items are counted in ints
    assert call(batch=0) == attn.ATTN_OK and call(max_kv=0) == attn.ATTN_OK


def call_evict(attn, **over):
    a = dict(k=kv(attn), v=kv(attn), w=sc4(attn), lens=P, keep=P, batch=4, heads=8, dk=128, dv=128,
             max_kv=500, max_keep=200, first=4, recent=16, ko=kv(attn, page_table=2 * P),
             vo=kv(attn, page_table=2 * P), wo=sc4(attn), kept=P, idx=P)
    a.update(over)
    return attn.lib().attn_evict_kv(ref(a["k"]), ref(a["v"]), ref(a["w"]), a["lens"], a["keep"],
                                    a["batch"], a["heads"], a["dk"], a["dv"], a["max_kv"],
                                    a["max_keep"], a["first"], a["recent"], ref(a["ko"]),
                                    ref(a["vo"]), ref(a["wo"]), a["kept"], a["idx"], None)


def test_evict_refusals(attn):  # noqa: F811
    INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
    call = lambda **o: call_evict(attn, **o)   # noqa: E731
    out = lambda **o: kv(attn, **{**dict(page_table=2 * P), **o})   # noqa: E731
    for over in (dict(k=None), dict(v=None), dict(vo=None), dict(ko=None), dict(w=None),
                 dict(lens=None), dict(keep=None), dict(idx=None), dict(lens=P + 1),
                 dict(keep=P + 2), dict(kept=P + 2), dict(idx=P + 2), dict(batch=-1), dict(heads=0),
                 dict(dk=0), dict(dv=0), dict(max_kv=-1), dict(max_kv=513), dict(max_keep=-1),
                 dict(max_keep=513), dict(first=-1), dict(recent=-1)):
        assert call(**over) == INV, over
    for over in (dict(base=None), dict(base=P + 8), dict(reserved=1), dict(page_size=0),
                 dict(num_pages=0), dict(token_stride=1028), dict(token_stride=64),
                 dict(head_stride=64), dict(page_stride=0), dict(max_pages=0),
                 dict(page_table=None, page_size=100)):
        assert call(k=kv(attn, **over)) == INV and call(v=kv(attn, **over)) == INV, over
        assert call(ko=out(**over)) == INV and call(vo=out(**over)) == INV, over
    for name in ("w", "wo"):
        for over in (dict(base=None), dict(base=P + 2), dict(block_tokens=16), dict(reserved=1),
                     dict(page_stride=0), dict(block_stride=0), dict(head_stride=0)):
            assert call(**{name: sc4(attn, **over)}) == INV, over
    for over in (dict(dk=100), dict(dv=100), dict(heads=257, dk=8, dv=8), dict(batch=2049),
                 dict(max_kv=2 ** 31 - 1), dict(k=kv(attn, page_size=48)),
                 dict(ko=out(page_size=48)), dict(v=kv(attn, page_table=3 * P)),
                 dict(vo=out(page_table=3 * P)), dict(vo=out(num_pages=9))):
        assert call(**over) == UNS, over
    wide = dict(head_stride=2048, token_stride=8 * 2048, page_stride=64 * 8 * 2048)
    assert call(dk=1032, k=kv(attn, **wide), ko=out(**wide)) == UNS
    assert call(batch=0) == attn.ATTN_OK


def tensors():
    """Arguments that fit one another, on the CPU: refused for that alone."""
    t = dict(x=torch.zeros(2, 2, 128, dtype=torch.bfloat16),
             q=torch.zeros(2, 4, 128, dtype=torch.bfloat16), lens=torch.ones(2, dtype=torch.int32),
             table=torch.zeros(2, 2, dtype=torch.int32),
             c4=torch.zeros(4, 64, 2, 64, dtype=torch.uint8),
             e=torch.zeros(4, 64, 2, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu),
             s=torch.ones(4, 64, 2), c=torch.zeros(4, 64, 2, 128, dtype=torch.bfloat16),
             lse=torch.zeros(2, 4), w=torch.zeros(4, 64, 2), idx=None, kept=None)
    t["keep"] = t["lens"].clone()
    return t


def bad_e(e, kind):
    base = torch.zeros(4 * 64 * 2 * 8 + 8, dtype=torch.uint8)
    view = {"channels apart": base[:4096].view(4, 64, 2, 8)[..., ::2],
            "odd address": base[1:2049].view(4, 64, 2, 4),
            "odd stride": base.as_strided((4, 64, 2, 4), (64 * 2 * 5, 10, 5, 1))}[kind]
    return view.view(torch.uint8).view(torch.float8_e8m0fnu) if kind != "channels apart" else \
        base[:4096].view(torch.float8_e8m0fnu).view(4, 64, 2, 8)[..., ::2]


def runs(attn):
    a = dict(max_kv_len=128)
    return {
        "append": lambda t: attn.attn_append_kv_fp4(t["x"], t["x"], t["c4"], t.get("v4", t["c4"]),
                                                    t["e"], t["s"], t["lens"],
                                                    page_table=t["table"], **a),
        "decode": lambda t: attn.attn_decode_fp4(t["q"], t["c4"], t.get("v4", t["c4"]), t["e"],
                                                 t["s"], t["lens"], group=2, scale=0.1,
                                                 page_table=t["table"], **a),
        "weights": lambda t: attn.attn_key_weights(t["q"], t["c"], t["lse"], t["lens"], t["w"],
                                                   group=2, scale=0.1, page_table=t["table"], **a),
        "evict": lambda t: attn.attn_evict_kv(t["c"], t.get("v", t["c"]), t["w"], t["lens"],
                                              t["keep"], t.get("ko", t["c"]), t.get("vo", t["c"]),
                                              t.get("wo"), max_keep=64, page_table=t["table"],
                                              out_page_table=t.get("otable", t["table"]),
                                              kept_len=t["kept"], indices=t["idx"], **a)}


BAD = {
    "append": [("c4", lambda t: t.float()), ("c4", lambda t: t[..., :32]), ("x", lambda t: t[:, :1]),
               ("e", lambda t: t.view(torch.uint8)), ("e", lambda t: t[:, :32]),
               ("e", lambda t: t[..., :2]), ("s", lambda t: t.half()), ("s", lambda t: t[:3]),
               ("lens", lambda t: t.long()), ("table", lambda t: t[:1]),
               ("v4", lambda t: torch.zeros(4, 64, 1, 64, dtype=torch.uint8))],
    "decode": [("c4", lambda t: t.float()), ("c4", lambda t: t[..., :32]), ("q", lambda t: t.float()),
               ("q", lambda t: t[:, :2]), ("e", lambda t: t.view(torch.uint8)),
               ("e", lambda t: t[:, :32]), ("s", lambda t: t.double()), ("s", lambda t: t[:, :, :1]),
               ("lens", lambda t: t[:1]), ("table", lambda t: t[:1])],
    "weights": [("q", lambda t: t.float()), ("q", lambda t: t.transpose(0, 1)),
                ("q", lambda t: t[..., :64].contiguous()), ("c", lambda t: t.float()),
                ("c", lambda t: t[:, :, :1]), ("lse", lambda t: t.double()),
                ("lse", lambda t: t[:, :2]), ("lse", lambda t: t.t().contiguous().t()),
                ("w", lambda t: t.half()), ("w", lambda t: t[:, :32]), ("lens", lambda t: t.long()),
                ("table", lambda t: t[:1])],
    "evict": [("c", lambda t: t.float()), ("v", lambda t: None), ("vo", lambda t: None),
              ("v", lambda t: torch.zeros(4, 64, 1, 128, dtype=torch.bfloat16)),
              ("ko", lambda t: torch.zeros(4, 64, 1, 128, dtype=torch.bfloat16)),
              ("vo", lambda t: torch.zeros(4, 64, 2, 64, dtype=torch.bfloat16)),
              ("w", lambda t: t.half()), ("w", lambda t: t[:3]),
              ("wo", lambda t: torch.zeros(4, 64, 1)), ("keep", lambda t: t.long()),
              ("keep", lambda t: t[:1]), ("lens", lambda t: t.float()), ("table", lambda t: t[:1]),
              ("otable", lambda t: torch.zeros(1, 2, dtype=torch.int32)),
              ("kept", lambda t: torch.zeros(2, dtype=torch.int64)),
              ("idx", lambda t: torch.zeros(2, 2, 63, dtype=torch.int32))],
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_binding_refusals(attn, name):  # noqa: F811
    run = runs(attn)[name]
    with pytest.raises(ValueError, match="on the GPU"):   # that they are on the CPU alone
        t = tensors()
        run(t)
    for i, (key, change) in enumerate(BAD[name]):
        t = tensors()
        t[key] = change(t.get(key))
        with pytest.raises((ValueError, TypeError)) as err:
            run(t)
        assert "on the GPU" not in str(err.value), (i, key, err.value)
    if name in ("append", "decode"):
        for kind in ("channels apart", "odd address", "odd stride"):
            t = tensors()
            t["e"] = bad_e(t["e"], kind)
            with pytest.raises(ValueError, match="contiguous and 4-byte aligned"):
                run(t)
