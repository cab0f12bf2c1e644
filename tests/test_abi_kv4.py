"""Host checks of the 4-bit cache calls: every call below returns before its first CUDA call."""
import ctypes

import pytest
import torch

import sparse_attention_long_head_b200 as vs


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


CACHE = dict(pool=_fake(0x100000), n_pages=100, table=_fake(0x2000), tld=8, lens=_fake(0x3000), B=3, max_len=500,
             Hkv=2, d=128, ws=_fake(0x40000), wsb=1 << 30)


def _append(**kw):
    a = CACHE | dict(K=_fake(), V=_fake(), dtype=0, T=50, cu=_fake(0x5000), max_new=30, kvs=256, seen=None, Hq=4,
                     Av=None, acc=None, pos=None, ld=0) | kw
    return vs.lib().vs_kv4_append(a["K"], a["V"], a["dtype"], a["T"], a["cu"], a["max_new"], a["kvs"], a["pool"],
                                  a["n_pages"], a["table"], a["tld"], a["lens"], a["seen"], a["B"], a["max_len"],
                                  a["Hq"], a["Hkv"], a["d"], a["Av"], a["acc"], a["pos"], a["ld"], a["ws"], a["wsb"],
                                  None)


def _read(**kw):
    a = CACHE | dict(K=_fake(), V=_fake(), T=50, cu=_fake(0x5000), max_read=30, kvs=256, start=None) | kw
    return vs.lib().vs_kv4_read(a["pool"], a["n_pages"], a["table"], a["tld"], a["lens"], a["start"], a["B"],
                                a["max_len"], a["Hkv"], a["d"], a["cu"], a["max_read"], a["T"], a["K"], a["V"],
                                a["kvs"], a["ws"], a["wsb"], None)


def _decode(**kw):
    a = CACHE | dict(Q=_fake(), dtype=0, qs=512, Hq=4, scale=0.0, window=0, sinks=0, acc_in=None, acc_out=None, ld=0,
                     O=_fake(), lse=None) | kw
    return vs.lib().vs_kv4_decode_attn_fwd(a["Q"], a["dtype"], a["qs"], a["pool"], a["n_pages"], a["table"], a["tld"],
                                           a["lens"], a["B"], a["max_len"], a["Hq"], a["Hkv"], a["d"], a["scale"],
                                           a["window"], a["sinks"], a["acc_in"], a["acc_out"], a["ld"], a["O"],
                                           a["lse"], a["ws"], a["wsb"], None)


def _evict(**kw):
    a = CACHE | dict(seen=_fake(), acc=_fake(0x6000), pos=_fake(0x7000), ld=500, keep=100, sinks=4, recent=50,
                     lens_out=_fake(0x8000), acc_out=_fake(0x9000), pos_out=_fake(0xa000), ldo=100) | kw
    return vs.lib().vs_kv4_evict(a["pool"], a["n_pages"], a["table"], a["tld"], a["lens"], a["seen"], a["B"],
                                 a["max_len"], a["Hkv"], a["d"], a["acc"], a["pos"], a["ld"], a["keep"], a["sinks"],
                                 a["recent"], a["lens_out"], a["acc_out"], a["pos_out"], a["ldo"], a["ws"], a["wsb"],
                                 None)


@pytest.mark.parametrize("call", [_append, _read, _decode, _evict])
def test_cache_arguments(call):
    for bad in ("pool", "table", "lens"):
        assert call(**{bad: None}) == vs.VS_ERR_INVALID_ARG, bad
    for bad in ("n_pages", "B", "max_len", "Hkv", "tld"):
        assert call(**{bad: 0}) == vs.VS_ERR_INVALID_ARG, bad
    assert call(max_len=513) == vs.VS_ERR_INVALID_ARG  # eight pages hold 512
    assert call(d=96) == vs.VS_ERR_UNSUPPORTED
    assert call(pool=_fake(0x100008)) == vs.VS_ERR_UNSUPPORTED
    assert call(max_len=(1 << 24) + 1, tld=1 << 20) == vs.VS_ERR_UNSUPPORTED
    assert call(B=40000) == vs.VS_ERR_UNSUPPORTED
    assert call(ws=None) == vs.VS_ERR_WORKSPACE
    assert call(ws=_fake(0x40010)) == vs.VS_ERR_WORKSPACE
    assert call(wsb=128) == vs.VS_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_append, _read])
def test_append_and_read_arguments(call):
    for bad in ("K", "V", "cu"):
        assert call(**{bad: None}) == vs.VS_ERR_INVALID_ARG, bad
    assert call(T=0) == vs.VS_ERR_INVALID_ARG
    assert call(kvs=248) == vs.VS_ERR_INVALID_ARG
    assert call(kvs=260) == vs.VS_ERR_UNSUPPORTED
    assert call(K=_fake(0x10008)) == vs.VS_ERR_UNSUPPORTED
    most = "max_new" if call is _append else "max_read"
    assert call(**{most: 0}) == vs.VS_ERR_INVALID_ARG
    assert call(**{most: 1 << 26}) == vs.VS_ERR_UNSUPPORTED  # 2^26 * 2 * 16 pieces


def test_append_arguments():
    assert _append(dtype=vs.VS_FP32) == vs.VS_ERR_UNSUPPORTED
    assert _append(dtype=9) == vs.VS_ERR_INVALID_ARG
    assert _append(Hq=3) == vs.VS_ERR_INVALID_ARG
    assert _append(Av=_fake()) == vs.VS_ERR_INVALID_ARG  # weights without a place for them
    assert _append(acc=_fake(), ld=0) == vs.VS_ERR_INVALID_ARG


def test_decode_arguments():
    for bad in ("Q", "O"):
        assert _decode(**{bad: None}) == vs.VS_ERR_INVALID_ARG, bad
    assert _decode(dtype=vs.VS_FP32) == vs.VS_ERR_UNSUPPORTED
    assert _decode(dtype=9) == vs.VS_ERR_INVALID_ARG
    assert _decode(Hq=3) == vs.VS_ERR_INVALID_ARG
    assert _decode(qs=500) == vs.VS_ERR_INVALID_ARG
    assert _decode(qs=516) == vs.VS_ERR_UNSUPPORTED
    assert _decode(Q=_fake(0x10008)) == vs.VS_ERR_UNSUPPORTED
    assert _decode(O=_fake(0x10008)) == vs.VS_ERR_UNSUPPORTED
    assert _decode(scale=-1.0) == vs.VS_ERR_INVALID_ARG
    assert _decode(scale=float("nan")) == vs.VS_ERR_INVALID_ARG
    assert _decode(window=-1) == vs.VS_ERR_INVALID_ARG
    assert _decode(window=5, sinks=-1) == vs.VS_ERR_INVALID_ARG
    assert _decode(sinks=4) == vs.VS_ERR_INVALID_ARG  # sinks of no window
    assert _decode(acc_in=_fake()) == vs.VS_ERR_INVALID_ARG
    assert _decode(acc_out=_fake(), ld=499) == vs.VS_ERR_INVALID_ARG
    assert _decode(B=32767, max_len=1 << 24, tld=1 << 18) == vs.VS_ERR_UNSUPPORTED
    small = vs.vs_kv4_decode_workspace_size(3, 4, 2, 128, 500)
    assert _decode(wsb=small - 1) == vs.VS_ERR_WORKSPACE
    more = vs.vs_kv4_decode_workspace_size(3, 4, 2, 128, 500, True)
    assert more >= small + 4 * 3 * 4 * 512
    assert _decode(acc_out=_fake(), ld=500, wsb=more - 1) == vs.VS_ERR_WORKSPACE


def test_evict_arguments():
    for bad in ("seen", "acc", "pos", "lens_out", "acc_out", "pos_out"):
        assert _evict(**{bad: None}) == vs.VS_ERR_INVALID_ARG, bad
    for out, of in (("lens_out", "lens"), ("acc_out", "acc"), ("pos_out", "pos")):
        same = {"lens": 0x3000, "acc": 0x6000, "pos": 0x7000}[of]
        assert _evict(**{out: _fake(same)}) == vs.VS_ERR_INVALID_ARG, out  # in place
    assert _evict(keep=0) == vs.VS_ERR_INVALID_ARG
    assert _evict(sinks=-1) == vs.VS_ERR_INVALID_ARG
    assert _evict(recent=-1) == vs.VS_ERR_INVALID_ARG
    assert _evict(sinks=60, recent=41) == vs.VS_ERR_INVALID_ARG
    assert _evict(ld=499) == vs.VS_ERR_INVALID_ARG
    assert _evict(ldo=99) == vs.VS_ERR_INVALID_ARG
    assert _evict(max_len=(1 << 18) + 1, tld=1 << 13, ld=1 << 20) == vs.VS_ERR_UNSUPPORTED
    assert _evict(wsb=vs.vs_kv4_evict_workspace_size(3, 2, 500, 100) - 1) == vs.VS_ERR_WORKSPACE


def test_page_bytes_and_binding_checks():
    assert vs.vs_kv4_page_bytes(8, 128) == 8 * 9216 and vs.vs_kv4_page_bytes(1, 64) == 4608
    assert vs.vs_kv4_page_bytes(0, 128) == 0 and vs.vs_kv4_page_bytes(2, 96) == 0
    table = torch.zeros((2, 4), dtype=torch.int32)
    pool = vs.kv4_pool(3, 2, 64, device="cpu")
    assert pool.shape == (3, 2, 4608)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # more slots than the table's four pages hold
        vs.vs_kv4_decode_attn_fwd(q, pool, table, table[:, 0].contiguous(), 257, q, None, vs.workspace(256, "cpu"))
    with pytest.raises(AssertionError):  # heads with a gap between them
        vs.vs_kv4_decode_attn_fwd(torch.zeros((2, 8, 64), dtype=torch.bfloat16)[:, ::2], pool, table, table[:, 0].contiguous(),
                                  256, q, None, vs.workspace(256, "cpu"))
    with pytest.raises(ValueError):
        vs.vs_kv4_decode_attn_fwd(q, torch.zeros((3, 2, 100), dtype=torch.uint8), table, table[:, 0].contiguous(), 256, q, None,
                                  vs.workspace(256, "cpu"))


def test_binding_checks_types_and_shapes():
    """What would be read or written out of range is refused before the call."""
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pool, ws = vs.kv4_pool(3, 2, 64, device="cpu"), vs.workspace(1 << 20, "cpu")
    q, kv = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    acc, pos = torch.zeros((2, 2, 256)), torch.zeros((2, 2, 256), dtype=torch.int32)
    for kw in (dict(lse=torch.zeros((2, 4))), dict(lse=torch.zeros((4, 2), dtype=torch.float64)),
               dict(acc_out=acc[:1]), dict(acc_out=acc.double()), dict(acc_out=acc[..., :255]), dict(acc_out=acc, acc_in=acc[:, :1]),
               dict(lens=lens[:1]), dict(lens=lens.long()), dict(table=table[:1])):
        a = dict(lens=lens, table=table, lse=None, acc_in=None, acc_out=None) | kw
        with pytest.raises(AssertionError):
            vs.vs_kv4_decode_attn_fwd(q, pool, a["table"], a["lens"], 256, q.clone(), a["lse"], ws,
                                      acc_in=a["acc_in"], acc_out=a["acc_out"])
    for kw in (dict(acc=acc[:1]), dict(pos=pos[:, :1]), dict(acc=pos), dict(pos=pos.long()), dict(cu=cu.long()),
               dict(n_tokens=lens[:1]), dict(A_v=torch.zeros((4, 4)), acc=acc), dict(lens=lens[:1])):
        a = dict(cu=cu, lens=lens, n_tokens=None, A_v=None, acc=None, pos=None) | kw
        with pytest.raises(AssertionError):
            vs.vs_kv4_append(kv, kv, a["cu"], 5, pool, table, a["lens"], ws, n_tokens=a["n_tokens"], A_v=a["A_v"],
                             acc=a["acc"], pos=a["pos"])
    with pytest.raises(AssertionError):
        vs.vs_kv4_read(pool, table, lens, lens[:1], cu, 5, kv, kv.clone(), ws)
    for kw in (dict(acc=acc[:1]), dict(pos=acc), dict(lens_out=lens[:1]), dict(acc_out=acc[:, :1]),
               dict(pos_out=pos[..., :99]), dict(acc=acc[..., :255]), dict(n_tokens=lens.long())):
        a = dict(n_tokens=lens, acc=acc, pos=pos, lens_out=lens.clone(), acc_out=acc.clone(), pos_out=pos.clone()) | kw
        with pytest.raises(AssertionError):
            vs.vs_kv4_evict(pool, table, lens, a["n_tokens"], 256, a["acc"], a["pos"], 100, 4, 50, a["lens_out"],
                            a["acc_out"], a["pos_out"], ws)


def test_window_binding_checks_shapes():
    q, k = torch.zeros((8, 4, 64), dtype=torch.bfloat16), torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    ws = vs.workspace(256, "cpu")
    for args in ((q, k[:7], k[:7], q.clone(), None), (q, k, k[:, :1], q.clone(), None), (q, k, k, q[:7].clone(), None),
                 (q, k, k, q.clone(), torch.zeros((8, 4))), (q, k, k, q.clone(), torch.zeros((4, 7)))):
        with pytest.raises(AssertionError):
            vs.vs_window_attn_fwd(*args[:3], 5, 1, *args[3:], ws)
