"""Host checks of the sliding-window attention: every call below returns before its first CUDA call."""
import ctypes

import sparse_attention_long_head_b200 as vs


def _fake(addr=0x10000):
    return ctypes.c_void_p(addr)


def test_window_host_validation():
    L = vs.lib()
    f = _fake
    base = dict(Q=f(0x1000), K=f(0x2000), V=f(0x3000), dtype=0, T=1000, B=3, cu=f(0x9000), maxn=500,
                Hq=4, Hkv=2, d=128, qs=512, kvs=256, scale=0.0, window=64, sinks=4, O=f(0x8000),
                lse=None, ws=f(0x10000), wsb=256)

    def single(**kw):
        a = base | kw
        return L.vs_window_attn_fwd(a["Q"], a["K"], a["V"], a["dtype"], a["maxn"], a["Hq"], a["Hkv"],
                                    a["d"], a["qs"], a["kvs"], a["scale"], a["window"], a["sinks"],
                                    a["O"], a["lse"], a["ws"], a["wsb"], None)

    def varlen(**kw):
        a = base | kw
        return L.vs_window_attn_fwd_varlen(a["Q"], a["K"], a["V"], a["dtype"], a["T"], a["B"], a["cu"],
                                           a["maxn"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["kvs"],
                                           a["scale"], a["window"], a["sinks"], a["O"], a["lse"],
                                           a["ws"], a["wsb"], None)

    for call in (single, varlen):
        for bad in ("Q", "K", "V", "O"):
            assert call(**{bad: None}) == vs.VS_ERR_INVALID_ARG, bad
        assert call(window=0) == vs.VS_ERR_INVALID_ARG
        assert call(window=-5) == vs.VS_ERR_INVALID_ARG
        assert call(sinks=-1) == vs.VS_ERR_INVALID_ARG
        assert call(Hkv=3) == vs.VS_ERR_INVALID_ARG
        assert call(maxn=0) == vs.VS_ERR_INVALID_ARG
        assert call(scale=-1.0) == vs.VS_ERR_INVALID_ARG
        assert call(scale=float("nan")) == vs.VS_ERR_INVALID_ARG
        assert call(dtype=vs.VS_FP32) == vs.VS_ERR_UNSUPPORTED
        assert call(dtype=7) == vs.VS_ERR_INVALID_ARG
        assert call(d=96, qs=384, kvs=192) == vs.VS_ERR_UNSUPPORTED
        assert call(qs=516) == vs.VS_ERR_UNSUPPORTED
        assert call(Q=f(0x1008)) == vs.VS_ERR_UNSUPPORTED
        assert call(maxn=(1 << 24) + 1) == vs.VS_ERR_UNSUPPORTED
        assert call(ws=None) == vs.VS_ERR_WORKSPACE
        assert call(wsb=128) == vs.VS_ERR_WORKSPACE
        assert call(ws=f(0x10010)) == vs.VS_ERR_WORKSPACE
    assert varlen(cu=None) == vs.VS_ERR_INVALID_ARG
    assert varlen(B=0) == vs.VS_ERR_INVALID_ARG
    assert varlen(T=0) == vs.VS_ERR_INVALID_ARG
    assert varlen(B=1 << 20, maxn=1 << 24) == vs.VS_ERR_UNSUPPORTED
